"""Rotation and append (bitlinear_rope_append) against a plain 64-bit form."""
import pytest
import torch

import ternary_weight_w1_b200 as bl
from tests.paged_cases import Step, frequencies

pytestmark = pytest.mark.gpu

CANARY = 0.4375


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    bl.lib()
    yield
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_OK, 0)


def check(step, norm=False, interleaved=False, theta=10000.0, eps=1e-5, **kw):
    f = frequencies(step.d, theta)
    gains = {}
    if norm:
        gen = torch.Generator().manual_seed(1)
        gains = {n: (torch.rand(step.d, generator=gen) + 0.5).cuda() for n in ("q_gain", "k_gain")}
    out = torch.full((step.rows, step.hq, step.d), CANARY, dtype=torch.bfloat16, device="cuda")
    before = [c.clone().view(torch.int16) for c in (step.k_cache, step.v_cache)]
    step.append(f, q_out=out, eps=eps, interleaved=interleaved, **gains, **kw)
    q, q_tol = step.rotated(step.q, f, gains.get("q_gain"), eps, interleaved)
    k, k_tol = step.rotated(step.k, f, gains.get("k_gain"), eps, interleaved)
    placed = torch.zeros(step.k_cache.shape[0], step.page, dtype=torch.bool, device="cuda")
    written = torch.zeros(step.rows, dtype=torch.bool, device="cuda")
    for s, at, n, kv in step.spans():
        pos = torch.arange(kv - n, kv, device="cuda")
        ok = pos >= 0
        rows, pos = torch.arange(at, at + n, device="cuda")[ok], pos[ok]
        written[rows] = True
        page, slot = step.table[s].long()[pos // step.page], pos % step.page
        placed[page, slot] = True
        assert ((step.k_cache[page, :, slot].double() - k[rows]).abs() <= k_tol[rows]).all()
        assert torch.equal(step.v_cache[page, :, slot], step.v[rows])
    assert ((out.double() - q).abs() <= q_tol)[written].all()
    assert (out[~written] == CANARY).all()
    for c, b in zip((step.k_cache, step.v_cache), before):     # no other slot is touched
        same = c.view(torch.int16) == b
        assert same.transpose(1, 2)[~placed].all()


@pytest.mark.parametrize("heads", [(4, 2, 64), (20, 5, 128), (3, 1, 128), (64, 8, 128), (5, 5, 64)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(heads, norm, interleaved):
    check(Step([(1, 1), (1, 700), (40, 50), (0, 9), (3, 3)], heads, 16, seed=1, spare=4, front=2),
          norm, interleaved)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page):
    check(Step([(page + 3, 2 * page + 1), (1, page), (1, page + 1)], (4, 2, 64), page, seed=2))


def test_far_positions():
    # fp32 products would be off by a hundredth of a turn here
    step = Step([(5, 131072), (1, 99991)], (2, 1, 128), 256, seed=3)
    check(step, theta=500000.0)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 1000, 1100])
def test_sequence_counts(n):
    lens = [(i % 3, 20 + i % 7) for i in range(n)]
    check(Step(lens, (2, 1, 64), 16, seed=n, spare=1), norm=True)


def test_many_rows():
    check(Step([(5000, 5003), (0, 0), (1, 12), (900, 900)], (4, 2, 64), 64, seed=4), norm=True)


def test_rows_before_position_zero_are_skipped():
    check(Step([(9, 4), (2, 0), (3, 3)], (4, 2, 64), 16, seed=5))


@pytest.mark.parametrize("lens", [[], [(0, 0)], [(0, 5), (0, 0)]])
def test_nothing_to_do(lens):
    check(Step(lens, spare=3, front=1))


def test_one_gain_only():
    for name in ("q_gain", "k_gain"):
        step = Step([(3, 40)], (4, 2, 64), 16, seed=6)
        f, g = frequencies(64), torch.linspace(0.5, 1.5, 64, device="cuda")
        out = step.append(f, eps=1e-5, **{name: g})
        q, q_tol = step.rotated(step.q, f, g if name == "q_gain" else None, 1e-5)
        k, k_tol = step.rotated(step.k, f, g if name == "k_gain" else None, 1e-5)
        assert ((out.double() - q).abs() <= q_tol).all()
        page = step.table[0].long()[torch.arange(37, 40, device="cuda") // 16]
        got = step.k_cache[page, :, torch.arange(37, 40, device="cuda") % 16].double()
        assert ((got - k).abs() <= k_tol).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_parts_of_a_fused_projection_in_place(interleaved):
    # q, k and v are column ranges of one buffer; q is rotated where it stands
    step = Step([(1, 8), (20, 30)], (4, 2, 64), 16, seed=7)
    fused = torch.cat((step.q.flatten(1), step.k.flatten(1), step.v.flatten(1)), 1)
    f = frequencies(64)
    q, q_tol = step.rotated(step.q, f, interleaved=interleaved)
    kept = fused[:, 256:].clone()
    qv = fused[:, :256]
    out = step.append(f, q=qv, k=fused[:, 256:384], v=fused[:, 384:].view(step.rows, 2, 64),
                      q_out=qv, interleaved=interleaved)
    assert out is qv and torch.equal(fused[:, 256:], kept)
    assert ((out.reshape(q.shape).double() - q).abs() <= q_tol).all()


def test_captured_step():
    step = Step([(1, 30), (1, 50)], (4, 2, 64), 16, seed=8)
    f, out = frequencies(64), torch.empty_like(step.q)
    step.append(f, q_out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.append(f, q_out=out)
    step.lens = [(1, 17), (1, 49)]
    step.kv_len.copy_(torch.tensor([17, 49], dtype=torch.int32))
    g.replay()
    q, tol = step.rotated(step.q, f)
    assert ((out.double() - q).abs() <= tol).all()


def test_bad_indexes_are_reported_and_not_used():
    # CPU reading first: every index passes view() or page_of() before an access
    for what, value in (("table", -2), ("table", 10 ** 6), ("kv_len", 10 ** 6), ("kv_len", -3),
                        ("q_start", 10 ** 6)):
        step = Step([(2, 150), (2, 90)], (4, 2, 64), 16, seed=9)
        kept = step.k_cache.clone()
        if what == "table":
            step.table[1, 5] = value                   # positions 80 .. 95
        elif what == "kv_len":
            step.kv_len[1] = value
        else:
            step.q_start[2] = value
        step.append(frequencies(64))
        status, word = bl.bitlinear_get_fault()
        assert status == bl.BITLINEAR_ERR_INDEX and word == 2, (what, value, status, word)
        if what == "table":                            # only sequence 0's two tokens were stored
            changed = (step.k_cache.view(torch.int16) != kept.view(torch.int16)).any(-1).any(1)
            assert changed.sum() == 2
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_OK, 0)


@pytest.mark.parametrize("bad", ["one token more than the table holds", "far behind the table",
                                 "most negative", "end behind the rows", "start before the rows"])
@pytest.mark.parametrize("page", [16, 64])
def test_a_sequence_of_bad_lengths_stores_nothing(bad, page):
    # every column of the table holds a page of the cache, so that a length cut to
    # what exists would find a place: nothing may be stored there
    step = Step([(3, 3 * page), (2, 3 * page), (4, 2 * page + 5)], (4, 2, 64), page, seed=10,
                extra_cols=0)
    f = frequencies(64)
    want = [c.clone() for c in (step.k_cache, step.v_cache)]
    good = Step([(3, 3 * page), (2, 3 * page), (4, 2 * page + 5)], (4, 2, 64), page, seed=10,
                extra_cols=0)
    good.append(f)
    stored = {0: 3, 1: 2, 2: 4}
    if bad == "end behind the rows":
        step.q_start[3] = 10 ** 6
        del stored[2]
    elif bad == "start before the rows":
        step.q_start[0] = -7
        del stored[0]
    else:
        step.kv_len[1] = {"one token more than the table holds": 3 * page + 1,
                          "far behind the table": 2 ** 31 - 1, "most negative": -2 ** 31}[bad]
        del stored[1]
    for s, n in stored.items():                        # what the good sequences store
        kv = step.lens[s][1]
        pos = torch.arange(kv - n, kv, device="cuda")
        at, slot = good.table[s].long()[pos // page], pos % page
        for w, c in zip(want, (good.k_cache, good.v_cache)):
            w[at, :, slot] = c[at, :, slot]
    step.append(f)
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_ERR_INDEX, 2)
    for c, w in zip((step.k_cache, step.v_cache), want):
        assert (c.view(torch.int16) != w.view(torch.int16)).sum().item() == 0
