"""Attention over the paged cache (bitlinear_paged_attention) against a plain
64-bit form, at the shapes, masks and index patterns where it can go wrong."""
import math

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


def check(step, window=0, scale=None, max_q_len=None):
    y = torch.full((step.rows, step.hq, step.d), CANARY, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((step.rows, step.hq), device="cuda")
    need = bl.bitlinear_workspace_bytes_attention(step.rows, len(step.lens), step.hq, step.hkv,
                                                  step.d)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")   # no initialisation needed
    out = step.attend(y=y, lse=lse, workspace=ws, window=window, scale=scale, max_q_len=max_q_len)
    assert out is y
    step.check_attention(y, lse, CANARY, scale, window)
    return y, lse


# heads: groups of 1, 2, 3, 4, 5, 8, 12, 16 and 20 query heads per key head
HEADS = [(4, 4, 64), (4, 2, 64), (6, 2, 128), (20, 5, 128), (5, 1, 64), (8, 1, 128), (24, 2, 128),
         (16, 1, 64), (20, 1, 128)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_single_tokens(heads, page):
    check(Step([(1, 1), (1, 700), (1, 31), (1, 32), (1, 33), (1, 129)], heads, page, seed=1),
          max_q_len=1)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(page, d):
    lens = [(1, page - 1), (1, page), (1, page + 1), (3, 3 * page + 5), (40, 2 * page + 7)]
    check(Step(lens, (8, 2, d), page, seed=2))


@pytest.mark.parametrize("heads", HEADS)
def test_drafts(heads):
    check(Step([(5, 5), (2, 300), (4, 63), (5, 1000)], heads, 32, seed=3), max_q_len=5)


@pytest.mark.parametrize("q,kv", [(1, 4099), (2, 2), (7, 7), (16, 16), (33, 33), (64, 200),
                                  (127, 127), (128, 128), (129, 129), (255, 300), (300, 1000),
                                  (513, 513)])
@pytest.mark.parametrize("heads", [(8, 2, 64), (20, 5, 128), (3, 3, 128), (6, 1, 64)])
def test_chunk_lengths(q, kv, heads):
    check(Step([(q, kv)], heads, 64, seed=q + kv))


@pytest.mark.parametrize("heads", [(8, 2, 64), (20, 5, 128)])
@pytest.mark.parametrize("page", [16, 128])
def test_mixed_batch(heads, page):
    lens = [(1, 77), (200, 333), (1, 1), (0, 50), (1, 1500), (90, 90), (0, 0), (5, 2000)]
    step = Step(lens, heads, page, seed=5, spare=9, front=3)
    check(step)
    check(step, max_q_len=200)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 64, 100, 129, 5000])
@pytest.mark.parametrize("heads", [(8, 2, 64), (20, 5, 128)])
def test_window(window, heads):
    check(Step([(1, 900), (40, 300), (1, 20), (150, 150), (3, 65)], heads, 16, seed=6),
          window=window)


def test_pages_in_front_of_the_window_are_not_needed():
    # a server frees them: their table entries are gone, their slots rewritten
    step = Step([(1, 900), (40, 700), (300, 900)], (8, 2, 64), 16, seed=7)
    window, want = 100, None
    want = step.attention(window=window)
    for s, at, n, kv in step.spans():
        gone = max(0, kv - n - window + 1) // 16
        step.k_cache[step.table[s, :gone].long()] = math.nan
        step.v_cache[step.table[s, :gone].long()] = math.nan
        step.table[s, :gone] = -1
    y = step.attend(window=window)
    off = (y.double() - want[0]).abs()
    assert (off <= want[1]).all()


def test_rows_that_see_nothing():
    # more rows than the cache holds: the first ones stand before position 0
    step = Step([(10, 4), (3, 0), (50, 20), (1, 0), (300, 130)], (8, 2, 64), 16, seed=8)
    y, lse = check(step)
    none = torch.isinf(lse[:, 0])
    assert none.sum() == 6 + 3 + 30 + 1 + 170 and (y[none] == 0).all()


@pytest.mark.parametrize("lens", [[], [(0, 0)], [(0, 5), (0, 0)]])
def test_nothing_to_do(lens):
    step = Step(lens, spare=2)
    y = torch.full((2, 4, 64), CANARY, dtype=torch.bfloat16, device="cuda")
    step.attend(y=y)
    assert (y == CANARY).all()


@pytest.mark.parametrize("scale", [1e-3, 0.5, 4.0])
def test_scale(scale):
    # at the largest a row's weight sits on one key, far above the others
    check(Step([(1, 500), (70, 400)], (8, 2, 64), 32, seed=9), scale=scale)


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("q", [1, 80])
def test_scores_that_grow_and_fall_along_the_keys(rising, q):
    # every tile of keys raises the running maximum, or none after the first
    step = Step([(q, 1500)], (4, 1, 64), 64, seed=10)
    ramp = torch.linspace(0.05, 4.0, 1500)
    ramp = (ramp if rising else ramp.flip(0)).cuda()
    direction = torch.randn(64, generator=torch.Generator().manual_seed(3)).cuda()
    at = step.table[0].long()[:-(-1500 // 64)]
    k = (ramp[:, None] * direction).to(torch.bfloat16)
    full = torch.full((len(at) * 64, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    full[:1500] = k
    step.k_cache[at, 0] = full.view(len(at), 64, 64)
    step.q[:] = direction.to(torch.bfloat16)
    check(step, scale=1.0)


def test_large_and_small_values():
    step = Step([(1, 300), (60, 260)], (4, 2, 128), 16, seed=11)
    step.v_cache.mul_(1e30)
    check(step)
    step.v_cache.mul_(1e-38)
    step.q.mul_(1e-20)
    check(step)


def test_many_sequences():
    gen = torch.Generator().manual_seed(4)
    lens = [(int(n > 2), int(kv)) for n, kv in zip(torch.randint(0, 12, (1100,), generator=gen),
                                                   torch.randint(1, 90, (1100,), generator=gen))]
    check(Step(lens, (4, 1, 64), 16, seed=12), max_q_len=1)


def test_five_thousand_sequences():
    lens = [(1, 1 + i % 5) for i in range(5000)] + [(40, 60)]
    check(Step(lens, (2, 1, 64), 16, seed=24))


@pytest.mark.parametrize("heads", [(130, 1, 64), (200, 2, 64), (128, 1, 128)])
def test_many_heads_per_key_head(heads):
    # a token of more rows than half an item of the chunk kernel is cut anywhere
    check(Step([(1, 70), (3, 40), (20, 33)], heads, 16, seed=25))


def test_one_long_sequence_among_short_ones():
    check(Step([(1, 5), (1, 40000), (1, 3), (1, 64)], (8, 2, 128), 128, seed=13), max_q_len=1)


def test_shared_prefix_pages():
    step = Step([(1, 130), (6, 140), (30, 150)], (4, 2, 64), 16, seed=14)
    step.table[1:, :8] = step.table[0, :8]         # 128 positions in common
    check(step)


def test_strided_queries_and_outputs():
    # queries as the front part of a fused projection's rows, outputs into a
    # wider buffer, two-dimensional rows
    step = Step([(1, 77), (40, 90), (3, 3)], (4, 2, 64), 16, seed=15)
    wide = torch.full((step.rows, 640), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:320] = step.q.flatten(1)
    out = torch.full((step.rows, 512), CANARY, dtype=torch.bfloat16, device="cuda")
    y = step.attend(q=wide[:, 64:320], y=out[:, 128:384])
    step.check_attention(y)
    assert (out[:, :128] == CANARY).all() and (out[:, 384:] == CANARY).all()
    assert torch.equal(step.attend(q=wide[:, 64:320].view(step.rows, 4, 64)).flatten(1), y)


@pytest.mark.parametrize("offset", [8, 24])
def test_rows_aligned_to_sixteen_bytes_only(offset):
    step = Step([(1, 77), (90, 100)], (4, 2, 64), 16, seed=26)
    wide = torch.full((step.rows, 256 + 40), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, offset:offset + 256] = step.q.flatten(1)
    out = torch.full((step.rows, 256 + 40), CANARY, dtype=torch.bfloat16, device="cuda")
    step.check_attention(step.attend(q=wide[:, offset:offset + 256],
                                     y=out[:, offset:offset + 256]))
    assert (out[:, :offset] == CANARY).all() and (out[:, offset + 256:] == CANARY).all()


@pytest.mark.parametrize("q", [1, 150])
def test_a_cache_of_more_than_two_to_the_32_elements(q):
    step = Step([(q, 300), (1, 90)], (8, 2, 128), 64, seed=27)
    pages = step.k_cache.shape[0]
    first = 2 ** 32 // (2 * 64 * 128)                  # its elements are past 32 bits
    caches = []
    for c in (step.k_cache, step.v_cache):
        big = torch.empty((first + pages, 2, 64, 128), dtype=torch.bfloat16, device="cuda")
        big[first:] = c
        caches.append(big)
    table = torch.where(step.table >= 0, step.table + first, step.table)
    y = bl.bitlinear_paged_attention(step.q, *caches, step.q_start, step.kv_len, table)
    step.check_attention(y)
    # and the append reaches the same places
    f = torch.zeros(64, device="cuda")                 # no rotation: the keys as they are
    bl.bitlinear_rope_append(step.q, step.k, step.v, *caches, step.q_start, step.kv_len, table, f)
    page = table[0].long()[torch.arange(300 - q, 300, device="cuda") // 64]
    slot = torch.arange(300 - q, 300, device="cuda") % 64
    assert torch.equal(caches[0][page, :, slot], step.k[:q])
    assert torch.equal(caches[1][page, :, slot], step.v[:q])


def test_a_hint_that_is_too_small_only_costs_time():
    step = Step([(1, 50), (130, 200), (20, 20)], (8, 2, 64), 16, seed=16)
    check(step, max_q_len=1)


def test_same_bits_every_time():
    step = Step([(1, 3000), (200, 700), (1, 64), (12, 900)], (20, 5, 128), 64, seed=17)
    first = step.attend()
    for _ in range(3):
        assert torch.equal(step.attend().view(torch.int16), first.view(torch.int16))


def test_captured_step_follows_the_lengths_on_the_device():
    # one graph, captured for the largest step, replayed while tokens arrive
    step = Step([(2, 40), (60, 400), (1, 200)], (8, 2, 64), 16, seed=18)
    y = torch.zeros((step.rows, 8, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(bl.bitlinear_workspace_bytes_attention(step.rows, 3, 8, 2, 64),
                     dtype=torch.uint8, device="cuda")
    step.attend(y=y, workspace=ws)                     # outside the capture first
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.attend(y=y, workspace=ws)
    for lens in ([(2, 40), (60, 400), (1, 200)], [(1, 33), (60, 60), (0, 0)],
                 [(0, 40), (1, 399), (1, 17)], [(0, 0), (0, 0), (63, 180)]):
        start = torch.tensor([0] + [n for n, _ in lens]).cumsum(0)
        step.q_start.copy_(start.to(torch.int32))
        step.kv_len.copy_(torch.tensor([kv for _, kv in lens], dtype=torch.int32))
        step.lens = lens
        step.live = torch.arange(step.rows, device="cuda") < int(start[-1])
        y.fill_(CANARY)
        graph.replay()
        step.check_attention(y, canary=CANARY)


def test_two_graphs_share_a_workspace_one_after_the_other():
    a = Step([(1, 5000)], (8, 2, 128), 64, seed=19)
    b = Step([(100, 300), (1, 4000)], (20, 5, 128), 32, seed=20)
    need = max(bl.bitlinear_workspace_bytes_attention(s.rows, len(s.lens), s.hq, s.hkv, s.d)
               for s in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for s in (a, b):
        y = torch.zeros((s.rows, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
        s.attend(y=y, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.attend(y=y, workspace=ws)
        outs.append(y)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        (a, b)[i].check_attention(outs[i])


def test_replays_in_a_row_on_one_workspace():
    # flags and parts of one replay are never taken for another's
    steps = [Step([(300, 900), (1, 2000)], (8, 2, 64), 16, seed=28),
             Step([(700, 700)], (4, 1, 128), 64, seed=29)]
    need = max(bl.bitlinear_workspace_bytes_attention(s.rows, len(s.lens), s.hq, s.hkv, s.d)
               for s in steps)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for s in steps:
        y = torch.zeros((s.rows, s.hq, s.d), dtype=torch.bfloat16, device="cuda")
        s.attend(y=y, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.attend(y=y, workspace=ws)
        outs.append(y)
        graphs.append(g)
    first = [o.clone() for o in outs]
    for i, s in enumerate(steps):
        s.check_attention(first[i])
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for n in range(150):
        i = (n * 7 // 3) % 2
        outs[i].fill_(CANARY)
        graphs[i].replay()
        wrong += (outs[i].view(torch.int16) != first[i].view(torch.int16)).sum()
    assert wrong.item() == 0


def test_streams():
    # two steps on two streams at once, each with what the call allocates
    steps = [Step([(1, 3000), (64, 500)], (8, 2, 64), 16, seed=21),
             Step([(1, 2500), (1, 100)], (20, 5, 128), 64, seed=22)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(6):
        for i in (0, 1):
            outs[i].append(steps[i].attend(stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        steps[i].check_attention(outs[i][0])
        assert all(torch.equal(o.view(torch.int16), outs[i][0].view(torch.int16)) for o in outs[i])


@pytest.mark.parametrize("q", [1, 100])
def test_bad_indexes_are_reported_and_not_used(q):
    # CPU reading first: every index passes view() or page_of() before an access
    good = Step([(q, 150), (q, 90)], (8, 2, 64), 16, seed=23)
    lives = torch.zeros(good.rows, dtype=torch.bool, device="cuda")
    lives[:q] = True                                   # sequence 0 is untouched below
    for what, value in (("table", -5), ("table", 10 ** 6), ("kv_len", 10 ** 6), ("kv_len", -3),
                        ("q_start", 10 ** 6)):
        step = Step([(q, 150), (q, 90)], (8, 2, 64), 16, seed=23)
        if what == "table":
            step.table[1, 2] = value
        elif what == "kv_len":
            step.kv_len[1] = value
        else:
            step.q_start[2] = value
        y = step.attend()
        status, word = bl.bitlinear_get_fault()
        assert status == bl.BITLINEAR_ERR_INDEX and word == 2, (what, value, status, word)
        good.check_attention(y, rows=lives)
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_OK, 0)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("heads", [(16, 16, 64), (32, 16, 64), (20 * 12, 12, 64)])
def test_short_and_long_sequences_in_two_launches(heads, window):
    # enough sequences and key heads of 64 channels that the short ones get a launch
    # of their own; among them lengths on both sides of its 16 (or 32) rows
    lens = [(1, 1 + 37 * i % 300) for i in range(34)] + [
        (8, 90), (9, 90), (16, 16), (17, 500), (0, 7), (32, 40), (33, 33), (130, 200), (1, 0),
        (2, 64), (3, 1)]
    lens = lens[::2] + lens[1::2]
    step = Step(lens, heads, 16, seed=21, spare=3)
    check(step, window=window)
    check(step, window=window, max_q_len=130)


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("q,heads", [(17, (2, 2, 128)), (5, (8, 2, 128)), (8, (8, 2, 128)),
                                     (3, (21, 3, 128)), (1, (40, 2, 128)), (2, (128, 1, 128)),
                                     (1, (129, 1, 128)), (32, (1, 1, 128))])
def test_a_few_rows_of_128_channels(q, heads, window):
    check(Step([(q, q), (q, 1000), (1, 129), (q, 128), (0, 9), (q, q + 63)], heads, 32, seed=22),
          window=window, max_q_len=q)


@pytest.mark.parametrize("kv", [64, 65, 127, 128, 129, 191, 192, 193, 449])
@pytest.mark.parametrize("window", [0, 1, 63, 64, 65, 128])
def test_ends_and_windows_about_the_steps_of_sixty_four_keys(kv, window):
    # first and last steps that hold one key, all keys or none that a row sees
    for heads in ((4, 1, 64), (2, 2, 64), (4, 1, 128)):
        check(Step([(kv, kv), (33, kv), (min(kv, 200), kv + 64)], heads, 16, seed=kv), window=window)


def test_prompts_on_two_streams():
    # both fill the GPU and join split items while the other one's blocks come and go
    steps = [Step([(700, 900), (300, 1500)], (20, 5, 128), 64, seed=31),
             Step([(900, 900), (1, 3000), (250, 2000)], (40, 10, 64), 16, seed=32)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for i in (0, 1):
            outs[i].append(steps[i].attend(stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        steps[i].check_attention(outs[i][0])
        assert all(torch.equal(o.view(torch.int16), outs[i][0].view(torch.int16)) for o in outs[i])


@pytest.mark.parametrize("q", [2, 100])
def test_starts_that_fall_are_reported(q):
    # sequences that overlap write the same rows: nothing out of range, and a fault
    step = Step([(q, 150), (q, 150), (q, 150)], (8, 2, 64), 16, seed=33)
    step.q_start[2] = 0
    y = step.attend()
    torch.cuda.synchronize()
    assert bl.bitlinear_get_fault()[0] == bl.BITLINEAR_ERR_INDEX
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64)])
@pytest.mark.parametrize("n", [32, 33, 65, 600])
def test_chunks_among_many_sequences(n, heads):
    # above 32 sequences the deal's sums stand in shared memory that the first
    # queries are copied to
    lens = [(1 + 89 * i % 40, 40 + 53 * i % 90) for i in range(n)]
    step = Step(lens, heads, 16, seed=34)
    y, _ = check(step)
    for _ in range(3):
        assert torch.equal(step.attend().view(torch.int16), y.view(torch.int16))


def test_prompts_on_many_streams_beside_decoding():
    # blocks that join parts hold their SMs while the other launches, of both
    # kernels and two priorities, take those that come free
    steps = [Step([(500 + 90 * i, 700 + 200 * i), (60, 900)], heads, 64, seed=40 + i)
             for i, heads in enumerate([(20, 5, 128), (8, 2, 64), (8, 1, 128)])]
    steps += [Step([(1, 20000), (1, 9000)], (8, 2, 128), 128, seed=44),
              Step([(1, 30000)], (8, 2, 64), 64, seed=45)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(priority=-(i % 2)) for i in range(len(steps))]
    outs = [[] for _ in steps]
    for _ in range(12):
        for s, st, o in zip(steps, streams, outs):
            o.append(s.attend(stream=st))
    torch.cuda.synchronize()
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_OK, 0)
    for s, o in zip(steps, outs):
        s.check_attention(o[0])
        assert all(torch.equal(x.view(torch.int16), o[0].view(torch.int16)) for x in o)


def timed_out(step, worker, **kw):
    """A call in which `worker` waits in vain for 2 ms: a fault, every row of a head
    complete or as it was, and the next call on the workspace right."""
    y = torch.full((step.rows, step.hq, step.d), CANARY, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.rows, step.hq), CANARY, device="cuda")
    ws = torch.empty(bl.bitlinear_workspace_bytes_attention(
        step.rows, len(step.lens), step.hq, step.hkv, step.d), dtype=torch.uint8, device="cuda")
    rc = bl.bitlinear_paged_attention_inject_timeout(
        step.q, step.k_cache, step.v_cache, step.q_start, step.kv_len, step.table, worker, 2000,
        y=y, lse=lse, workspace=ws, **kw)
    assert rc == bl.BITLINEAR_OK
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_ERR_TIMEOUT, 1)
    want, tol, want_lse, lse_tol = step.attention()
    kept = (y == CANARY).all(-1)
    right = ((y.double() - want).abs() <= tol).all(-1)
    assert (kept | right)[step.live].all() and kept[~step.live].all()
    assert kept[step.live].any()
    assert (lse[kept] == CANARY).all()
    done = ~kept & step.live[:, None]
    assert ((lse.double() - want_lse).abs() <= lse_tol)[done].all()
    y.fill_(CANARY)
    step.attend(y=y, lse=lse, workspace=ws, **kw)
    step.check_attention(y, lse, CANARY)
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_OK, 0)


@pytest.mark.parametrize("worker", [0, 1, 5])
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64)])
def test_a_wait_that_runs_out_in_the_kernel_for_few_rows(heads, worker):
    # single sequences' keys on many workers, and sequences whole on one
    for lens in ([(1, 9000), (1, 40)], [(1, 30 + i) for i in range(300)]):
        timed_out(Step(lens, heads, 16, seed=50, spare=2), worker, max_q_len=1)


@pytest.mark.parametrize("worker", [0, 1, 7])
@pytest.mark.parametrize("heads", [(20, 5, 128), (8, 2, 64)])
def test_a_wait_that_runs_out_in_the_kernel_for_many_rows(heads, worker):
    # neighbours wait for the worker's part of an item, in the kernel or behind it
    for lens in ([(700, 900), (300, 1500)], [(130, 6000)], [(100, 130)] * 70):
        timed_out(Step(lens, heads, 64, seed=51, spare=2), worker)


@pytest.mark.parametrize("lens", [[(1, 300), (1, 17)], [(70, 90), (1, 40)]])
def test_python_and_compiled_marshalling_make_the_same_calls(lens, monkeypatch):
    f = frequencies(64)
    gain = torch.linspace(0.5, 1.5, 64, device="cuda")
    got = []
    for calls in (bl._fast(), bl._NoFastCalls):
        monkeypatch.setattr(bl, "_fast_calls", calls)
        step = Step(lens, (8, 2, 64), 16, seed=46, spare=1)
        wide = torch.cat((step.q.flatten(1), step.k.flatten(1), step.v.flatten(1)), 1)
        lse = torch.zeros((step.rows, 8), device="cuda")
        q = step.append(f, q=wide[:, :512], k=wide[:, 512:640], v=wide[:, 640:].view(-1, 2, 64),
                        q_gain=gain, eps=1e-5, interleaved=True)
        y = step.attend(q=q, lse=lse, window=50, scale=0.2, max_q_len=70)
        z = step.attend(q=q.view(-1, 8, 64), stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        got.append([t.view(torch.int16)[step.live] for t in (q, y, z, lse)] +
                   [c.view(torch.int16) for c in (step.k_cache, step.v_cache)])
        with pytest.raises(ValueError, match="rows"):
            step.attend(q=q, y=y[:1])
        with pytest.raises(bl.BitLinearError):
            step.attend(q=q, scale=-1.0)
    assert bl._fast().__name__ == "_NoFastCalls"
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_other_python_threads_run_during_a_call(tmp_path):
    # the extension's calls bound to a function that waits until another thread of
    # the interpreter has run (two seconds at most)
    import ctypes
    import subprocess
    import threading
    src = tmp_path / "wait.c"
    src.write_text("""
#include <time.h>
static volatile int go, in;
int inside(void) { return in; }
void set(int v) { go = v; in = 0; }
int call(void) {
    struct timespec t = {0, 1000000};
    in = 1;
    for (int i = 0; i < 2000 && !go; ++i) nanosleep(&t, 0);
    return go ? 0 : 2;
}
""")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(src), "-o", str(tmp_path / "wait.so")],
                   check=True)
    wait = ctypes.CDLL(str(tmp_path / "wait.so"))
    address = ctypes.cast(wait.call, ctypes.c_void_p).value
    L, fast = bl.lib(), bl._fast()
    step, f = Step([(1, 30)], (8, 2, 64), 16, seed=47), frequencies(64)
    real = [ctypes.cast(n, ctypes.c_void_p).value
            for n in (L.bitlinear_rope_append, L.bitlinear_paged_attention)]
    fast.bind(address, address)
    try:
        for call in (lambda: step.append(f), step.attend):
            wait.set(0)

            def other():
                while not wait.inside():
                    pass
                wait.set(1)

            thread = threading.Thread(target=other, daemon=True)
            thread.start()
            call()                                     # raises when the other never ran
            thread.join(timeout=10)
            assert not thread.is_alive()
    finally:
        fast.bind(*real)
    step.check_attention(step.attend())


def test_queries_and_outputs_side_by_side_and_on_top_of_each_other():
    step = Step([(1, 77), (40, 90)], (4, 2, 64), 16, seed=48)
    wide = torch.full((step.rows, 768), CANARY, dtype=torch.bfloat16, device="cuda")
    wide[:, 256:512] = step.q.flatten(1)
    for at in (0, 512):                                # their ranges overlap, no element does
        step.check_attention(step.attend(q=wide[:, 256:512], y=wide[:, at:at + 256]))
        assert torch.equal(wide[:, 256:512], step.q.flatten(1))
    for y in (wide[:, 256:512], wide[:, 248:504], wide[:, 264:520], wide[:, 8:264]):
        with pytest.raises(bl.BitLinearError) as e:
            step.attend(q=wide[:, 256:512], y=y)
        assert e.value.status == bl.BITLINEAR_ERR_ARG
    # the append's queries: q, k and v in one buffer, the output over one of them
    flat = torch.full((step.rows * 776,), CANARY, dtype=torch.bfloat16, device="cuda")
    fused = flat[:step.rows * 768].view(step.rows, 768)
    fused[:, :512] = torch.cat((step.q.flatten(1), step.k.flatten(1), step.v.flatten(1)), 1)
    kept = flat.clone()
    parts = dict(q=fused[:, :256], k=fused[:, 256:384], v=fused[:, 384:512])
    for out in (fused[:, 8:264], fused[:, 264:520], fused[:, 504:760],
                flat.as_strided((step.rows, 256), (776, 1))):
        with pytest.raises(bl.BitLinearError) as e:
            step.append(frequencies(64), q_out=out, **parts)
        assert e.value.status == bl.BITLINEAR_ERR_ARG
    assert torch.equal(flat, kept)
    step.append(frequencies(64), q_out=fused[:, 512:], **parts)
    want, tol = step.rotated(step.q, frequencies(64))
    assert ((fused[:, 512:].reshape(want.shape).double() - want).abs() <= tol).all()
    assert torch.equal(fused[:, :512], kept[:step.rows * 768].view(step.rows, 768)[:, :512])


def test_host_tensors_are_named_on_another_stream_too():
    step, stream = Step([(1, 30)], (8, 2, 64), 16, seed=49), torch.cuda.Stream()
    for call in (lambda q: step.attend(q=q, stream=stream),
                 lambda q: step.append(frequencies(64), q=q, stream=stream)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(step.q.cpu())
