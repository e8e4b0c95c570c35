"""The attention block (bitlinear_attn_forward) against its single calls at other
layouts: the ~2B decoder's layer, heads of 128 channels, interleaved pairs, fp32
tokens, and enough rows for the tensor-core projections."""
import pytest
import torch

import workloads
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


_layers = {}


def layer(K, heads):
    """(packed, gamma) of q, k, v and o, and gains, packed once per layout."""
    if (K, heads) not in _layers:
        hq, hkv, d = heads
        shapes = ((hq * d, K), (hkv * d, K), (hkv * d, K), (K, hq * d))
        proj = []
        for i, (n, k) in enumerate(shapes):
            p, g = bl.bitlinear_pack_weights(workloads.latent_weights(n, k, 30 + i))
            proj.append((torch.from_numpy(p).cuda(), g))
        gains = [torch.from_numpy(workloads.norm_gains(n, 40 + i)).cuda()
                 for i, n in enumerate((K, K, K, hq * d, d, d))]
        _layers[K, heads] = proj, gains
    return _layers[K, heads]


def steps(lens, heads, page, seed, spare):
    """Two equal steps whose caches hold finite values everywhere."""
    for _ in range(2):
        step = Step(lens, heads, page, seed=seed, spare=spare)
        step.k_cache.nan_to_num_(0.25)
        step.v_cache.nan_to_num_(0.25)
        yield step


# the 2B decoder's layer (20 heads on 5 of 128, 2560 wide), its widths with heads of
# 64, one key head for all, and as many as queries; model widths that differ from the
# heads' and widths on both sides of the others' blocks
LAYOUTS = [(2560, (20, 5, 128)), (2560, (40, 10, 64)), (640, (8, 1, 128)), (256, (4, 4, 64)),
           (1152, (6, 3, 128))]
STEPS = [[(1, 700)], [(1, 33), (1, 900), (1, 1)], [(5, 77), (3, 300)], [(130, 130), (1, 64), (2, 2)],
         [(0, 9), (260, 300), (0, 0), (1, 5000)]]


@pytest.mark.parametrize("K,heads", LAYOUTS)
@pytest.mark.parametrize("lens", STEPS)
@pytest.mark.parametrize("norm,interleaved,dtype", [(False, True, torch.bfloat16),
                                                    (True, False, torch.float32),
                                                    (True, True, torch.float32)])
def test_block_is_its_calls(K, heads, lens, norm, interleaved, dtype):
    hq, hkv, d = heads
    proj, gains = layer(K, heads)
    one, two = steps(lens, heads, 32, 7, spare=2)
    f, hint = frequencies(d, 500000.0), max(n for n, _ in lens)
    x = torch.from_numpy(workloads.activations_f32(one.rows, K, 3)).cuda().to(dtype)
    y = torch.full((one.rows, K), CANARY, dtype=torch.bfloat16, device="cuda")
    got = bl.bitlinear_attn_forward(
        x, *proj, hq, one.k_cache, one.v_cache, one.q_start, one.kv_len, one.table, f,
        gains=gains[:4] if norm else (None,) * 4, head_gains=gains[4:] if norm else (None, None),
        eps=1e-5, interleaved=interleaved, window=200, max_q_len=hint, y=y)
    assert got is y

    problems = [(x, p, g, n, None) for (p, g), n in zip(proj, (hq * d, hkv * d, hkv * d))]
    ws = torch.empty(bl.bitlinear_workspace_bytes_grouped(problems), dtype=torch.uint8,
                     device="cuda")
    if norm:
        q, k, v = bl.bitlinear_forward_grouped_rmsnorm(problems, gains[:3], eps=1e-5,
                                                       workspace=ws)
    else:
        q, k, v = bl.bitlinear_forward_grouped(problems, workspace=ws)
    head_gains = dict(q_gain=gains[4], k_gain=gains[5]) if norm else {}
    q = two.append(f, q=q, k=k, v=v, eps=1e-5, interleaved=interleaved, **head_gains)
    a = two.attend(q=q, window=200, max_q_len=hint)
    p, g = proj[3]
    want = (bl.bitlinear_forward_rmsnorm(a, p, g, K, gains[3], eps=1e-5) if norm
            else bl.bitlinear_forward(a, p, g, K))
    live = one.live
    assert torch.equal(y[live].view(torch.int16), want[live].view(torch.int16))
    for c, e in ((one.k_cache, two.k_cache), (one.v_cache, two.v_cache)):
        assert torch.equal(c.view(torch.int16), e.view(torch.int16))
    two.q = q.view(two.rows, hq, d)
    two.check_attention(a, window=200)


@pytest.mark.parametrize("T", [1, 61])
def test_captured_decode_step_of_the_2b_layer(T):
    # one graph of the block, replayed while every sequence gets its next token
    K, heads = LAYOUTS[0]
    proj, _ = layer(K, heads)
    lens = [(1, 40 + 13 * i % 400) for i in range(T)]
    one, two = steps(lens, heads, 64, 8, spare=0)
    f = frequencies(heads[2])
    x = torch.from_numpy(workloads.activations_f32(T, K, 5)).cuda().to(torch.bfloat16)
    y = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(bl.bitlinear_workspace_bytes_attn(T, K, T, *heads), dtype=torch.uint8,
                     device="cuda")

    def call(step, y, **kw):
        return bl.bitlinear_attn_forward(x, *proj, heads[0], step.k_cache, step.v_cache,
                                         step.q_start, step.kv_len, step.table, f, max_q_len=1,
                                         y=y, **kw)

    call(two, torch.empty_like(y))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(one, y, workspace=ws)
    for back in (3, 2, 1):
        kv = torch.tensor([n - back for _, n in lens], dtype=torch.int32)
        one.kv_len.copy_(kv)
        two.kv_len.copy_(kv)
        graph.replay()
        want = call(two, torch.empty_like(y))
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_blocks_on_two_streams_at_once():
    # a prompt's and a decode step's, each with what the call allocates
    K, heads = LAYOUTS[0]
    proj, gains = layer(K, heads)
    f = frequencies(heads[2])
    work = []
    for i, lens in enumerate(([(300, 300), (90, 500)], [(1, 60 * n) for n in range(1, 12)])):
        one, two = steps(lens, heads, 64, 20 + i, spare=0)
        x = torch.from_numpy(workloads.activations_f32(one.rows, K, 6 + i)).cuda()
        work.append((one, two, x.to(torch.bfloat16)))

    def call(step, x, stream=None):
        return bl.bitlinear_attn_forward(x, *proj, heads[0], step.k_cache, step.v_cache,
                                         step.q_start, step.kv_len, step.table, f,
                                         gains=gains[:4], stream=stream)

    want = [call(two, x) for _, two, x in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(8):
        for i, (one, _, x) in enumerate(work):
            outs[i].append(call(one, x, streams[i]))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(y.view(torch.int16), w.view(torch.int16)) for y in o)


def test_a_block_of_no_rows():
    K, heads = LAYOUTS[0]
    proj, _ = layer(K, heads)
    step = Step([(0, 30)], heads, 64, seed=9)
    kept = step.k_cache.clone()
    y = bl.bitlinear_attn_forward(torch.empty((0, K), dtype=torch.bfloat16, device="cuda"), *proj,
                                  heads[0], step.k_cache, step.v_cache, step.q_start, step.kv_len,
                                  step.table, frequencies(heads[2]))
    assert y.shape == (0, K)
    assert torch.equal(step.k_cache.view(torch.int16), kept.view(torch.int16))
