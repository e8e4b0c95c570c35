"""The attention block of a decoder layer (bitlinear_attn_forward): the run of the
projections, the rotation that appends, the attention and the o projection as a
model makes it, prompt first and tokens after it."""
import numpy as np
import pytest
import torch

import oracle
import workloads
import ternary_weight_w1_b200 as bl
from tests.paged_cases import Step, frequencies

pytestmark = pytest.mark.gpu

K, HEADS = 384, (6, 2, 64)          # model width; 6 query heads on 2 key heads of 64


@pytest.fixture(scope="module", autouse=True)
def cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    bl.lib()
    yield
    assert bl.bitlinear_get_fault() == (bl.BITLINEAR_OK, 0)


class Layer:
    def __init__(self, seed, norm=False, head_norm=False):
        hq, hkv, d = HEADS
        shapes = ((hq * d, K), (hkv * d, K), (hkv * d, K), (K, hq * d))
        self.latent = [workloads.latent_weights(n, k, seed + i) for i, (n, k) in enumerate(shapes)]
        packed = [bl.bitlinear_pack_weights(w) for w in self.latent]
        self.proj = [(torch.from_numpy(p).cuda(), g) for p, g in packed]
        self.gains = tuple(torch.from_numpy(workloads.norm_gains(k, seed + i)).cuda() if norm
                           else None for i, (_, k) in enumerate(shapes))
        self.head_gains = tuple(torch.from_numpy(workloads.norm_gains(d, seed + i)).cuda()
                                if head_norm else None for i in (7, 8))
        self.f = frequencies(d)

    def tokens(self, n, seed, dtype=torch.bfloat16):
        x = torch.from_numpy(workloads.activations_f32(n, K, seed)).cuda()
        return x.to(dtype)

    def block(self, step, x, **kw):
        return bl.bitlinear_attn_forward(x, *self.proj, HEADS[0], step.k_cache, step.v_cache,
                                         step.q_start, step.kv_len, step.table, self.f,
                                         gains=self.gains, head_gains=self.head_gains, **kw)

    def apart(self, step, x, **kw):
        """The same by the single calls."""
        hq, hkv, d = HEADS
        problems = [(x, p, g, n, None) for (p, g), n in zip(self.proj, (hq * d, hkv * d, hkv * d))]
        need = bl.bitlinear_workspace_bytes_grouped(problems)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        if self.gains[0] is not None:
            q, k, v = bl.bitlinear_forward_grouped_rmsnorm(problems, self.gains[:3], workspace=ws)
        else:
            q, k, v = bl.bitlinear_forward_grouped(problems, workspace=ws)
        q = step.append(self.f, q=q, k=k, v=v, q_gain=self.head_gains[0],
                        k_gain=self.head_gains[1])
        a = step.attend(q=q, **kw)
        (p, g), gain = self.proj[3], self.gains[3]
        if gain is not None:
            return bl.bitlinear_forward_rmsnorm(a, p, g, K, gain), q, a
        return bl.bitlinear_forward(a, p, g, K), q, a


def filled(step, seed):
    """A step whose cache holds finite values wherever a sequence has tokens."""
    step.k_cache[step.k_cache.isnan()] = 0
    step.v_cache[step.v_cache.isnan()] = 0
    return step


@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 300), (1, 17)], [(5, 90), (1, 33)],
                                  [(70, 70)], [(40, 100), (1, 200), (0, 0), (3, 3)]])
@pytest.mark.parametrize("norm", [False, True])
def test_block_is_its_calls(lens, norm):
    layer = Layer(50, norm=norm, head_norm=norm)
    one, two = (filled(Step(lens, HEADS, 16, seed=4), 4) for _ in range(2))
    x = layer.tokens(one.rows, 9)
    y = layer.block(one, x, window=64)
    want, q, a = layer.apart(two, x, window=64)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    assert torch.equal(one.k_cache.view(torch.int16), two.k_cache.view(torch.int16))
    assert torch.equal(one.v_cache.view(torch.int16), two.v_cache.view(torch.int16))
    # the attention of the run against the plain 64-bit form on the run's cache
    two.q = q.view(two.rows, HEADS[0], HEADS[2])
    two.check_attention(a, window=64)


def test_projections_against_the_oracle():
    # one token: v of a one-token sequence is what the attention returns, so the
    # block is the o BitLinear of the v BitLinear, which the oracle computes
    layer = Layer(60)
    step = Step([(1, 1)], HEADS, 16, seed=5)
    x = layer.tokens(1, 3)
    y = layer.block(step, x)
    orc = oracle.default()
    bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    v = orc.forward(bits, layer.latent[2], gamma=np.float32(layer.proj[2][1]))["y"]
    v = v.reshape(HEADS[1], 1, HEADS[2]).repeat(HEADS[0] // HEADS[1], 1).reshape(1, -1)
    want = orc.forward(np.ascontiguousarray(v), layer.latent[3],
                       gamma=np.float32(layer.proj[3][1]))["y"]
    assert np.array_equal(y.view(torch.int16).cpu().numpy().view(np.uint16), want)


@pytest.mark.parametrize("parts", [[30], [13, 17], [1] * 6 + [24], [29, 1]])
def test_prompt_in_parts_then_tokens(parts):
    # however a prompt is cut, its cache and its last row's attention are the
    # same up to the order of the sums
    layer = Layer(70)
    x = layer.tokens(32, 11)
    parts = parts + [1, 1]
    step = Step([(1, 32)], HEADS, 16, seed=6)          # its pages; the cache starts empty
    step.k_cache.fill_(float("nan"))
    step.v_cache.fill_(float("nan"))
    done = 0
    for n in parts:
        step.q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        step.kv_len = torch.tensor([done + n], dtype=torch.int32, device="cuda")
        step.lens, step.rows = [(n, done + n)], n
        step.live = torch.ones(n, dtype=torch.bool, device="cuda")
        _, q, a = layer.apart(step, x[done:done + n].contiguous())
        step.q = q.view(n, HEADS[0], HEADS[2])
        step.check_attention(a)
        done += n
    assert done == 32
    whole = Step([(32, 32)], HEADS, 16, seed=6)
    layer.block(whole, x)
    assert torch.equal(step.keys(0, step.k_cache), whole.keys(0, whole.k_cache))
    assert torch.equal(step.keys(0, step.v_cache), whole.keys(0, whole.v_cache))


def test_fp32_tokens_padding_and_a_given_workspace():
    layer = Layer(80)
    lens = [(1, 20), (9, 40)]
    step = filled(Step(lens, HEADS, 16, seed=7, spare=3), 7)
    x = layer.tokens(step.rows, 12, torch.float32)
    need = bl.bitlinear_workspace_bytes_attn(step.rows, K, 2, *HEADS)
    y = layer.block(step, x)
    again = filled(Step(lens, HEADS, 16, seed=7, spare=3), 7)
    out = torch.empty_like(y)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert layer.block(again, x, y=out, workspace=ws) is out
    assert torch.equal(out[:10].view(torch.int16), y[:10].view(torch.int16))


def test_captured_block():
    layer = Layer(90)
    step = filled(Step([(1, 40), (1, 90)], HEADS, 16, seed=8), 8)
    x, y = layer.tokens(2, 13), torch.zeros((2, K), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(bl.bitlinear_workspace_bytes_attn(2, K, 2, *HEADS), dtype=torch.uint8,
                     device="cuda")
    layer.block(step, x, y=y, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.block(step, x, y=y, workspace=ws)
    want = y.clone()
    for _ in range(3):
        y.zero_()
        g.replay()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
