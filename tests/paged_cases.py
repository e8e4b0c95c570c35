"""A step's sequences on a paged cache, and the plain 64-bit forms of the two
operators on it (test infrastructure; it shares no code with the library).

Every slot of the cache that no sequence's position owns holds a NaN, and so
do the rows of q, k and v that belong to no sequence: an operator that lets one
into a result fails its comparison."""
import math

import torch

import ternary_weight_w1_b200 as bl

HALF_BF16 = 2.0 ** -8          # half a step of bf16, relative to the value


class Step:
    """Sequences of (new tokens, tokens in the cache with these)."""

    def __init__(self, lens, heads=(4, 2, 64), page=16, seed=0, spare=0, front=0, extra_cols=1,
                 q_scale=2.0, device="cuda"):
        self.lens, self.page, self.front = list(lens), page, front
        self.hq, self.hkv, self.d = heads
        gen = torch.Generator().manual_seed(seed)
        q_len = [q for q, _ in self.lens]
        need = [-(-kv // page) for _, kv in self.lens]
        self.rows = front + sum(q_len) + spare
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=gen).tolist()
        table = torch.full((len(need), max(need, default=0) + extra_cols), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            for c in range(n):
                table[s, c] = order.pop()
        start = [front]
        for n in q_len:
            start.append(start[-1] + n)

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=gen) * scale).to(torch.bfloat16).to(device)

        self.q = normal(self.rows, self.hq, self.d, scale=q_scale)
        self.k, self.v = normal(self.rows, self.hkv, self.d), normal(self.rows, self.hkv, self.d)
        live = torch.zeros(self.rows, dtype=torch.bool)
        live[front:start[-1]] = True
        for t in (self.q, self.k, self.v):
            t[~live.to(device)] = math.nan
        self.k_cache = normal(pages, self.hkv, page, self.d)
        self.v_cache = normal(pages, self.hkv, page, self.d)
        owned = torch.zeros((pages, page), dtype=torch.bool)
        for s, (_, kv) in enumerate(self.lens):
            for c in range(need[s]):
                owned[table[s, c], :min(page, kv - c * page)] = True
        for c in (self.k_cache, self.v_cache):
            c.masked_fill_(~owned.to(device)[:, None, :, None], math.nan)
        self.table, self.live = table.to(device), live.to(device)
        self.q_start = torch.tensor(start, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor([kv for _, kv in self.lens], dtype=torch.int32, device=device)
        self.device = device

    def keys(self, s, cache):
        """[kv][hkv][d] in 64 bits."""
        kv = self.lens[s][1]
        pages = self.table[s, :-(-kv // self.page)].long()
        return cache[pages].transpose(1, 2).reshape(-1, self.hkv, self.d)[:kv].double()

    def spans(self):
        at = self.front
        for s, (n, kv) in enumerate(self.lens):
            yield s, at, n, kv
            at += n

    # ------------------------------------------------------------- attention

    def attend(self, **kw):
        return bl.bitlinear_paged_attention(kw.pop("q", self.q), self.k_cache, self.v_cache,
                                            self.q_start, self.kv_len, self.table, **kw)

    def attention(self, scale=None, window=0):
        """(y, tolerance of y, lse, tolerance of lse), rows of no sequence NaN.

        The kernel rounds every weight p to bf16 (half a step each, so the sum
        moves by at most 2^-8 sum p |v|) and the output once (2^-8 |y|). Its
        fp32 parts: a score is a sum of d products, off by at most
        d 2^-24 sum |q k| before the scale, and its exponent's argument is
        rounded twice more at magnitude |s| scale log2 e, together below
        4 d 2^-24 b with b the row's largest scale sum |q k|; ex2 is off by
        2^-22 relative; sums over n keys by n 2^-23 relative."""
        scale = self.d ** -0.5 if scale is None else scale
        shape = (self.rows, self.hq, self.d)
        y = torch.full(shape, math.nan, dtype=torch.float64, device=self.device)
        tol, lse, lse_tol = torch.zeros_like(y), y[..., 0].clone(), torch.zeros_like(y[..., 0])
        g = self.hq // self.hkv
        for s, at, n, kv in self.spans():
            if n == 0:
                continue
            k, v = (self.keys(s, c).repeat_interleave(g, 1) for c in (self.k_cache, self.v_cache))
            q = self.q[at:at + n].double()
            pos = torch.arange(kv - n, kv, device=self.device)[:, None]
            j = torch.arange(kv, device=self.device)
            seen = j <= pos
            if window:
                seen &= j > pos - window
            sc = torch.einsum("qhd,khd->hqk", q, k) * scale
            b = torch.einsum("qhd,khd->hqk", q.abs(), k.abs()) * scale * seen
            b = b.amax(-1, keepdim=True) if kv else torch.zeros_like(q[:, :, :1]).transpose(0, 1)
            sc = sc.masked_fill(~seen, -math.inf)
            top = sc.amax(-1, keepdim=True) if kv else b - math.inf
            p = torch.exp(sc - top.clamp(min=-1e300))
            total = p.sum(-1, keepdim=True)
            p = torch.where(total > 0, p / total, 0.0)
            out = torch.einsum("hqk,khd->qhd", p, v)
            size = torch.einsum("hqk,khd->qhd", p, v.abs())
            fp32 = 4 * self.d * 2.0 ** -24 * b + 2.0 ** -21 + (kv + 64) * 2.0 ** -23
            y[at:at + n] = out
            tol[at:at + n] = HALF_BF16 * (out.abs() + size) * 1.01 + size * fp32.permute(1, 0, 2)
            lse[at:at + n] = (top + torch.log(total))[..., 0].T
            lse_tol[at:at + n] = (fp32[..., 0] + 2.0 ** -22 * top[..., 0].abs().clamp(max=1e6)).T
        return y, tol, lse, lse_tol

    def check_attention(self, y, lse=None, canary=None, scale=None, window=0, rows=None):
        """Every row of every sequence against the plain form; the other rows
        still hold ``canary``."""
        want, tol, want_lse, lse_tol = self.attention(scale, window)
        live = self.live if rows is None else rows
        y = y.reshape(self.rows, self.hq, self.d)
        off = (y[live].double() - want[live]).abs()
        assert torch.isfinite(y[live]).all()
        worst = (off - tol[live]).max().item() if off.numel() else 0.0
        assert worst <= 0, (worst, (off / tol[live].clamp(min=1e-30)).max().item())
        if canary is not None:
            assert (y[~self.live] == canary).all()
        if lse is not None:
            none = torch.isinf(want_lse[live])
            assert torch.equal(torch.isinf(lse[live]) & (lse[live] < 0), none)
            far = (lse[live].double() - want_lse[live]).abs()[~none] - lse_tol[live][~none]
            assert far.numel() == 0 or far.max().item() <= 0, far.max().item()

    # ---------------------------------------------------------------- append

    def append(self, inv_freq, **kw):
        return bl.bitlinear_rope_append(kw.pop("q", self.q), kw.pop("k", self.k),
                                        kw.pop("v", self.v), self.k_cache, self.v_cache,
                                        self.q_start, self.kv_len, self.table, inv_freq, **kw)

    def rotated(self, x, inv_freq, gain=None, eps=bl.RMSNORM_EPS, interleaved=False):
        """(rotated rows in 64 bits, tolerance): half a step of the value's
        bf16 rounding, and 2^-19 of the pair's size for the fp32 parts (the
        norm's sum of d squares, root and division, the gain, cosine and sine
        each a few 2^-23, and the pair's three roundings)."""
        x = x.double()
        if gain is not None:
            x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double()
        out, size = torch.full_like(x, math.nan), torch.zeros_like(x)
        i = torch.arange(self.d // 2, device=self.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + self.d // 2)
        for s, at, n, kv in self.spans():
            pos = torch.arange(kv - n, kv, device=self.device).double()
            ang = torch.outer(pos, inv_freq.double())[:, None]
            xa, xb = x[at:at + n][..., a], x[at:at + n][..., b]
            out[at:at + n, :, a] = xa * ang.cos() - xb * ang.sin()
            out[at:at + n, :, b] = xb * ang.cos() + xa * ang.sin()
            size[at:at + n, :, a] = xa.abs() + xb.abs()
            size[at:at + n, :, b] = xa.abs() + xb.abs()
        return out, HALF_BF16 * out.abs() + 2.0 ** -19 * size


def frequencies(d, theta=10000.0, device="cuda"):
    i = torch.arange(d // 2, dtype=torch.float64)
    return (theta ** (-2.0 * i / d)).to(torch.float32).to(device)
