"""The attention half of a decoder layer on a paged key/value cache: the cases
on which the two operators are measured, and their plain forms.

  append     bitlinear_rope_append: the queries and keys of the step's new
             tokens, optionally RMS-normalised per head, are rotated by their
             positions; the queries go to q_out, the keys and the values into
             the pages of their sequences.
  attention  bitlinear_paged_attention: the new tokens of every sequence attend
             to the sequence's keys in the cache up to their own position.

A step's sequences: sequence s owns the query rows q_start[s] .. q_start[s + 1]
and, with these, kv_len[s] tokens in the cache, so its row i stands at position
kv_len[s] - q_len[s] + i. Position j of sequence s is slot j % page of page
page_table[s][j // page]; a cache is [pages][kv_heads][page][head_dim].

Head layouts: 20 query heads on 5 key heads of 128 are the ~2B decoder's
(2560 and 640 wide), 64 on 8 of 128 the large sweep's 8192-wide layer; 40 on
10 of 64 are the 2B widths with the other common head size.
"""
import math
import random

import torch

own = False

LAYOUTS = ((20, 5, 128), (64, 8, 128), (40, 10, 64), (16, 16, 64), (24, 2, 128))
PAGES = (16, 32, 64, 128)
MOST_FLOPS = 4.2e12         # of one pass: no drawn case is above the largest listed
MOST_BYTES = 2.2e9
MOST_SCORES = 1.3e9         # padded scores of one key head in the plain form
ROPE_THETA = 500000.0
NORM_EPS = 1e-6


def _case(name, op, layout, page, chunks=0, q_min=1, q_max=1, tokens=0, ctx_min=0, ctx_max=0,
          lens=1, spare=0, **more):
    """`chunks` sequences of q_min .. q_max new tokens and `tokens` sequences
    of one, each behind ctx_min .. ctx_max tokens that the cache holds already
    (drawn from `lens`); `spare` rows follow the last sequence."""
    hq, hkv, d = layout
    c = dict(name=name, op=op, q_heads=hq, kv_heads=hkv, head_dim=d, page=page, chunks=chunks,
             q_min=q_min, q_max=q_max, tokens=tokens, ctx_min=ctx_min, ctx_max=ctx_max,
             lens=lens, spare=spare)
    c.update(more)
    return c


def _attention(name, layout, page, window=0, **kw):
    return _case(name, "attention", layout, page, window=window, **kw)


def _append(name, layout, page, norm=False, interleaved=False, **kw):
    return _case(name, "append", layout, page, norm=norm, interleaved=interleaved, **kw)


def listed():
    b2, large, narrow = LAYOUTS[:3]
    return [
        # one user's next token in the ~2B decoder: the time to the answer counts
        _attention("attend_token", b2, 64, tokens=1, ctx_min=700, ctx_max=700),
        # a full decode batch of the 2B decoder over its 4096-token context,
        # padded to a captured batch size
        _attention("attend_batch", b2, 64, tokens=61, ctx_min=1, ctx_max=4095, spare=3),
        # a few documents of 128k tokens being answered, wide layer
        _attention("attend_tokens_long", large, 128, tokens=4, ctx_min=120000, ctx_max=131071),
        # a loaded server's decode batch, wide layer
        _attention("attend_batch_large", large, 64, tokens=96, ctx_min=500, ctx_max=9500),
        # drafted tokens being verified, five a sequence, small heads and pages
        _attention("attend_draft", narrow, 16, chunks=24, q_min=5, q_max=5, ctx_min=30,
                   ctx_max=4000),
        # the 2048-token prompt of the 2B decoder, from an empty cache
        _attention("attend_prompt", b2, 64, chunks=1, q_min=2048, q_max=2048),
        # a scheduler's mixed step: one chunk of a prompt beside decoding users
        _attention("attend_mixed", b2, 32, chunks=1, q_min=1021, q_max=1021, tokens=47,
                   ctx_min=200, ctx_max=3000),
        # a chunk in the middle of a long document, wide layer: the largest
        _attention("attend_chunk_long", large, 128, chunks=1, q_min=4096, q_max=4096,
                   ctx_min=28672, ctx_max=28672),
        # ragged prompts under a sliding window, small heads
        _attention("attend_window", narrow, 16, chunks=4, q_min=1500, q_max=4000, window=1024),
        # one token of the 2B decoder
        _append("append_token", b2, 64, tokens=1, ctx_min=700, ctx_max=700),
        # a decode batch with normalised queries and keys
        _append("append_batch", b2, 64, norm=True, tokens=61, ctx_min=1, ctx_max=4095, spare=3),
        # prompts of the wide layer, far positions among them, pairs interleaved
        _append("append_prompts", large, 128, norm=True, interleaved=True, chunks=5, q_min=1000,
                q_max=5000, ctx_min=0, ctx_max=120000),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        layout, page = rng.choice(LAYOUTS), rng.choice(PAGES)
        kw = dict(lens=rng.randrange(1 << 30), spare=rng.choice((0, 0, 1, 7)))
        kind = rng.choice(("tokens", "draft", "chunks", "mixed"))
        ctx = _log_int(rng, 1, 131000)
        kw["ctx_min"], kw["ctx_max"] = rng.choice((0, ctx // 3, ctx)), ctx
        if kind in ("tokens", "mixed"):
            kw["tokens"] = _log_int(rng, 1, 256)
        if kind == "draft":
            kw.update(chunks=_log_int(rng, 1, 64), q_min=1, q_max=rng.randint(2, 12))
        elif kind != "tokens":
            q = _log_int(rng, 13, 8192)
            kw.update(chunks=_log_int(rng, 1, 8), q_min=rng.choice((q // 4 + 1, q)), q_max=q)
        if rng.random() < 0.35:
            c = _append(None, layout, page, norm=rng.random() < 0.5,
                        interleaved=rng.random() < 0.5, **kw)
        else:
            window = _log_int(rng, 16, 8192) if rng.random() < 0.25 else 0
            c = _attention(None, layout, page, window=window, **kw)
        del c["name"]
        w, (ql, kl) = work(c), _lengths(c)
        cached = sum(-(-k // page) for k in kl) * page * c["kv_heads"] * c["head_dim"] * 4
        padded = len(ql) * max(ql) * max(kl) * (c["q_heads"] // c["kv_heads"])
        if (w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES and padded <= MOST_SCORES
                and len(ql) * max(kl) <= 4e6 and cached <= 5e9):
            return c


def _lengths(case):
    """The sequences' new tokens and their tokens in the cache with these; the
    chunks stand between the single tokens as a scheduler would mix them."""
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["chunks"])]
    q += [1] * case["tokens"]
    rng.shuffle(q)
    return q, [n + rng.randint(case["ctx_min"], case["ctx_max"]) for n in q]


def _seen(q, kv, window):
    """(query, key) pairs of one sequence, and its keys that any query sees."""
    first = kv - q
    if not window or window >= kv:
        return q * first + q * (q + 1) // 2, kv
    short = max(0, min(q, window - first))            # rows that see fewer than `window` keys
    pairs = short * first + short * (short + 1) // 2 + (q - short) * window
    return pairs, min(kv, q + window - 1)


def work(case):
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    ql, kl = _lengths(case)
    n = sum(ql)
    table = sum(4 * -(-k // case["page"]) for k in kl) + 8 * len(ql) + 4
    if case["op"] == "append":
        per = 7 if case["norm"] else 3
        return {"bytes": 4 * n * (hq + 2 * hkv) * d + 2 * d
                + (8 * d if case["norm"] else 0) + 8 * len(ql) + 4 * n,
                "flops": per * n * (hq + hkv) * d}
    pairs, keys = (sum(v) for v in zip(*(_seen(q, k, case["window"]) for q, k in zip(ql, kl))))
    return {"bytes": 4 * keys * hkv * d + 4 * n * hq * d + table, "flops": 4 * pairs * hq * d}


def prepare(case, seed):
    hq, hkv, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    ql, kl = _lengths(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    rows = sum(ql) + case["spare"]

    def normal(*shape, scale=1.0):
        t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        return t.normal_(0.0, scale, generator=gen)

    need = [-(-k // page) for k in kl]
    pages = sum(need) + 3
    table = torch.full((len(ql), max(need) + 1), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=host).to(torch.int32)
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    start = [0]
    for n in ql:
        start.append(start[-1] + n)
    st = {
        "op": case["op"], "max_q_len": max(ql), "max_kv_len": max(kl),
        "q_start": torch.tensor(start, dtype=torch.int32, device="cuda"),
        "kv_len": torch.tensor(kl, dtype=torch.int32, device="cuda"),
        "page_table": table.cuda(),
        "k_cache": normal(pages, hkv, page, d), "v_cache": normal(pages, hkv, page, d),
        # attention logits of trained layers have a spread of a few units
        "q": normal(rows, hq, d, scale=2.5),
        "q_out": torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda"),
    }
    if case["op"] == "append":
        st["k"], st["v"] = normal(rows, hkv, d), normal(rows, hkv, d)
        i = torch.arange(d // 2, dtype=torch.float64)
        st["inv_freq"] = (ROPE_THETA ** (-2.0 * i / d)).to(torch.float32).cuda()
        st["interleaved"] = case["interleaved"]
        gain = lambda: torch.empty(d, device="cuda").uniform_(0.5, 1.5, generator=gen)  # noqa: E731
        st["q_gain"], st["k_gain"] = (gain(), gain()) if case["norm"] else (None, None)
    else:
        st["window"] = case["window"]
        if own:
            import ternary_weight_w1_b200 as bl
            st["workspace"] = torch.empty(
                bl.bitlinear_workspace_bytes_attention(rows, len(ql), hq, hkv, d),
                dtype=torch.uint8, device="cuda")
    return st


def run(state):
    if state["op"] == "append":
        return _append_own(state) if own else _append_plain(state)
    return _attention_own(state) if own else _attention_plain(state)


def _append_own(st):
    import ternary_weight_w1_b200 as bl
    bl.bitlinear_rope_append(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                             st["q_start"], st["kv_len"], st["page_table"], st["inv_freq"],
                             q_out=st["q_out"], q_gain=st["q_gain"], k_gain=st["k_gain"],
                             eps=NORM_EPS, interleaved=st["interleaved"])
    return st["q_out"], st["k_cache"], st["v_cache"]


def _attention_own(st):
    import ternary_weight_w1_b200 as bl
    return bl.bitlinear_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["q_start"],
                                        st["kv_len"], st["page_table"], window=st["window"],
                                        max_q_len=st["max_q_len"], y=st["q_out"],
                                        workspace=st["workspace"])


def _rotate(x, gain, cos, sin, interleaved):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS) * gain
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return y.to(torch.bfloat16)


def _append_plain(st):
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    page = st["k_cache"].shape[2]
    n = st["q"].shape[0]
    t = torch.arange(n, device="cuda")
    s = torch.searchsorted(q_start[1:], t, right=True)
    live = s < kv_len.numel()                      # rows of a sequence
    s = s.clamp(max=kv_len.numel() - 1)
    pos = kv_len[s] - q_start[s + 1] + t
    angle = pos.double()[:, None] * st["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _rotate(st["q"], st["q_gain"], cos, sin, st["interleaved"])
    k = _rotate(st["k"], st["k_gain"], cos, sin, st["interleaved"])
    st["q_out"].copy_(torch.where(live[:, None, None], q, st["q_out"]))
    s, pos, k, v = s[live], pos[live], k[live], st["v"][live]
    at = st["page_table"][s, pos // page].long()
    st["k_cache"][at, :, pos % page] = k
    st["v_cache"][at, :, pos % page] = v
    return st["q_out"], st["k_cache"], st["v_cache"]


def _attention_plain(st):
    q_start, kv_len, q = st["q_start"].long(), st["kv_len"].long(), st["q"]
    _, kv_heads, page, d = st["k_cache"].shape
    group = q.shape[1] // kv_heads
    q_len = q_start[1:] - q_start[:-1]
    i = torch.arange(st["max_q_len"], device="cuda")
    j = torch.arange(st["max_kv_len"], device="cuda")
    row = (q_start[:-1, None] + i).clamp(max=q.shape[0] - 1)               # [S][q]
    live = i < q_len[:, None]
    pos = (kv_len - q_len)[:, None] + i
    hidden = j > pos[..., None]                                            # [S][q][kv]
    if st["window"]:
        hidden |= j <= pos[..., None] - st["window"]
    at = st["page_table"].long().clamp(min=0)[:, j // page], j % page      # [S][kv]
    cached = (j < kv_len[:, None])[..., None]
    heads = []
    for h in range(kv_heads):      # one key head's scores at a time fit in memory
        k = st["k_cache"][at[0], h, at[1]].float().where(cached, 0.0)      # [S][kv][d]
        v = st["v_cache"][at[0], h, at[1]].float().where(cached, 0.0)
        x = q[:, h * group:(h + 1) * group].float()[row].transpose(1, 2)   # [S][g][q][d]
        p = x @ (k.transpose(1, 2) / math.sqrt(d))[:, None]
        p.masked_fill_(hidden[:, None], -math.inf)
        top = p.amax(-1, keepdim=True).clamp(min=-3e38)
        p.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        heads.append(((p @ v[:, None]) / total.clamp(min=1e-30)).transpose(1, 2)[live])
    st["q_out"][row[live]] = torch.cat(heads, 1).to(q.dtype)
    return st["q_out"]


def exact(case, seed):
    return (_append_exact if case["op"] == "append" else _attention_exact)(case, seed)


def _append_exact(case, seed):
    st = prepare(case, seed)
    ql, kl = _lengths(case)
    page, d = case["page"], case["head_dim"]
    q_out = torch.zeros_like(st["q"], dtype=torch.float64)
    caches = st["k_cache"].double(), st["v_cache"].double()
    even = torch.arange(0, d, 2, device="cuda") if case["interleaved"] else torch.arange(d // 2, device="cuda")
    odd = even + (1 if case["interleaved"] else d // 2)
    begin = 0
    for s, (n, kv) in enumerate(zip(ql, kl)):
        rows = slice(begin, begin + n)
        begin += n
        pos = torch.arange(kv - n, kv, device="cuda")
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer(pos.double(), st["inv_freq"].double()))[:, None]

        def rotated(x, gain):
            x = x[rows].double()
            if gain is not None:
                x = x / (x.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * gain.double()
            z = torch.complex(x[..., even], x[..., odd]) * turn
            y = torch.empty_like(x)
            y[..., even], y[..., odd] = z.real, z.imag
            return y

        q_out[rows] = rotated(st["q"], st["q_gain"])
        slots = st["page_table"][s].long()[pos // page], pos % page
        for cache, new in zip(caches, (rotated(st["k"], st["k_gain"]), st["v"][rows].double())):
            cache[slots[0], :, slots[1]] = new
    return q_out, *caches


def _attention_exact(case, seed):
    st = prepare(case, seed)
    ql, kl = _lengths(case)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    y = torch.zeros_like(st["q"], dtype=torch.float64)
    begin = 0
    for s, (n, kv) in enumerate(zip(ql, kl)):
        pages = st["page_table"][s, :-(-kv // case["page"])].long()
        q = st["q"][begin:begin + n].double().unflatten(1, (hkv, hq // hkv))
        for h in range(hkv):
            k, v = (c[pages, h].flatten(0, 1)[:kv].double() for c in (st["k_cache"], st["v_cache"]))
            for a in range(0, n, 512):
                b = min(n, a + 512)
                last = kv - n + b                                  # keys this block can see
                p = torch.arange(kv - n + a, last, device="cuda")[:, None] - torch.arange(last, device="cuda")
                seen = (p >= 0) & (p < (case["window"] or kv + 1))
                w = torch.einsum("qgd,kd->gqk", q[a:b, h], k[:last]) / d ** 0.5
                w = w.masked_fill(~seen, -math.inf).softmax(-1)
                y[begin + a:begin + b].unflatten(1, (hkv, hq // hkv))[:, h] = torch.einsum(
                    "gqk,kd->qgd", w, v[:last])
        begin += n
    return y
