"""The paged-cache operators refuse bad arguments on the host: every check here
returns before the library touches CUDA."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import ternary_weight_w1_b200 as bl

FAKE = 1 << 20          # a 256-byte-aligned non-null address; never dereferenced
BIG = 1 << 40


class KVCache(ctypes.Structure):
    _fields_ = [("k_dev", ctypes.c_void_p), ("v_dev", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("page", ctypes.c_int64), ("head_dim", ctypes.c_int64)]


class Seqs(ctypes.Structure):
    _fields_ = [("q_start_dev", ctypes.c_void_p), ("kv_len_dev", ctypes.c_void_p),
                ("page_table_dev", ctypes.c_void_p), ("seqs", ctypes.c_int64),
                ("table_cols", ctypes.c_int64)]


def descriptors(kw):
    c = dict(k=FAKE, v=FAKE, pages=10, kv_heads=2, page=16, head_dim=64)
    s = dict(q_start=FAKE, kv_len=FAKE, table=FAKE, seqs=1, cols=4)
    for d in (c, s):
        d.update({n: kw.pop(n) for n in list(kw) if n in d})
    return (KVCache(c["k"], c["v"], c["pages"], c["kv_heads"], c["page"], c["head_dim"]),
            Seqs(s["q_start"], s["kv_len"], s["table"], s["seqs"], s["cols"]))


def append(**kw):
    cache, seqs = descriptors(kw)
    a = dict(q=FAKE, qs=256, kk=FAKE, ks=128, vv=FAKE, vs=128, T=3, heads=4,
             cache=ctypes.addressof(cache), sq=ctypes.addressof(seqs), f=FAKE, inter=0, qg=None,
             kg=None, eps=1e-6, out=FAKE, os=256, stream=None)
    a.update(kw)
    return bl.lib().bitlinear_rope_append(*a.values())


def attend(**kw):
    cache, seqs = descriptors(kw)
    a = dict(q=FAKE, qs=256, T=3, heads=4, cache=ctypes.addressof(cache),
             sq=ctypes.addressof(seqs), scale=0.125, window=0, max_q=0, y=FAKE, ys=256, lse=None,
             ws=FAKE, wsb=BIG, stream=None)
    a.update(kw)
    return bl.lib().bitlinear_paged_attention(*a.values())


SHARED = [
    (dict(cache=None), bl.BITLINEAR_ERR_ARG),
    (dict(sq=None), bl.BITLINEAR_ERR_ARG),
    (dict(k=None), bl.BITLINEAR_ERR_ARG),
    (dict(v=None), bl.BITLINEAR_ERR_ARG),
    (dict(q_start=None), bl.BITLINEAR_ERR_ARG),
    (dict(kv_len=None), bl.BITLINEAR_ERR_ARG),
    (dict(table=None), bl.BITLINEAR_ERR_ARG),
    (dict(q=None), bl.BITLINEAR_ERR_ARG),
    (dict(T=-1), bl.BITLINEAR_ERR_ARG),
    (dict(heads=0), bl.BITLINEAR_ERR_ARG),
    (dict(kv_heads=0), bl.BITLINEAR_ERR_ARG),
    (dict(pages=0), bl.BITLINEAR_ERR_ARG),
    (dict(cols=0), bl.BITLINEAR_ERR_ARG),
    (dict(seqs=-1), bl.BITLINEAR_ERR_ARG),
    (dict(heads=3), bl.BITLINEAR_ERR_SHAPE),              # not a multiple of the key heads
    (dict(heads=65538, qs=65538 * 64), bl.BITLINEAR_ERR_SHAPE),
    (dict(head_dim=96), bl.BITLINEAR_ERR_SHAPE),
    (dict(head_dim=256), bl.BITLINEAR_ERR_SHAPE),
    (dict(head_dim=0), bl.BITLINEAR_ERR_SHAPE),
    (dict(page=8), bl.BITLINEAR_ERR_SHAPE),
    (dict(page=24), bl.BITLINEAR_ERR_SHAPE),
    (dict(page=512), bl.BITLINEAR_ERR_SHAPE),
    (dict(page=-16), bl.BITLINEAR_ERR_SHAPE),
    (dict(page=0), bl.BITLINEAR_ERR_SHAPE),
    (dict(seqs=16385), bl.BITLINEAR_ERR_SHAPE),
    (dict(T=1 << 29), bl.BITLINEAR_ERR_SHAPE),
    (dict(T=1 << 62), bl.BITLINEAR_ERR_SHAPE),
    (dict(cols=1 << 27), bl.BITLINEAR_ERR_SHAPE),
    (dict(pages=1 << 27), bl.BITLINEAR_ERR_SHAPE),
    (dict(pages=1 << 62), bl.BITLINEAR_ERR_SHAPE),
    (dict(kv_heads=1 << 40, heads=1 << 40), bl.BITLINEAR_ERR_SHAPE),
    (dict(qs=255), bl.BITLINEAR_ERR_SHAPE),               # rows would overlap
    (dict(qs=260), bl.BITLINEAR_ERR_ALIGN),
    (dict(q=FAKE + 8), bl.BITLINEAR_ERR_ALIGN),
    (dict(k=FAKE + 8), bl.BITLINEAR_ERR_ALIGN),
    (dict(v=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    (dict(q_start=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    (dict(kv_len=FAKE + 1), bl.BITLINEAR_ERR_ALIGN),
    (dict(table=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    # no token or no sequence: nothing to do, no pointer is needed
    (dict(T=0), bl.BITLINEAR_OK),
    (dict(seqs=0), bl.BITLINEAR_OK),
    (dict(T=0, q=None, k=None, v=None, q_start=None, kv_len=None, table=None), bl.BITLINEAR_OK),
]


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("kw,status", SHARED)
def test_shared_refusals(call, kw, status):
    assert call(**dict(kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kk=None), bl.BITLINEAR_ERR_ARG),
    (dict(vv=None), bl.BITLINEAR_ERR_ARG),
    (dict(f=None), bl.BITLINEAR_ERR_ARG),
    (dict(out=None), bl.BITLINEAR_ERR_ARG),
    (dict(inter=2), bl.BITLINEAR_ERR_ARG),
    (dict(qg=FAKE, eps=0.0), bl.BITLINEAR_ERR_ARG),
    (dict(kg=FAKE, eps=float("nan")), bl.BITLINEAR_ERR_ARG),
    (dict(kg=FAKE, eps=float("inf")), bl.BITLINEAR_ERR_ARG),
    (dict(ks=64), bl.BITLINEAR_ERR_SHAPE),
    (dict(vs=-128), bl.BITLINEAR_ERR_SHAPE),
    (dict(vs=132), bl.BITLINEAR_ERR_ALIGN),
    (dict(kk=FAKE + 4), bl.BITLINEAR_ERR_ALIGN),
    (dict(out=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    (dict(f=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    (dict(qg=FAKE + 1), bl.BITLINEAR_ERR_ALIGN),
    (dict(kg=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
])
def test_append_refusals(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), bl.BITLINEAR_ERR_ARG),
    (dict(scale=0.0), bl.BITLINEAR_ERR_ARG),
    (dict(scale=-1.0), bl.BITLINEAR_ERR_ARG),
    (dict(scale=float("nan")), bl.BITLINEAR_ERR_ARG),
    (dict(scale=float("inf")), bl.BITLINEAR_ERR_ARG),
    (dict(scale=3e38), bl.BITLINEAR_ERR_ARG),             # its product with log2 e overflows
    (dict(window=-1), bl.BITLINEAR_ERR_ARG),
    (dict(max_q=-1), bl.BITLINEAR_ERR_ARG),
    (dict(ys=128), bl.BITLINEAR_ERR_SHAPE),
    (dict(ys=257), bl.BITLINEAR_ERR_ALIGN),
    (dict(y=FAKE + 8), bl.BITLINEAR_ERR_ALIGN),
    (dict(lse=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    (dict(ws=None), bl.BITLINEAR_ERR_WORKSPACE),
    (dict(wsb=64), bl.BITLINEAR_ERR_WORKSPACE),
    (dict(ws=FAKE + 128), bl.BITLINEAR_ERR_ALIGN),
])
def test_attention_refusals(kw, status):
    assert attend(**kw) == status


def test_attention_workspace_bytes():
    size_max = ctypes.c_size_t(-1).value
    ws = bl.bitlinear_workspace_bytes_attention
    assert 0 < ws(1, 1, 20, 5, 128) < 16 << 20
    assert ws(1, 1, 20, 5, 128) <= ws(100, 1, 20, 5, 128) <= ws(5000, 1, 20, 5, 128) < 256 << 20
    assert ws(0, 1, 20, 5, 128) == 0 and ws(1, 0, 20, 5, 128) == 0
    for bad in ((-1, 1, 20, 5, 128), (1, 1, 20, 3, 128), (1, 1, 20, 5, 80), (1, 16385, 20, 5, 128),
                (1 << 40, 1, 20, 5, 128)):
        assert ws(*bad) == size_max


def host_step():
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k_cache=c, v_cache=c.clone(),
                q_start=i(2), kv_len=i(1), page_table=i(1, 4))


def test_binding_refuses_host_tensors_and_wrong_shapes():
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for call in (lambda a: bl.bitlinear_paged_attention(**a),
                 lambda a: bl.bitlinear_rope_append(k=kv, v=kv, inv_freq=torch.zeros(32), **a)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(host_step())
        with pytest.raises(ValueError, match="pages"):
            call(dict(host_step(), k_cache=torch.zeros(4, 64)))
        with pytest.raises(ValueError, match="page_table"):
            call(dict(host_step(), page_table=torch.zeros(4, dtype=torch.int32)))
        with pytest.raises(bl.BitLinearError) as e:
            call(dict(host_step(), k_cache=torch.zeros(4, 2, 16, 80, dtype=torch.bfloat16)))
        assert e.value.status == bl.BITLINEAR_ERR_SHAPE


class Projection(ctypes.Structure):
    _fields_ = [("packed_dev", ctypes.c_void_p), ("gamma", ctypes.c_float),
                ("gain_dev", ctypes.c_void_p)]


def block(**kw):
    cache, seqs = descriptors(kw)
    gains = kw.pop("gains", (None,) * 4)
    proj = [Projection(kw.pop("packed", FAKE) if i == 3 else FAKE, 1.0, g)
            for i, g in enumerate(gains)]
    a = dict(x=FAKE, xdt=0, M=3, K=256, q=ctypes.addressof(proj[0]), kk=ctypes.addressof(proj[1]),
             vv=ctypes.addressof(proj[2]), o=ctypes.addressof(proj[3]), heads=4,
             cache=ctypes.addressof(cache), sq=ctypes.addressof(seqs), f=FAKE, inter=0, qg=None,
             kg=None, eps=1e-6, scale=0.125, window=0, max_q=0, y=FAKE, ws=FAKE, wsb=BIG,
             stream=None)
    a.update(kw)
    return bl.lib().bitlinear_attn_forward(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), bl.BITLINEAR_ERR_ARG),
    (dict(o=None), bl.BITLINEAR_ERR_ARG),
    (dict(packed=None), bl.BITLINEAR_ERR_ARG),
    (dict(x=None), bl.BITLINEAR_ERR_ARG),
    (dict(y=None), bl.BITLINEAR_ERR_ARG),
    (dict(f=None), bl.BITLINEAR_ERR_ARG),
    (dict(k=None), bl.BITLINEAR_ERR_ARG),
    (dict(M=-1), bl.BITLINEAR_ERR_ARG),
    (dict(K=0), bl.BITLINEAR_ERR_ARG),
    (dict(xdt=5), bl.BITLINEAR_ERR_DTYPE),
    (dict(K=200), bl.BITLINEAR_ERR_SHAPE),
    (dict(K=65536 + 128), bl.BITLINEAR_ERR_SHAPE),
    (dict(heads=3, kv_heads=3), bl.BITLINEAR_ERR_SHAPE),      # 192 wide: no multiple of 128
    (dict(heads=2048), bl.BITLINEAR_ERR_SHAPE),               # 131072 wide
    (dict(gains=(FAKE, None, FAKE, None)), bl.BITLINEAR_ERR_ARG),
    (dict(gains=(None, None, None, FAKE), eps=0.0), bl.BITLINEAR_ERR_ARG),
    (dict(kg=FAKE, eps=-1.0), bl.BITLINEAR_ERR_ARG),
    (dict(gains=(FAKE, FAKE, FAKE + 4, None)), bl.BITLINEAR_ERR_ALIGN),
    (dict(scale=0.0), bl.BITLINEAR_ERR_ARG),
    (dict(window=-1), bl.BITLINEAR_ERR_ARG),
    (dict(max_q=-1), bl.BITLINEAR_ERR_ARG),
    (dict(inter=3), bl.BITLINEAR_ERR_ARG),
    (dict(x=FAKE + 2), bl.BITLINEAR_ERR_ALIGN),
    (dict(y=FAKE + 8), bl.BITLINEAR_ERR_ALIGN),
    (dict(ws=None), bl.BITLINEAR_ERR_WORKSPACE),
    (dict(wsb=1000), bl.BITLINEAR_ERR_WORKSPACE),
    (dict(ws=FAKE + 16), bl.BITLINEAR_ERR_ALIGN),
    (dict(M=0), bl.BITLINEAR_OK),
    (dict(seqs=0), bl.BITLINEAR_OK),
])
def test_block_refusals(kw, status):
    assert block(**dict(kw)) == status


def test_block_workspace_bytes():
    size_max = ctypes.c_size_t(-1).value
    ws = bl.bitlinear_workspace_bytes_attn
    assert ws(0, 2560, 1, 20, 5, 128) == 0
    assert ws(1, 2560, 1, 20, 5, 128) >= bl.bitlinear_workspace_bytes_attention(1, 1, 20, 5, 128)
    assert ws(100, 2560, 1, 20, 5, 128) > 100 * (2 * 2560 + 2 * 640) * 2
    for bad in ((1, 2500, 1, 20, 5, 128), (1, 2560, 1, 3, 3, 64), (1, 2560, 1, 20, 5, 32),
                (-1, 2560, 1, 20, 5, 128)):
        assert ws(*bad) == size_max


@pytest.mark.parametrize("worker,timeout_us", [(-1, 1000), (0, 0), (0, -1), (0, 10 ** 7 + 1)])
def test_inject_timeout_refuses_bad_workers_and_limits(worker, timeout_us):
    cache, seqs = descriptors({})
    rc = bl.lib().bitlinear_paged_attention_inject_timeout(
        FAKE, 256, 3, 4, ctypes.addressof(cache), ctypes.addressof(seqs), 0.125, 0, 0, 2 * FAKE,
        256, None, FAKE, BIG, None, worker, timeout_us)
    assert rc == bl.BITLINEAR_ERR_ARG


def without(modules, code):
    """Runs `code` in a Python where importing any of `modules` fails."""
    block = f"import sys; sys.modules.update(dict.fromkeys({modules!r}))\n"
    return subprocess.run([sys.executable, "-c", block + code], capture_output=True, text=True,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_calls_work_without_the_compiled_marshalling():
    # missing, or built for another Python or torch: the ctypes path takes every call
    r = without(["ternary_weight_w1_b200._fastcall"], """
import warnings
import torch
import ternary_weight_w1_b200 as bl
c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
i = lambda *s: torch.zeros(s, dtype=torch.int32)
x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for call in (lambda: bl.bitlinear_paged_attention(x, c, c, i(2), i(1), i(1, 4)),
                 lambda: bl.bitlinear_rope_append(x, x, x, c, c, i(2), i(1), i(1, 4), i(32))):
        try:
            call()
        except ValueError as e:
            print(e)
print(len(seen), seen[0].category.__name__)
""")
    assert r.returncode == 0, r.stderr
    *refusals, last = r.stdout.splitlines()
    assert len(refusals) == 2 and all("CUDA tensor" in line for line in refusals)
    assert last == "1 RuntimeWarning"              # said once


def test_the_library_builds_without_torch():
    r = without(["torch"], """
from ternary_weight_w1_b200 import build
print(build.build(), build.build_fastcall(force=True))
""")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [bl.LIB_PATH, "None"]


@pytest.mark.parametrize("call,kw", [
    (attend, dict()),                                     # y is q
    (attend, dict(T=1)),
    (attend, dict(y=FAKE + 16)),
    (attend, dict(y=FAKE + 2 * 512)),                     # q's last row
    (attend, dict(qs=512, ys=512, y=FAKE + 2 * 240)),     # a part of a wide buffer, 16 too near
    (attend, dict(qs=512, ys=256, y=FAKE + 2 * 768)),
    (append, dict(kk=2 * FAKE, vv=3 * FAKE, os=512)),     # in place, with another stride
    (append, dict(kk=2 * FAKE, vv=3 * FAKE, out=FAKE + 512)),
    (append, dict(kk=2 * FAKE, vv=3 * FAKE, out=2 * FAKE + 16)),
    (append, dict(kk=2 * FAKE, vv=3 * FAKE, out=3 * FAKE - 512)),
])
def test_outputs_that_share_memory_with_inputs(call, kw):
    assert call(**kw) == bl.BITLINEAR_ERR_ARG
