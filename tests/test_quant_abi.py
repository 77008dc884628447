"""Refusals of the quantised cache's and the modified scores' entry points,
without a GPU: every bad argument is rejected on the host, before a launch."""
from __future__ import annotations

import ctypes

import pytest
import torch

INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_cache_22_gb300 import build
    build.build()
    import paged_kv_cache_22_gb300 as m
    m.library()
    return m


def test_tile_bytes(pkv):
    assert pkv.quant_tile_bytes(128, 16, "int8") == 16 * (128 + 4)
    assert pkv.quant_tile_bytes(64, 8, "fp4") == 8 * (32 + 4 + 4)
    assert pkv.quant_cache_shape(5, 3, 32, 128, "fp4") == (5, 3, 32 * (64 + 8 + 4))
    for d, bs in ((96, 16), (128, 12), (0, 16), (128, 64)):
        assert pkv.library().pkv_quant_tile_bytes(d, bs, 0) == 0
        with pytest.raises(ValueError):
            pkv.quant_tile_bytes(d, bs, "int8")
    assert pkv.library().pkv_quant_tile_bytes(128, 16, 2) == 0
    with pytest.raises(ValueError, match="unknown quantised format"):
        pkv.quant_tile_bytes(128, 16, "int4")


def qdesc(pkv, nb=8, bs=16, hkv=2, d=128, fmt=0):
    return pkv.QuantDesc(nb, bs, hkv, d, fmt)


def test_write_refusals(pkv):
    f = pkv.library().pkv_kv_quantize_and_cache

    def call(k=P, v=P, dt=1, n=4, kc=P, vc=P, desc=None, slots=P):
        d = ctypes.byref(desc) if desc is not None else None
        return f(k, v, dt, n, kc, vc, d, slots, None)

    ok = qdesc(pkv)
    assert call() == INVALID                                  # no descriptor
    assert call(n=-1, desc=ok) == INVALID
    assert call(dt=2, desc=ok) == UNSUPPORTED                 # fp8 source
    for bad in (qdesc(pkv, d=96), qdesc(pkv, bs=4), qdesc(pkv, nb=0), qdesc(pkv, hkv=0), qdesc(pkv, fmt=3)):
        assert call(desc=bad) == INVALID
    for name in ("k", "v", "kc", "vc"):
        assert call(desc=ok, **{name: None}) == INVALID
        assert call(desc=ok, **{name: ODD}) == INVALID        # 8-byte aligned only
    assert call(desc=ok, slots=None) == INVALID
    assert call(desc=ok, slots=ctypes.c_void_p(0x1004)) == INVALID
    assert call(k=None, v=None, n=0, kc=None, vc=None, desc=ok, slots=None) == 0  # nothing to do


def test_gather_refusals(pkv):
    f = pkv.library().pkv_gather_kv_quant

    def call(ko=P, vo=P, dt=1, kc=P, vc=P, desc=None, tb=P, mb=4, ln=P, cu=P, n=2, total=9, mx=9):
        d = ctypes.byref(desc) if desc is not None else None
        return f(ko, vo, dt, kc, vc, d, tb, mb, ln, cu, n, total, mx, None)

    ok = qdesc(pkv, fmt=1)
    assert call() == INVALID
    assert call(desc=ok, dt=2) == UNSUPPORTED
    for kw in (dict(mb=0), dict(n=-1), dict(total=-1), dict(mx=-1), dict(ko=None), dict(vo=ODD), dict(kc=ODD),
               dict(vc=None), dict(tb=None), dict(ln=None), dict(cu=None), dict(cu=ctypes.c_void_p(0x1004)),
               dict(tb=ctypes.c_void_p(0x1002)), dict(ln=ctypes.c_void_p(0x1002))):
        assert call(desc=ok, **kw) == INVALID, kw
    assert call(desc=ok, n=65536) == UNSUPPORTED
    for kw in (dict(n=0), dict(total=0), dict(mx=0)):
        assert call(desc=ok, **kw) == 0


def attend(pkv, which, desc, out=P, q=P, dt=1, qs=None, n=2, total=2, mq=1, hq=8, kc=P, vc=P, tb=P, mb=4, ln=P, mx=64,
           scale=0.1, kv=1.0, opts=None, ws=P, wb=1 << 30):
    f = getattr(pkv.library(), "pkv_paged_attention_" + which)
    d = ctypes.byref(desc) if desc is not None else None
    o = ctypes.byref(opts) if opts is not None else None
    more = (kv,) if which == "scored" else ()
    return f(out, q, dt, qs, n, total, mq, hq, kc, vc, d, tb, mb, ln, mx, scale, *more, o, ws, wb, None)


@pytest.mark.parametrize("which", ["scored", "quant"])
def test_attention_refusals(pkv, which):
    def desc(**kw):
        return qdesc(pkv, **kw) if which == "quant" else pkv.CacheDesc(kw.get("nb", 8), kw.get("bs", 16),
                                                                        kw.get("hkv", 2), kw.get("d", 128), 1)

    nan, inf = float("nan"), float("inf")
    ok = desc()
    assert attend(pkv, which, None) == INVALID
    for bad in (desc(d=96), desc(bs=64), desc(nb=0), desc(hkv=0)):
        assert attend(pkv, which, bad) == INVALID
    for kw in (dict(n=-1), dict(total=-1), dict(hq=7), dict(hq=0), dict(mb=0), dict(mx=-1), dict(scale=nan),
               dict(scale=inf), dict(total=3), dict(qs=P, mq=-1), dict(qs=P, mq=0), dict(out=None), dict(q=None),
               dict(q=ODD), dict(out=ODD), dict(kc=None), dict(vc=ODD), dict(tb=None), dict(ln=None),
               dict(ln=ctypes.c_void_p(0x1002)), dict(qs=ctypes.c_void_p(0x1002))):
        assert attend(pkv, which, ok, **kw) == INVALID, kw
    S = pkv.ScoreOpts
    for o in (S(-1.0, None, None, 0, 0), S(nan, None, None, 0, 0), S(inf, None, None, 0, 0), S(0.0, None, None, -1, 0),
              S(0.0, None, None, 4, -1), S(0.0, 0x1002, None, 0, 0), S(0.0, None, 0x1002, 0, 0)):
        assert attend(pkv, which, ok, opts=o) == INVALID
    assert attend(pkv, which, ok, dt=0) == UNSUPPORTED        # fp32 queries
    assert attend(pkv, which, ok, n=1 << 20, total=4, qs=P, mq=1 << 20, hq=64) == UNSUPPORTED  # too many chunks
    assert attend(pkv, which, ok, n=0, total=0) == 0
    assert attend(pkv, which, ok, n=2, total=0, qs=P) == 0


def test_scored_cache_types(pkv):
    assert attend(pkv, "scored", pkv.CacheDesc(8, 16, 2, 128, 0)) == UNSUPPORTED  # fp32 cache
    assert attend(pkv, "scored", pkv.CacheDesc(8, 16, 2, 128, 5)) == INVALID
    f8 = pkv.CacheDesc(8, 16, 2, 128, 2)
    for kv in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(pkv, "scored", f8, kv=kv) == INVALID


def test_workspace_bytes(pkv):
    f = pkv.library().pkv_scored_workspace_bytes
    for bad in ((-1, 1, 8, 2, 128), (2, -1, 8, 2, 128), (2, 1, 7, 2, 128), (2, 1, 8, 2, 96), (2, 1, 0, 2, 128),
                (2, 1, 8, 0, 128)):
        assert f(*bad) == 0


def test_bindings_refuse_before_any_device_work(pkv):
    d, bs = 64, 16
    kc = torch.zeros(pkv.quant_cache_shape(4, 2, bs, d, "int8"), dtype=torch.uint8)
    x = torch.zeros((3, 2, d), dtype=torch.bfloat16)
    sl = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        pkv.kv_quantize_and_cache(x.half(), x.half(), kc, kc, sl, bs)
    with pytest.raises(TypeError):
        pkv.kv_quantize_and_cache(x, x, kc, kc, sl.int(), bs)
    with pytest.raises(ValueError):
        pkv.kv_quantize_and_cache(x, x, kc, kc, sl[:2], bs)            # one slot per token
    with pytest.raises(ValueError):
        pkv.kv_quantize_and_cache(x, x, kc, kc, sl, bs, "fp4")         # a cache of another format
    with pytest.raises(ValueError):
        pkv.kv_quantize_and_cache(x[:, :1], x[:, :1], kc, kc, sl, bs)  # another head count
    with pytest.raises(ValueError):
        pkv.kv_quantize_and_cache(x, x, kc, kc, sl, bs)                # host tensors
    q = torch.zeros((2, 4, d), dtype=torch.bfloat16)
    tb, ln = torch.zeros((2, 3), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    bf = torch.zeros((4, 2, bs, d), dtype=torch.bfloat16)
    calls = [lambda **kw: pkv.paged_attention_scored(kw.pop("out", q), kw.pop("q", q), bf, bf, kw.pop("tb", tb),
                                                     kw.pop("ln", ln), 0.1, **kw),
             lambda **kw: pkv.paged_attention_quant(kw.pop("out", q), kw.pop("q", q), kc, kc, kw.pop("tb", tb),
                                                    kw.pop("ln", ln), 0.1, bs, **kw)]
    for call in calls:
        for kw, err in ((dict(out=q.float()), ValueError), (dict(out=q[:1]), ValueError), (dict(tb=tb.long()), TypeError),
                        (dict(tb=tb[:1]), ValueError), (dict(ln=ln.long()), TypeError),
                        (dict(q_start=torch.zeros(2, dtype=torch.int32)), ValueError),
                        (dict(alibi_slopes=torch.zeros(3)), ValueError),
                        (dict(alibi_slopes=torch.zeros(4, dtype=torch.float64)), TypeError),
                        (dict(prefix_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
                        (dict(out=q[:1], q=q[:1]), ValueError), (dict(), ValueError)):
            with pytest.raises(err):
                call(**kw)
    with pytest.raises(ValueError):
        pkv.paged_attention_scored(q, q, bf, bf[:, :1], tb, ln, 0.1)
