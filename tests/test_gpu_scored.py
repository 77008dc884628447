"""Attention with modified scores and attention over quantised caches on the
GPU, every row against the formula in 64 bits over the cache's own values.

Tolerance of an output o with value range V = max |V[t]| over its sequence and
kv head: the bf16 rounding of the result, 2^-8 |o|, plus what the rounding of
the weights moves a convex combination by.  fp8 and quantised caches hold a
weight in fp16 (2^-11 of it), bf16 caches in two bf16 parts (2^-17); the scores
come from exact products summed in fp32, their errors (and those of exp2,
tanh) are below 2^-12 of a weight at these sizes.  So 2^-8 |o| + 2^-10 V and
2^-8 |o| + 2^-11 V.  Calls with 128 or more query rows per (sequence, kv head)
hold a weight over a bf16 cache in one bf16 part (2^-8 of it): 2^-8 |o| +
(2^-8 + 2^-11) V."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests._quant import attention_row, e4m3_values, slots_for, tables_for

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_22_gb300 as m
    m.library()
    return m


class Problem:
    """A filled, poisoned cache of any kind with query rows, and its values."""

    def __init__(self, pkv, kind, d, bs, hq, hkv, lens, rows=None, seed=0, kv=None, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.pkv, self.kind, self.d, self.bs, self.hq, self.hkv, self.lens = pkv, kind, d, bs, hq, hkv, list(lens)
        self.rows = rows
        self.tables, self.pool = tables_for(lens, bs, g)
        n = sum(lens)
        k = torch.randn(n, hkv, d, generator=g)
        k[..., ::17] *= 3
        v = torch.randn(n, hkv, d, generator=g)
        if kv is not None:
            k, v = kv(k, v)
        q_rows = len(lens) if rows is None else sum(rows)
        self.q = torch.randn(q_rows, hq, d, generator=g).to(torch.bfloat16)
        self.q_start = None if rows is None else torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32)
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.kv_scale = 1.0
        slots = slots_for(lens, self.tables, bs).to(DEV)
        k, v = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
        ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
        mx = max(max(lens), 1)
        if kind in ("int8", "fp4"):
            self.kc = torch.full(pkv.quant_cache_shape(self.pool, hkv, bs, d, kind), 0xFF, dtype=torch.uint8, device=DEV)
            self.vc = self.kc.clone()
            pkv.kv_quantize_and_cache(k, v, self.kc, self.vc, slots, bs, kind)
            ko, vo = pkv.gather_kv_quant(self.kc, self.vc, self.tables.to(DEV), ln, bs, d, kind, mx, out_dtype=torch.float32)
            self.K, self.V = ko.double().cpu().numpy(), vo.double().cpu().numpy()
        else:
            dt = torch.bfloat16 if kind == "bf16" else torch.uint8
            self.kc = torch.full((self.pool * hkv * bs * d * (2 if kind == "bf16" else 1),), 0xFF, dtype=torch.uint8,
                                 device=DEV).view(dt).view(self.pool, hkv, bs, d)
            self.vc = self.kc.clone()
            if kind == "fp8":
                self.kv_scale = 0.03
            pkv.kv_reshape_and_cache(k, v, self.kc, self.vc, slots, self.kv_scale)
            ko, vo = pkv.gather_kv(self.kc, self.vc, self.tables.to(DEV), ln, mx)
            if kind == "fp8":
                t = e4m3_values() * self.kv_scale
                self.K, self.V = t[ko.cpu().numpy()], t[vo.cpu().numpy()]
            else:
                self.K, self.V = ko.double().cpu().numpy(), vo.double().cpu().numpy()
        assert pkv.get_device_error() == 0

    def run(self, out=None, tables=None, lens=None, workspace=None, stream=None, max_q=None, q_start=None,
            max_seq_len=None, **opts):
        pkv = self.pkv
        q = self.q.to(DEV)
        out = torch.full_like(q, 7.0) if out is None else out
        tables = (self.tables if tables is None else tables).to(DEV)
        ln = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32, device=DEV)
        qs = self.q_start if q_start is None else q_start
        self.bound = max_q or max(self.rows or [1])
        opts = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in opts.items()}
        kw = dict(q_start=None if qs is None else qs.to(DEV), max_q=max_q, workspace=workspace, stream=stream,
                  max_seq_len=max_seq_len or max(max(self.lens), 1), **opts)
        if self.kind in ("int8", "fp4"):
            pkv.paged_attention_quant(out, q, self.kc, self.vc, tables, ln, self.scale, self.bs, self.kind, **kw)
        else:
            pkv.paged_attention_scored(out, q, self.kc, self.vc, tables, ln, self.scale, kv_scale=self.kv_scale, **kw)
        return out

    def expected(self, softcap=0.0, alibi_slopes=None, window=0, sinks=0, prefix_lens=None, missing=None):
        """(rows, V ranges) in 64 bits."""
        want = np.zeros((self.q.shape[0], self.hq, self.d))
        vmax = np.zeros((self.q.shape[0], self.hq, 1))
        q = self.q.double().numpy()
        g = self.hq // self.hkv
        at = base = 0
        for s, L in enumerate(self.lens):
            T = 1 if self.rows is None else self.rows[s]
            for i in range(T):
                p = L - T + i
                for h in range(self.hq if L else 0):
                    K, V = self.K[base: base + L, h // g], self.V[base: base + L, h // g]
                    want[at + i, h] = attention_row(
                        q[at + i, h], K, V, p, L, self.scale, softcap,
                        float(alibi_slopes[h]) if alibi_slopes is not None else 0.0, window, sinks,
                        max(0, int(prefix_lens[s])) if prefix_lens is not None else 0, (missing or {}).get(s, ()))
                    vmax[at + i, h] = np.abs(V).max()
            at += T
            base += L
        return want, vmax

    def weights(self):
        if self.kind != "bf16":
            return 2.0 ** -10
        tiled = self.rows is not None and self.bound * (self.hq // self.hkv) >= 128
        return 2.0 ** -11 + (2.0 ** -8 if tiled else 0.0)

    def check(self, got, want, vmax, what=""):
        torch.cuda.synchronize()
        got = got.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN in other places"
        tol = 2.0 ** -8 * np.abs(want) + self.weights() * vmax
        over = np.nan_to_num(np.abs(got - want) - tol)
        i = np.unravel_index(over.argmax(), over.shape)
        assert over.max() <= 0, f"{what}: at {i}: {got[i]} for {want[i]}, tolerance {tol[i]}"


def slopes(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1, dtype=torch.float32) / hq)


KINDS = ["bf16", "fp8", "int8", "fp4"]
SHAPES = [  # d, bs, hq, hkv
    (128, 16, 8, 2), (64, 16, 6, 2), (128, 32, 7, 1), (128, 8, 10, 2), (64, 32, 16, 1), (64, 8, 3, 3), (128, 16, 34, 2),
]
OPTS = {
    "plain": {},
    "cap": dict(softcap=5.0),
    "alibi": dict(alibi=True),
    "window": dict(window=21, sinks=3),
    "all": dict(softcap=20.0, alibi=True, window=33, sinks=0, prefix=True),
}


def options(o, hq, lens):
    o = dict(o)
    if o.pop("alibi", False):
        o["alibi_slopes"] = slopes(hq)
    if o.pop("prefix", False):
        o["prefix_lens"] = torch.tensor([(-2, 0, 1, 17, 40, 10 ** 6)[i % 6] for i in range(len(lens))], dtype=torch.int32)
    return o


@pytest.mark.parametrize("opt", list(OPTS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bs%d_q%d_kv%d" % s)
@pytest.mark.parametrize("kind", KINDS)
def test_decode(pkv, kind, shape, opt):
    d, bs, hq, hkv = shape
    lens = [1, 2, 0, 15, 16, 17, 33, 100, 203]
    p = Problem(pkv, kind, d, bs, hq, hkv, lens, seed=d + bs)
    o = options(OPTS[opt], hq, lens)
    p.check(p.run(**o), *p.expected(**o), f"{kind} {shape} {opt}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("opt", list(OPTS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bs%d_q%d_kv%d" % s)
@pytest.mark.parametrize("kind", KINDS)
def test_several_tokens(pkv, kind, shape, opt):
    """Chunks of one to many tokens; sequences without any; whole prompts."""
    d, bs, hq, hkv = shape
    lens, rows = [5, 40, 64, 90, 1, 30], [5, 3, 0, 21, 1, 30]
    p = Problem(pkv, kind, d, bs, hq, hkv, lens, rows, seed=d + bs + 1)
    o = options(OPTS[opt], hq, lens)
    want = p.expected(**o)
    p.check(p.run(**o), *want, f"{kind} {shape} {opt}")
    p.check(p.run(max_q=max(rows) + 19, **o), *want, "a larger bound")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_verification_over_cut_segments(pkv, kind):
    """A few tokens of long sequences: segments cut between many warps."""
    lens, rows = [3001, 1500, 4], [4, 2, 4]
    p = Problem(pkv, kind, 128, 16, 8, 2, lens, rows, seed=4)
    for o in ({}, dict(softcap=30.0, alibi_slopes=slopes(8), window=700, sinks=5)):
        p.check(p.run(**o), *p.expected(**o), kind)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_long_chunk(pkv, kind):
    """A prompt chunk with hundreds of rows per kv head."""
    lens, rows = [260, 131], [130, 131]
    p = Problem(pkv, kind, 128, 16, 8, 2, lens, rows, seed=14)
    for o in ({}, dict(softcap=10.0, window=50, prefix_lens=torch.tensor([60, 0], dtype=torch.int32))):
        p.check(p.run(**o), *p.expected(**o), kind)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("opt", list(OPTS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bs%d_q%d_kv%d" % s)
@pytest.mark.parametrize("kind", KINDS)
def test_tiles_of_query_rows(pkv, kind, shape, opt):
    """Calls whose bound asks for 128-row tiles: ragged chunks of zero rows to
    several tiles, over one to several steps of 128 positions."""
    d, bs, hq, hkv = shape
    lens, rows = [300, 129, 128, 1, 77, 515], [90, 1, 128, 1, 0, 3]
    p = Problem(pkv, kind, d, bs, hq, hkv, lens, rows, seed=d + bs + 2)
    o = options(OPTS[opt], hq, lens)
    p.check(p.run(**o), *p.expected(**o), f"{kind} {shape} {opt}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("rows", [32, 48])
def test_tiles_of_many_long_sequences(pkv, rows):
    """More CTAs than run at once, fed as fast as memory gives: K or V may come
    late while the softmax is a step ahead of its products.  (128 and 192 rows
    per kv head: CTAs of one tile and of two.)"""
    hq, hkv, d, bs = 32, 8, 128, 16
    lens = [2048 - 16 * ((37 * i) % 64) - i % 5 for i in range(64)]
    g = torch.Generator(device=DEV).manual_seed(rows)
    tables, pool = tables_for(lens, bs, torch.Generator().manual_seed(rows))
    n = sum(lens)
    k, v = (torch.randn(n, hkv, d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(64 * rows, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    kc = torch.full((pool, hkv, bs, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = kc.clone()
    pkv.kv_reshape_and_cache(k, v, kc, vc, slots_for(lens, tables, bs).to(DEV), 1.0)
    q_start = torch.arange(65, dtype=torch.int32, device=DEV) * rows
    out = torch.empty_like(q)
    for _ in range(3):
        out.fill_(7)
        pkv.paged_attention_scored(out, q, kc, vc, tables.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                   1 / math.sqrt(d), q_start=q_start, max_q=rows, max_seq_len=2048)
        assert pkv.get_device_error() == 0
        at = 0
        for s, L in enumerate(lens):
            K, V = k[at: at + L].double(), v[at: at + L].double()
            Q = q[s * rows: (s + 1) * rows].double().reshape(rows, hkv, hq // hkv, d)
            z = torch.einsum("tkgd,nkd->tkgn", Q, K) / math.sqrt(d)
            seen = torch.arange(L, device=DEV)[None] <= torch.arange(L - rows, L, device=DEV)[:, None]
            w = torch.softmax(z.masked_fill(~seen[:, None, None], -math.inf), -1)
            want = torch.einsum("tkgn,nkd->tkgd", w, V).reshape(rows, hq, d)
            vmax = V.abs().amax((0, 2)).repeat_interleave(hq // hkv)[None, :, None]
            over = (out[s * rows: (s + 1) * rows].double() - want).abs() - 2.0 ** -8 * want.abs() - (2.0 ** -8 + 2.0 ** -11) * vmax
            assert over.max().item() <= 0, (s, L)
            at += L


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_whose_maximum_grows(pkv, kind):
    """Scores that rise along the keys, by more than 2^8 between the halves of
    a step and between steps: every rescale is taken."""
    def kv(k, v):
        t = torch.arange(k.shape[0], dtype=torch.float32)
        return k * 0.01 + (t // 64)[:, None, None] * 0.35, v

    p = Problem(pkv, kind, 128, 16, 4, 1, [400], [200], seed=3, kv=kv)
    p.q = p.q.abs() * 0.5
    for o in ({}, dict(softcap=400.0)):
        want, vmax = p.expected(**o)
        p.check(p.run(**o), want, vmax, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [8, 32])
def test_tiles_leave_out_bad_and_freed_blocks(pkv, kind, bs):
    lens, rows, W = [500, 200], [60, 70], 90
    p = Problem(pkv, kind, 128, bs, 8, 2, lens, rows, seed=5)
    tables = p.tables.clone()
    tables[0, 1:(500 - 60 - W) // bs] = -9       # before every row's window, past the sinks
    want = p.expected(window=W, sinks=3)
    p.check(p.run(tables=tables, window=W, sinks=3), *want, kind)
    assert pkv.get_device_error() == 0
    tables = p.tables.clone()
    tables[1, 2] = p.pool
    got = p.run(tables=tables)
    assert pkv.get_device_error() == pkv.DEVERR_BAD_BLOCK_ID
    p.check(got, *p.expected(missing={1: range(2 * bs, 3 * bs)}), kind)


@pytest.mark.parametrize("kind", ["int8", "fp4"])
def test_row_scales_of_any_size(pkv, kind):
    """Rows of V whose magnitudes differ by up to 2^40, the largest weights on
    the smallest rows; rows of zeros.  The tolerance is the largest |V|."""
    def kv(k, v):
        e = (torch.arange(k.shape[0]) * 7 % 41 - 20).float()
        v = v * torch.exp2(e)[:, None, None]
        v[::11] = 0
        k[1::11] = 0
        return k * torch.where(e < 0, 2.0, 0.5)[:, None, None], v

    for only in (None, 0):
        p = Problem(pkv, kind, 128, 16, 8, 2, [400, 37], seed=6, kv=kv if only is None else lambda k, v: (k, v * 0))
        p.check(p.run(), *p.expected(), kind)
    # every row small: nothing is lost against the rows' own size
    p = Problem(pkv, kind, 64, 16, 8, 2, [300], seed=6, kv=lambda k, v: (k * 1e-4, v * 1e-20))
    p.check(p.run(), *p.expected(), kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mag", [1e-30, 1e-4, 300.0, 1e30])
def test_queries_of_any_size(pkv, kind, mag):
    """One row of q scaled, the others not: each row keeps its precision."""
    p = Problem(pkv, kind, 128, 16, 8, 1, [50], seed=2, scale=0.02)
    if mag > 100:
        p.K *= 1  # scores of one kept position only: the softmax is one-hot
    p.q[:, 3] = (p.q[:, 3].float() * mag).to(torch.bfloat16)
    got = p.run()
    want, vmax = p.expected()
    keep = np.ones(8, bool)
    if mag > 100:  # z differs by far more than its error: the largest wins alone; compared below
        keep[3] = False
        x = p.q[0, 3].double().numpy() @ p.K[:, 0].T
        order = np.sort(x)
        assert order[-1] - order[-2] > 2.0 ** -9 * np.abs(x).max()
        want[0, 3] = p.V[x.argmax(), 0]
        if p.scale * (order[-1] - order[-2]) > 40:
            keep[3] = True
    p.check(got[:, keep], want[:, keep], vmax[:, keep], kind)


def test_softcap_of_any_size(pkv):
    """A cap far above the scores changes nothing; a small one saturates."""
    p = Problem(pkv, "bf16", 128, 16, 4, 1, [300], seed=3)
    for cap in (1e-3, 0.5, 50.0, 1e4, 1e8, 1e30):
        p.check(p.run(softcap=cap), *p.expected(softcap=cap), f"cap {cap}")


@pytest.mark.parametrize("kind", KINDS)
def test_negative_and_zero_scale(pkv, kind):
    for scale in (-0.1, 0.0):
        p = Problem(pkv, kind, 64, 16, 4, 2, [70, 3], seed=3, scale=scale)
        p.check(p.run(softcap=4.0), *p.expected(softcap=4.0), f"{kind} {scale}")
        p = Problem(pkv, kind, 64, 16, 4, 1, [170, 40], [60, 33], seed=3, scale=scale)
        for o in ({}, dict(softcap=4.0)):
            p.check(p.run(**o), *p.expected(**o), f"{kind} {scale} tiles")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_freed_blocks_outside_the_window(pkv, kind, bs):
    """Table entries of blocks no row attends may hold anything."""
    L, W, S = 500, 70, 5
    p = Problem(pkv, kind, 64, bs, 4, 2, [L], seed=3)
    want = p.expected(window=W, sinks=S)
    tables = p.tables.clone()
    tables[0, -(-S // bs): (L - W) // bs] = -5
    p.check(p.run(tables=tables, window=W, sinks=S), *want, kind)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_bad_blocks_are_left_out(pkv, kind, bs):
    """A bad id inside the attended range is flagged, its positions left out;
    a sequence with no good block gets a zero row."""
    lens = [100, 40, 20]
    p = Problem(pkv, kind, 64, bs, 4, 2, lens, seed=5)
    tables = p.tables.clone()
    tables[0, 1] = p.pool
    tables[1, :] = -1
    assert pkv.get_device_error() == 0
    got = p.run(tables=tables)
    assert pkv.get_device_error() == pkv.DEVERR_BAD_BLOCK_ID
    want, vmax = p.expected(missing={0: range(bs, 2 * bs), 1: range(40)})
    p.check(got, want, vmax, kind)
    assert (got[1] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_masked_places_may_hold_anything(pkv, kind):
    """NaN and infinities in rows outside a decode's window do not reach it."""
    lens, W = [90, 47], 20
    p = Problem(pkv, kind, 128, 16, 4, 2, lens, seed=5)
    want = p.expected(window=W)
    d = p.d
    bad = torch.full((1, 2, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    inf = torch.full_like(bad, float("inf"))
    for s, L in enumerate(lens):
        for t in (0, 3, L - W - 1):
            slot = torch.tensor([int(p.tables[s, t // 16]) * 16 + t % 16], dtype=torch.int64, device=DEV)
            x = bad if t % 2 else inf
            if kind in ("int8", "fp4"):
                pkv.kv_quantize_and_cache(x, x, p.kc, p.vc, slot, 16, kind)
            else:
                pkv.kv_reshape_and_cache(bad, bad, p.kc, p.vc, slot, p.kv_scale)
    p.check(p.run(window=W), *want, kind)
    # attended, they show
    got = p.run()
    assert torch.isnan(got).all()


class Loose(Problem):
    """Calls whose bound of query tokens is far above the rows: enough of them
    for the 128-row tiles at any number of sequences."""

    def run(self, *args, **kw):
        if self.rows is not None and kw.get("max_q") is None:
            kw["max_q"] = 1 << 14
        return super().run(*args, **kw)


@pytest.fixture
def loose(monkeypatch):
    monkeypatch.setitem(globals(), "Problem", Loose)


@pytest.mark.parametrize("opt", list(OPTS))
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bs%d_q%d_kv%d" % s)
@pytest.mark.parametrize("kind", KINDS)
def test_tiles_at_a_loose_bound(pkv, loose, kind, shape, opt):
    test_tiles_of_query_rows(pkv, kind, shape, opt)


@pytest.mark.parametrize("kind", KINDS)
def test_tile_cases_at_a_loose_bound(pkv, loose, kind):
    test_long_chunk(pkv, kind)
    test_verification_over_cut_segments(pkv, kind)
    test_tiles_whose_maximum_grows(pkv, kind)
    test_negative_and_zero_scale(pkv, kind)
    for bs in (8, 32):
        test_tiles_leave_out_bad_and_freed_blocks(pkv, kind, bs)


@pytest.mark.parametrize("kind", KINDS)
def test_tile_row_scales_and_queries_of_any_size(pkv, loose, kind):
    """Prompt rows over K and V rows of very different sizes; query rows scaled
    far down or up."""
    def kv(k, v):
        e = (torch.arange(k.shape[0]) * 7 % 41 - 20).float()
        v = v * torch.exp2(e)[:, None, None] if kind in ("int8", "fp4") else v
        v[::11] = 0
        k[1::11] = 0
        return k * torch.where(e < 0, 2.0, 0.5)[:, None, None], v

    p = Problem(pkv, kind, 128, 16, 8, 2, [400, 70], [140, 37], seed=6, kv=kv)
    p.check(p.run(), *p.expected(), kind)
    p = Problem(pkv, kind, 64, 16, 8, 1, [150], [90], seed=2, scale=0.02)
    p.q[:, 3] = (p.q[:, 3].float() * 1e-30).to(torch.bfloat16)
    p.q[:, 5] = (p.q[:, 5].float() * 1e-4).to(torch.bfloat16)
    p.check(p.run(), *p.expected(), kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [0.5, 12.0, 30.0, 80.0, 1e4, 1e30])
def test_tiles_capped(pkv, loose, kind, cap):
    """Scores far below the cap, near it and above: each form of the tanh."""
    p = Problem(pkv, kind, 128, 16, 4, 1, [450, 300], [130, 70], seed=9)
    p.check(p.run(softcap=cap), *p.expected(softcap=cap), f"{kind} {cap}")


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_flag_bad_lengths(pkv, kind):
    """The other sequences' rows are right, the bad ones' left as they were."""
    lens, rows = [50, 30, 60], [3, 30, 9]
    p = Loose(pkv, kind, 64, 16, 4, 2, lens, rows, seed=5)
    want, vmax = p.expected()
    at = [0, 3, 33, 42]
    for ln in ([50, 7, 60], [50, -1, 60], [50, 10 ** 9, 60]):
        got = p.run(lens=ln)
        assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
        for s in range(3):
            r = slice(at[s], at[s + 1])
            if s == 1:
                assert (got[r] == 7).all()
            else:
                p.check(got[r], want[r], vmax[r], f"{ln} sequence {s}")
    for qs in ([0, 3, 33, 45], [0, 3, 1, 10], [-3, 3, 33, 42]):
        got = p.run(q_start=torch.tensor(qs, dtype=torch.int32))
        assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
        bad = [s for s in range(3) if qs[s] < 0 or qs[s + 1] < qs[s] or qs[s + 1] > 42]
        touched = {r for s in range(3) if s not in bad for r in range(qs[s], qs[s + 1])}
        assert all((got[r] == 7).all() for r in range(42) if r not in touched)
    # padding rows behind the last sequence
    p.q = torch.cat([p.q, p.q[:5]])
    got = p.run()
    p.check(got[:42], want[:42], vmax[:42])
    assert (got[42:] == 7).all()
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_masked_places_may_hold_anything(pkv, kind):
    """NaN and infinities at positions that no row of a chunk attends, in
    blocks of which others are."""
    lens, rows, W = [300, 130], [70, 40], 50
    p = Loose(pkv, kind, 128, 16, 8, 2, lens, rows, seed=8)
    opts = [dict(window=W), dict(window=W, sinks=2, alibi_slopes=slopes(8)), dict(window=W, softcap=30.0)]
    wants = [p.expected(**o) for o in opts]
    for s, L in enumerate(lens):
        for t, x in ((2, "nan"), (5, "inf"), (L - rows[s] - W, "-inf"), (L - rows[s] - W - 1, "nan")):
            slot = torch.tensor([int(p.tables[s, t // 16]) * 16 + t % 16], dtype=torch.int64, device=DEV)
            x = torch.full((1, 2, 128), float(x), dtype=torch.bfloat16, device=DEV)
            if kind in ("int8", "fp4"):
                pkv.kv_quantize_and_cache(x, x, p.kc, p.vc, slot, 16, kind)
            else:
                pkv.kv_reshape_and_cache(x, x, p.kc, p.vc, slot, p.kv_scale)
    for o, want in zip(opts, wants):
        p.check(p.run(**o), *want, f"{kind} {o}")
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("max_q", [None, 1 << 14], ids=["columns", "tiles"])
@pytest.mark.parametrize("kind", ["int8", "fp4"])
def test_a_nan_row_shows_where_it_is_attended(pkv, kind, max_q):
    """A quantised row of NaN: rows of a chunk before its position, or whose
    window has left it, keep their values."""
    L, T, W, bad = 120, 80, 30, 75
    p = Problem(pkv, kind, 128, 16, 8, 2, [L], [T], seed=8)
    want, vmax = p.expected(window=W)
    x = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    slot = torch.tensor([int(p.tables[0, bad // 16]) * 16 + bad % 16], dtype=torch.int64, device=DEV)
    pkv.kv_quantize_and_cache(x, x, p.kc, p.vc, slot, 16, kind)
    seen = [r for r in range(T) if bad <= L - T + r < bad + W]
    want[seen] = np.nan
    p.check(p.run(max_q=max_q, window=W), want, vmax, kind)


@pytest.mark.parametrize("kind", KINDS)
def test_tiles_of_many_short_sequences(pkv, kind):
    """More sequences than are sorted by length; a few rows each, some none."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(1, 40, (300,), generator=g).tolist()
    rows = [min(n, r) for n, r in zip(lens, torch.randint(0, 6, (300,), generator=g).tolist())]
    p = Problem(pkv, kind, 64, 8, 2, 1, lens, rows, seed=4)
    p.check(p.run(max_q=100, softcap=6.0), *p.expected(softcap=6.0), kind)
    assert pkv.get_device_error() == 0


def test_tiles_streams_and_graphs(pkv):
    """Calls on two streams at once, and two graphs replayed side by side with
    inputs changed in between."""
    ps = [Loose(pkv, "fp4", 128, 16, 8, 2, [700, 90, 5], [150, 40, 5], seed=1),
          Loose(pkv, "bf16", 128, 16, 8, 2, [500, 300], [200, 1], seed=2)]
    os = [dict(softcap=9.0), dict(window=100, alibi_slopes=slopes(8).to(DEV))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wants = [p.expected(**{k: v.cpu() if torch.is_tensor(v) else v for k, v in o.items()}) for p, o in zip(ps, os)]
    torch.cuda.synchronize()
    got = [[p.run(stream=st, **o) for p, o, st in zip(ps, os, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for outs in got:
        for p, x, want in zip(ps, outs, wants):
            p.check(x, *want)

    graphs = []
    for p, o in zip(ps, os):
        q, out = p.q.to(DEV), torch.zeros_like(p.q, device=DEV)
        tb, ln, qs = p.tables.to(DEV), torch.tensor(p.lens, dtype=torch.int32, device=DEV), p.q_start.to(DEV)
        kw = dict(q_start=qs, max_q=1 << 14, max_seq_len=max(p.lens), **o)

        def call():
            if p.kind == "fp4":
                pkv.paged_attention_quant(out, q, p.kc, p.vc, tb, ln, p.scale, p.bs, p.kind, **kw)
            else:
                pkv.paged_attention_scored(out, q, p.kc, p.vc, tb, ln, p.scale, **kw)
        call()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        graphs.append((gr, q, out, tb, ln, qs))
    for p, (_, q, *_) in zip(ps, graphs):
        p.q = -p.q
        q.copy_(p.q)
    wants = [p.expected(**{k: v.cpu() if torch.is_tensor(v) else v for k, v in o.items()}) for p, o in zip(ps, os)]
    for _ in range(5):
        for gr in graphs:
            gr[2].zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr[0].replay()
        torch.cuda.synchronize()
        for p, gr, want in zip(ps, graphs, wants):
            p.check(gr[2], *want)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_bad_lengths(pkv, kind):
    """Decode: a negative length gives a zero row, one beyond the bound is
    clipped; several tokens: the sequence's rows are left as they were."""
    lens = [50, 30, 60]
    p = Problem(pkv, kind, 64, 16, 4, 2, lens, seed=5)
    want, vmax = p.expected()
    assert pkv.get_device_error() == 0
    got = p.run(lens=[50, -4, 60])
    assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
    want[1] = 0
    p.check(got, want, vmax, kind)
    got = p.run(lens=[50, 30, 10 ** 6], max_seq_len=60)
    assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
    want, vmax = p.expected()
    p.check(got, want, vmax, kind)

    p = Problem(pkv, kind, 64, 16, 4, 2, lens, rows=[3, 30, 9], seed=5)
    want, vmax = p.expected()
    at = [0, 3, 33, 42]
    cases = [dict(max_q=8), dict(lens=[50, 7, 60]), dict(lens=[50, -1, 60])]
    for kw in cases:
        got = p.run(**kw)
        assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
        keep = [0, 2] if "lens" in kw else [0]
        for s in range(3):
            r = slice(at[s], at[s + 1])
            if s in keep:
                p.check(got[r], want[r], vmax[r], f"{kw} sequence {s}")
            else:
                assert (got[r] == 7).all(), f"{kw} sequence {s}"
    # offsets past the rows there are, decreasing, negative
    for qs in ([0, 3, 33, 45], [0, 3, 1, 10], [-3, 3, 33, 42]):
        got = p.run(q_start=torch.tensor(qs, dtype=torch.int32), max_q=30)
        assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
        bad = [s for s in range(3) if qs[s] < 0 or qs[s + 1] < qs[s] or qs[s + 1] > 42]
        touched = {r for s in range(3) if s not in bad for r in range(qs[s], qs[s + 1])}
        for r in range(42):
            if r not in touched:
                assert (got[r] == 7).all()


def test_rows_of_no_sequence_are_left(pkv):
    p = Problem(pkv, "bf16", 64, 16, 4, 2, [50, 30], rows=[3, 4], seed=5)
    p.q = torch.cat([p.q, p.q[:5]])  # padding rows behind the last sequence
    p.rows = [3, 4]
    want, vmax = p.expected()
    got = p.run(max_q=4)
    p.check(got[:7], want[:7], vmax[:7])
    assert (got[7:] == 7).all()


def test_streams_graphs_and_workspaces(pkv):
    """Two calls at once on two streams, a captured and replayed one with new
    inputs in between, and one workspace shared with plain decode."""
    a = Problem(pkv, "int8", 128, 16, 8, 2, [3000, 700, 5], seed=1)
    b = Problem(pkv, "bf16", 128, 16, 8, 2, [2500, 900], seed=2)
    wa, wb = a.expected(softcap=9.0), b.expected(window=300)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(a.run(softcap=9.0, stream=s1), b.run(window=300, stream=s2)) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in got:
        a.check(x, *wa)
        b.check(y, *wb)

    # two graphs, replayed side by side, with their inputs changed before
    def captured(p, **o):
        kw = dict(q_start=None, max_seq_len=max(p.lens), **o)
        q, out = p.q.to(DEV), torch.zeros_like(p.q, device=DEV)
        tb, ln = p.tables.to(DEV), torch.tensor(p.lens, dtype=torch.int32, device=DEV)

        def call():
            if p.kind == "int8":
                pkv.paged_attention_quant(out, q, p.kc, p.vc, tb, ln, p.scale, p.bs, p.kind, **kw)
            else:
                pkv.paged_attention_scored(out, q, p.kc, p.vc, tb, ln, p.scale, **kw)
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        return g, q, out

    ga, qa, oa = captured(a, softcap=9.0)
    gb, qb, ob = captured(b, window=300)
    for p, q in ((a, qa), (b, qb)):
        p.q = -p.q
        q.copy_(p.q)
    wa, wb = a.expected(softcap=9.0), b.expected(window=300)
    torch.cuda.synchronize()
    for _ in range(10):
        oa.zero_()
        ob.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        torch.cuda.synchronize()
        a.check(oa, *wa)
        b.check(ob, *wb)

    # the decode's merge counters in a shared workspace stay zero
    ws = pkv.DecodeWorkspace()
    q, out = b.q.to(DEV), torch.zeros_like(b.q, device=DEV)
    ln = torch.tensor(b.lens, dtype=torch.int32, device=DEV)
    plain = b.expected()
    for engine in ("cuda_cores", "tensor_cores"):
        with pkv.decode_engine(engine):
            for _ in range(3):
                b.check(b.run(workspace=ws, window=300), *wb)
                out.zero_()
                pkv.paged_attention_decode(out, q, b.kc, b.vc, b.tables.to(DEV), ln, b.scale, max_seq_len=2500, workspace=ws)
                b.check(out, *plain)
    assert pkv.get_device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_a_prompt_then_decode_steps(pkv, fmt):
    """As a serving loop uses them: a prompt quantised and attended in chunks
    (prefix visible in both directions), then tokens one at a time, with the
    cache read back at the end."""
    d, bs, hq, hkv, cap = 128, 16, 8, 2, 30.0
    g = torch.Generator().manual_seed(11)
    lens, chunk, steps, pre = [45, 71], 24, 3, [10, 30]
    total = [n + steps for n in lens]
    tables, pool = tables_for(total, bs, g)
    kc = torch.full(pkv.quant_cache_shape(pool, hkv, bs, d, fmt), 0xFF, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    k = [torch.randn(n, hkv, d, generator=g).to(torch.bfloat16) for n in total]
    v = [torch.randn(n, hkv, d, generator=g).to(torch.bfloat16) for n in total]
    q = [torch.randn(n, hq, d, generator=g).to(torch.bfloat16) for n in total]
    outs = [torch.zeros(n, hq, d) for n in total]
    prefix = torch.tensor(pre, dtype=torch.int32, device=DEV)
    tb = tables.to(DEV)
    done = [0, 0]

    def step(new):
        at = [list(range(done[s], done[s] + new[s])) for s in range(2)]
        slots = [int(tables[s, p // bs]) * bs + p % bs for s in range(2) for p in at[s]]
        cat = lambda x: torch.cat([x[s][at[s]] for s in range(2)]).to(DEV)  # noqa: E731
        pkv.kv_quantize_and_cache(cat(k), cat(v), kc, vc, torch.tensor(slots, dtype=torch.int64, device=DEV), bs, fmt)
        for s in range(2):
            done[s] += new[s]
        ln = torch.tensor(done, dtype=torch.int32, device=DEV)
        qs = torch.tensor([0, new[0], new[0] + new[1]], dtype=torch.int32, device=DEV)
        one = new == [1, 1]
        x = cat(q)
        out = torch.full_like(x, 7.0)
        pkv.paged_attention_quant(out, x, kc, vc, tb, ln, 0.09, bs, fmt, q_start=None if one else qs, max_q=max(new),
                                  softcap=cap, prefix_lens=prefix, max_seq_len=max(total))
        out = out.float().cpu()
        for s in range(2):
            outs[s][at[s]] = out[:new[0]] if s == 0 else out[new[0]:]
        return [list(a) for a in at]

    seen = []  # (rows, length when they were computed) per sequence
    while any(done[s] < lens[s] for s in range(2)):
        at = step([min(chunk, lens[s] - done[s]) for s in range(2)])
        seen.append((at, list(done)))
    for _ in range(steps):
        at = step([1, 1])
        seen.append((at, list(done)))
    ln = torch.tensor(total, dtype=torch.int32, device=DEV)
    ko, vo = pkv.gather_kv_quant(kc, vc, tb, ln, bs, d, fmt, max(total), out_dtype=torch.float32)
    assert pkv.get_device_error() == 0
    K, V = ko.double().cpu().numpy(), vo.double().cpu().numpy()
    base = [0, total[0]]
    for at, now in seen:
        for s in range(2):
            for p in at[s]:
                for h in range(hq):
                    Ks, Vs = (x[base[s]: base[s] + now[s], h // 4] for x in (K, V))
                    want = attention_row(q[s][p, h].double().numpy(), Ks, Vs, p, now[s], 0.09, cap, prefix=pre[s])
                    got = outs[s][p, h].double().numpy()
                    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(Vs).max()).all()
