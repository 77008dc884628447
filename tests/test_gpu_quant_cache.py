"""The quantised paged cache on the GPU: tokens quantised as they are written
(byte for byte against a plain quantiser) and read back (the exact values,
rounded once)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests._quant import e4m3_values, quantise_row, read_row, slots_for, tables_for, write_row

pytestmark = pytest.mark.gpu
DEV = "cuda"
POISON = 0xFF


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_22_gb300 as m
    m.library()
    return m


def rows(T, hkv, d, seed, dtype):
    """Token rows with the values a quantiser can go wrong at: zeros, negative
    zeros, tiny and huge rows, one large element, ties, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, hkv, d, generator=g)
    x[..., ::17] *= 4
    if T > 12:
        x[1] = 0
        x[2] = -0.0
        x[3] *= 1e-26          # below the smallest stored magnitude (bf16 and fp32 hold it)
        x[4] *= 1e-20
        x[5] = 3e38 * torch.sign(x[5])
        x[6, 0, 3] = float("inf")
        x[7, -1, d - 1] = float("nan")
        x[8, :, 1:] = 0
        x[9] = torch.arange(d, dtype=torch.float32) - 63.5    # halves: ties of the integer grid when a = 127 / 2 ...
        x[9, :, 0] = 127
        x[10, :, :] = 0
        x[10, :, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
        x[11, :, 16:32] = 1e-6   # a group whose scale rounds to zero beside large ones
    return x.to(dtype)


def expected(k, slots, shape, bs, fmt):
    c = np.full(shape, POISON, np.uint8)
    for t, slot in enumerate(slots.tolist()):
        if slot < 0:
            continue
        for h in range(shape[1]):
            write_row(c[slot // bs, h], slot % bs, k[t, h].float().numpy(), bs, fmt)
    return c


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d,bs,hkv,T,src", [(128, 16, 8, 37, torch.bfloat16), (64, 16, 3, 50, torch.float32),
                                            (128, 8, 1, 61, torch.float32), (64, 32, 5, 29, torch.bfloat16),
                                            (128, 32, 2, 1, torch.bfloat16), (64, 8, 4, 13, torch.float32)])
def test_write_is_byte_exact(pkv, fmt, d, bs, hkv, T, src):
    nb = -(-T // bs) + 4
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(nb * bs, generator=g)[:T].to(torch.int64)
    if T > 12:
        slots[0] = -1  # padding
    k, v = rows(T, hkv, d, 5, src), rows(T, hkv, d, 6, src)
    shape = pkv.quant_cache_shape(nb, hkv, bs, d, fmt)
    kc = torch.full(shape, POISON, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, POISON)
    pkv.kv_quantize_and_cache(k.to(DEV), v.to(DEV), kc, vc, slots.to(DEV), bs, fmt)
    assert pkv.get_device_error() == 0
    for got, x in ((kc, k), (vc, v)):
        want = expected(x, slots, shape, bs, fmt)
        diff = np.argwhere(got.cpu().numpy() != want)
        assert diff.size == 0, f"{len(diff)} bytes differ, the first at {diff[0]}"


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_codes_at_rounding_borders(pkv, fmt):
    """Rows built so that many quotients lie next to a border of the code grid
    (scaled half steps, off by one unit in the last place of binary32)."""
    d, bs, hkv, T = 128, 16, 2, 64
    g = torch.Generator().manual_seed(3)
    s = torch.rand(T, hkv, 1, generator=g) * 0.1 + 1e-3
    if fmt == "int8":
        n = torch.randint(-126, 126, (T, hkv, d), generator=g).float() + 0.5
        n[..., 0] = 127
    else:
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        n = mids[torch.randint(0, 7, (T, hkv, d), generator=g)]
        n[..., ::16] = 6.0
        s = s * 2.0 ** torch.randint(-3, 4, (T, hkv, 1), generator=g)
    x = n * s
    bump = torch.randint(-1, 2, x.shape, generator=g, dtype=torch.int32)
    x = (x.view(torch.int32) + bump).view(torch.float32)
    slots = torch.arange(T, dtype=torch.int64)
    shape = pkv.quant_cache_shape(T // bs, hkv, bs, d, fmt)
    kc = torch.full(shape, POISON, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, POISON)
    pkv.kv_quantize_and_cache(x.to(DEV), (-x).contiguous().to(DEV), kc, vc, slots.to(DEV), bs, fmt)
    assert np.array_equal(kc.cpu().numpy(), expected(x, slots, shape, bs, fmt))
    assert np.array_equal(vc.cpu().numpy(), expected(-x, slots, shape, bs, fmt))


@pytest.mark.parametrize("size", [1e-20, 1.0, 1e35])
def test_group_scales_at_rounding_borders(pkv, size):
    """Groups whose largest element puts m / (6 s) next to the middle between
    two e4m3 codes (off by one unit in the last place of binary32)."""
    d, bs, hkv, T = 128, 16, 2, 64
    rng = np.random.default_rng(8)
    grid = e4m3_values()[:127].astype(np.float32)
    a = (rng.uniform(0.5, 1.0, (T, hkv, 1)) * size).astype(np.float32)
    s6 = np.float32(6) * (a * np.float32(1 / 2688))
    i = rng.integers(0, 126, (T, hkv, d // 16))
    m = ((grid[i] + grid[i + 1]) / 2 * s6).astype(np.float32)
    m = (m.view(np.int32) + rng.integers(-1, 2, m.shape, dtype=np.int32)).view(np.float32)
    x = (rng.uniform(-1, 1, (T, hkv, d // 16, 16)).astype(np.float32) * m[..., None]).astype(np.float32)
    x[..., 5] = m
    x[:, :, 0, 0] = a[..., 0]
    x = torch.from_numpy(x.reshape(T, hkv, d))
    assert (x.abs().amax(-1) == torch.from_numpy(a[..., 0])).all()
    slots = torch.arange(T, dtype=torch.int64)
    shape = pkv.quant_cache_shape(T // bs, hkv, bs, d, "fp4")
    kc = torch.full(shape, POISON, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, POISON)
    pkv.kv_quantize_and_cache(x.to(DEV), (-x).contiguous().to(DEV), kc, vc, slots.to(DEV), bs, "fp4")
    assert np.array_equal(kc.cpu().numpy(), expected(x, slots, shape, bs, "fp4"))
    assert np.array_equal(vc.cpu().numpy(), expected(-x, slots, shape, bs, "fp4"))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
def test_quantisation_error_is_within_the_format(pkv, fmt):
    """int8: half a step, a / 254 (and a rounding of binary32); fp4: an element
    is off by at most half the largest gap of e2m1 (1) times its group's step
    plus what saturation cuts, the group scale being off by 2^-4 at most."""
    d, bs = 128, 16
    x = rows(40, 4, d, 9, torch.float32)[12:]
    for r in x.reshape(-1, d).numpy():
        tile = np.zeros(bs * (row := (d if fmt == "int8" else d // 2)) + (bs * d // 16 if fmt == "fp4" else 0) + 4 * bs, np.uint8)
        write_row(tile, 5, r, bs, fmt)
        got, a = read_row(tile, 5, d, bs, fmt), np.abs(r).max()
        if fmt == "int8":
            assert np.abs(got - r).max() <= a / 254 * (1 + 1e-5)
        else:
            m = np.abs(r.reshape(-1, 16)).max(1)
            step = m / 6 * (1 + 2.0 ** -4) + a / 2688 * 2.0 ** -9
            assert (np.abs(got - r).reshape(-1, 16) <= (step * (1 + 6 * 2.0 ** -4))[:, None]).all()


def test_bad_slots_are_flagged_and_skipped(pkv):
    d, bs, hkv, nb = 64, 16, 2, 3
    shape = pkv.quant_cache_shape(nb, hkv, bs, d, "int8")
    kc = torch.full(shape, POISON, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, POISON)
    x = rows(3, hkv, d, 1, torch.bfloat16)
    slots = torch.tensor([nb * bs, 5, -7], dtype=torch.int64)
    assert pkv.get_device_error() == 0
    pkv.kv_quantize_and_cache(x.to(DEV), x.to(DEV), kc, vc, slots.to(DEV), bs, "int8")
    assert pkv.get_device_error() == pkv.DEVERR_BAD_SLOT
    slots[0] = -1
    assert np.array_equal(kc.cpu().numpy(), expected(x, slots, shape, bs, "int8"))
    pkv.kv_quantize_and_cache(x[:0].to(DEV), x[:0].to(DEV), kc, vc, slots[:0].to(DEV), bs, "int8")  # no token


def same(got: torch.Tensor, want: np.ndarray, dtype) -> None:
    w = torch.from_numpy(want.astype(np.float32)).to(dtype)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(w))
    assert torch.equal(torch.nan_to_num(got.cpu().float()), torch.nan_to_num(w.float()))


@pytest.mark.parametrize("fmt", ["int8", "fp4"])
@pytest.mark.parametrize("d,bs,hkv,dtype", [(128, 16, 8, torch.bfloat16), (64, 8, 3, torch.float32),
                                            (128, 32, 1, torch.float32), (64, 32, 2, torch.bfloat16)])
def test_gather_returns_the_stored_values(pkv, fmt, d, bs, hkv, dtype):
    lens = [1, 0, bs, bs + 1, 77, 2 * bs - 1]
    g = torch.Generator().manual_seed(8)
    tables, pool = tables_for(lens, bs, g)
    slots = slots_for(lens, tables, bs)
    k, v = rows(sum(lens), hkv, d, 3, torch.float32), rows(sum(lens), hkv, d, 4, torch.float32)
    shape = pkv.quant_cache_shape(pool, hkv, bs, d, fmt)
    kc = torch.full(shape, POISON, dtype=torch.uint8, device=DEV)
    vc = torch.full_like(kc, POISON)
    pkv.kv_quantize_and_cache(k.to(DEV), v.to(DEV), kc, vc, slots.to(DEV), bs, fmt)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ko, vo = pkv.gather_kv_quant(kc, vc, tables.to(DEV), ln, bs, d, fmt, max(lens), out_dtype=dtype)
    assert pkv.get_device_error() == 0
    for got, x in ((ko, k), (vo, v)):
        want = np.empty((sum(lens), hkv, d))
        for t in range(sum(lens)):
            for h in range(hkv):
                codes, groups, s = quantise_row(x[t, h].numpy(), fmt)
                tile = np.zeros(shape[2], np.uint8)
                write_row(tile, 0, x[t, h].numpy(), bs, fmt)
                want[t, h] = read_row(tile, 0, d, bs, fmt)
        same(got, want, dtype)


def test_gather_flags_bad_blocks_lengths_and_room(pkv):
    d, bs, hkv, fmt = 64, 16, 2, "fp4"
    lens = [20, 33, 40]
    tables, pool = tables_for(lens, bs, torch.Generator().manual_seed(1))
    slots = slots_for(lens, tables, bs)
    x = rows(sum(lens), hkv, d, 3, torch.bfloat16)
    kc = torch.full(pkv.quant_cache_shape(pool, hkv, bs, d, fmt), POISON, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    pkv.kv_quantize_and_cache(x.to(DEV), x.to(DEV), kc, vc, slots.to(DEV), bs, fmt)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 20, 53, 93], dtype=torch.int64, device=DEV)
    good, _ = pkv.gather_kv_quant(kc, vc, tables.to(DEV), ln, bs, d, fmt, 40, cu_seq_lens=cu, total_tokens=93)
    assert pkv.get_device_error() == 0

    def call(tables, ln, max_len, total):
        """Through the C ABI, into outputs that hold a known value."""
        import ctypes
        ko = torch.full((93, hkv, d), 7.0, dtype=torch.bfloat16, device=DEV)
        vo = ko.clone()
        desc = pkv.QuantDesc(pool, bs, hkv, d, 1)
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        tb = tables.to(DEV)
        st = pkv.library().pkv_gather_kv_quant(p(ko), p(vo), 1, p(kc), p(vc), ctypes.byref(desc), p(tb), tb.shape[1],
                                               p(ln), p(cu), 3, total, max_len, None)
        assert st == 0
        torch.cuda.synchronize()
        return ko

    def equal(a, b):  # bit for bit (some rows are NaN)
        return torch.equal(a.view(torch.int16), b.view(torch.int16))

    bad = tables.clone()
    bad[1, 1] = pool  # positions 16..31 of sequence 1
    got = call(bad, ln, 40, 93)
    assert pkv.get_device_error() == pkv.DEVERR_BAD_BLOCK_ID
    assert (got[36:52] == 7).all() and equal(got[:36], good[:36]) and equal(got[52:], good[52:])
    got = call(tables, ln, 35, 93)  # sequence 2 is longer than the bound
    assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
    assert equal(got[:88], good[:88]) and (got[88:] == 7).all()
    got = call(tables, ln, 40, 80)  # sequence 2 passes the rows there are
    assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
    assert equal(got[:80], good[:80]) and (got[80:] == 7).all()
    neg = ln.clone()
    neg[0] = -3
    got = call(tables, neg, 40, 93)
    assert pkv.get_device_error() == pkv.DEVERR_BAD_SEQ_LEN
    assert (got[:20] == 7).all() and equal(got[20:], good[20:])
