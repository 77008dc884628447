"""What is measured of the quantised paged cache and of attention with modified scores.

Operators (plain form here; the library's calls where ``own`` is true):

* ``write_read``: new tokens' K and V are quantised into their slots of a paged cache
  (``kv_quantize_and_cache``), then every sequence is read back as contiguous values
  (``gather_kv_quant``);
* ``quant``: attention over a quantised paged cache (``paged_attention_quant``), one query
  token per sequence or several;
* ``scored``: attention over a bf16 or fp8-e4m3 paged cache (``paged_attention_scored``) whose
  scores are capped by a tanh, biased by distance, limited to a window or opened over a prefix.

The layout of a quantised (block, kv head) tile, a run of bytes in ``[num_blocks, Hkv, tile]``:
``bs`` rows of codes (int8: D bytes, code + 128; fp4: D / 2 bytes, two e2m1 codes per byte, the
even element in the low half), 16-byte chunk c of row r stored at position
``c ^ ((r * row_bytes // 128) % (row_bytes // 16))``; fp4: ``bs`` rows of D / 16 e4m3 group
scales; ``bs`` row scales in binary32.
"""
import math

import torch

own = False

CAPACITY = 8 * 32768 * 8 * 128  # elements of one cache (K or V) of the largest case
UNUSED = 0x7FFFFFFF             # table entries past a sequence's last block
TINY = 2.0 ** -80               # rows below this magnitude are stored as zeros


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the four short sequences of the smallest workload: latency of two launches
        dict(name="write_read fp4 tiny", op="write_read", fmt="fp4", src="f32", hkv=4, d=64, bs=16, seqs=4, lo=1, hi=100),
        # a chunked prefill's caches filled and exported
        dict(name="write_read int8 prompts", op="write_read", fmt="int8", src="bf16", hkv=8, d=128, bs=16, seqs=8,
             lo=1024, hi=4096),
        # the long-context batch, every token
        dict(name="write_read fp4 long", op="write_read", fmt="fp4", src="bf16", hkv=8, d=128, bs=16, seqs=8, lo=32768,
             hi=32768),
        # the decode batch of the benchmark on an int8 cache
        dict(name="quant decode int8", op="quant", fmt="int8", hq=32, hkv=8, d=128, bs=16, seqs=64, lo=128, hi=2048,
             t_lo=0, t_hi=0, cap=0.0, alibi=False, window=0, sinks=0, prefix=False),
        # long contexts on a 4-bit cache, where its bytes count most
        dict(name="quant decode fp4 long", op="quant", fmt="fp4", hq=32, hkv=8, d=128, bs=16, seqs=8, lo=32768, hi=32768,
             t_lo=0, t_hi=0, cap=0.0, alibi=False, window=0, sinks=0, prefix=False),
        # speculative verification, four tokens of each sequence
        dict(name="quant verify int8", op="quant", fmt="int8", hq=32, hkv=8, d=128, bs=16, seqs=64, lo=128, hi=2048,
             t_lo=4, t_hi=4, cap=0.0, alibi=False, window=0, sinks=0, prefix=False),
        # a 512-token chunk of a prompt over a 4-bit cache
        dict(name="quant chunk fp4", op="quant", fmt="fp4", hq=32, hkv=8, d=128, bs=16, seqs=8, lo=1024, hi=4096,
             t_lo=512, t_hi=512, cap=0.0, alibi=False, window=0, sinks=0, prefix=False),
        # one request alone: latency
        dict(name="scored decode single", op="scored", fmt="bf16", hq=8, hkv=2, d=64, bs=16, seqs=1, lo=300, hi=300,
             t_lo=0, t_hi=0, cap=30.0, alibi=False, window=0, sinks=0, prefix=False),
        # a layer of a capped model with a sliding window, 128 requests of skewed lengths
        dict(name="scored decode cap window", op="scored", fmt="bf16", hq=64, hkv=8, d=128, bs=16, seqs=128, lo=16,
             hi=8192, t_lo=0, t_hi=0, cap=50.0, alibi=False, window=4096, sinks=0, prefix=False),
        # distance bias, one query head per kv head, odd counts, fp8 cache
        dict(name="scored decode fp8 alibi", op="scored", fmt="fp8", hq=12, hkv=12, d=64, bs=16, seqs=37, lo=100, hi=3001,
             t_lo=0, t_hi=0, cap=0.0, alibi=True, window=0, sinks=0, prefix=False),
        # chunked prefill of a capped model
        dict(name="scored chunk cap", op="scored", fmt="bf16", hq=32, hkv=8, d=128, bs=16, seqs=8, lo=1024, hi=4096,
             t_lo=512, t_hi=512, cap=50.0, alibi=False, window=0, sinks=0, prefix=False),
        # ragged prompts with a prefix all rows see, distance bias and a window; odd group of 7 heads
        dict(name="scored ragged prefix", op="scored", fmt="bf16", hq=14, hkv=2, d=128, bs=32, seqs=5, lo=700, hi=2500,
             t_lo=1, t_hi=699, cap=0.0, alibi=True, window=1000, sinks=4, prefix=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write_read", "quant", "quant", "scored", "scored"])
    d, bs = rng.choice([64, 128]), rng.choice([8, 16, 32])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 8])
    seqs = _log(rng, 1, 128)
    most = max(1, min(32768, CAPACITY // 4 // (seqs * hkv * d)))
    hi = _log(rng, 1, most)
    lo = rng.choice([0, 1, max(1, hi // 16), hi])
    if op == "write_read":
        return dict(op=op, fmt=rng.choice(["int8", "fp4"]), src=rng.choice(["bf16", "f32"]), hkv=hkv, d=d, bs=bs,
                    seqs=seqs, lo=max(1, lo), hi=hi)
    fmt = rng.choice(["int8", "fp4"]) if op == "quant" else rng.choice(["bf16", "bf16", "fp8"])
    if op == "scored":  # the shapes that the library's bf16 and fp8 caches come in
        bs = bs if fmt == "bf16" and d == 128 else 16
    hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    t_lo = t_hi = 0
    if rng.random() < 0.5:
        lo = max(1, lo)
        rows = max(1, (1 << 31) // (seqs * hq * hi * 2))  # scores of the plain form, per row of one sequence
        t_hi = _log(rng, 1, max(1, min(1024, hi, rows)))
        t_lo = rng.choice([1, t_hi])
    return dict(op=op, fmt=fmt, hq=hq, hkv=hkv, d=d, bs=bs, seqs=seqs, lo=lo, hi=hi, t_lo=t_lo, t_hi=t_hi,
                cap=rng.choice([0.0, 30.0, 50.0]), alibi=rng.random() < 0.4,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), sinks=rng.choice([0, 4]),
                prefix=t_hi > 0 and rng.random() < 0.4)


def _spread(n, lo, hi, step):
    """n whole numbers over [lo, hi], the same for every seed (work() needs them); the first is hi."""
    return [hi - int((i * step) % 1.0 * (hi - lo + 1)) for i in range(n)]


def _lens(c):
    return _spread(c["seqs"], c["lo"], c["hi"], 0.6180339887)


def _rows(c):
    """Query tokens of each sequence (one each for decode)."""
    if not c["t_hi"]:
        return [1] * c["seqs"]
    return [min(t, n) for t, n in zip(_spread(c["seqs"], c["t_lo"], c["t_hi"], 0.7548776662), _lens(c))]


def _prefixes(c):
    return [n // 3 for n in _lens(c)] if c["prefix"] else [0] * c["seqs"]


def _tile(fmt, d, bs):
    row = d if fmt == "int8" else d // 2
    return bs * row + (bs * d // 16 if fmt == "fp4" else 0) + 4 * bs


# ------------------------------------------------------------------ work
def _attended(c, n, t, pre):
    """(positions that some row attends, (row, position) pairs attended) of a sequence of n tokens, t rows."""
    w = c["window"] or n
    pairs, lo, low = 0, n, 0
    for i in range(t):
        p = n - t + i
        if p < 0:
            continue
        first = max(0, p + 1 - w)
        always = max(min(c["sinks"] if c["window"] else 0, p + 1), min(pre, n))
        pairs += always + max(0, p + 1 - max(first, always))
        lo, low = min(lo, first), max(low, always)
    return (n if low >= lo else low + n - lo) if n and t else 0, pairs


def work(c):
    lens = _lens(c)
    blocks = sum(-(-n // c["bs"]) for n in lens)
    if c["op"] == "write_read":
        rows = 2 * sum(lens) * c["hkv"]
        e = 4 if c["src"] == "f32" else 2
        rec = _tile(c["fmt"], c["d"], c["bs"]) / c["bs"]
        # source read, records written, values written (in the source's type)
        return {"bytes": rows * (2 * e * c["d"] + rec) + 8 * sum(lens) + 4 * blocks, "flops": rows * c["d"] * 4}
    e = {"bf16": 2 * c["d"], "fp8": c["d"]}.get(c["fmt"]) or _tile(c["fmt"], c["d"], c["bs"]) / c["bs"]
    at = [_attended(c, n, t, p) for n, t, p in zip(lens, _rows(c), _prefixes(c))]
    return {"bytes": 2 * c["hkv"] * e * sum(a for a, _ in at) + 4 * sum(_rows(c)) * c["hq"] * c["d"] + 4 * blocks,
            "flops": max(1, 4 * c["d"] * c["hq"] * sum(p for _, p in at))}


# ------------------------------------------------------------------ the quantised rows, plain
def _quantise_int8(x):
    """Rows [..., D] in binary32 -> (codes + 128 as uint8, row scales)."""
    a = x.abs().amax(-1)
    s = torch.where(a < TINY, torch.zeros_like(a), a / 127)
    bad = ~torch.isfinite(a)
    q = torch.where((s > 0)[..., None] & ~bad[..., None], torch.round(x / s[..., None]), torch.zeros_like(x))
    return (q + 128).to(torch.uint8), torch.where(bad, torch.full_like(s, float("nan")), s)


def _quantise_fp4(x):
    """Rows [..., D] in binary32 -> (codes as uint8 0..15 [..., D], e4m3 group scales [..., D / 16], row scales)."""
    g = x.unflatten(-1, (-1, 16))
    m = g.abs().amax(-1)
    a = m.amax(-1)
    bad = ~torch.isfinite(a)
    s = torch.where((a < TINY) | bad, torch.zeros_like(a), a / 2688)
    u = torch.where((s > 0)[..., None], m / (6 * s)[..., None], torch.zeros_like(m))
    t = u.clamp(max=448.0).to(torch.float8_e4m3fn)
    step = t.to(torch.float32) * s[..., None]
    y = torch.where((step > 0)[..., None], g / step[..., None], torch.zeros_like(g))
    v = y.abs()
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5))
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    return code.flatten(-2), t, torch.where(bad, torch.full_like(s, float("nan")), s)


def _chunk_order(d, bs, fmt, device):
    row = d if fmt == "int8" else d // 2
    r = torch.arange(bs, device=device)[:, None]
    return torch.arange(row // 16, device=device)[None, :] ^ ((r * row // 128) % (row // 16))  # [bs, chunks]


def _tiles(x, fmt):
    """Token rows of whole tiles [n, bs, D] -> records [n, tile] (bytes)."""
    n, bs, d = x.shape
    if fmt == "int8":
        codes, s = _quantise_int8(x)
        parts = [s.contiguous().view(torch.uint8).reshape(n, 4 * bs)]
    else:
        nib, t, s = _quantise_fp4(x)
        codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
        parts = [t.contiguous().view(torch.uint8).reshape(n, -1), s.contiguous().view(torch.uint8).reshape(n, 4 * bs)]
    c = codes.reshape(n, bs, -1, 16)
    order = _chunk_order(d, bs, fmt, x.device)[None, :, :, None].expand_as(c)
    return torch.cat([torch.gather(c, 2, order).reshape(n, -1)] + parts, -1)  # the order is its own inverse


def _values(rec, d, bs, fmt):
    """Records [..., tile] -> values [..., bs, D] in binary32."""
    lead = rec.shape[:-1]
    rec = rec.reshape(-1, rec.shape[-1])
    n, row = rec.shape[0], d if fmt == "int8" else d // 2
    c = rec[:, : bs * row].reshape(n, bs, row // 16, 16)
    c = torch.gather(c, 2, _chunk_order(d, bs, fmt, rec.device)[None, :, :, None].expand_as(c)).reshape(n, bs, row)
    s = rec[:, -4 * bs:].contiguous().view(torch.float32)[..., None]
    if fmt == "int8":
        return ((c.to(torch.float32) - 128) * s).reshape(*lead, bs, d)
    nib = torch.stack([c & 15, c >> 4], -1).reshape(n, bs, d).to(torch.int32)
    mag, exp = (nib & 1).to(torch.float32), (nib >> 1) & 3
    v = torch.where(exp == 0, mag * 0.5, (1 + 0.5 * mag) * torch.exp2((exp - 1).to(torch.float32)))
    v = torch.where(nib >= 8, -v, v)
    t = rec[:, bs * row: bs * row + bs * d // 16].contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    return ((v.unflatten(-1, (-1, 16)) * t.reshape(n, bs, -1, 1)).flatten(-2) * s).reshape(*lead, bs, d)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, spread):
    """N(0, 1) values; `spread` gives a few of the last axis' channels larger magnitudes, as keys have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    if spread:
        x[..., :: 17] *= 4
    return x


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lens, bs, d, hkv = _lens(c), c["bs"], c["d"], c["hkv"]
    nb = [-(-n // bs) for n in lens]
    pool = max(1, sum(nb))
    ids = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    tables = torch.full((len(lens), max(1, max(nb))), UNUSED, dtype=torch.int32)
    at = 0
    ids_host = ids.cpu()
    for i, n in enumerate(nb):
        tables[i, :n] = ids_host[at: at + n]
        at += n
    s = dict(case=dict(c), tables=tables.cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             max_len=max(1, max(lens)))
    if c["op"] == "write_read":
        total = sum(lens)
        dt = torch.float32 if c["src"] == "f32" else torch.bfloat16
        s["k"] = _normal(gen, (total, hkv, d), True).to(dt)
        s["v"] = _normal(gen, (total, hkv, d), False).to(dt)
        slots = torch.empty(total, dtype=torch.int64)
        t64 = tables.to(torch.int64)
        at = 0
        for i, n in enumerate(lens):
            p = torch.arange(n)
            slots[at: at + n] = t64[i, p // bs] * bs + p % bs
            at += n
        s["slots"] = slots.cuda()
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int64, device="cuda")
        s["total"] = total
        s["k_cache"] = torch.zeros((pool, hkv, _tile(c["fmt"], d, bs)), dtype=torch.uint8, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        return s
    rows = _rows(c)
    s["rows"], s["total_q"], s["max_q"] = rows, sum(rows), max(rows)
    s["q"] = _normal(gen, (sum(rows), c["hq"], d), False).to(torch.bfloat16)
    s["out"] = torch.zeros_like(s["q"])
    if c["t_hi"]:
        s["q_start"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device="cuda")
    shape = (pool, hkv, bs, d)
    k, v = _normal(gen, shape, c["op"] == "quant"), _normal(gen, shape, False)
    s["kv_scale"] = 1.0
    if c["op"] == "quant":
        s["k_cache"], s["v_cache"] = (_tiles(x.reshape(-1, bs, d), c["fmt"]).reshape(pool, hkv, -1) for x in (k, v))
    elif c["fmt"] == "fp8":
        s["kv_scale"] = 6.0 / 448
        s["k_cache"], s["v_cache"] = ((x / s["kv_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                                      for x in (k, v))
    else:
        s["k_cache"], s["v_cache"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(d)
    if c["alibi"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["hq"] + 1, device="cuda", dtype=torch.float32) / c["hq"])
    if c["prefix"]:
        s["prefix"] = torch.tensor(_prefixes(c), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ the pass
def run(s):
    c = s["case"]
    if c["op"] == "write_read":
        if own:
            import paged_kv_cache_22_gb300 as pkv
            pkv.kv_quantize_and_cache(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], c["bs"], c["fmt"])
            return pkv.gather_kv_quant(s["k_cache"], s["v_cache"], s["tables"], s["lens"], c["bs"], c["d"], c["fmt"],
                                       s["max_len"], out_dtype=s["k"].dtype, cu_seq_lens=s["cu"], total_tokens=s["total"])
        return tuple(_plain_write_read(s, s[x], s[x + "_cache"]) for x in "kv")
    if own:
        import paged_kv_cache_22_gb300 as pkv
        more = dict(q_start=s.get("q_start"), max_q=s["max_q"] if c["t_hi"] else None, softcap=c["cap"],
                    alibi_slopes=s.get("slopes"), window=c["window"], sinks=c["sinks"], prefix_lens=s.get("prefix"),
                    max_seq_len=s["max_len"])
        if c["op"] == "quant":
            return pkv.paged_attention_quant(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                             s["scale"], c["bs"], c["fmt"], **more)
        return pkv.paged_attention_scored(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                          s["scale"], kv_scale=s["kv_scale"], **more)
    return _plain_attention(s)


def _plain_write_read(s, x, cache):
    c = s["case"]
    bs, d, fmt = c["bs"], c["d"], c["fmt"]
    blk, off = s["slots"] // bs, s["slots"] % bs
    # every token as a one-row tile: its codes, group scales and row scale, then moved to their places
    row = d if fmt == "int8" else d // 2
    flat = _tiles(x.to(torch.float32).reshape(-1, 1, d), fmt).reshape(x.shape[0], c["hkv"], -1)
    chunk = torch.arange(row // 16, device=x.device)
    place = off[:, None] * row + (chunk[None, :] ^ ((off * row // 128) % (row // 16))[:, None]) * 16
    place = (place[:, :, None] + torch.arange(16, device=x.device)).reshape(-1, row)
    parts = [place]
    if fmt == "fp4":
        parts.append(bs * row + off[:, None] * (d // 16) + torch.arange(d // 16, device=x.device))
    parts.append(cache.shape[-1] - 4 * bs + off[:, None] * 4 + torch.arange(4, device=x.device))
    place = torch.cat(parts, 1)[:, None, :]
    head = torch.arange(c["hkv"], device=x.device)[None, :, None]
    cache[blk[:, None, None], head, place] = flat
    # read back, token by token of each sequence
    vals = _values(cache, d, bs, fmt)  # [pool, hkv, bs, d]
    return vals[blk[:, None], torch.arange(c["hkv"], device=x.device)[None, :], off[:, None]].to(x.dtype)


def _plain_kv(s, cache, ids):
    """Values [B, hkv, tokens, d] in binary32 of the blocks `ids` [B, nb]."""
    c = s["case"]
    x = cache[ids]
    if c["op"] == "quant":
        x = _values(x, c["d"], c["bs"], c["fmt"])
    elif c["fmt"] == "fp8":
        x = x.view(torch.float8_e4m3fn).to(torch.float32) * s["kv_scale"]
    else:
        x = x.to(torch.float32)
    return x.transpose(1, 2).flatten(2, 3)  # [B, hkv, nb * bs, d]


def _plain_attention(s):
    c = s["case"]
    B, hkv, g, d = c["seqs"], c["hkv"], c["hq"] // c["hkv"], c["d"]
    dev = s["q"].device
    ids = torch.where(s["tables"] == UNUSED, torch.zeros_like(s["tables"]), s["tables"]).to(torch.int64)
    n = s["lens"].to(torch.int64)
    T = s["max_q"]
    start = s["q_start"][:-1].to(torch.int64) if c["t_hi"] else torch.arange(B, device=dev)
    rows = s["q_start"].diff().to(torch.int64) if c["t_hi"] else torch.ones_like(n)
    i = torch.arange(T, device=dev)
    real = i[None, :] < rows[:, None]
    at = torch.where(real, start[:, None] + i[None, :], torch.zeros_like(real, dtype=torch.int64))
    q = s["q"][at].to(torch.float32).reshape(B, T, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, g * T, d)
    K, V = _plain_kv(s, s["k_cache"], ids), _plain_kv(s, s["v_cache"], ids)
    t = torch.arange(K.shape[2], device=dev)
    pos = n[:, None] - rows[:, None] + i[None, :]                                   # [B, T]
    keep = t[None, None] <= pos[..., None]
    if c["window"]:
        keep &= (t[None, None] > pos[..., None] - c["window"]) | (t < c["sinks"])
    if c["prefix"]:
        keep |= t[None, None] < s["prefix"][:, None, None]
    keep &= t[None, None] < n[:, None, None]
    V = torch.where((t[None] < n[:, None])[:, None, :, None], V, torch.zeros_like(V))
    x = torch.matmul(q, K.transpose(2, 3)).reshape(B, hkv, g, T, -1) * s["scale"]
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    if c["alibi"]:
        far = (pos[..., None] - t[None, None]).abs().to(torch.float32)
        x = x - s["slopes"].reshape(1, hkv, g, 1, 1) * far[:, None, None]
    x = x.masked_fill(~keep[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.reshape(B, hkv, g * T, -1), V).reshape(B, hkv, g, T, d).permute(0, 3, 1, 2, 4)
    s["out"][at[real]] = o.reshape(B, T, c["hq"], d)[real].to(torch.bfloat16)
    return s["out"]


# ------------------------------------------------------------------ in 64 bits
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e4m3(code):
    """e4m3 codes -> values in 64 bits."""
    code = code.to(torch.int64)
    e, m = (code >> 3) & 15, (code & 7).to(torch.float64)
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.to(torch.float64) - 10))
    v = torch.where((code & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(code >= 128, -v, v)


def _exact_token(rec, r, d, bs, fmt):
    """Values in 64 bits of row r[i] of record rec[i, head]: [n, hkv, d]."""
    row = d if fmt == "int8" else d // 2
    j = torch.arange(row, device=rec.device)
    twist = (r * row // 128) % (row // 16)
    at = r[:, None] * row + (((j // 16)[None] ^ twist[:, None]) * 16 + (j % 16)[None])
    codes = torch.gather(rec, 2, at[:, None].expand(-1, rec.shape[1], -1))
    f = rec.shape[2] - 4 * bs + 4 * r[:, None] + torch.arange(4, device=rec.device)
    scale = torch.gather(rec, 2, f[:, None].expand(-1, rec.shape[1], -1)).contiguous().view(torch.float32).to(torch.float64)
    if fmt == "int8":
        return (codes.to(torch.float64) - 128.0) * scale
    look = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float64, device=rec.device)
    v = torch.empty(*codes.shape[:2], d, dtype=torch.float64, device=rec.device)
    v[..., 0::2], v[..., 1::2] = look[(codes % 16).to(torch.int64)], look[(codes // 16).to(torch.int64)]
    f = bs * row + r[:, None] * (d // 16) + torch.arange(d // 16, device=rec.device)
    t = _e4m3(torch.gather(rec, 2, f[:, None].expand(-1, rec.shape[1], -1)))
    return v * t.repeat_interleave(16, 2) * scale


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "write_read":
        return tuple(_exact_stored(s[x], c["fmt"]) for x in "kv")
    lens, rows, pre = _lens(c), _rows(c), _prefixes(c)
    bs, hkv, g, d = c["bs"], c["hkv"], c["hq"] // c["hkv"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, T) in enumerate(zip(lens, rows)):
        if n and T:
            t = torch.arange(n, device="cuda")
            blk = s["tables"][b, t // bs].to(torch.int64)
            kv = []
            for cache in (s["k_cache"], s["v_cache"]):
                if c["op"] == "quant":
                    kv.append(_exact_token(cache[blk], t % bs, d, bs, c["fmt"]))
                elif c["fmt"] == "fp8":
                    kv.append(_e4m3(cache[blk, :, t % bs]) * s["kv_scale"])
                else:
                    kv.append(cache[blk, :, t % bs].to(torch.float64))
            pos = torch.arange(n - T, n, device="cuda")[:, None]
            w = c["window"] or n + 1
            ok = (t[None] <= pos) & ((t[None] > pos - w) | (t[None] < (c["sinks"] if c["window"] else 0)))
            ok |= (t < pre[b])[None]
            for h in range(hkv):
                q = s["q"][at: at + T, h * g: (h + 1) * g].to(torch.float64).transpose(0, 1)       # [g, T, d]
                x = torch.einsum("gtd,nd->gtn", q, kv[0][:, h]) * s["scale"]
                if c["cap"]:
                    x = torch.tanh(x / c["cap"]) * c["cap"]
                if c["alibi"]:
                    x -= s["slopes"][h * g: (h + 1) * g].to(torch.float64)[:, None, None] * (pos - t[None]).abs()
                p = torch.softmax(x.masked_fill(~ok, float("-inf")), -1)
                out[at: at + T, h * g: (h + 1) * g] = torch.einsum("gtn,nd->gtd", p, kv[1][:, h]).transpose(0, 1)
        at += T
    return out


def _exact_stored(x, fmt):
    """What the cache holds of the rows x: the codes come from binary32 divisions, by definition; the values in 64 bits."""
    parts = []
    for y in x.to(torch.float32).split(32768):
        if fmt == "int8":
            s = y.abs().amax(-1, keepdim=True) / 127
            q = torch.nan_to_num(torch.round(y / s))
            parts.append(q.to(torch.float64) * s.to(torch.float64))
            continue
        y = y.reshape(*y.shape[:-1], -1, 16)
        top = y.abs().amax((-1, -2), keepdim=True) / 2688
        u = torch.nan_to_num(y.abs().amax(-1, keepdim=True) / (6 * top)).to(torch.float64)
        e = torch.floor(torch.log2(u.clamp(min=2.0 ** -6))).clamp(max=8) - 3   # e4m3: four significant bits, ties to even
        t = torch.clamp(torch.round(u * torch.exp2(-e)) * torch.exp2(e), max=448.0)
        r = torch.nan_to_num(y / (t.to(torch.float32) * top), posinf=0.0, neginf=0.0).to(torch.float64)
        e = torch.floor(torch.log2(r.abs().clamp(min=1.0))).clamp(max=2) - 1   # e2m1: two significant bits
        v = torch.clamp(torch.round(r * torch.exp2(-e)) * torch.exp2(e), -6.0, 6.0)
        parts.append((v * t * top.to(torch.float64)).reshape(*y.shape[:-2], -1))
    return torch.cat(parts)
