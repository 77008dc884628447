// attn_cols.cuh -- paged attention with modified scores (softcap, distance
// bias, window, prefix) over bf16, fp8-e4m3 and quantised (int8, fp4) caches,
// for one query token per sequence or several (pkv_paged_attention_scored,
// pkv_paged_attention_quant).
//
// For a query row at position p, over the positions t it attends (pkv.h):
//   out = sum_t softmax(z)_t V[t],  z_t = cap(scale * q . K[t]) - slope * |p - t|
// accumulated with an online softmax in base-2 units and split over the keys
// with a log-sum-exp merge of the parts.
//
// The query rows are the COLUMNS of both contractions: S^T = K Q^T has the 16
// tokens of a step as the m16 rows of mma.sync m16n8k16 and 8 (or 16) query
// rows as its columns, O^T += V^T P^T has 16 head dims as rows.  With the
// query rows as the m16 operand instead, a decode of 4 or 8 heads per kv head
// leaves half of every MMA empty; here a tile takes half the MMAs, and the
// accumulators (D x 8 instead of D x 16) and the query fragments half the
// registers, so that more warps fit an SM.
//
//  * Work: (sequence, chunk of NC = 8 NT query rows, kv head) segments of
//    tiles (16 tokens; 32 for blocks of 32), laid end to end and cut into
//    equal ranges, one per one-warp CTA.  A query row is (token, head of the
//    kv head's group), token-major.  A tile no row of the chunk attends is
//    not in the stream.
//  * Tiles land in a ring of shared-memory stages: bf16 and fp8 by tensor
//    copy, quantised tiles (codes, group scales, row scales) by one bulk copy.
//  * K fragments: bf16 through ldmatrix; codes by 16-byte loads, a lane (g, t)
//    = (lane / 4, lane % 4) taking D / 4 consecutive dims of rows g and g + 8,
//    widened exactly to fp16 (e4m3 and e2m1 by conversion, int8 by placing
//    the byte in the mantissa of 1024 and subtracting).  The k order this
//    gives is also q's.  An fp4 group scale (e4m3) multiplies the fp16 code
//    exactly: at most 2 + 4 significant bits.
//  * V fragments: bf16 through ldmatrix.trans; codes by loads of the lane's
//    D / 8 dims of tokens 2t, 2t + 1, 2t + 8, 2t + 9, interleaved by bytes or
//    half bytes.  Row r of m-tile j is then dim (D / 8) g + 2j (r = g) or
//    (D / 8) g + 2j + 1 (r = g + 8).
//  * P^T: a lane's probabilities (token g or g + 8, columns 2t, 2t + 1) become
//    the B operand by one 8x8 transpose (movmatrix) per 8 tokens.
//  * Row scales of a quantised cache never touch the codes.  K's multiplies
//    the score.  V's multiplies the probability before it is rounded to fp16:
//    w = 2^(z + log2(s_v) - m) with m a running maximum of z + log2(s_v), so
//    that the largest weight, not the largest probability, sits near one and
//    scales of any size keep 11 bits; the sum takes the probability w / s_v,
//    in fp32.
//  * bf16 caches: P is a bf16 head plus a bf16 remainder (16 bits, two MMAs);
//    fp8 and quantised caches: one fp16 operand (11 bits).  A weight rounded
//    to 11 bits moves an output by at most 2^-11 max|V|, an eighth of the
//    rounding of the bf16 output.
//  * The maximum is lazy: m moves only when some score passes it by more than
//    2^8, a warp-uniform branch; weights stay below 2^8.
//
// Measured (attention and merge; share of the measured copy bandwidth): bf16,
// 128 sequences of up to 8192 tokens, 64 heads on 8, cap, window: 250 us, 0.97,
// HBM.  Codes are bound by the instructions that widen and multiply them (35-41
// % of issue slots, 8-16 warps per SM): int8, 64 sequences of up to 2048, 32
// heads on 8: 36 us, 0.61 (four tokens each, 16 columns: 51 us, 0.44); fp4, 8
// of 32768: 76 us, 0.63; fp8, D 64, a head per kv head: 28 us, 0.50.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "decode_tc.cuh"
#include "quant_layout.cuh"

namespace pkv {
namespace cols {

enum Kind { kBf16 = 0, kFp8 = 1, kInt8 = 2, kFp4 = 3 };

struct Args {
  unsigned int* err;
  __nv_bfloat16* out;
  const __nv_bfloat16* q;
  const int32_t* q_start;  // null: one row per sequence
  const uint8_t* k_cache;  // quantised caches (the others come through tensor maps)
  const uint8_t* v_cache;
  const int32_t* block_tables;
  int64_t table_stride;
  const int32_t* seq_lens;
  int num_seqs, total_q, max_q, num_q_heads, num_kv_heads, group, num_blocks, len_clip;
  int chunks;       // chunks of NC rows per (sequence, kv head), from max_q
  float qk_scale;   // scale * log2(e) (* kv_scale for fp8 caches)
  float out_scale;  // 1 (kv_scale for fp8 caches)
  float cap;        // softcap * log2(e); 0 = none
  float inv_cap;    // 1 / cap
  const float* slopes;
  const int32_t* prefix_lens;
  int window, sinks;
  int by_length;    // 128-row tiles: the longest sequences first
  float* partials;  // [2 * CTAs][slot_floats(NC, D)]
  struct Cut* cuts; // [CTAs]
};

// A segment cut between warps, described by the warp that ends it (parts 0: none).
struct Cut {
  int parts;              // pieces of the segment, on consecutive warps
  uint32_t slot0, first;  // partial slot of the first piece; its warp
  int row0;               // first query row of q / out of the chunk's sequence
  int r0, rows, head0;    // first row of the chunk, rows of the (sequence, kv head), first query head
  int pad;
};

template <int KIND, int D, int BS>
struct Geo {
  static constexpr bool REC = KIND == kInt8 || KIND == kFp4;  // quantised records
  static constexpr int ROW = KIND == kBf16 ? 2 * D : (KIND == kFp4 ? D / 2 : D);
  static constexpr int IB = ROW >= 128 ? 128 : ROW;  // bytes of a swizzled line part
  static constexpr int CPB = IB / 16;
  // Tokens per tile: 32 for codes (two independent products per step of the
  // loop, and its fixed costs spread over twice the tokens), 16 for bf16, whose
  // tiles are two to four times larger (HBM sets the pace there).
  static constexpr int WANT = KIND == kBf16 ? 16 : 32;
  static constexpr int BPT = BS < WANT ? WANT / BS : 1;  // blocks per tile
  static constexpr int TOK = BS * BPT;               // tokens per tile
  static constexpr int STEPS = TOK / 16;             // m16 rows of tokens per tile
  static constexpr int NI = 2 * STEPS;               // tokens of a tile per lane
  static constexpr int BLOCK = REC ? quant_tile_bytes(D, BS, KIND == kFp4) : BS * ROW;  // one block's bytes of K or V
  static constexpr int CACHE = BPT * BLOCK;
  static constexpr int STAGE = 2 * CACHE;            // K then V
  static constexpr int KS = D / 16;                  // k-steps of q.K
  static constexpr int MT = D / 16;                  // m-tiles of V^T P^T
  // bytes from a token's code row, group scales and row scale to those of the
  // token 8 rows on, and 16 rows on (the next step)
  static constexpr int R8 = BS == 8 ? BLOCK : 8 * IB, R16 = BS == 32 ? 16 * IB : 16 / BS * BLOCK;
  static constexpr int G8 = BS == 8 ? BLOCK : D / 2, G16 = BS == 32 ? D : 16 / BS * BLOCK;
  static constexpr int S8 = BS == 8 ? BLOCK : 32, S16 = BS == 32 ? 64 : 16 / BS * BLOCK;
  static constexpr int DPL = D / 4;                  // codes: dims of a K row per lane
  static constexpr int DL = D / 8;                   // codes: dims of a V row per lane
  // Stages per warp: two (four of the smallest): the other warps of the SM keep
  // the copies going, and shared memory decides how many those are.
  static constexpr int NS = STAGE <= 2560 ? 4 : 2;
  static_assert(REC || STAGE % 1024 == 0, "tensor copies keep the swizzle phase");
};

__host__ __device__ constexpr int slot_floats(int NC, int D) { return NC * D + 2 * NC; }

// A chunk of query rows of a sequence and the tiles its rows attend: tiles
// [0, na) and [wt, nt) (na == wt when nothing is left out).
struct Chunk {
  int L, T, q0;       // length, query tokens, first row of q (and out)
  int r0;             // first row of the chunk within the (sequence, kv head)
  int hi_min, hi_max; // positions + 1 of the chunk's first and last token
  int lo_min;         // first position of the first token's window
  int a_max;          // tokens below it may be attended whatever the window
  int na, wt, nt;
  __device__ __forceinline__ int tiles() const { return nt - (wt - na); }
  __device__ __forceinline__ int tile(int j) const { return j < na ? j : j + (wt - na); }
};

// The chunk `v % chunks` of sequence v / chunks; false (and no tile) when it
// has no row or no position.  Bad lengths are flagged.
template <int NC, int TOK>
__device__ __forceinline__ Chunk chunk_of(const Args& a, int v) {
  Chunk c;
  int s = v, ci = 0;
  if (a.chunks > 1) {
    s = v / a.chunks;
    ci = v % a.chunks;
  }
  c.L = __ldg(a.seq_lens + s);
  const bool bad_len = c.L < 0 || c.L > a.len_clip;
  c.na = c.wt = c.nt = 0;
  c.r0 = ci * NC;
  if (a.q_start) {
    c.q0 = __ldg(a.q_start + s);
    const int64_t T = (int64_t)__ldg(a.q_start + s + 1) - c.q0;
    if (bad_len || T < 0 || T > c.L || T > a.max_q || c.q0 < 0 || c.q0 + T > a.total_q) {
      raise_error(a.err, PKV_DEVERR_BAD_SEQ_LEN);
      c.T = 0;
    } else {
      c.T = (int)T;
    }
  } else {
    if (bad_len) {
      raise_error(a.err, PKV_DEVERR_BAD_SEQ_LEN);
      c.L = c.L < 0 ? 0 : a.len_clip;
    }
    c.q0 = s;
    c.T = 1;
  }
  const int rows = c.T * a.group;
  if (c.r0 >= rows || c.L <= 0) return c;
  const int i0 = c.r0 / a.group, i1 = (min(c.r0 + NC, rows) - 1) / a.group;
  c.hi_min = c.L - c.T + i0 + 1;
  c.hi_max = c.L - c.T + i1 + 1;
  c.lo_min = a.window > 0 ? max(0, c.hi_min - a.window) : 0;
  int pre = a.prefix_lens ? __ldg(a.prefix_lens + s) : 0;
  pre = min(max(pre, 0), c.L);
  c.a_max = max(min(a.sinks, c.hi_max), pre);
  c.nt = (max(c.hi_max, c.a_max) + TOK - 1) / TOK;
  c.na = (c.a_max + TOK - 1) / TOK;
  c.wt = c.lo_min / TOK;
  if (c.wt <= c.na) c.na = c.wt = 0;  // one run
  return c;
}

// What a query row (column) attends: positions [0, a) and [lo, hi).
struct Col {
  int a, lo, hi;
  float slope;  // distance bias, base 2
};

// The stream's T tiles over N warps: the first T % N warps take one more.
// Counts are 32-bit (the host refuses a call whose bound passes 2^31 tiles).
struct Split {
  uint32_t T, per, rem;
  __device__ __forceinline__ Split(uint32_t t, uint32_t n) : T(t), per(t / n), rem(t - t / n * n) {}
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * per + min(w, rem); }
  __device__ __forceinline__ uint32_t owner(uint32_t u) const {
    const uint32_t cut = rem * (per + 1);
    return u < cut ? u / (per + 1) : rem + (u - cut) / per;
  }
};

// Walk over the (chunk, kv head) segments of a range of the tile stream.
struct Walk {
  int v, h;        // chunk index over all sequences, kv head
  Chunk c;
  int nb;          // tiles of the segment
  uint32_t base;   // first tile of chunk v in the stream
  int jb, je;      // piece = tiles [jb, je) of the segment
  bool done;
  __device__ __forceinline__ uint32_t seg() const { return base + (uint32_t)h * nb; }
};

template <int KIND, int D, int BS, int NT>
struct Smem {
  using GE = Geo<KIND, D, BS>;
  static constexpr int kStages = 0;
  static constexpr int kQ = GE::NS * GE::STAGE;                   // [NC][D] bf16: the next piece's query rows
  static constexpr int kBars = (kQ + 8 * NT * D * 2 + 15) / 16 * 16;
  static constexpr int kOk = kBars + 8 * GE::NS;                  // bit b: block b of the stage is there
  static constexpr int kWalks = (kOk + 4 * GE::NS + 15) / 16 * 16;  // this piece's, the next one's, the copies'
  static constexpr int kCols = kWalks + 3 * (int)sizeof(Walk);    // [NC] column limits
  static constexpr int kBytes = kCols + 8 * NT * (int)sizeof(Col);
  // CTAs per SM that shared memory allows (1 KiB of it per CTA is the
  // system's), at most 16: the register budget follows
  static constexpr int kFit = 233472 / (kBytes + 1024);
  static constexpr int kCtas = NT == 2 ? 8 : (kFit > 16 ? 16 : kFit);
};

template <int NC, int TOK>
__device__ __forceinline__ void settle(Walk& w, const Args& a, uint32_t u1) {
  const int vs = a.num_seqs * a.chunks;
  while (!w.done) {
    if (w.nb > 0 && w.h < a.num_kv_heads) {
      const int left = (int)(u1 - w.seg());
      if (left <= 0) {
        w.done = true;
        return;
      }
      w.je = min(left, w.nb);
      if (w.jb < w.je) return;
      w.jb = 0;
      ++w.h;
      continue;
    }
    w.base += (uint32_t)w.nb * a.num_kv_heads;
    w.h = 0;
    w.jb = 0;
    if (++w.v >= vs || w.base >= u1) {
      w.done = true;
      return;
    }
    w.c = chunk_of<NC, TOK>(a, w.v);
    w.nb = w.c.tiles();
  }
}

template <int NC, int TOK>
__device__ __forceinline__ void next_piece(Walk& w, const Args& a, uint32_t u1) {
  if (w.je < w.nb) {  // the range ended inside this segment
    w.done = true;
    return;
  }
  w.jb = 0;
  ++w.h;
  settle<NC, TOK>(w, a, u1);
}

// Tiles of the whole stream (every lane of a warp).
template <int NC, int TOK>
__device__ __forceinline__ uint32_t total_tiles(const Args& a, int lane) {
  const int vs = a.num_seqs * a.chunks;
  uint32_t mine = 0;
  for (int v = lane; v < vs; v += 32) mine += chunk_of<NC, TOK>(a, v).tiles();
  return __reduce_add_sync(0xffffffffu, mine) * a.num_kv_heads;
}

// The walk on the first piece of the range [u0, u1), u0 < u1.
template <int NC, int TOK>
__device__ __forceinline__ Walk walk_from(const Args& a, uint32_t u0, uint32_t u1, int lane) {
  Walk w;
  w.done = true;
  const int vs = a.num_seqs * a.chunks;
  uint32_t run = 0;
  for (int v = 0; v < vs; v += 32) {
    const uint32_t n = v + lane < vs ? (uint32_t)chunk_of<NC, TOK>(a, v + lane).tiles() * a.num_kv_heads : 0;
    uint32_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const uint32_t excl = run + incl - n;
    const unsigned hit = __ballot_sync(0xffffffffu, excl <= u0 && u0 < excl + n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.v = v + src;
      w.base = __shfl_sync(0xffffffffu, excl, src);
      w.c = chunk_of<NC, TOK>(a, w.v);
      w.nb = w.c.tiles();
      const uint32_t off = u0 - w.base;
      w.h = (int)(off / (uint32_t)w.nb);
      w.jb = (int)(off - (uint32_t)w.h * w.nb);
      w.done = false;
      settle<NC, TOK>(w, a, u1);
      return w;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  return w;
}

// The partial slot of a cut piece: two per warp, the first for a piece that
// starts the warp's range, the second for a later one.
template <int NC, int D>
__device__ __forceinline__ float* slot_of(const Args& a, const Walk& w, uint32_t gw, uint32_t u0) {
  const uint32_t k = w.seg() + w.jb == u0 ? 2 * gw : 2 * gw + 1;
  return a.partials + (size_t)k * slot_floats(NC, D);
}

// ----------------------------------------------------------------------------
// Element conversions.
// ----------------------------------------------------------------------------
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four int8 codes (+ 128) -> two exact fp16 pairs: 0x6400 | u is 1024 + u.
__device__ __forceinline__ void i8x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = hadd2(__byte_perm(w, 0x64646464u, 0x4140), 0xE480E480u);  // - 1152
  hi = hadd2(__byte_perm(w, 0x64646464u, 0x4342), 0xE480E480u);
}
// Eight e2m1 codes -> four exact fp16 pairs, one per byte (low half first).
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t (&f)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
      : "r"(w));
}
// Two e4m3 codes (low 16 bits) -> an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap * tanh(x / cap), x and cap in base-2 units.  tanh(u) = 1 - 2 / (1 + e^2u)
// loses what u has below 2^-23 of one, so small |u| take the odd series to
// u^7 (next term 62/2835 u^9: below 2^-20 of u at the border 1/4).
__device__ __forceinline__ float soft_cap(float x, float cap, float inv_cap) {
  const float u = x * inv_cap;
  const float u2 = u * u;
  const float small = u * fmaf(u2, fmaf(u2, fmaf(u2, -0.05396825397f, 0.13333333333f), -0.33333333333f), 1.f);
  const float e = fast_exp2(u * 2.885390081777927f);  // e^2u
  const float big = fmaf(-2.f, fast_rcp(1.f + e), 1.f);
  return cap * (fabsf(u) < 0.25f ? small : big);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// log2 of the smallest row scale a stored row can have is above this (a zero
// row has scale 0; its codes are 0 too, so any weight will do).
constexpr float kMinLogScale = -96.f;
constexpr float kSlack = 8.f;  // a score may pass the running maximum by this (base 2)

// ----------------------------------------------------------------------------
// The kernel: one warp per CTA.
// ----------------------------------------------------------------------------
template <int KIND, int D, int BS, int NT>
__global__ void __launch_bounds__(32, Smem<KIND, D, BS, NT>::kCtas)
    attn_cols_kernel(const __grid_constant__ Args a, const __grid_constant__ TmaMaps maps) {
  using GE = Geo<KIND, D, BS>;
  using SM = Smem<KIND, D, BS, NT>;
  constexpr int NC = 8 * NT, TOK = GE::TOK, NS = GE::NS, KS = GE::KS, MT = GE::MT;
  constexpr bool REC = GE::REC, BF = KIND == kBf16;
  extern __shared__ __align__(1024) uint8_t cols_smem[];
  uint8_t* const smem = cols_smem;
  const int lane = threadIdx.x, g = lane >> 2, t = lane & 3;
  const uint32_t smem_s = smem_addr(smem);
  if (!REC && (smem_s & 1023u)) {
    if (lane == 0) raise_error(a.err, PKV_DEVERR_SMEM_ALIGN);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SM::kBars);
  uint32_t* stage_ok = reinterpret_cast<uint32_t*>(smem + SM::kOk);
  // a dependent merge grid may start its own planning now; it waits for this
  // grid to finish before it reads a partial
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NS; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  __syncwarp();

  const uint32_t gw = blockIdx.x, NW = gridDim.x;
  // decode rows of empty sequences are zero
  if (!a.q_start) {
    for (uint32_t s = gw; s < (uint32_t)a.num_seqs; s += NW) {
      if (__ldg(a.seq_lens + s) > 0 && a.len_clip > 0) continue;
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)s * a.num_q_heads * D);
      for (int i = lane; i < a.num_q_heads * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
    }
  }
  const Split split(total_tiles<NC, TOK>(a, lane), NW);
  const uint32_t u0 = split.start(gw), u1 = split.start(gw + 1);
  if (u0 >= u1) {
    if (lane == 0) a.cuts[gw].parts = 0;
    return;
  }
  // The walks live in shared memory (every lane would hold the same words of
  // them in registers): [0] and [1] the piece in work and the next, [2] the
  // piece being copied.
  Walk* const walks = reinterpret_cast<Walk*>(smem + SM::kWalks);
  Col* const col_s = reinterpret_cast<Col*>(smem + SM::kCols);
  {
    const Walk w = walk_from<NC, TOK>(a, u0, u1, lane);
    if (lane == 0) {
      walks[0] = walks[2] = w;
      // a range that starts inside a segment and reaches its end: this warp
      // leaves the merge grid the segment's description
      Cut c{};
      if (w.jb > 0 && w.seg() + w.nb <= u1) {
        c.first = split.owner(w.seg());
        c.parts = (int)(gw - c.first + 1);
        c.slot0 = w.seg() != split.start(c.first) ? 2 * c.first + 1 : 2 * c.first;
        c.row0 = w.c.q0;
        c.r0 = w.c.r0;
        c.rows = w.c.T * a.group;
        c.head0 = w.h * a.group;
      }
      a.cuts[gw] = c;
    }
  }
  __syncwarp();

  // ---------------------------------------------------------------- issue side
  const Walk& cw = walks[2];
  int cj = cw.jb, issued = 0;
  bool more = true;  // tiles left to copy
  // id of block b of the j-th tile of the walk's segment; kNoBlock where a tile
  // of several blocks has one that no row attends (its entry may hold anything)
  constexpr int32_t kNoBlock = INT32_MIN;
  const int32_t* table;
  auto set_table = [&]() { table = a.block_tables + (size_t)(a.chunks > 1 ? cw.v / a.chunks : cw.v) * a.table_stride; };
  auto block_id = [&](int j, int b) -> int32_t {
    const int e = cw.c.tile(j) * GE::BPT + b;
    if (GE::BPT > 1 && e * BS >= cw.c.a_max && (e * BS >= cw.c.hi_max || (e + 1) * BS <= cw.c.lo_min)) return kNoBlock;
    return __ldg(table + e);
  };
  set_table();
  int32_t next_id[GE::BPT];
#pragma unroll
  for (int b = 0; b < GE::BPT; ++b) next_id[b] = block_id(cj, b);
  auto issue_next = [&]() {
    if (!more) return;
    const int st = issued % NS;
    uint8_t* dst = smem + st * GE::STAGE;
    uint32_t ok = 0;
#pragma unroll
    for (int b = 0; b < GE::BPT; ++b)
      if (next_id[b] >= 0 && next_id[b] < a.num_blocks) ok |= 1u << b;
    if (elect_one()) {
      const int h = cw.h;
#pragma unroll
      for (int b = 0; b < GE::BPT; ++b)
        if (!(ok >> b & 1) && next_id[b] != kNoBlock) raise_error(a.err, PKV_DEVERR_BAD_BLOCK_ID);
      stage_ok[st] = ok;
      mbar_arrive_expect_tx(&bars[st], (uint32_t)(__popc(ok) * 2 * GE::BLOCK));
#pragma unroll
      for (int b = 0; b < GE::BPT; ++b) {
        if (!(ok >> b & 1)) continue;
        uint8_t* kd = dst + b * GE::BLOCK;
        uint8_t* vd = kd + GE::CACHE;
        if constexpr (REC) {
          const size_t off = ((size_t)next_id[b] * a.num_kv_heads + h) * GE::BLOCK;
          bulk_g2s(kd, a.k_cache + off, GE::BLOCK, &bars[st]);
          bulk_g2s(vd, a.v_cache + off, GE::BLOCK, &bars[st]);
        } else if constexpr (GE::ROW > GE::IB) {
          tma_load_4d(kd, &maps.k, 0, h * BS, 0, next_id[b], &bars[st]);
          tma_load_4d(vd, &maps.v, 0, h * BS, 0, next_id[b], &bars[st]);
        } else {
          tma_load_3d(kd, &maps.k, 0, h * BS, next_id[b], &bars[st]);
          tma_load_3d(vd, &maps.v, 0, h * BS, next_id[b], &bars[st]);
        }
      }
    }
    __syncwarp();
    ++issued;
    if (++cj >= cw.je) {
      Walk w = cw;
      next_piece<NC, TOK>(w, a, u1);
      __syncwarp();
      if (lane == 0) walks[2] = w;
      __syncwarp();
      cj = w.jb;
      more = !w.done;
      if (more) set_table();
    }
    if (more) {
#pragma unroll
      for (int b = 0; b < GE::BPT; ++b) next_id[b] = block_id(cj, b);
    }
  };
  // the query rows of a chunk (16 bytes per lane and copy)
  auto issue_q = [&](const Walk& w) {
    const int rows = w.c.T * a.group;
#pragma unroll
    for (int i = lane; i < NC * (D / 8); i += 32) {
      const int col = i / (D / 8), r = w.c.r0 + col;
      if (r < rows) {
        const int64_t row = ((int64_t)w.c.q0 + r / a.group) * a.num_q_heads + w.h * a.group + r % a.group;
        cp_async16(smem + SM::kQ + (col * (D / 8) + i % (D / 8)) * 16, a.q + row * D + (i % (D / 8)) * 8);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  issue_q(walks[0]);
#pragma unroll 1
  for (int i = 0; i < NS; ++i) issue_next();

  // ---------------------------------------------------------------- fragment offsets
  // Byte offset in a cache's tile of 16-byte chunk c of row r (of the first step).
  auto chunk_at = [](int r, int c) -> uint32_t {
    const int rb = r % BS;
    return (uint32_t)((r / BS) * GE::BLOCK + (c / GE::CPB) * (BS * GE::IB) + rb * GE::IB +
                      (((c % GE::CPB) ^ ((rb * GE::IB / 128) & (GE::CPB - 1))) << 4));
  };
  // What a lane reads of a stage, as offsets kept over the whole range; the
  // rows 8 and 16 further on are constants away (the swizzle repeats).
  uint32_t kx, vx, vx1 = 0, kg = 0, vg = 0;
  if constexpr (BF) {
    // ldmatrix rows; chunk 2k + (lane's half): the even part is XORed in
    kx = chunk_at((lane & 7) + 8 * ((lane >> 3) & 1), lane >> 4);
    vx = GE::CACHE + chunk_at((lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1);
  } else {
    constexpr int CB = KIND == kFp4 ? GE::DPL / 2 : GE::DPL, VB = KIND == kFp4 ? GE::DL / 2 : GE::DL;
    kx = chunk_at(g, CB * t / 16) + CB * t % 16;
    vx = GE::CACHE + chunk_at(2 * t, VB * g / 16) + VB * g % 16;
    vx1 = GE::CACHE + chunk_at(2 * t + 1, VB * g / 16) + VB * g % 16;
    if constexpr (KIND == kFp4) {
      kg = BS * GE::ROW + g * (D / 16) + GE::DPL / 16 * t;
      vg = GE::CACHE + BS * GE::ROW + 2 * t * (D / 16) + g * GE::DL / 16;
    }
  }
  const uint32_t rx = GE::BLOCK - 4 * BS + 4 * g;  // row scale of token g

  int consumed = 0, waited = 0, piece = 0;  // (piece: its walk's slot)
  bool alive = true;

#pragma unroll 1
  for (bool last = false; !last; ++piece) {
    const Walk& wk = walks[piece & 1];
    // ---- the piece's query fragments and per-column limits
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    const int rows = wk.c.T * a.group;
    uint32_t qb[NT][KS][2];
    float2 qmul[NT];  // score units of columns 2t, 2t + 1
    {
      const uint8_t* qs = smem + SM::kQ;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int col = 8 * n + g;
        const bool have = wk.c.r0 + col < rows;
        const uint8_t* qr = qs + col * D * 2;
        if constexpr (BF) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qb[n][k][0] = have ? *reinterpret_cast<const uint32_t*>(qr + (16 * k + 2 * t) * 2) : 0u;
            qb[n][k][1] = have ? *reinterpret_cast<const uint32_t*>(qr + (16 * k + 2 * t + 8) * 2) : 0u;
          }
          qmul[n] = make_float2(a.qk_scale, a.qk_scale);
        } else {
          // fp16, each column scaled by a power of two that brings its
          // largest |q| into [2^14, 2^15); the factor goes to the score
          uint32_t raw[KS][2];
          uint32_t mx = 0;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint2 v = have ? *reinterpret_cast<const uint2*>(qr + (GE::DPL * t + 4 * k) * 2) : make_uint2(0, 0);
            raw[k][0] = v.x;
            raw[k][1] = v.y;
            mx = __vmaxu2(mx, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu));
          }
          mx = max(mx & 0xFFFFu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // exponent field e of the largest: shift by 14 - (e - 127); a zero
          // or subnormal row, an infinity and a NaN keep a shift in range
          const int e = min(max((int)(mx >> 7), 20), 254);
          const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
          const float down = a.qk_scale * __uint_as_float((uint32_t)(e - 14) << 23);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 f = bf16x2_to_f2(raw[k][i]);
              qb[n][k][i] = pack_f16x2(f.x * up, f.y * up);
            }
          }
          qmul[n].x = __shfl_sync(0xffffffffu, down, 8 * t);
          qmul[n].y = __shfl_sync(0xffffffffu, down, 8 * t + 4);
        }
      }
    }
    if (lane < NC) {  // rows past the last take the last's limits (their results are dropped)
      const int r = min(wk.c.r0 + lane, rows - 1);
      const int hi = wk.c.L - wk.c.T + r / a.group + 1;
      const int pre = a.prefix_lens ? min(__ldg(a.prefix_lens + wk.v / a.chunks), wk.c.L) : 0;
      Col c;
      c.hi = hi;
      c.lo = a.window > 0 ? max(0, hi - a.window) : 0;
      c.a = max(min(a.sinks, hi), pre);
      c.slope = a.slopes ? __ldg(a.slopes + wk.h * a.group + r % a.group) * 1.4426950408889634f : 0.f;
      col_s[lane] = c;
    }
    {  // the next piece's query rows while this one runs
      Walk nx = wk;
      next_piece<NC, TOK>(nx, a, u1);
      last = nx.done;
      if (lane == 0) walks[(piece + 1) & 1] = nx;
      __syncwarp();
      if (!last) issue_q(nx);
    }
    const int jb = wk.jb, je = wk.je, L = wk.c.L, na = wk.c.na, gap = wk.c.wt - wk.c.na;

    // positions every column attends / some column attends (in the window)
    const int all_lo = a.window > 0 ? max(0, wk.c.hi_max - a.window) : 0, all_hi = wk.c.hi_min;

    float o[NT][MT][4];
    float2 m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < MT; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = make_float2(-CUDART_INF_F, -CUDART_INF_F);
      l[n] = make_float2(0.f, 0.f);
    }

#pragma unroll 1
    for (int j = jb; j < je; ++j) {
      const int st = consumed % NS;
      bool ok = false;
      if (alive && consumed < issued) {
        ok = mbar_wait_bounded(&bars[st], (consumed / NS) & 1, a.err);
        waited = consumed + 1;
        if (!ok) alive = false;
      }
      const int tb = (j < na ? j : j + gap) * TOK;  // first position of the tile
      // positions of the tile that exist and were copied, one bit each
      uint32_t there = low_bits(L - tb < TOK ? L - tb : TOK);
      const uint32_t blocks = ok ? stage_ok[st] : 0u;
#pragma unroll
      for (int b = 0; b < GE::BPT; ++b)
        if (!(blocks >> b & 1)) there &= ~(low_bits(BS) << (b * (BS & 31)));
      const bool inner = there == low_bits(TOK) && tb >= all_lo && tb + TOK <= all_hi;

      // ---- S^T = K Q^T per step of 16 tokens; two chains of k-steps where
      // there is one step
      constexpr int STEPS = GE::STEPS, CH = STEPS == 1 ? 2 : 1, NI = GE::NI;
      const uint32_t stage = smem_s + st * GE::STAGE;
      float s2[STEPS][CH][NT][4];
#pragma unroll
      for (int step = 0; step < STEPS; ++step) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int n = 0; n < NT; ++n) s2[step][c][n][0] = s2[step][c][n][1] = s2[step][c][n][2] = s2[step][c][n][3] = 0.f;
        if constexpr (BF) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            uint32_t r[4];
            ldsm_x4(((stage + kx) ^ (uint32_t)(2 * k % GE::CPB << 4)) + step * GE::R16 + 2 * k / GE::CPB * (BS * GE::IB), r);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_k16_rows16<false>(s2[step][k % CH][n], r[0], r[1], r[2], r[3], qb[n][k][0], qb[n][k][1]);
          }
        } else {
          constexpr int CB = KIND == kFp4 ? GE::DPL / 2 : GE::DPL;  // code bytes of a row per lane: 8, 16 or 32
          uint32_t kw[2][CB / 4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = stage + kx + step * GE::R16 + i * GE::R8;
            if constexpr (CB >= 16) {
#pragma unroll
              for (int c = 0; c < CB / 16; ++c) {  // (the lane's second chunk is its first one's neighbour)
                const uint4 v = lds128(c ? ((stage + step * GE::R16 + i * GE::R8) + (kx ^ 16u)) : at);
                kw[i][4 * c] = v.x; kw[i][4 * c + 1] = v.y; kw[i][4 * c + 2] = v.z; kw[i][4 * c + 3] = v.w;
              }
            } else {
              const uint2 v = lds64(at);
              kw[i][0] = v.x; kw[i][1] = v.y;
            }
          }
          if constexpr (KIND == kFp4) {
            constexpr int GPL = GE::DPL / 16;  // groups of a row per lane: 2 or 1
            uint32_t gs[2][GPL];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t at = stage + kg + step * GE::G16 + i * GE::G8;
              const uint32_t two = e4m3x2_to_f16x2(GPL == 2 ? lds16(at) : lds8(at));
              gs[i][0] = __byte_perm(two, 0, 0x1010);
              if constexpr (GPL == 2) gs[i][1] = __byte_perm(two, 0, 0x3232);
            }
#pragma unroll
            for (int w = 0; w < CB / 4; ++w) {
              uint32_t f0[4], f1[4];
              e2m1x8_to_f16x2x4(kw[0][w], f0);
              e2m1x8_to_f16x2x4(kw[1][w], f1);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f0[e] = hmul2(f0[e], gs[0][w / 2]);
                f1[e] = hmul2(f1[e], gs[1][w / 2]);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_k16_rows16<true>(s2[step][h % CH][n], f0[2 * h], f1[2 * h], f0[2 * h + 1], f1[2 * h + 1],
                                       qb[n][2 * w + h][0], qb[n][2 * w + h][1]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t a0, a1, a2, a3;
              if constexpr (KIND == kFp8) {
                e4m3x4_to_f16x2x2(kw[0][k], a0, a2);
                e4m3x4_to_f16x2x2(kw[1][k], a1, a3);
              } else {
                i8x4_to_f16x2x2(kw[0][k], a0, a2);
                i8x4_to_f16x2x2(kw[1][k], a1, a3);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_k16_rows16<true>(s2[step][k % CH][n], a0, a1, a2, a3, qb[n][k][0], qb[n][k][1]);
            }
          }
        }
      }

      // ---- scores of tokens g + 8 i, column pairs (2t, 2t + 1): z (base 2),
      // log2 of V's row scale, its inverse
      float ksc[NI], vlg[NI], vis[NI];
      if constexpr (REC) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const uint32_t at = stage + rx + i / 2 * GE::S16 + i % 2 * GE::S8;
          ksc[i] = __uint_as_float(lds32(at));
          const float lg = fast_log2(__uint_as_float(lds32(at + GE::CACHE)));
          vlg[i] = lg < kMinLogScale ? kMinLogScale : lg;  // (a NaN scale stays NaN)
          vis[i] = fast_exp2(-vlg[i]);
        }
      }
      float2 z[NI][NT];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int k = 2 * (i % 2);
          float2 x = make_float2(s2[i / 2][0][n][k], s2[i / 2][0][n][k + 1]);
          if constexpr (CH == 2) x = __fadd2_rn(x, make_float2(s2[i / 2][CH - 1][n][k], s2[i / 2][CH - 1][n][k + 1]));
          x = __fmul2_rn(x, qmul[n]);
          if constexpr (REC) x = __fmul2_rn(x, make_float2(ksc[i], ksc[i]));
          z[i][n] = x;
        }
      if (a.cap > 0.f) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            z[i][n] = make_float2(soft_cap(z[i][n].x, a.cap, a.inv_cap), soft_cap(z[i][n].y, a.cap, a.inv_cap));
      }
      if (a.slopes) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const Col c0 = col_s[8 * n + 2 * t], c1 = col_s[8 * n + 2 * t + 1];
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int pos = tb + g + 8 * i + 1;
            z[i][n].x = fmaf(-c0.slope, fabsf((float)(c0.hi - pos)), z[i][n].x);
            z[i][n].y = fmaf(-c1.slope, fabsf((float)(c1.hi - pos)), z[i][n].y);
          }
        }
      }
      if constexpr (REC) {  // z + log2(s_v): what the weight is a power of
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) z[i][n] = __fadd2_rn(z[i][n], make_float2(vlg[i], vlg[i]));
      }
      if (!inner) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const Col c0 = col_s[8 * n + 2 * t], c1 = col_s[8 * n + 2 * t + 1];
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int tk = g + 8 * i, pos = tb + tk;
            const bool have = there >> tk & 1;
            z[i][n].x = have && (pos < c0.a || (pos >= c0.lo && pos < c0.hi)) ? z[i][n].x : -CUDART_INF_F;
            z[i][n].y = have && (pos < c1.a || (pos >= c1.lo && pos < c1.hi)) ? z[i][n].y : -CUDART_INF_F;
          }
        }
        if constexpr (REC) {
#pragma unroll
          for (int i = 0; i < NI; ++i) vis[i] = vis[i] < CUDART_INF_F ? vis[i] : 1.f;  // beside a masked scale that is no number
        }
      }
      bool grow = false;
      float2 mx[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mx[n] = z[0][n];
#pragma unroll
        for (int i = 1; i < NI; ++i) mx[n] = make_float2(fmaxf(mx[n].x, z[i][n].x), fmaxf(mx[n].y, z[i][n].y));
        grow = grow || mx[n].x > m[n].x + kSlack || mx[n].y > m[n].y + kSlack;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int sh = 4; sh <= 16; sh <<= 1) {
            mx[n].x = fmaxf(mx[n].x, __shfl_xor_sync(0xffffffffu, mx[n].x, sh));
            mx[n].y = fmaxf(mx[n].y, __shfl_xor_sync(0xffffffffu, mx[n].y, sh));
          }
          const float2 mn = make_float2(fmaxf(m[n].x, mx[n].x), fmaxf(m[n].y, mx[n].y));
          const float2 alpha = make_float2(mn.x > m[n].x ? fast_exp2(m[n].x - mn.x) : 1.f,
                                           mn.y > m[n].y ? fast_exp2(m[n].y - mn.y) : 1.f);
          m[n] = mn;
          l[n] = __fmul2_rn(l[n], alpha);
#pragma unroll
          for (int jm = 0; jm < MT; ++jm) {
            o[n][jm][0] *= alpha.x; o[n][jm][1] *= alpha.y;
            o[n][jm][2] *= alpha.x; o[n][jm][3] *= alpha.y;
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 nm = make_float2(m[n].x == -CUDART_INF_F ? 0.f : -m[n].x, m[n].y == -CUDART_INF_F ? 0.f : -m[n].y);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const float2 d = __fadd2_rn(z[i][n], nm);
          z[i][n] = make_float2(fast_exp2(d.x), fast_exp2(d.y));  // the weight; the probability is the weight / s_v
          l[n] = REC ? ffma2(z[i][n], make_float2(vis[i], vis[i]), l[n]) : __fadd2_rn(l[n], z[i][n]);
        }
      }

      // rows of V that no column attends may hold anything: they become zero
      // (0 * NaN is NaN)
      uint32_t vkeep = 0xFFFFFFFFu;  // bit k: token k of the tile
      if (!inner) vkeep = there & (low_bits(wk.c.a_max - tb) | (low_bits(wk.c.hi_max - tb) & ~low_bits(wk.c.lo_min - tb)));

#pragma unroll
      for (int step = 0; step < STEPS; ++step) {
        // ---- P^T as the B operand: columns = query rows, k = tokens
        uint32_t pb[NT][2], pr[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 w = z[2 * step + i][n];
            const uint32_t h = BF ? pack_bf16x2(w.x, w.y) : pack_f16x2(w.x, w.y);
            pb[n][i] = movmatrix_t(h);
            if constexpr (BF) {
              const float2 f = bf16x2_to_f2(h);
              pr[n][i] = movmatrix_t(pack_bf16x2(w.x - f.x, w.y - f.y));
            }
          }

        // ---- O^T += V^T P^T
        auto kept = [&](int tk) -> bool { return vkeep >> (16 * step + tk) & 1; };
        if constexpr (BF) {
          const uint32_t k0 = (kept(2 * t) ? 0xFFFFu : 0u) | (kept(2 * t + 1) ? 0xFFFF0000u : 0u);
          const uint32_t k1 = (kept(2 * t + 8) ? 0xFFFFu : 0u) | (kept(2 * t + 9) ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int jm = 0; jm < MT; ++jm) {
            uint32_t r[4];
            ldsm_x4_t(((stage + vx) ^ (uint32_t)(2 * jm % GE::CPB << 4)) + step * GE::R16 + 2 * jm / GE::CPB * (BS * GE::IB), r);
            if (!inner) {
              r[0] &= k0; r[1] &= k0; r[2] &= k1; r[3] &= k1;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_k16_rows16<false>(o[n][jm], r[0], r[1], r[2], r[3], pb[n][0], pb[n][1]);
              mma_k16_rows16<false>(o[n][jm], r[0], r[1], r[2], r[3], pr[n][0], pr[n][1]);
            }
          }
        } else {
          // the lane's dims of tokens 2t, 2t + 1, 2t + 8, 2t + 9
          constexpr int VB = KIND == kFp4 ? GE::DL / 2 : GE::DL, W = VB / 4;
          uint32_t X[4][W];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = stage + (i % 2 ? vx1 : vx) + step * GE::R16 + i / 2 * GE::R8;
            if constexpr (W == 4) {
              const uint4 v = lds128(at);
              X[i][0] = v.x; X[i][1] = v.y; X[i][2] = v.z; X[i][3] = v.w;
            } else if constexpr (W == 2) {
              const uint2 v = lds64(at);
              X[i][0] = v.x; X[i][1] = v.y;
            } else {
              X[i][0] = lds32(at);
            }
          }
          if constexpr (KIND == kFp4) {
            uint32_t gv[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint32_t at = stage + vg + step * GE::G16 + p * GE::G8;
              uint32_t s0 = lds8(at), s1 = lds8(at + D / 16);
              if (!inner) {  // an unwritten scale may be NaN
                s0 = kept(2 * t + 8 * p) ? s0 : 0u;
                s1 = kept(2 * t + 8 * p + 1) ? s1 : 0u;
              }
              gv[p] = e4m3x2_to_f16x2(s0 | s1 << 8);
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
              // half byte k of a row's word is dim 8w + k: pair the tokens
              uint32_t ev[2][4], od[2][4];  // [token pair][byte]: even dims, odd dims
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t x0 = X[2 * p][w], x1 = X[2 * p + 1][w];
                e2m1x8_to_f16x2x4((x0 & 0x0F0F0F0Fu) | (x1 << 4 & 0xF0F0F0F0u), ev[p]);
                e2m1x8_to_f16x2x4((x0 >> 4 & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u), od[p]);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  ev[p][b] = hmul2(ev[p][b], gv[p]);
                  od[p][b] = hmul2(od[p][b], gv[p]);
                }
              }
#pragma unroll
              for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_k16_rows16<true>(o[n][4 * w + b], ev[0][b], od[0][b], ev[1][b], od[1][b], pb[n][0], pb[n][1]);
            }
          } else {
            if constexpr (KIND == kFp8) {
              if (!inner) {  // an unwritten code may be NaN (int8 codes are numbers)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                  for (int w = 0; w < W; ++w) X[i][w] = kept(2 * t + 8 * (i / 2) + i % 2) ? X[i][w] : 0u;
              }
            }
#pragma unroll
            for (int w = 0; w < W; ++w) {
              // byte k of a row's word is dim 4w + k: pair the tokens, then widen
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7362 : 0x5140;
                const uint32_t p0 = __byte_perm(X[0][w], X[1][w], sel), p1 = __byte_perm(X[2][w], X[3][w], sel);
                uint32_t a0, a1, a2, a3;
                if constexpr (KIND == kFp8) {
                  e4m3x4_to_f16x2x2(p0, a0, a1);
                  e4m3x4_to_f16x2x2(p1, a2, a3);
                } else {
                  i8x4_to_f16x2x2(p0, a0, a1);
                  i8x4_to_f16x2x2(p1, a2, a3);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                  mma_k16_rows16<true>(o[n][2 * w + h], a0, a1, a2, a3, pb[n][0], pb[n][1]);
              }
            }
          }
        }
      }
      __syncwarp();  // every lane is done with this stage before it is refilled
      ++consumed;
      if (alive) issue_next();
    }

    // ------------------------------------------------------------ piece end
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int sh = 4; sh <= 16; sh <<= 1) {
        l[n].x += __shfl_xor_sync(0xffffffffu, l[n].x, sh);
        l[n].y += __shfl_xor_sync(0xffffffffu, l[n].y, sh);
      }
    if (jb == 0 && je == wk.nb) {
      // the whole segment: the output rows
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float inv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) inv[e] = (e ? l[n].y : l[n].x) == 0.f ? 0.f : a.out_scale / (e ? l[n].y : l[n].x);
        auto out_row = [&](int col) -> __nv_bfloat16* {
          const int r = wk.c.r0 + col;
          return a.out + (((int64_t)wk.c.q0 + r / a.group) * a.num_q_heads + wk.h * a.group + r % a.group) * D;
        };
        if constexpr (BF) {
          // m-tile j, row half i: (dim, columns 2t, 2t + 1) -> (column g, dims 2t, 2t + 1)
          const bool have = wk.c.r0 + 8 * n + g < rows;
          __nv_bfloat16* dst = have ? out_row(8 * n + g) : nullptr;
#pragma unroll
          for (int jm = 0; jm < MT; ++jm)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t v = movmatrix_t(pack_bf16x2(o[n][jm][2 * i] * inv[0], o[n][jm][2 * i + 1] * inv[1]));
              if (have) *reinterpret_cast<uint32_t*>(dst + 16 * jm + 8 * i + 2 * t) = v;
            }
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (wk.c.r0 + 8 * n + 2 * t + e < rows) {
              __nv_bfloat16* dst = out_row(8 * n + 2 * t + e) + GE::DL * g;
              uint32_t pk[MT];
#pragma unroll
              for (int jm = 0; jm < MT; ++jm) pk[jm] = pack_bf16x2(o[n][jm][e] * inv[e], o[n][jm][2 + e] * inv[e]);
#pragma unroll
              for (int w = 0; w < MT; w += 4)
                *reinterpret_cast<uint4*>(dst + 2 * w) = make_uint4(pk[w], pk[w + 1], pk[w + 2], pk[w + 3]);
            }
          }
        }
      }
    } else {
      // cut between warps: the unnormalised part, for the merge grid
      float* ps = slot_of<NC, D>(a, wk, gw, u0);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = 8 * n + 2 * t + e;
          if constexpr (BF) {
#pragma unroll
            for (int jm = 0; jm < MT; ++jm) {
              ps[col * D + 16 * jm + g] = o[n][jm][e];
              ps[col * D + 16 * jm + 8 + g] = o[n][jm][2 + e];
            }
          } else {
#pragma unroll
            for (int jm = 0; jm < MT; jm += 2)
              *reinterpret_cast<float4*>(ps + col * D + GE::DL * g + 2 * jm) =
                  make_float4(o[n][jm][e], o[n][jm][2 + e], o[n][jm + 1][e], o[n][jm + 1][2 + e]);
          }
          if (g == 0) {
            ps[NC * D + col] = e ? m[n].y : m[n].x;
            ps[NC * D + NC + col] = e ? l[n].y : l[n].x;
          }
        }
    }
    __syncwarp();  // the walk's slot is written again two pieces on
  }

  // Leave no copy in flight (only possible after a timeout).
  for (int k = waited; k < issued; ++k) mbar_wait_bounded(&bars[k % NS], (k / NS) & 1, a.err);
}

// ----------------------------------------------------------------------------
// The merge of cut segments: CTA gw takes the one that warp gw of the attention
// grid described, if any.  (A CTA per warp of that grid, of which few have
// work, measured 2 to 4 us less than four CTAs per SM that look at several
// descriptions each: a segment's merge is a chain of latencies, and segments
// must not queue.)  The segment's columns are spread over the warps; where
// there are fewer columns than warps, several warps share a column's parts.
// ----------------------------------------------------------------------------
inline int merge_warps(int cols) { return cols > 4 ? 8 : 4; }

template <int D, int NT>
__global__ void __launch_bounds__(256) merge_cols_kernel(const __grid_constant__ Args a) {
  constexpr int NC = 8 * NT, SLOT = slot_floats(NC, D), V = D / 32;
  const int MW = blockDim.x / 32;
  constexpr int kRound = 8;  // parts in flight per warp
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  __shared__ float part_s[8][D + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4* cp = reinterpret_cast<const int4*>(a.cuts + blockIdx.x);
  const int4 c0 = __ldcg(cp), c1 = __ldcg(cp + 1);
  const int n = c0.x, row0 = c0.w, r0 = c1.x, head0 = c1.z;
  if (n == 0) return;
  const uint32_t slot0 = (uint32_t)c0.y, first = (uint32_t)c0.z;
  const int cols = min(NC, c1.y - r0);
  const int share = cols >= MW ? 1 : MW / cols, at_once = MW / share;  // warps per column, columns at once
  auto part = [&](int i) -> const float* { return a.partials + (size_t)(i == 0 ? slot0 : 2 * (first + i)) * SLOT; };
  for (int base = 0; base < cols; base += at_once) {
    const int col = base + warp / share, who = warp % share;
    const bool have = col < cols && warp / share < at_once;
    float num[V], den = 0.f, M = -CUDART_INF_F;
#pragma unroll
    for (int d = 0; d < V; ++d) num[d] = 0.f;
    if (have) {
      for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(part(i) + NC * D + col));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      if (M == -CUDART_INF_F) M = 0.f;
      // parts who, who + share, ...: 32 factors at a time, one per lane
      for (int i0 = who; i0 < n; i0 += 32 * share) {
        const int i = i0 + lane * share;
        float f = 0.f;
        if (i < n) {
          const float* p = part(i) + NC * D + col;
          f = fast_exp2(__ldcg(p) - M);
          den = fmaf(f, __ldcg(p + NC), den);
        }
        const int cnt = min(32, (n - i0 + share - 1) / share);
        for (int k0 = 0; k0 < cnt; k0 += kRound) {
          Vec x[kRound];
#pragma unroll
          for (int k = 0; k < kRound; ++k)
            if (k0 + k < cnt) x[k] = __ldcg(reinterpret_cast<const Vec*>(part(i0 + (k0 + k) * share) + col * D) + lane);
#pragma unroll
          for (int k = 0; k < kRound; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
            if (k0 + k < cnt) {
              const float* xv = reinterpret_cast<const float*>(&x[k]);
#pragma unroll
              for (int d = 0; d < V; ++d) num[d] = fmaf(fk, xv[d], num[d]);
            }
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    if (share > 1) {  // the column's shares, all relative to the same maximum
#pragma unroll
      for (int d = 0; d < V; ++d) part_s[warp][V * lane + d] = num[d];
      if (lane == 0) part_s[warp][D] = den;
      __syncthreads();
      if (have && who == 0) {
        for (int k = 1; k < share; ++k) {
#pragma unroll
          for (int d = 0; d < V; ++d) num[d] += part_s[warp + k][V * lane + d];
          den += part_s[warp + k][D];
        }
      }
      __syncthreads();
    }
    if (have && who == 0) {
      const float inv = den == 0.f ? 0.f : a.out_scale / den;
      const int r = r0 + col;
      __nv_bfloat16* dst = a.out + ((int64_t)(row0 + r / a.group) * a.num_q_heads + head0 + r % a.group) * D + V * lane;
      if constexpr (V == 4) {
        store4<__nv_bfloat16>(dst, num[0] * inv, num[1] * inv, num[2] * inv, num[3] * inv);
      } else {
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(num[0] * inv, num[1] * inv);
      }
    }
  }
}

// A compiled instance: its kernels and launch shape.
struct Kernel {
  const void* fn = nullptr;
  const void* merge = nullptr;
  int smem = 0, tok = 0;
};

template <int KIND, int D, int BS, int NT>
Kernel kernel_info() {
  return Kernel{reinterpret_cast<const void*>(&attn_cols_kernel<KIND, D, BS, NT>),
                reinterpret_cast<const void*>(&merge_cols_kernel<D, NT>),
                Smem<KIND, D, BS, NT>::kBytes, Geo<KIND, D, BS>::TOK};
}

// One translation unit per kind and head_dim.
template <int KIND, int D>
Kernel pick(int bs, int nt) {
  if (bs == 8) return nt == 1 ? kernel_info<KIND, D, 8, 1>() : kernel_info<KIND, D, 8, 2>();
  if (bs == 16) return nt == 1 ? kernel_info<KIND, D, 16, 1>() : kernel_info<KIND, D, 16, 2>();
  return nt == 1 ? kernel_info<KIND, D, 32, 1>() : kernel_info<KIND, D, 32, 2>();
}

Kernel pick_bf16_64(int bs, int nt);
Kernel pick_bf16_128(int bs, int nt);
Kernel pick_fp8_64(int bs, int nt);
Kernel pick_fp8_128(int bs, int nt);
Kernel pick_int8_64(int bs, int nt);
Kernel pick_int8_128(int bs, int nt);
Kernel pick_fp4_64(int bs, int nt);
Kernel pick_fp4_128(int bs, int nt);

}  // namespace cols
}  // namespace pkv
