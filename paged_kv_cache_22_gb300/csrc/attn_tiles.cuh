// attn_tiles.cuh -- paged attention with modified scores for many query rows
// per (sequence, kv head) (prompt chunks), on the 5th-generation tensor cores:
// two 128-row query tiles per CTA that share one stream of K and V.  The
// operation and the kinds of cache are those of attn_cols.cuh.
//
// Per step of 64 positions and tile x of the two:
//   S_x = Q_x K^T    M 128, N 64, K = D   (tcgen05.mma, operands in shared memory)
//   P_x = 2^(z - m)  eight softmax warps per tile, two threads per row (32
//                    columns each); P_x goes back to tensor memory, each half
//                    over its own columns of S_x, as the A operand of
//   O_x += P_x V     M 128, N = D, K = 64
// S_x has two buffers: S_x(j + 1) is issued before the P_x(j) of the running
// softmax is waited for, so the softmax warps, which set the pace, find their
// next scores ready (with one buffer they waited 1100 of the 2700 clocks of a
// step; now 330).  The order of the tensor pipe alone keeps S_x(j + 1) off the
// P_x(j - 1) that it overwrites.  Steps of 128 positions with one buffer, which
// is all that 512 columns of tensor memory hold, took 2630 clocks per 64.
//
// The maximum m of a row is lazy: it moves only when a score passes it by more
// than 2^8 (weights stay below 2^8).  Each step the two warps of the same 32
// rows vote (one barrier with an OR) whether any row's must; the two threads of
// a row exchange their maxima only then, and wait for the product before it only
// to rescale O_x.  (A vote of all 256 threads of a tile: 219 us instead of 214
// for the bf16 chunk below.)
//
// Tensor memory: S_0, S_1 at columns 0 and 128 (two buffers of 64 each), O_0,
// O_1 at 256 and 256 + D.
//
// Warps: 0-7 and 8-15 bring Q, then softmax of tiles 0 and 1 (column half
// (w / 4) % 2); 17 and 19 the MMAs of tiles 0 and 1 (beside the softmax warps an
// MMA takes its issuing warp longer than the tensor pipe: one warp for both
// tiles left the pipe idle); 16 and 18 the copies of K and V; 20-23 widen codes
// to fp16 operands (fp8 and quantised caches), 32 rows of K or V each (two warps
// for all of it: 550 us instead of 284 for the chunk below, MMAs waiting; with all
// of a warp's codes loaded before the first is widened 233).
//
// Measured (8 sequences of 1024-4096 tokens, 512 query tokens each, 32 heads
// on 8, D 128): 209 us for bf16 with a cap (827 TF/s; 43 % of what a large
// library product reaches), 229 us for a 4-bit cache.  A step of 64 positions
// takes some 2200 clocks, of which the two tiles' products need 1280 and the
// softmax's arithmetic 1100 (exponents 512, multiply-adds and conversions the
// rest); what is over is latency within a step that two warps per scheduler and
// tile do not hide.  Each CTA adds 3 us before its first product, and CTAs of
// 27-82 us leave the last tenth of the call with idle SMs although the longest
// start first (247 us before they did, and before Q and O went through shared
// memory in whole lines).
//
// softcap: cap * tanh(x / cap) through a quadratic in (x / cap)^2 while every
// score of a warp's step is below cap / 4, a cubic below cap / 2 (relative error
// 6e-7), else through e^2u.  (Below cap / 4 the cubic took 219 us, the quadratic
// 205.)  They are evaluated where the exponent is formed: |cap * tanh(x / cap)| <=
// |x| bounds the scores for the vote on the maximum.
//
// bf16 caches: tensor copies land in the operand layout, P is one bf16 operand
// (a weight keeps 8 bits, as in pkv_paged_attention_multi: a remainder would
// double the products; an output moves by at most 2^-8 max|V|).  Codes: raw
// tiles land in a ring of steps of each cache, four warps widen them exactly; q
// is fp16, each row scaled by a power of two (the factor goes to its scores); P
// is one fp16 operand.  Row scales never touch the codes: K's multiplies the
// score's column, V's is added to the score as its base-2 logarithm (weight w),
// and the row sum takes w / s_v.
#pragma once

#include "attn_cols.cuh"
#include "attn_tc05.cuh"

namespace pkv {
namespace tiles {

using cols::Args;
using cols::kBf16;
using cols::kFp4;
using cols::kFp8;
using cols::kInt8;

constexpr int kStep = 64;       // positions per step
constexpr int kHalf = 32;       // columns of S per softmax thread
constexpr int kTile = 128;      // query rows per tile (TMEM lanes)
constexpr int kSpan = 128;      // bytes of a swizzle span
constexpr int kMaxSmem = 232448;
constexpr int kOkRing = 16;     // steps whose block bits are kept (more than the copies run ahead)

template <int KIND, int D, int BS>
struct Geo {
  static constexpr bool BF = KIND == kBf16;
  static constexpr bool REC = KIND == kInt8 || KIND == kFp4;
  static constexpr int SPANS = D / 64;
  // bf16 has no warps that widen codes, and more registers for the rest (95 for
  // 80: the chunk above 215 -> 209 us)
  static constexpr int kThreads = BF ? 640 : 768;
  static constexpr int NB = kStep / BS;                       // blocks per step
  static constexpr int OP = SPANS * kStep * kSpan;            // one operand tile of K or V
  static constexpr int NS = BF ? (D == 128 ? 4 : 8) : 3;      // operand stages of K, of V
  static constexpr int ROW = BF ? 2 * D : (KIND == kFp4 ? D / 2 : D);
  static constexpr int RAW = BF ? 0 : cols::Geo<KIND, D, BS>::BLOCK;  // one block of one cache
  static constexpr int kQ = 0;                                // [tile][span][128 rows][128 B]
  static constexpr int kK = 2 * SPANS * kTile * kSpan;
  static constexpr int kV = kK + NS * OP;
  static constexpr int kRaw = kV + NS * OP;
  // Row scales as columns: K's, the logarithm and the inverse of V's.  Two
  // stages more than the operands have: when the products of step j have freed
  // K's operand stage, the softmax may still read the scales of step j - 1.
  static constexpr int NCS = NS + 2;
  static constexpr int kColBytes = REC ? 3 * NCS * kStep * 4 : 0;
  static constexpr int kXch = 2 * 2 * kTile * 4;              // a float per softmax thread: row maxima, sums
  static constexpr int kTail = kColBytes + kXch + 2 * kTile * 4 + 1024;  // and q scales, barriers, words
  static constexpr int NR0 = RAW ? (kMaxSmem - kRaw - kTail) / RAW : 0;
  static constexpr int BPG = BS < 32 ? 32 / BS : 1;           // blocks of 32 rows
  static constexpr int NG = NR0 / (2 * NB) > 6 ? 6 : NR0 / (2 * NB);  // steps of raw K, of raw V
  static constexpr int NR = RAW ? 2 * NG * NB : 0;            // raw slots
  static constexpr int kCol = kRaw + NR * RAW;
  static constexpr int kX = kCol + kColBytes;
  static constexpr int kQmul = kX + kXch;                     // [2 * 128] score units of a row
  static constexpr int kBar = (kQmul + 2 * kTile * 4 + 15) / 16 * 16;
  static constexpr int kNumBars = 4 * NS + 13 + 4 * (RAW ? NG : 0);
  static constexpr int kOk = kBar + 8 * kNumBars;
  static constexpr int kTmem = kOk + 4 * 2 * kOkRing;         // of K's blocks, of V's
  static constexpr int kBytes = kTmem + 16;
  static constexpr int CPR = ROW >= 128 ? 8 : ROW / 16;       // raw: chunks of a swizzled row
  static_assert(kBytes <= kMaxSmem, "shared memory");
  static_assert(BF || NG >= 2, "raw ring");
  static_assert(NS + (BF ? 0 : NG) + 3 < kOkRing, "block bits");
};

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
               ::"r"(d), "r"(a_tmem), "l"(b), "r"(id), "r"(acc));
}

// 16 columns of packed operands.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float maxabs3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// OR over the threads of a named barrier, which they all reach.
__device__ __forceinline__ bool any_of(int barrier, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(barrier), "r"(threads), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }

// tanh(u) / u as a cubic in u^2 for |u| < 1/2, a quadratic for |u| < 1/4 (fits
// of least relative error, 5.5e-7 and 4e-7); beyond, the exponential.
constexpr float kSeriesMax = 0.5f, kShortMax = 0.25f;
constexpr float kQ0 = 0.9999995827674866f, kQ1 = -0.33321908116340637f, kQ2 = 0.12841613590717316f;
constexpr float kC0 = 0.999999463558197f, kC1 = -0.33326318860054016f, kC2 = 0.13190296292304993f,
                kC3 = -0.04440222680568695f;

// S -> S tanh(u) / u, u = S k1 small: the capped score in units of S.
__device__ __forceinline__ void cap_series(float (&v)[32], float k1) {
  const float k2 = k1 * k1;
  const float2 c1 = f2(kC1 * k2), c2 = f2(kC2 * k2 * k2), c3 = f2(kC3 * k2 * k2 * k2);
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const float2 y = make_float2(v[c], v[c + 1]), u = __fmul2_rn(y, y);
    const float2 z = __fmul2_rn(y, ffma2(u, ffma2(u, ffma2(u, c3, c2), c1), f2(kC0)));
    v[c] = z.x;
    v[c + 1] = z.y;
  }
}
__device__ __forceinline__ float max32(const float (&v)[32]) {
  float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F;
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    m0 = max3(m0, v[c], v[c + 1]);
    m1 = max3(m1, v[c + 2], v[c + 3]);
  }
  return fmaxf(m0, m1);
}
__device__ __forceinline__ float maxabs32(const float (&v)[32]) {
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int c = 0; c < 32; c += 4) {
    m0 = maxabs3(m0, v[c], v[c + 1]);
    m1 = maxabs3(m1, v[c + 2], v[c + 3]);
  }
  return fmaxf(m0, m1);
}

template <int KIND, int D, int BS>
__global__ void __launch_bounds__(Geo<KIND, D, BS>::kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ Args a, const __grid_constant__ TmaMaps maps) {
  using namespace tc05;
  using G = Geo<KIND, D, BS>;
  constexpr bool BF = G::BF, REC = G::REC;
  constexpr int NS = G::NS, NB = G::NB, SPANS = G::SPANS, NR = G::NR;
  extern __shared__ __align__(1024) uint8_t tile_smem[];
  uint8_t* const sm = tile_smem;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int g = a.group;

  // ---- the CTA's rows and the positions they attend
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + G::kTmem);
  int s = blockIdx.z;
  if (a.by_length) {  // CTAs start in the order of their index: the longest sequences come first
    for (int i = tid; i < a.num_seqs; i += G::kThreads) {
      const int n = __ldg(a.seq_lens + i);
      int rank = 0;
      for (int k = 0; k < a.num_seqs; ++k) {
        const int m = __ldg(a.seq_lens + k);
        rank += m > n || (m == n && k < i);
      }
      if (rank == s) tslot[1] = i;
    }
    __syncthreads();
    s = tslot[1];
  }
  const int kvh = blockIdx.x % a.num_kv_heads, tile_pair = (gridDim.x - 1 - blockIdx.x) / a.num_kv_heads;  // later rows attend more
  const int q0 = __ldg(a.q_start + s);
  const int64_t T64 = (int64_t)__ldg(a.q_start + s + 1) - q0;
  const int L = __ldg(a.seq_lens + s);
  if (L < 0 || L > a.len_clip || T64 < 0 || T64 > L || T64 > a.max_q || q0 < 0 || q0 + T64 > a.total_q) {
    if (tid == 0 && kvh == 0 && tile_pair == 0) raise_error(a.err, PKV_DEVERR_BAD_SEQ_LEN);
    return;  // its rows are left alone
  }
  const int T = (int)T64, rows = T * g;
  const int row0 = tile_pair * 2 * kTile;
  if (row0 >= rows) return;
  if (smem_addr(sm) & 1023u) {
    if (tid == 0) raise_error(a.err, PKV_DEVERR_SMEM_ALIGN);
    return;
  }
  const int nx = rows - row0 > kTile ? 2 : 1;  // tiles with rows
  const int i0 = row0 / g, i1 = (min(row0 + 2 * kTile, rows) - 1) / g;
  const int hi_min = L - T + i0 + 1, hi_max = L - T + i1 + 1;
  const int lo_min = a.window > 0 ? max(0, hi_min - a.window) : 0;
  const int pre = a.prefix_lens ? min(max(__ldg(a.prefix_lens + s), 0), L) : 0;
  const int a_max = max(min(a.sinks, hi_max), pre);
  const int nt = (max(hi_max, a_max) + kStep - 1) / kStep;
  int na = (a_max + kStep - 1) / kStep, wt = lo_min / kStep;
  if (wt <= na) na = wt = 0;
  const int steps = nt - (wt - na);
  // First position of step j.  With a distance bias the last positions come
  // first: scores then fall from step to step, where a steep slope would raise
  // the maximum, and rescale O, at each (ragged prompts, 14 heads: 62 us instead of 51).
  const bool backward = a.slopes != nullptr;
  auto base_of = [&](int j) -> int {
    const int i = backward ? steps - 1 - j : j;
    return (i < na ? i : i + (wt - na)) * kStep;
  };
  const int32_t* table = a.block_tables + (size_t)s * a.table_stride;

  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + G::kBar);
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_empty + NS;
  uint64_t* v_empty = v_full + NS;
  uint64_t* s_ready = v_empty + NS;  // [tile][buffer]
  uint64_t* p_ready = s_ready + 4;   // [tile][buffer]: a softmax may be a step ahead of its products
  uint64_t* o_ready = p_ready + 4;   // [2] the products of a step are in O
  uint64_t* o_done = o_ready + 2;    // [2]
  uint64_t* q_ready = o_done + 2;    // the operands Q and the rows' factors
  uint64_t* raw_full = q_ready + 1;  // [2][NG]
  uint64_t* raw_empty = raw_full + 2 * G::NG;
  uint32_t* ok_bits = reinterpret_cast<uint32_t*>(sm + G::kOk);
  float* ksc_s = reinterpret_cast<float*>(sm + G::kCol);  // [NCS][128]
  float* vlg_s = ksc_s + G::NCS * kStep;
  float* vis_s = vlg_s + G::NCS * kStep;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&k_full[i], BF ? 1 : 2);
      mbar_init(&k_empty[i], nx);
      mbar_init(&v_full[i], BF ? 1 : 2);
      mbar_init(&v_empty[i], nx);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_ready[2 * i], 1);
      mbar_init(&s_ready[2 * i + 1], 1);
      mbar_init(&p_ready[2 * i], 8);
      mbar_init(&p_ready[2 * i + 1], 8);
      mbar_init(&o_ready[i], 1);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(q_ready, 16);
    if constexpr (!BF) {
      for (int i = 0; i < 2 * G::NG; ++i) {
        mbar_init(&raw_full[i], 1);
        mbar_init(&raw_empty[i], 2);
      }
    }
    fence_mbar_init();
  }
  if (w == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tslot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tslot;

  // whether some row of the CTA attends a position of the block
  auto wanted = [&](int first, int len) -> bool {
    return first < a_max || (first < hi_max && first + len > lo_min);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.err));
  };

  if (w >= 16) {
    if (w == 16 || w == 18) {
      // ---- copies of K or V: block b of a step by lane b, the next step's ids
      // already in flight.  bf16 goes to the operand, codes to the raw ring.
      constexpr int N = BF ? NS : G::NG;
      const int v = w == 18;
      auto load_id = [&](int j) -> int32_t {
        const int first = base_of(j) + lane * BS;
        return j < steps && lane < NB && wanted(first, BS) ? __ldg(table + first / BS) : INT32_MIN;
      };
      uint64_t* const fulls = BF ? (v ? v_full : k_full) : raw_full + v * G::NG;
      uint64_t* const empties = BF ? (v ? v_empty : k_empty) : raw_empty + v * G::NG;
      const TmaMap* const map = v ? &maps.v : &maps.k;
      int32_t id = load_id(0);
      int armed = 0;
      for (int j = 0; j < steps; ++j) {
        const int32_t nid = load_id(j + 1);
        const bool good = id >= 0 && id < a.num_blocks;
        const uint32_t ok = __ballot_sync(0xffffffffu, good);
        const uint32_t bad = __ballot_sync(0xffffffffu, !good && id != INT32_MIN);
        const int st = j % N;
        uint64_t* const full = fulls + st;
        if (!wait_all(empties + st, ((j / N) & 1) ^ 1)) break;
        armed = j + 1;
        if (lane == 0) {
          if (bad && !v) raise_error(a.err, PKV_DEVERR_BAD_BLOCK_ID);
          ok_bits[v * kOkRing + j % kOkRing] = ok;
          mbar_arrive_expect_tx(full, (uint32_t)(__popc(ok) * (BF ? BS * D * 2 : G::RAW)));
        }
        __syncwarp();
        if (good) {
          if constexpr (BF) {
            uint8_t* const dst = sm + (v ? G::kV : G::kK) + st * G::OP + lane * (BS * kSpan);
#pragma unroll
            for (int sp = 0; sp < SPANS; ++sp) tma_span_tile(dst + sp * (kStep * kSpan), map, sp * 64, kvh * BS, id, full);
          } else {
            uint8_t* const dst = sm + G::kRaw + ((v * G::NG + st) * NB + lane) * G::RAW;
            if constexpr (REC)
              bulk_g2s(dst, (v ? a.v_cache : a.k_cache) + ((size_t)id * a.num_kv_heads + kvh) * G::RAW, G::RAW, full);
            else
              tma_load_3d(dst, map, 0, kvh * BS, id, full);
          }
        }
        __syncwarp();
        id = nid;
      }
      // no copy may land after the CTA is gone
      for (int j = max(0, armed - N); j < armed; ++j)
        if (!wait_all(fulls + j % N, (j / N) & 1)) break;
    } else if (!BF && w >= 20) {
      // ---- widen codes, raw rows -> fp16 operand rows: each warp 32 of a
      // step's rows of one cache.  A thread widens 16 codes (unit k) of a row
      // at a time; eight neighbouring lanes take four units of the rows r and
      // r ^ 5, which puts both their loads of codes and their two stores each on
      // all banks (swizzled positions c ^ r of the chunks, c of one half for
      // a load, of one parity for a store).
      constexpr int BPG = G::BPG, NG = G::NG, QPI = D == 128 ? 2 : 4;
      const int c = w >= 22, half = w & 1, k = (lane & 3) + (D == 128 ? lane >> 1 & 4 : 0), c0 = 2 * (k % 4);
      const int q = D == 128 ? lane >> 4 : lane >> 3, alt = lane & 4 ? 5 : 0;
      uint64_t* const empties = c ? v_empty : k_empty;
      uint64_t* const fulls = c ? v_full : k_full;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        const int st = j % NS, cs = j % G::NCS, slot = j % NG;
        if (!wait_all(&empties[st], ((j / NS) & 1) ^ 1) || !wait_all(&raw_full[c * NG + slot], (j / NG) & 1)) break;
        const uint32_t ok = ok_bits[c * kOkRing + j % kOkRing] >> (half * BPG);
        uint8_t* const op = sm + (c ? G::kV : G::kK) + st * G::OP + (k / 4) * (kStep * kSpan) + 32 * half * kSpan;
        const uint8_t* const raws = sm + G::kRaw + ((c * NG + slot) * NB + half * BPG) * G::RAW;
        // all codes first: their loads' latency is paid once (a unit at a time,
        // unrolled by four, the fp4 chunk took 279 us instead of 233)
        constexpr int U = 16 / QPI;
        uint4 y4[KIND == kFp4 ? 1 : U];
        uint2 y2[KIND == kFp4 ? U : 1];
        uint32_t ts[KIND == kFp4 ? U : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int rr = 2 * (u * QPI + q) ^ alt, p = rr % BS, b = rr / BS;  // row of the 32, of its block
          const uint8_t* raw = raws + b * G::RAW;
          if constexpr (KIND == kFp4) {
            y2[u] = *reinterpret_cast<const uint2*>(raw + p * G::ROW + 16 * quant_chunk(p, k / 2, G::ROW) + 8 * (k & 1));
            ts[u] = raw[BS * G::ROW + p * (D / 16) + k];
          } else {
            constexpr int M = G::CPR - 1;
            y4[u] = *reinterpret_cast<const uint4*>(raw + p * G::ROW + ((k ^ ((p * G::ROW / 128) & M)) << 4));
          }
        }
        // V rows that no row attends, or that were not copied, are zero (0 * NaN
        // is NaN); K rows may hold anything (their scores are masked)
        const int first = base_of(j) + 32 * half;
        const bool whole = !c || ((ok & ((1u << BPG) - 1)) == (1u << BPG) - 1 &&
                                  (first + 32 <= a_max || (first >= lo_min && first + 32 <= hi_max)));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int rr = 2 * (u * QPI + q) ^ alt, b = rr / BS;
          uint32_t h8[8];
          if constexpr (KIND == kFp4) {
            uint32_t f[4];
            const uint32_t t2 = cols::e4m3x2_to_f16x2(ts[u] | ts[u] << 8);
            cols::e2m1x8_to_f16x2x4(y2[u].x, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) h8[e] = cols::hmul2(f[e], t2);
            cols::e2m1x8_to_f16x2x4(y2[u].y, f);
#pragma unroll
            for (int e = 0; e < 4; ++e) h8[4 + e] = cols::hmul2(f[e], t2);
          } else {
            const uint32_t y[4] = {y4[u].x, y4[u].y, y4[u].z, y4[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (KIND == kFp8) e4m3x4_to_f16x2x2(y[e], h8[2 * e], h8[2 * e + 1]);
              else cols::i8x4_to_f16x2x2(y[e], h8[2 * e], h8[2 * e + 1]);
            }
          }
          if (!whole && (!(ok >> b & 1) || !wanted(first + rr, 1))) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h8[e] = 0u;
          }
          uint8_t* dst = op + rr * kSpan;
          *reinterpret_cast<uint4*>(dst + ((c0 ^ (rr & 7)) << 4)) = make_uint4(h8[0], h8[1], h8[2], h8[3]);
          *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ (rr & 7)) << 4)) = make_uint4(h8[4], h8[5], h8[6], h8[7]);
        }
        if constexpr (REC) {  // the 32 rows' scales, one per lane
          const float sc = *reinterpret_cast<const float*>(raws + lane / BS * G::RAW + G::RAW - 4 * BS + 4 * (lane % BS));
          const int col = cs * kStep + 32 * half + lane;
          if (!c) {
            ksc_s[col] = sc;
          } else {
            const float lg0 = cols::fast_log2(sc), lg = lg0 < cols::kMinLogScale ? cols::kMinLogScale : lg0;
            vlg_s[col] = lg;
            vis_s[col] = lg == lg ? fast_exp2(-lg) : 1.f;  // (any finite factor will do beside a NaN weight)
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[c * NG + slot]);
          mbar_arrive(&fulls[st]);
        }
      }
    } else if (w == 17 || (w == 19 && nx == 2)) {
      // ---- the MMAs of a tile.  The loop is unrolled over the operand stages
      // so that every descriptor is a constant, and runs warp-wide with values
      // the compiler sees as uniform: issued from one lane with descriptors in
      // vector registers, an MMA cost 85 clocks.  What arrives early is waited
      // for first: V of this step and K of the next before the tile's P.
      constexpr uint32_t id_s = idesc_f16kind(kTile, kStep, BF, false);
      constexpr uint32_t id_o = idesc_f16kind(kTile, D, BF, true);
      const int t = __shfl_sync(0xffffffffu, (int)(w == 19), 0), n = __shfl_sync(0xffffffffu, steps, 0);
      const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dq = sw128_desc(smem_addr(sm + G::kQ) + t * (SPANS * kTile * kSpan), 16, 1024);
      const uint64_t dk = sw128_desc(smem_addr(sm + G::kK), 16, 1024);
      const uint64_t dv = sw128_desc(smem_addr(sm + G::kV), kStep * kSpan, 1024);  // MN-major
      const uint32_t s_t = base + t * 2 * kStep, o_t = base + 256 + t * D;
      auto issue_s = [&](int st, int buf) {
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_bf16(s_t + buf * kStep, dq + (uint64_t)((k / 4 * (kTile * kSpan) + k % 4 * 32) >> 4),
                     dk + (uint64_t)((st * G::OP + k / 4 * (kStep * kSpan) + k % 4 * 32) >> 4), id_s, k > 0);
          mma_commit(&s_ready[2 * t + buf]);
          mma_commit(&k_empty[st]);
        }
        __syncwarp();
      };
      bool ok = n > 0 && wait_all(q_ready, 0) && wait_all(&k_full[0], 0);
      if (ok) {
        fence_after_sync();
        issue_s(0, 0);
      }
#pragma unroll 1
      for (int j0 = 0, par = 0; ok && j0 < n; j0 += NS, par ^= 1) {
#pragma unroll
        for (int st = 0; st < NS; ++st) {
          const int j = j0 + st;
          if (!ok || j >= n) break;
          const bool more = j + 1 < n;
          const int buf = j & 1;
          if (more) {
            ok = wait_all(&k_full[(st + 1) % NS], st + 1 == NS ? par ^ 1 : par);
            if (!ok) break;
            fence_after_sync();
            issue_s((st + 1) % NS, buf ^ 1);
          }
          ok = wait_all(&v_full[st], par) && wait_all(&p_ready[2 * t + buf], (j >> 1) & 1);
          if (!ok) break;
          fence_after_sync();
          if (elect_one()) {
            const uint32_t p_t = s_t + buf * kStep;
            if (j == 0)
              mma_ts(o_t, p_t, dv, id_o, 0u);
            else
              mma_ts(o_t, p_t, dv + (uint64_t)((st * G::OP) >> 4), id_o, 1u);
#pragma unroll
            for (int k = 1; k < kStep / 16; ++k)
              mma_ts(o_t, p_t + (k / 2) * kHalf + 8 * (k % 2), dv + (uint64_t)((st * G::OP + k * 16 * kSpan) >> 4), id_o, 1u);
            mma_commit(&v_empty[st]);
            mma_commit(more ? &o_ready[t] : &o_done[t]);
          }
          __syncwarp();
        }
      }
      // every MMA issued has completed before TMEM is released: the softmax
      // warps wait for o_done; after a timeout this drains what was issued
      if (!ok && n > 0) {
        if (elect_one()) mma_commit(&o_done[t]);
        __syncwarp();
        wait_all(&o_done[t], 0);
      }
    }
  } else {
    // ---- the query rows, D / 8 lanes per row: K-major, 128-byte swizzle
    float* const qmul_s = reinterpret_cast<float*>(sm + G::kQmul);
    {
      constexpr int LPR = D / 8, RPW = 32 / LPR, IT = 2 * kTile / (16 * RPW);
      const int c = lane % LPR;
      const uint32_t sign = a.qk_scale < 0.f ? 0x80008000u : 0u;  // a negative scale's sign goes to q
      uint4 v[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int R = row0 + (i * 16 + w) * RPW + lane / LPR, tok = R / g;
        v[i] = make_uint4(0, 0, 0, 0);
        if (R < rows)
          v[i] = __ldg(reinterpret_cast<const uint4*>(a.q + ((size_t)(q0 + tok) * a.num_q_heads + kvh * g + R - tok * g) * D) + c);
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int r = (i * 16 + w) * RPW + lane / LPR;  // of both tiles
        uint4 q = v[i];
        float qmul = fabsf(a.qk_scale);
        if constexpr (!BF) {  // fp16: the row's largest |q| brought into [2^14, 2^15)
          uint32_t mx = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu), __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
          mx = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int e = min(max((int)(mx >> 7), 20), 254);
          const float up = __uint_as_float((uint32_t)(268 - e) << 23);
          qmul *= __uint_as_float((uint32_t)(e - 14) << 23);
          const float2 f0 = bf16x2_to_f2(q.x), f1 = bf16x2_to_f2(q.y), f2_ = bf16x2_to_f2(q.z), f3 = bf16x2_to_f2(q.w);
          q = make_uint4(pack_f16x2(f0.x * up, f0.y * up), pack_f16x2(f1.x * up, f1.y * up), pack_f16x2(f2_.x * up, f2_.y * up),
                         pack_f16x2(f3.x * up, f3.y * up));
        }
        q.x ^= sign; q.y ^= sign; q.z ^= sign; q.w ^= sign;
        // (kept above zero: a masked score, -inf times this, has to stay -inf)
        if (c == 0) qmul_s[r] = fmaxf(qmul, 0x1p-120f);
        *reinterpret_cast<uint4*>(sm + G::kQ + (r / kTile * SPANS + c / 8) * (kTile * kSpan) + r % kTile * kSpan +
                                  ((c % 8 ^ (r & 7)) << 4)) = q;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    }
    // ---- the softmax threads: tile x, column half h, row r of the tile
    const int x = w >> 3, h = (w >> 2) & 1, r = (w & 3) * 32 + lane;
    const int pair = 1 + x * 4 + (w & 3);  // barrier of the two warps of the same 32 rows
    if (x < nx) {
      int hi = 0, lo = 0, al = 0, my_row = -1, my_head = 0;
      const int R = row0 + x * kTile + r;
      if (R < rows) {
        const int tok = R / g;
        my_row = q0 + tok;
        my_head = kvh * g + R % g;
        hi = L - T + tok + 1;
        lo = a.window > 0 ? max(0, hi - a.window) : 0;
        al = max(min(a.sinks, hi), pre);
      }
      // A warp whose wait gave up goes on without waiting (and writes no
      // output): the tile's warps meet at barriers, and none may be left there.
      bool ok = mbar_wait_bounded(q_ready, 0, a.err);
      const uint32_t lane_base = tmem + ((uint32_t)((w & 3) * 32) << 16);
      const uint32_t s_col0 = lane_base + x * 2 * kStep + h * kHalf;  // S, and P over it, of even steps
      const uint32_t o_col = lane_base + 256 + x * D + h * (D / 2);
      float* const xch = reinterpret_cast<float*>(sm + G::kX) + x * 2 * kTile;  // [2 halves][128 rows]
      const float qmul = qmul_s[x * kTile + r];  // base-2 score units per unit of S (>= 0)
      const float slope = a.slopes && my_row >= 0 ? __ldg(a.slopes + my_head) * 1.4426950408889634f : 0.f;
      const float k1 = qmul * a.inv_cap;  // S -> u = z / cap
      constexpr uint32_t kAll = NB == 32 ? 0xFFFFFFFFu : (1u << NB) - 1u;
      float m = -CUDART_INF_F;
      float2 l2 = f2(0.f);
      // positions every row of the warp attends: [0, all_al) and [all_lo, all_hi)
      const int all_hi = __reduce_min_sync(0xffffffffu, my_row < 0 ? 0x7FFFFFFF : hi);
      const int all_lo = __reduce_max_sync(0xffffffffu, my_row < 0 ? 0 : lo);
      const int all_al = __reduce_min_sync(0xffffffffu, my_row < 0 ? 0x7FFFFFFF : al);
      for (int j = 0; j < steps; ++j) {
        const int t0 = base_of(j), st = j % NS, cs = j % G::NCS, th = t0 + h * kHalf;  // first position of the step, of this half
        const uint32_t s_col = s_col0 + (j & 1) * kStep;
        ok = ok && mbar_wait_bounded(&s_ready[2 * x + (j & 1)], (j >> 1) & 1, a.err);
        if constexpr (REC) ok = ok && mbar_wait_bounded(&v_full[st], (j / NS) & 1, a.err);  // V's scales come with its codes
        __syncwarp();
        fence_after_sync();
        const uint32_t okb = ok_bits[j % kOkRing];
        const bool inner = ((t0 >= all_lo && t0 + kStep <= all_hi) || t0 + kStep <= all_al) && okb == kAll;  // no mask
        float v[kHalf];
        float4 kpre[REC ? kHalf / 4 : 1];  // (before S: their latency hides behind its load, 232 -> 228 us)
        if constexpr (REC) {
          const float4* ks = reinterpret_cast<const float4*>(ksc_s + cs * kStep + kHalf * h);
#pragma unroll
          for (int c = 0; c < kHalf / 4; ++c) kpre[c] = ks[c];
        }
        tmem_ld32(s_col, v);
        if constexpr (REC) {
#pragma unroll
          for (int c = 0; c < kHalf / 4; ++c) {
            const float4 k4 = kpre[c];
            const float2 e = __fmul2_rn(make_float2(v[4 * c], v[4 * c + 1]), make_float2(k4.x, k4.y));
            const float2 f = __fmul2_rn(make_float2(v[4 * c + 2], v[4 * c + 3]), make_float2(k4.z, k4.w));
            v[4 * c] = e.x; v[4 * c + 1] = e.y; v[4 * c + 2] = f.x; v[4 * c + 3] = f.y;
          }
        }
        float mul = qmul, mt = 0.f;  // z = v * mul
        bool late = false, brief = false;  // the cap is applied where the exponent is formed, as a quadratic
        if (a.cap > 0.f) {
          const float big = maxabs32(v);
          const bool series = __all_sync(0xffffffffu, big * k1 < kSeriesMax);
          late = series && inner && !REC && !a.slopes;
          if (late) {
            mt = big * qmul;
            brief = __all_sync(0xffffffffu, big * k1 < kShortMax);
          } else if (series) {
            cap_series(v, k1);
          } else {
#pragma unroll
            for (int c = 0; c < kHalf; ++c) v[c] = cols::soft_cap(v[c] * qmul, a.cap, a.inv_cap);
            mul = 1.f;
          }
        }
        if (a.slopes) {  // z - slope |p - t|; p = hi - 1
          const float far = (float)(th - (hi - 1));
          if (t0 + kStep <= all_hi) {  // t <= p: slope (t - p), packed
            const float2 at = f2(slope * far);
#pragma unroll
            for (int c = 0; c < kHalf; c += 2) {
              const float2 b = ffma2(f2(slope), make_float2((float)c, (float)(c + 1)), at);
              const float2 e = ffma2(make_float2(v[c], v[c + 1]), f2(mul), b);
              v[c] = e.x; v[c + 1] = e.y;
            }
          } else {
#pragma unroll
            for (int c = 0; c < kHalf; ++c) v[c] = fmaf(v[c], mul, -slope * fabsf(far + (float)c));
          }
          mul = 1.f;
        }
        if constexpr (REC) {
          const float4* lg = reinterpret_cast<const float4*>(vlg_s + cs * kStep + kHalf * h);
#pragma unroll
          for (int c = 0; c < kHalf / 4; ++c) {
            const float4 l4 = lg[c];
            const float2 e = ffma2(make_float2(v[4 * c], v[4 * c + 1]), f2(mul), make_float2(l4.x, l4.y));
            const float2 f = ffma2(make_float2(v[4 * c + 2], v[4 * c + 3]), f2(mul), make_float2(l4.z, l4.w));
            v[4 * c] = e.x; v[4 * c + 1] = e.y; v[4 * c + 2] = f.x; v[4 * c + 3] = f.y;
          }
          mul = 1.f;
        }
        if (!inner) {
          uint32_t keep = low_bits(al - th) | (low_bits(hi - th) & ~low_bits(lo - th));
#pragma unroll
          for (int b = 0; b < kHalf / BS; ++b)
            if (!(okb >> (h * kHalf / BS + b) & 1)) keep &= ~(low_bits(BS) << (b * (BS & 31)));
#pragma unroll
          for (int c = 0; c < kHalf; ++c) v[c] = keep >> c & 1 ? v[c] : -CUDART_INF_F;
        }
        if (!late) mt = max32(v) * mul;
        if (any_of(pair, 64, mt > m + cols::kSlack)) {
          if (late) {  // the bound was not enough: the scores themselves
            cap_series(v, k1);
            mt = max32(v) * mul;
            late = false;
          }
          xch[h * kTile + r] = mt;
          asm volatile("barrier.cta.sync %0, 64;" ::"r"(pair) : "memory");
          mt = fmaxf(mt, xch[(h ^ 1) * kTile + r]);
          asm volatile("barrier.cta.sync %0, 64;" ::"r"(pair) : "memory");  // read before the next exchange
          float factor = 1.f;
          if (mt > m + cols::kSlack) {
            factor = m == -CUDART_INF_F ? 0.f : fast_exp2(m - mt);
            m = mt;
            l2 = __fmul2_rn(l2, f2(factor));
          }
          if (j > 0 && __any_sync(0xffffffffu, factor != 1.f)) {  // this half of the row's O
            ok = ok && mbar_wait_bounded(&o_ready[x], (j - 1) & 1, a.err);
            __syncwarp();
            fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[16];
              tmem_ld16(o_col + 16 * c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= factor;
              tmem_st16u(o_col + 16 * c, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        const float nm = m == -CUDART_INF_F ? 0.f : -m;
        float2 l3 = f2(0.f);
        // the weights out of the exponents' arguments, packed over S
        auto weigh = [&](auto arg) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < kHalf; c += 4) {
            float2 d0 = arg(c), d1 = arg(c + 2);
            d0 = make_float2(fast_exp2(d0.x), fast_exp2(d0.y));
            d1 = make_float2(fast_exp2(d1.x), fast_exp2(d1.y));
            if constexpr (REC) {
              const float4 is = reinterpret_cast<const float4*>(vis_s + cs * kStep + kHalf * h)[c / 4];
              l2 = ffma2(d0, make_float2(is.x, is.y), l2);
              l3 = ffma2(d1, make_float2(is.z, is.w), l3);
            } else {
              l2 = __fadd2_rn(l2, d0);
              l3 = __fadd2_rn(l3, d1);
            }
            pk[c / 2] = BF ? pack_bf16x2(d0.x, d0.y) : pack_f16x2(d0.x, d0.y);
            pk[c / 2 + 1] = BF ? pack_bf16x2(d1.x, d1.y) : pack_f16x2(d1.x, d1.y);
          }
          tmem_st16u(s_col, pk);
        };
        if (late) {
          // z = S qmul (kC0 + u2 (kC1 + u2 (kC2 + u2 kC3))), u2 = (S k1)^2; the
          // quadratic takes a fifth off the multiply-adds of a weight
          const float k2 = k1 * k1;
          if (brief) {
            const float2 e0 = f2(kQ0 * qmul), e1 = f2(kQ1 * qmul * k2), e2 = f2(kQ2 * qmul * k2 * k2);
            weigh([&](int c) {
              const float2 y = make_float2(v[c], v[c + 1]), u = __fmul2_rn(y, y);
              return ffma2(y, ffma2(u, ffma2(u, e2, e1), e0), f2(nm));
            });
          } else {
            const float2 e0 = f2(kC0 * qmul), e1 = f2(kC1 * qmul * k2), e2 = f2(kC2 * qmul * k2 * k2),
                         e3 = f2(kC3 * qmul * k2 * k2 * k2);
            weigh([&](int c) {
              const float2 y = make_float2(v[c], v[c + 1]), u = __fmul2_rn(y, y);
              return ffma2(y, ffma2(u, ffma2(u, ffma2(u, e3, e2), e1), e0), f2(nm));
            });
          }
        } else {
          weigh([&](int c) { return ffma2(make_float2(v[c], v[c + 1]), f2(mul), f2(nm)); });
        }
        l2 = __fadd2_rn(l2, l3);
        if constexpr (BF) {
          // V rows that no row attends, or that were not copied, become zero
          // (by each tile's threads, before its own PV)
          const bool all_rows = okb == kAll && (t0 + kStep <= a_max || (t0 >= lo_min && t0 + kStep <= hi_max));
          if (!all_rows) {
            ok = ok && mbar_wait_bounded(&v_full[st], (j / NS) & 1, a.err);
            const int t = r % kStep, part = 2 * h + r / kStep;  // a quarter of a row's chunks per thread
            if (!(okb >> (t / BS) & 1) || !wanted(t0 + t, 1)) {
#pragma unroll
              for (int sp = 0; sp < SPANS; ++sp)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  *reinterpret_cast<uint4*>(sm + G::kV + st * G::OP + sp * (kStep * kSpan) + t * kSpan + 32 * part + 16 * c) =
                      make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[2 * x + (j & 1)]);
      }
      // the row's sum: both halves' shares
      if (ok && steps > 0) ok = mbar_wait_bounded(&o_done[x], 0, a.err);
      ok = __all_sync(0xffffffffu, ok);
      fence_after_sync();
      const float mine = l2.x + l2.y;
      xch[h * kTile + r] = mine;
      asm volatile("barrier.cta.sync %0, 64;" ::"r"(pair) : "memory");
      const float l = mine + xch[(h ^ 1) * kTile + r];
      const float inv = l == 0.f ? 0.f : a.out_scale / l;
      // The rows go out through the tile's place in Q, which no product reads any
      // more: D / 8 lanes per row then write whole lines (a lane per row took
      // 4 us per CTA, 32 lines per store).
      uint8_t* const rows_s = sm + G::kQ + x * (SPANS * kTile * kSpan);  // [128][D] bf16, chunk c of row r at c ^ (r % 8)
#pragma unroll 1
      for (int c = 0; c < D / 64; ++c) {
        float o[32];
        tmem_ld32(o_col + 32 * c, o);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(rows_s + r * (2 * D) + ((h * (D / 16) + 4 * c + i) ^ (r & 7)) * 16) =
              make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                         pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
      }
      if (any_of(9 + x, 256, !ok)) ok = false;
      if (ok) {
        constexpr int LPR = D / 8, RPI = 256 / LPR;
        const int c = lane % LPR;
#pragma unroll 4
        for (int i = 0; i < kTile / RPI; ++i) {
          const int rr = i * RPI + (tid & 255) / LPR, R = row0 + x * kTile + rr, tok = R / g;
          if (R < rows)
            *reinterpret_cast<uint4*>(a.out + ((size_t)(q0 + tok) * a.num_q_heads + kvh * g + R - tok * g) * D + 8 * c) =
                *reinterpret_cast<const uint4*>(rows_s + rr * (2 * D) + ((c ^ (rr & 7)) * 16));
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  if (w == 0) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

struct Kernel {
  const void* fn = nullptr;
  int smem = 0, threads = 0;
};

template <int KIND, int D, int BS>
Kernel kernel_info() {
  using G = Geo<KIND, D, BS>;
  return Kernel{reinterpret_cast<const void*>(&attn_tiles_kernel<KIND, D, BS>), G::kBytes, G::kThreads};
}

template <int KIND>
Kernel pick(int D, int bs) {
  if (D == 64) return bs == 8 ? kernel_info<KIND, 64, 8>() : bs == 16 ? kernel_info<KIND, 64, 16>() : kernel_info<KIND, 64, 32>();
  return bs == 8 ? kernel_info<KIND, 128, 8>() : bs == 16 ? kernel_info<KIND, 128, 16>() : kernel_info<KIND, 128, 32>();
}

Kernel pick_bf16(int D, int bs);
Kernel pick_fp8(int D, int bs);
Kernel pick_int8(int D, int bs);
Kernel pick_fp4(int D, int bs);

}  // namespace tiles
}  // namespace pkv
