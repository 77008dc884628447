// attn_tiles.cuh -- paged attention with modified scores for many query rows
// per (sequence, kv head) (prompt chunks), on the 5th-generation tensor cores:
// two 128-row query tiles per CTA that share one stream of K and V.  The
// operation and the kinds of cache are those of attn_cols.cuh.
//
// Per step of 128 positions and tile x of the two:
//   S_x = Q_x K^T    M 128, N 128, K = D   (tcgen05.mma, operands in shared memory)
//   P_x = 2^(z - m)  eight softmax warps per tile, two threads per row (64
//                    columns each); P_x goes back to tensor memory, each half
//                    over its own columns of S_x, as the A operand of
//   O_x += P_x V     M 128, N = D, K = 128
// The tensor pipe works on one tile while the other's softmax runs: PV_x(j)
// and S_x(j + 1) are issued together once P_x(j) is there, and their
// completion (one commit) is what the softmax of step j + 1 waits for, so it
// may also rescale O_x without another barrier.  P in tensor memory keeps its
// writes and reads off shared memory, whose 128 B/clock the operands of two
// 128x128x16 products already fill.
//
// The maximum m of a row is lazy: it moves only when a score passes it by more
// than 2^8 (weights stay below 2^8).  Each step the 256 threads of a tile vote
// (one barrier with an OR) whether any row's must; the two threads of a row
// exchange their maxima only then.  S is read twice, 32 columns at a time (for
// the maximum, then for the weights): a load of 32 columns by all 16 warps
// takes 72 cycles, while 64 scores held in registers spilled.
//
// Tensor memory: S_0, S_1 at columns 0 and 128, O_0, O_1 at 256 and 256 + D.
//
// Warps: 0-7 and 8-15 softmax of tiles 0 and 1 (column half (w / 4) % 2); 16
// the copies of K (bf16) or of all codes; 17 the MMAs; 18 the copies of V
// (bf16), or 18 and 19 widen codes to fp16 operands (fp8 and quantised caches).
//
// softcap: cap * tanh(x / cap) through a cubic in (x / cap)^2 while every score
// of a warp's step is below cap / 2 (relative error 6e-7), else through e^2u.
// The cubic is evaluated where the exponent is formed: |cap * tanh(x / cap)| <=
// |x| bounds the scores for the vote on the maximum.
//
// bf16 caches: tensor copies land in the operand layout, P is one bf16 operand
// (a weight keeps 8 bits, as in pkv_paged_attention_multi: a remainder would
// double the products; an output moves by at most 2^-9 max|V|).  Codes: raw
// tiles land in a ring of one block of one cache per slot, four warps widen
// them exactly; q is fp16, each row scaled by a power of two (the factor goes
// to its scores); P is one fp16 operand.  Row scales never touch the codes:
// K's multiplies the score's column, V's is added to the score as its base-2
// logarithm (weight w), and the row sum takes w / s_v.
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

constexpr int kStep = 128;      // positions per step
constexpr int kHalf = 64;       // columns of S per softmax thread
constexpr int kTile = 128;      // query rows per tile (TMEM lanes)
constexpr int kThreads = 640;
constexpr int kSpan = 128;      // bytes of a swizzle span
constexpr int kMaxSmem = 232448;
constexpr int kOkRing = 8;      // steps whose block bits are kept (more than the copies run ahead)

template <int KIND, int D, int BS>
struct Geo {
  static constexpr bool BF = KIND == kBf16;
  static constexpr bool REC = KIND == kInt8 || KIND == kFp4;
  static constexpr int SPANS = D / 64;
  static constexpr int NB = kStep / BS;                       // blocks per step
  static constexpr int OP = SPANS * kStep * kSpan;            // one operand tile of K or V
  static constexpr int NS = D == 128 ? 2 : 3;                 // operand stages of K, of V
  static constexpr int ROW = BF ? 2 * D : (KIND == kFp4 ? D / 2 : D);
  static constexpr int RAW = BF ? 0 : cols::Geo<KIND, D, BS>::BLOCK;  // one block of one cache
  static constexpr int kQ = 0;                                // [tile][span][128 rows][128 B]
  static constexpr int kK = kQ + 2 * SPANS * kTile * kSpan;
  static constexpr int kV = kK + NS * OP;
  static constexpr int kRaw = kV + NS * OP;
  // Row scales as columns: K's, the logarithm and the inverse of V's.  One
  // stage more than the operands have: the softmax of step j still reads K's
  // when the products have freed K's operand stage.
  static constexpr int NCS = NS + 1;
  static constexpr int kColBytes = REC ? 3 * NCS * kStep * 4 : 0;
  static constexpr int kXch = 2 * 2 * kTile * 4;              // a float per softmax thread: row maxima, sums
  static constexpr int kTail = kColBytes + kXch + 2 * kTile * 4 + 1024;  // and q scales, barriers, words
  static constexpr int NR0 = RAW ? (kMaxSmem - kRaw - kTail) / RAW : 0;
  static constexpr int NR = NR0 > 16 ? 16 : NR0;              // raw slots
  static constexpr int kCol = kRaw + NR * RAW;
  static constexpr int kX = kCol + kColBytes;
  static constexpr int kQmul = kX + kXch;                     // [2 * 128] score units of a row
  static constexpr int kBar = (kQmul + 2 * kTile * 4 + 15) / 16 * 16;
  static constexpr int kNumBars = 4 * NS + 6 + 2 * NR;
  static constexpr int kOk = kBar + 8 * kNumBars;
  static constexpr int kTmem = kOk + 4 * kOkRing;
  static constexpr int kBytes = kTmem + 16;
  static constexpr int CPR = ROW >= 128 ? 8 : ROW / 16;       // raw: chunks of a swizzled row
  static_assert(kBytes <= kMaxSmem, "shared memory");
  static_assert(BF || NR >= 4, "raw ring");
};

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
               ::"r"(d), "r"(a_tmem), "l"(b), "r"(id), "r"(acc));
}

// 32 columns of packed operands from registers into this thread's lane.
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]),
        "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]),
        "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

// 16 columns of packed operands.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
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

// tanh(u) / u as a cubic in u^2 for |u| < 1/2 (a fit of least relative error,
// 5.5e-7); beyond, the exponential.
constexpr float kSeriesMax = 0.5f;
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
__global__ void __launch_bounds__(kThreads, 1)
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
  const int s = blockIdx.z, kvh = blockIdx.y;
  const int q0 = __ldg(a.q_start + s);
  const int64_t T64 = (int64_t)__ldg(a.q_start + s + 1) - q0;
  const int L = __ldg(a.seq_lens + s);
  if (L < 0 || L > a.len_clip || T64 < 0 || T64 > L || T64 > a.max_q || q0 < 0 || q0 + T64 > a.total_q) {
    if (tid == 0 && kvh == 0 && blockIdx.x == 0) raise_error(a.err, PKV_DEVERR_BAD_SEQ_LEN);
    return;  // its rows are left alone
  }
  const int T = (int)T64, rows = T * g;
  const int row0 = blockIdx.x * 2 * kTile;
  if (row0 >= rows) return;
  if (smem_addr(sm) & 1023u) {
    if (tid == 0) raise_error(a.err, PKV_DEVERR_SMEM_ALIGN);
    return;
  }
  const int nx = rows - row0 > kTile ? 2 : 1;  // tiles with rows
  const int i0 = row0 / g, i1 = (min(row0 + 2 * kTile, rows) - 1) / g;
  const int hi_min = L - T + i0 + 1, hi_max = L - T + i1 + 1;
  const int lo_min = a.window > 0 ? max(0, hi_min - a.window) : 0;
  const int lo_max = a.window > 0 ? max(0, hi_max - a.window) : 0;
  const int pre = a.prefix_lens ? min(max(__ldg(a.prefix_lens + s), 0), L) : 0;
  const int a_max = max(min(a.sinks, hi_max), pre);
  const int nt = (max(hi_max, a_max) + kStep - 1) / kStep;
  int na = (a_max + kStep - 1) / kStep, wt = lo_min / kStep;
  if (wt <= na) na = wt = 0;
  const int steps = nt - (wt - na);
  auto base_of = [&](int j) -> int { return (j < na ? j : j + (wt - na)) * kStep; };
  const int32_t* table = a.block_tables + (size_t)s * a.table_stride;

  uint64_t* k_full = reinterpret_cast<uint64_t*>(sm + G::kBar);
  uint64_t* k_empty = k_full + NS;
  uint64_t* v_full = k_empty + NS;
  uint64_t* v_empty = v_full + NS;
  uint64_t* s_ready = v_empty + NS;  // [2]
  uint64_t* p_ready = s_ready + 2;   // [2]
  uint64_t* o_done = p_ready + 2;    // [2]
  uint64_t* raw_full = o_done + 2;   // [NR]
  uint64_t* raw_empty = raw_full + NR;
  uint32_t* ok_bits = reinterpret_cast<uint32_t*>(sm + G::kOk);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + G::kTmem);
  float* ksc_s = reinterpret_cast<float*>(sm + G::kCol);  // [NCS][128]
  float* vlg_s = ksc_s + G::NCS * kStep;
  float* vis_s = vlg_s + G::NCS * kStep;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&k_full[i], BF ? 1 : 2);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], BF ? 1 : 2);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_ready[i], 1);
      mbar_init(&p_ready[i], 8);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 2);
    }
    fence_mbar_init();
  }
  if (w == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tslot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- the softmax threads: tile x, column half h, row r of the tile
  const int x = w >> 3, h = (w >> 2) & 1, r = (w & 3) * 32 + lane;
  int hi = 0, lo = 0, al = 0, my_row = -1, my_head = 0;
  if (w < 16) {
    const int R = row0 + x * kTile + r;
    if (R < rows) {
      const int tok = R / g;
      my_row = q0 + tok;
      my_head = kvh * g + R % g;
      hi = L - T + tok + 1;
      lo = a.window > 0 ? max(0, hi - a.window) : 0;
      al = max(min(a.sinks, hi), pre);
    }
  }
  // the first half's threads bring their query rows: K-major, 128-byte swizzle
  float* const qmul_s = reinterpret_cast<float*>(sm + G::kQmul);
  if (w < 16 && h == 0) {
    const uint4* src = reinterpret_cast<const uint4*>(a.q + ((size_t)max(my_row, 0) * a.num_q_heads + my_head) * D);
    float qmul = fabsf(a.qk_scale);
    const uint32_t sign = a.qk_scale < 0.f ? 0x80008000u : 0u;  // a negative scale's sign goes to q
    float up = 1.f;
    if constexpr (!BF) {  // fp16: the row's largest |q| brought into [2^14, 2^15)
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 q = my_row >= 0 ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        mx = __vmaxu2(mx, __vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu));
        mx = __vmaxu2(mx, __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
      }
      mx = max(mx & 0xFFFFu, mx >> 16);
      const int e = min(max((int)(mx >> 7), 20), 254);
      up = __uint_as_float((uint32_t)(268 - e) << 23);
      qmul *= __uint_as_float((uint32_t)(e - 14) << 23);
    }
    // (kept above zero: a masked score, -inf times this, has to stay -inf)
    qmul_s[x * kTile + r] = fmaxf(qmul, 0x1p-120f);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      uint4 v = my_row >= 0 ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      if constexpr (!BF) {
        const float2 f0 = bf16x2_to_f2(v.x), f1 = bf16x2_to_f2(v.y), f2_ = bf16x2_to_f2(v.z), f3 = bf16x2_to_f2(v.w);
        v = make_uint4(pack_f16x2(f0.x * up, f0.y * up), pack_f16x2(f1.x * up, f1.y * up),
                       pack_f16x2(f2_.x * up, f2_.y * up), pack_f16x2(f3.x * up, f3.y * up));
      }
      v.x ^= sign; v.y ^= sign; v.z ^= sign; v.w ^= sign;
      const int sp = c / 8, cc = c % 8;
      *reinterpret_cast<uint4*>(sm + G::kQ + (x * SPANS + sp) * (kTile * kSpan) + r * kSpan + ((cc ^ (r & 7)) << 4)) = v;
    }
  }
  fence_proxy_async_smem();
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
    if (w == 16 || (BF && w == 18)) {
      // ---- copies: the table ids of a step on lanes 0 .. NB - 1, the next
      // step's already in flight
      auto load_id = [&](int j, int b) -> int32_t {
        const int first = base_of(j) + b * BS;
        return j < steps && b < NB && wanted(first, BS) ? __ldg(table + first / BS) : INT32_MIN;
      };
      int32_t id = load_id(0, lane);
      int armed = 0;
      for (int j = 0; j < steps; ++j) {
        const int32_t nid = load_id(j + 1, lane);
        const bool good = id >= 0 && id < a.num_blocks;
        const uint32_t ok = __ballot_sync(0xffffffffu, good);
        const uint32_t bad = __ballot_sync(0xffffffffu, !good && id != INT32_MIN);
        if (lane == 0 && w == 16) {
          if (bad) raise_error(a.err, PKV_DEVERR_BAD_BLOCK_ID);
          ok_bits[j % kOkRing] = ok;
        }
        if constexpr (BF) {
          const int st = j % NS, v = w == 18;
          if (!wait_all(v ? &v_empty[st] : &k_empty[st], ((j / NS) & 1) ^ 1)) break;
          armed = j + 1;
          uint64_t* full = v ? &v_full[st] : &k_full[st];
          const TmaMap* map = v ? &maps.v : &maps.k;
          uint8_t* dst = sm + (v ? G::kV : G::kK) + st * G::OP;
          if (elect_one()) mbar_arrive_expect_tx(full, (uint32_t)(__popc(ok) * BS * D * 2));
          __syncwarp();
#pragma unroll 1
          for (int b = 0; b < NB; ++b) {
            const int blk = __shfl_sync(0xffffffffu, id, b);
            if (!(ok >> b & 1)) continue;
            if (elect_one()) {
#pragma unroll
              for (int sp = 0; sp < SPANS; ++sp)
                tma_span_tile(dst + sp * (kStep * kSpan) + b * (BS * kSpan), map, sp * 64, kvh * BS, blk, full);
            }
            __syncwarp();
          }
        } else {
          bool live = true;
#pragma unroll 1
          for (int c = 0; live && c < 2; ++c) {
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
              const int i = (2 * j + c) * NB + b, sl = i % (NR ? NR : 1);
              const int blk = __shfl_sync(0xffffffffu, id, b);
              live = wait_all(&raw_empty[sl], ((i / (NR ? NR : 1)) & 1) ^ 1);
              if (!live) break;
              armed = i + 1;
              if (elect_one()) {
                uint8_t* dst = sm + G::kRaw + sl * G::RAW;
                if (ok >> b & 1) {
                  mbar_arrive_expect_tx(&raw_full[sl], G::RAW);
                  if constexpr (REC) {
                    bulk_g2s(dst, (c ? a.v_cache : a.k_cache) + ((size_t)blk * a.num_kv_heads + kvh) * G::RAW, G::RAW,
                             &raw_full[sl]);
                  } else {
                    tma_load_3d(dst, c ? &maps.v : &maps.k, 0, kvh * BS, blk, &raw_full[sl]);
                  }
                } else {
                  mbar_arrive(&raw_full[sl]);
                }
              }
              __syncwarp();
            }
          }
          if (!live) break;
        }
        id = nid;
      }
      // no copy may land after the CTA is gone
      if constexpr (BF) {
        uint64_t* full = w == 18 ? v_full : k_full;
        for (int j = max(0, armed - NS); j < armed; ++j)
          if (!wait_all(&full[j % NS], (j / NS) & 1)) break;
      } else {
        for (int i = max(0, armed - NR); i < armed; ++i)
          if (!wait_all(&raw_full[i % NR], (i / NR) & 1)) break;
      }
    } else if (w == 17) {
      // ---- MMA issue
      constexpr uint32_t id_s = idesc_f16kind(kTile, kStep, BF, false);
      constexpr uint32_t id_o = idesc_f16kind(kTile, D, BF, true);
      const uint64_t dq = sw128_desc(smem_addr(sm + G::kQ), 16, 1024);
      const uint64_t dk = sw128_desc(smem_addr(sm + G::kK), 16, 1024);
      const uint64_t dv = sw128_desc(smem_addr(sm + G::kV), kStep * kSpan, 1024);  // MN-major
      auto issue_s = [&](int x, int j, bool last_of_stage) {
        const int st = j % NS;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int sp = k / 4, ko = (k % 4) * 32;
            mma_bf16(tmem + x * kStep, dq + (uint64_t)(((x * SPANS + sp) * (kTile * kSpan) + ko) >> 4),
                     dk + (uint64_t)((st * G::OP + sp * (kStep * kSpan) + ko) >> 4), id_s, k > 0);
          }
          mma_commit(&s_ready[x]);
          if (last_of_stage) mma_commit(&k_empty[st]);
        }
        __syncwarp();
      };
      bool ok = steps > 0 && wait_all(&k_full[0], 0);
      if (ok) {
        fence_after_sync();
        for (int x = 0; x < nx; ++x) issue_s(x, 0, x == nx - 1);
      }
      for (int j = 0; ok && j < steps; ++j) {
        const int st = j % NS;
        for (int x = 0; ok && x < nx; ++x) {
          ok = wait_all(&p_ready[x], j & 1) && (x > 0 || wait_all(&v_full[st], (j / NS) & 1));
          if (!ok) break;
          fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k)
              mma_ts(tmem + 256 + x * D, tmem + x * kStep + (k / 4) * kHalf + 8 * (k % 4), dv + (uint64_t)((st * G::OP + k * 16 * kSpan) >> 4), id_o,
                     (j > 0 || k > 0) ? 1u : 0u);
            if (x == nx - 1) mma_commit(&v_empty[st]);
            if (j + 1 == steps) mma_commit(&o_done[x]);
          }
          __syncwarp();
          if (j + 1 < steps) {
            if (x == 0) {
              ok = wait_all(&k_full[(j + 1) % NS], ((j + 1) / NS) & 1);
              if (!ok) break;
              fence_after_sync();
            }
            issue_s(x, j + 1, x == nx - 1);
          }
        }
      }
      // every MMA issued has completed before TMEM is released: the softmax
      // warps wait for o_done; after a timeout this drains what was issued
      if (!ok && steps > 0) {
        if (elect_one()) mma_commit(&o_done[0]);
        __syncwarp();
        wait_all(&o_done[0], 0);
      }
    } else if (!BF && w >= 18) {
      // ---- widen codes: raw blocks -> fp16 operand rows.  A thread takes the
      // unit k of 16 codes of every kRows-th row, 32 rows at a time so that
      // several units' loads are in flight.
      constexpr int UPR = D / 16, kRows = 64 / UPR, UB = 32 / kRows, BPB = 32 / BS;  // BPB blocks per 32 rows
      const int ct = tid - 18 * 32, k = ct % UPR, p0 = ct / UPR;
      const int c0 = 2 * (k % 4);
      bool live = true;
      for (int j = 0; live && j < steps; ++j) {
        const int st = j % NS, cs = j % G::NCS, t0 = base_of(j);
#pragma unroll 1
        for (int c = 0; live && c < 2; ++c) {
          live = wait_all(c ? &v_empty[st] : &k_empty[st], ((j / NS) & 1) ^ 1);
          if (!live) break;
          uint8_t* op = sm + (c ? G::kV : G::kK) + st * G::OP + (k / 4) * (kStep * kSpan);
#pragma unroll 1
          for (int r0 = 0; r0 < kStep; r0 += 32) {
            const int i0 = (2 * j + c) * NB + r0 / BS;  // raw sequence number of the rows' first block
#pragma unroll
            for (int b = 0; b < BPB; ++b) live = live && wait_all(&raw_full[(i0 + b) % NR], ((i0 + b) / NR) & 1);
            if (!live) break;
            const uint32_t ok = ok_bits[j % kOkRing] >> (r0 / BS);
#pragma unroll
            for (int i = 0; i < UB; ++i) {
              const int rr = i * kRows + p0, p = rr % BS, b = rr / BS;  // row of the 32, of its block
              const int row = r0 + rr;
              const uint8_t* raw = sm + G::kRaw + ((i0 + b) % NR) * G::RAW;
              uint32_t h8[8];
              if constexpr (KIND == kFp4) {
                const uint2 v = *reinterpret_cast<const uint2*>(raw + p * G::ROW + 16 * quant_chunk(p, k / 2, G::ROW) + 8 * (k & 1));
                const uint32_t t = raw[BS * G::ROW + p * (D / 16) + k];
                uint32_t f[4];
                const uint32_t ts = cols::e4m3x2_to_f16x2(t | t << 8);
                cols::e2m1x8_to_f16x2x4(v.x, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) h8[e] = cols::hmul2(f[e], ts);
                cols::e2m1x8_to_f16x2x4(v.y, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) h8[4 + e] = cols::hmul2(f[e], ts);
              } else {
                constexpr int M = G::CPR - 1;
                const uint4 v = *reinterpret_cast<const uint4*>(raw + p * G::ROW + ((k ^ ((p * G::ROW / 128) & M)) << 4));
                const uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if constexpr (KIND == kFp8) e4m3x4_to_f16x2x2(y[e], h8[2 * e], h8[2 * e + 1]);
                  else cols::i8x4_to_f16x2x2(y[e], h8[2 * e], h8[2 * e + 1]);
                }
              }
              // V rows that no row attends, or that were not copied, are zero
              // (0 * NaN is NaN); K rows may hold anything (their scores are masked)
              if (c && (!(ok >> b & 1) || !wanted(t0 + row, 1))) {
#pragma unroll
                for (int e = 0; e < 8; ++e) h8[e] = 0u;
              }
              uint8_t* dst = op + row * kSpan;
              *reinterpret_cast<uint4*>(dst + ((c0 ^ (row & 7)) << 4)) = make_uint4(h8[0], h8[1], h8[2], h8[3]);
              *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ (row & 7)) << 4)) = make_uint4(h8[4], h8[5], h8[6], h8[7]);
            }
            if constexpr (REC) {
              if (ct < 32) {  // the 32 rows' scales, one per lane of the first warp
                const uint8_t* raw = sm + G::kRaw + ((i0 + ct / BS) % NR) * G::RAW;
                const float sc = *reinterpret_cast<const float*>(raw + G::RAW - 4 * BS + 4 * (ct % BS));
                if (!c) {
                  ksc_s[cs * kStep + r0 + ct] = sc;
                } else {
                  const float lg0 = cols::fast_log2(sc), lg = lg0 < cols::kMinLogScale ? cols::kMinLogScale : lg0;
                  vlg_s[cs * kStep + r0 + ct] = lg;
                  // any finite factor will do beside a NaN weight
                  vis_s[cs * kStep + r0 + ct] = lg == lg ? fast_exp2(-lg) : 1.f;
                }
              }
            }
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int b = 0; b < BPB; ++b) mbar_arrive(&raw_empty[(i0 + b) % NR]);
            }
          }
          if (!live) break;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(c ? &v_full[st] : &k_full[st]);
        }
      }
    }
  } else {
    if (x < nx) {
      const uint32_t lane_base = tmem + ((uint32_t)((w & 3) * 32) << 16);
      const uint32_t s_col = lane_base + x * kStep + h * kHalf;  // S, and P over it
      const uint32_t o_col = lane_base + 256 + x * D + h * (D / 2);
      float* const xch = reinterpret_cast<float*>(sm + G::kX) + x * 2 * kTile;  // [2 halves][128 rows]
      const float qmul = qmul_s[x * kTile + r];  // base-2 score units per unit of S (>= 0)
      const float slope = a.slopes && my_row >= 0 ? __ldg(a.slopes + my_head) * 1.4426950408889634f : 0.f;
      const float k1 = qmul * a.inv_cap;  // S -> u = z / cap
      constexpr uint32_t kAll = NB == 32 ? 0xFFFFFFFFu : (1u << NB) - 1u;
      float m = -CUDART_INF_F;
      float2 l2 = f2(0.f);
      // A warp whose wait gave up goes on without waiting (and writes no
      // output): the tile's warps meet at barriers, and none may be left there.
      bool ok = true;
      for (int j = 0; j < steps; ++j) {
        const int t0 = base_of(j), st = j % NS, cs = j % G::NCS, th = t0 + h * kHalf;  // first position of the step, of this half
        ok = ok && wait_all(&s_ready[x], j & 1);
        if constexpr (REC) ok = ok && wait_all(&v_full[st], (j / NS) & 1);  // V's scales come with its codes
        fence_after_sync();
        const uint32_t okb = ok_bits[j % kOkRing];
        // every position of the step attended by every row of the warp?
        const bool inner = __all_sync(0xffffffffu, my_row < 0 || (t0 >= lo && t0 + kStep <= hi)) && okb == kAll;
        // z of 32 columns (from th + 32 q) out of S, in units of `unit`
        const bool plain = !REC && !(a.cap > 0.f) && !a.slopes;
        const float unit = plain ? qmul : 1.f;
        auto score = [&](float (&v)[32], int q, bool series) {
          if constexpr (REC) {
            const float4* ks = reinterpret_cast<const float4*>(ksc_s + cs * kStep + kHalf * h + 32 * q);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 k4 = ks[c];
              const float2 e = __fmul2_rn(make_float2(v[4 * c], v[4 * c + 1]), make_float2(k4.x, k4.y));
              const float2 f = __fmul2_rn(make_float2(v[4 * c + 2], v[4 * c + 3]), make_float2(k4.z, k4.w));
              v[4 * c] = e.x; v[4 * c + 1] = e.y; v[4 * c + 2] = f.x; v[4 * c + 3] = f.y;
            }
          }
          float mul = qmul;
          if (a.cap > 0.f) {
            if (series) {
              cap_series(v, k1);
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = cols::soft_cap(v[c] * qmul, a.cap, a.inv_cap);
              mul = 1.f;
            }
          }
          if (a.slopes) {  // z - slope |p - t|; p = hi - 1
            const float far = (float)(th + 32 * q - (hi - 1));
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = fmaf(v[c], mul, -slope * fabsf(far + (float)c));
            mul = 1.f;
          }
          if constexpr (REC) {
            const float4* lg = reinterpret_cast<const float4*>(vlg_s + cs * kStep + kHalf * h + 32 * q);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float4 l4 = lg[c];
              const float2 e = ffma2(make_float2(v[4 * c], v[4 * c + 1]), f2(mul), make_float2(l4.x, l4.y));
              const float2 f = ffma2(make_float2(v[4 * c + 2], v[4 * c + 3]), f2(mul), make_float2(l4.z, l4.w));
              v[4 * c] = e.x; v[4 * c + 1] = e.y; v[4 * c + 2] = f.x; v[4 * c + 3] = f.y;
            }
          } else if (!plain && !a.slopes) {
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] *= mul;
          }
          if (!inner) {
            const int t32 = th + 32 * q;
            uint32_t keep = low_bits(al - t32) | (low_bits(hi - t32) & ~low_bits(lo - t32));
#pragma unroll
            for (int b = 0; b < 32 / BS; ++b)
              if (!(okb >> ((h * kHalf + 32 * q) / BS + b) & 1)) keep &= ~(low_bits(BS) << (b * (BS & 31)));
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = keep >> c & 1 ? v[c] : -CUDART_INF_F;
          }
        };
        bool series = false, late = false;
        float mt = -CUDART_INF_F;
        if (a.cap > 0.f) {
          float big = 0.f;
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            float v[32];
            tmem_ld32(s_col + 32 * q, v);
            if constexpr (REC) {
              const float* ks = ksc_s + cs * kStep + kHalf * h + 32 * q;
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] *= ks[c];
            }
            big = fmaxf(big, maxabs32(v));
          }
          series = __all_sync(0xffffffffu, big * k1 < kSeriesMax);
          late = series && inner && !REC && !a.slopes;  // cap where the exponent is formed
          if (late) mt = big * qmul;
        }
        auto exact_max = [&]() {
          float t = -CUDART_INF_F;
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            float v[32];
            tmem_ld32(s_col + 32 * q, v);
            score(v, q, series);
            t = fmaxf(t, max32(v));
          }
          return t * unit;
        };
        if (!late) mt = exact_max();
        if (any_of(1 + x, 256, mt > m + cols::kSlack)) {
          if (late) mt = exact_max();  // the bound was not enough: the scores themselves
          xch[h * kTile + r] = mt;
          asm volatile("barrier.cta.sync %0, 256;" ::"r"(1 + x) : "memory");
          mt = fmaxf(mt, xch[(h ^ 1) * kTile + r]);
          asm volatile("barrier.cta.sync %0, 256;" ::"r"(1 + x) : "memory");  // read before the next exchange
          float factor = 1.f;
          if (mt > m + cols::kSlack) {
            factor = m == -CUDART_INF_F ? 0.f : fast_exp2(m - mt);
            m = mt;
            l2 = __fmul2_rn(l2, f2(factor));
          }
          if (j > 0 && __any_sync(0xffffffffu, factor != 1.f)) {  // this half of the row's O
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              float o[32];
              tmem_ld32(o_col + 32 * c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= factor;
              tmem_st32(o_col + 32 * c, o);
            }
          }
        }
        const float nm = m == -CUDART_INF_F ? 0.f : -m;
        float2 l3 = f2(0.f);
        // weights of 32 columns: the exponents' arguments d, packed over S
        auto weigh = [&](int q, auto arg) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            float2 d0 = arg(c), d1 = arg(c + 2);
            d0 = make_float2(fast_exp2(d0.x), fast_exp2(d0.y));
            d1 = make_float2(fast_exp2(d1.x), fast_exp2(d1.y));
            if constexpr (REC) {
              const float4 is = reinterpret_cast<const float4*>(vis_s + cs * kStep + kHalf * h + 32 * q)[c / 4];
              l2 = ffma2(d0, make_float2(is.x, is.y), l2);
              l3 = ffma2(d1, make_float2(is.z, is.w), l3);
            } else {
              l2 = __fadd2_rn(l2, d0);
              l3 = __fadd2_rn(l3, d1);
            }
            pk[c / 2] = BF ? pack_bf16x2(d0.x, d0.y) : pack_f16x2(d0.x, d0.y);
            pk[c / 2 + 1] = BF ? pack_bf16x2(d1.x, d1.y) : pack_f16x2(d1.x, d1.y);
          }
          tmem_st16u(s_col + 16 * q, pk);
        };
        if (late) {
          // z = S qmul (kC0 + u2 (kC1 + u2 (kC2 + u2 kC3))), u2 = (S k1)^2
          const float k2 = k1 * k1;
          const float2 e0 = f2(kC0 * qmul), e1 = f2(kC1 * qmul * k2), e2 = f2(kC2 * qmul * k2 * k2),
                       e3 = f2(kC3 * qmul * k2 * k2 * k2);
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            float v[32];
            tmem_ld32(s_col + 32 * q, v);
            weigh(q, [&](int c) {
              const float2 y = make_float2(v[c], v[c + 1]), u = __fmul2_rn(y, y);
              return ffma2(y, ffma2(u, ffma2(u, ffma2(u, e3, e2), e1), e0), f2(nm));
            });
          }
        } else {
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            float v[32];
            tmem_ld32(s_col + 32 * q, v);
            score(v, q, series);
            weigh(q, [&](int c) { return ffma2(make_float2(v[c], v[c + 1]), f2(unit), f2(nm)); });
          }
        }
        l2 = __fadd2_rn(l2, l3);
        if constexpr (BF) {
          // V rows that no row attends, or that were not copied, become zero
          // (tile 0's threads, half a row each; PV of tile 1 is issued after tile 0's)
          const bool all_rows = okb == kAll && (t0 + kStep <= a_max || (t0 >= lo_min && t0 + kStep <= hi_max));
          if (x == 0 && !all_rows) {
            ok = ok && wait_all(&v_full[st], (j / NS) & 1);
            if (!(okb >> (r / BS) & 1) || !wanted(t0 + r, 1)) {
#pragma unroll
              for (int sp = 0; sp < SPANS; ++sp)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  *reinterpret_cast<uint4*>(sm + G::kV + st * G::OP + sp * (kStep * kSpan) + r * kSpan + 64 * h + 16 * c) =
                      make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[x]);
      }
      // the row's sum: both halves' shares
      if (ok && steps > 0) ok = wait_all(&o_done[x], 0);
      fence_after_sync();
      const float mine = l2.x + l2.y;
      xch[h * kTile + r] = mine;
      asm volatile("barrier.cta.sync %0, 256;" ::"r"(1 + x) : "memory");
      const float l = mine + xch[(h ^ 1) * kTile + r];
      const float inv = l == 0.f ? 0.f : a.out_scale / l;
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          float o[32];
          tmem_ld32(o_col + 32 * c, o);
          if (my_row >= 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.out + ((size_t)my_row * a.num_q_heads + my_head) * D + h * (D / 2) + 32 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                  pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
          }
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
  int smem = 0;
};

template <int KIND, int D, int BS>
Kernel kernel_info() {
  return Kernel{reinterpret_cast<const void*>(&attn_tiles_kernel<KIND, D, BS>), Geo<KIND, D, BS>::kBytes};
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
