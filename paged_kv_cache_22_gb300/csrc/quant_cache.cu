// quant_cache.cu -- the quantised paged cache: tokens quantised as they are
// written into their slots, and the cache read back as contiguous values.
// Formats and tile layout: quant_layout.cuh, pkv.h.
//
// Both are bound by HBM: one pass over the data, each thread a run of 16
// elements of one row (so that an fp4 group and its scale belong to one
// thread), the 4 or 8 threads of a row joined by shuffles for its maximum.
//
// Measured, 262144 tokens of 8 kv heads, D 128, bf16: write fp4 289 us (1.39 GB,
// 4.8 TB/s; conversions and maxima take two thirds of the issue slots; 308 us
// with exact reciprocals and a division per group), int8 292 us; read-back 244
// us (5.7 TB/s) and 271 us.  The measured copy bandwidth is 6.7 TB/s.
#include <cmath>

#include "kernels.h"
#include "pkv_device.cuh"
#include "quant_layout.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 16;  // elements per thread
constexpr int kTokens = 16;  // tokens of a head that consecutive rows of threads write

struct QuantWriteArgs {
  unsigned int* err;
  const void* k;
  const void* v;
  int num_tokens, num_kv_heads;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t num_slots;
  const int64_t* slot_mapping;
};

struct QuantGatherArgs {
  unsigned int* err;
  void* k_out;
  void* v_out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  int num_blocks, num_kv_heads;
  const int32_t* block_tables;
  int64_t table_stride;
  const int32_t* seq_lens;
  const int64_t* cu_seq_lens;
  int64_t total_tokens;
  int len_clip;
};

// 32 bytes of global memory in one access where the address allows it, past
// L1 (two accesses of 16 bytes touch half of a sector each).
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
// Streaming stores of 16 bytes: L2 joins the halves of a sector.  (One store
// of 32 bytes measured 263 us against 243 for the read-back of 262144 x 8 fp4
// rows, 268 against 271 for int8.)
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(static_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

// A run of 16 consecutive elements, held as it came (8 registers for bf16) and
// widened where it is used.
template <class Src>
struct Run;
template <>
struct Run<float> {
  uint32_t w[2][8];
  __device__ __forceinline__ void load(const float* p) {
    load32(p, w[0]);
    load32(p + 8, w[1]);
  }
  __device__ __forceinline__ float operator[](int i) const { return __uint_as_float(w[i / 8][i % 8]); }
  // The largest magnitude as its bits: the bits of magnitudes order as the
  // magnitudes do, infinity and then NaN above every finite one.
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i) m = max(m, w[i / 8][i % 8] & 0x7FFFFFFFu);
    return m;
  }
};
template <>
struct Run<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { load32(p, w); }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ uint32_t max_bits() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);  // both halves of a word at once
    return max(m << 16, m & 0xFFFF0000u);
  }
};

// Two binary32 values -> two e2m1 codes (lo in bits 0..3), to nearest even,
// saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t e2m1x8(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}
// 1 / x to one place (2^-23), for x and 1 / x normal.
__device__ __forceinline__ float near_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The codes are those of the binary32 quotient x / s.  A division costs about
// ten instructions, more than everything else a run needs, and a product with
// a reciprocal (itself a place off) differs from it by 2^-22 at most: it is used
// wherever that cannot change the code, away from the borders between codes.
// One run in a few thousand takes the division.

// 1.5 * 2^23 + 128: a float whose unit is 1, with the biased code in its low byte.
constexpr float kMagic = 12583040.f;

template <class R>
__device__ __forceinline__ void int8_codes(const R& x, float s, uint32_t (&w)[4]) {
  const float inv = near_rcp(s);
  // |x / s| <= 127 (1 + 2^-22), so that the quotient and the (unrounded) product
  // are within 127 (2^-23 + 2^-24) < 2^-15.4 of each other.  (Ties are not rare: with bf16 elements
  // 127 x / a is a ratio of small whole numbers.)
  constexpr float kNear = 0.5f - 0x1p-15f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float n[4], d[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float2 v = make_float2(x[4 * k + i], x[4 * k + i + 1]), c = make_float2(kMagic, kMagic);
      const float2 r = ffma2(v, make_float2(inv, inv), c);  // rounds x * inv to a whole number, ties to even
      const float2 e = ffma2(v, make_float2(inv, inv), ffma2(r, make_float2(-1.f, -1.f), c));
      n[i] = r.x; n[i + 1] = r.y;
      d[i] = e.x; d[i + 1] = e.y;
    }
    if (fmaxf(fmaxf(fabsf(d[0]), fabsf(d[1])), fmaxf(fabsf(d[2]), fabsf(d[3]))) > kNear) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (fabsf(d[i]) > kNear) n[i] = __fadd_rn(rintf(__fdiv_rn(x[4 * k + i], s)), kMagic);
    }
    const uint32_t lo = __byte_perm(__float_as_uint(n[0]), __float_as_uint(n[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(n[2]), __float_as_uint(n[3]), 0x0040);
    w[k] = __byte_perm(lo, hi, 0x5410);
  }
}

template <class R>
__device__ __forceinline__ void fp4_codes(const R& x, float step, uint32_t (&w)[2]) {
  // codes do not fall as the quotient grows: where a product a little below it
  // and one a little above (2^-21 either way) agree, it has that code too
  const float inv = near_rcp(step), lo = inv * (1.f - 0x1p-21f), hi = inv * (1.f + 0x1p-21f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[8], z[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 v = make_float2(x[8 * h + i], x[8 * h + i + 1]);
      const float2 a = __fmul2_rn(v, make_float2(lo, lo)), b = __fmul2_rn(v, make_float2(hi, hi));
      y[i] = a.x; y[i + 1] = a.y;
      z[i] = b.x; z[i + 1] = b.y;
    }
    w[h] = e2m1x8(y);
    const uint32_t diff = w[h] ^ e2m1x8(z);
    if (diff) {
#pragma unroll
      for (int i = 0; i < 4; ++i)  // the pair of byte i
        if (diff >> (8 * i) & 0xFFu)
          w[h] = (w[h] & ~(0xFFu << (8 * i))) |
                 e2m1x2(__fdiv_rn(x[8 * h + 2 * i], step), __fdiv_rn(x[8 * h + 2 * i + 1], step)) << (8 * i);
    }
  }
}

// One run of a row, quantised into its tile: codes, group scale, row scale.
template <int D, int BS, bool FP4, class R>
__device__ __forceinline__ void store_run(const R& x, uint32_t row_max, uint32_t run_m, int seg, int off,
                                          uint8_t* tile) {
  constexpr int ROW = quant_row_bytes(D, FP4);
  const bool bad = row_max >= 0x7F800000u;  // an infinity or a NaN in the row
  const float amax = __uint_as_float(row_max);
  const bool zero = bad || amax < kQuantTiny;
  const float s = zero ? 0.f : __fmul_rn(amax, FP4 ? 1.f / 2688.f : 1.f / 127.f);
  if constexpr (!FP4) {
    uint32_t w[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
    if (!zero) int8_codes(x, s, w);
    *reinterpret_cast<uint4*>(tile + off * ROW + 16 * quant_chunk(off, seg, ROW)) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t w[2] = {0u, 0u}, t = 0;
    if (!zero) {
      // the group scale, as the codes: by a product where both sides agree
      const float m = __uint_as_float(run_m), s6 = __fmul_rn(6.f, s), u = m * near_rcp(s6);
      const uint32_t both = __nv_cvt_float2_to_fp8x2(make_float2(u * (1.f - 0x1p-21f), u * (1.f + 0x1p-21f)), __NV_SATFINITE, __NV_E4M3);
      t = both & 0xFFu;
      if (t != both >> 8) t = __nv_cvt_float_to_fp8(__fdiv_rn(m, s6), __NV_SATFINITE, __NV_E4M3);
      __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)t, __NV_E4M3);
      const float step = __fmul_rn(__half2float(*reinterpret_cast<__half*>(&hr)), s);
      if (step > 0.f) fp4_codes(x, step, w);
    }
    *reinterpret_cast<uint2*>(tile + off * ROW + 16 * quant_chunk(off, seg / 2, ROW) + 8 * (seg % 2)) =
        make_uint2(w[0], w[1]);
    tile[BS * ROW + off * (D / 16) + seg] = (uint8_t)t;
  }
  if (seg == 0)
    reinterpret_cast<float*>(tile + BS * (ROW + quant_group_bytes(D, FP4)))[off] = bad ? __uint_as_float(0x7FC00000u) : s;
}

// One thread per run: the K and the V run of the same (token, head, segment).
template <class Src, int D, int BS, bool FP4>
__global__ void __launch_bounds__(kThreads, sizeof(Src) == 4 ? 3 : 5) kv_quantize_kernel(const __grid_constant__ QuantWriteArgs a) {
  constexpr int SEGS = D / kRun, TILE = quant_tile_bytes(D, BS, FP4);
  // Consecutive rows of threads are consecutive tokens of one head, kTokens at
  // a time: neighbours in a prompt are neighbours in a tile, so that a warp's
  // row scales (and an fp4 tile's group scales) are one access, not one each.
  constexpr uint32_t GROUP = kTokens * SEGS, PER_CTA = kThreads / GROUP;  // threads of a head's tokens
  const int seg = threadIdx.x % SEGS;
  const uint32_t hh = blockIdx.x * PER_CTA + threadIdx.x / GROUP;
  const uint32_t tg = hh / (uint32_t)a.num_kv_heads;
  const int h = (int)(hh - tg * (uint32_t)a.num_kv_heads);
  const int64_t t = (int64_t)tg * kTokens + threadIdx.x % GROUP / SEGS;
  const int64_t row = t * a.num_kv_heads + h;
  // a row's threads are SEGS consecutive lanes and end together; lanes without
  // a token stay for the shuffles
  const bool have = t < a.num_tokens;
  int64_t slot = -1;
  if (have) {
    slot = __ldg(a.slot_mapping + t);
    if (slot >= a.num_slots) {
      raise_error(a.err, PKV_DEVERR_BAD_SLOT);
      slot = -1;
    }
  }
  Run<Src> x[2] = {};
  uint32_t m[2], rm[2];
  if (have) {  // (a skipped token's row is read too: the loads do not wait for the slot)
    x[0].load(reinterpret_cast<const Src*>(a.k) + row * D + seg * kRun);
    x[1].load(reinterpret_cast<const Src*>(a.v) + row * D + seg * kRun);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    m[c] = x[c].max_bits();
    rm[c] = m[c];
#pragma unroll
    for (int o = SEGS / 2; o > 0; o >>= 1) rm[c] = max(rm[c], __shfl_xor_sync(0xffffffffu, rm[c], o));
  }
  if (slot < 0) return;
  const int64_t at = ((slot / BS) * a.num_kv_heads + h) * TILE;
  const int off = (int)(slot % BS);
  store_run<D, BS, FP4>(x[0], rm[0], m[0], seg, off, a.k_cache + at);
  store_run<D, BS, FP4>(x[1], rm[1], m[1], seg, off, a.v_cache + at);
}

__device__ __forceinline__ void store_vals(float* p, const float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(x[8 * i + k]);
    store32(p + 8 * i, w);
  }
}
__device__ __forceinline__ void store_vals(__nv_bfloat16* p, const float (&x)[kRun]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  store32(p, w);
}

// The 16 values of segment `seg` of row `off` of a tile.
template <int D, int BS, bool FP4>
__device__ __forceinline__ void load_vals(const uint8_t* tile, int off, int seg, float (&x)[kRun]) {
  constexpr int ROW = quant_row_bytes(D, FP4);
  const float s = __ldg(reinterpret_cast<const float*>(tile + BS * (ROW + quant_group_bytes(D, FP4))) + off);
  if constexpr (!FP4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(tile + off * ROW + 16 * quant_chunk(off, seg, ROW)));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kRun; ++i)  // 2^23 + byte, less 2^23 + 128: the code
      x[i] = __fmul_rn(__uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7540 + i % 4)) - 8388736.f, s);
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(tile + off * ROW + 16 * quant_chunk(off, seg / 2, ROW) + 8 * (seg % 2)));
    const uint32_t tc = __ldg(tile + BS * ROW + off * (D / 16) + seg);
    const __half2_raw tr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(tc | tc << 8), __NV_E4M3);
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t f[4];
      asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
          "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
          : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
          : "r"(w[i]));
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // code * group scale is exact in binary16 (six bits)
        const float2 y = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&f[k]), *reinterpret_cast<const __half2*>(&tr)));
        x[8 * i + 2 * k] = __fmul_rn(y.x, s);
        x[8 * i + 2 * k + 1] = __fmul_rn(y.y, s);
      }
    }
  }
}

// One CTA per table entry of a sequence: the block's rows of every head.
template <class Out, int D, int BS, bool FP4>
__global__ void __launch_bounds__(kThreads) gather_quant_kernel(const __grid_constant__ QuantGatherArgs a) {
  constexpr int SEGS = D / kRun, TILE = quant_tile_bytes(D, BS, FP4);
  const int s = blockIdx.y;
  int L = __ldg(a.seq_lens + s);
  if (L < 0 || L > a.len_clip) {
    if (threadIdx.x == 0 && blockIdx.x == 0) raise_error(a.err, PKV_DEVERR_BAD_SEQ_LEN);
    L = L < 0 ? 0 : a.len_clip;
  }
  const int64_t row0 = __ldg(a.cu_seq_lens + s);
  const int seg = threadIdx.x % SEGS, lane_row = threadIdx.x / SEGS;
  for (int64_t j = blockIdx.x; j * BS < L; j += gridDim.x) {
    const int32_t blk = __ldg(a.block_tables + s * a.table_stride + j);
    if (blk < 0 || blk >= a.num_blocks) {
      if (threadIdx.x == 0) raise_error(a.err, PKV_DEVERR_BAD_BLOCK_ID);
      continue;
    }
    for (int r = lane_row; r < a.num_kv_heads * BS; r += kThreads / SEGS) {
      const int h = r / BS, off = r % BS;
      const int64_t p = j * BS + off, tok = row0 + p;
      if (p >= L) continue;
      if (row0 < 0 || tok >= a.total_tokens) {
        raise_error(a.err, PKV_DEVERR_BAD_SEQ_LEN);
        continue;
      }
      const int64_t at = ((int64_t)blk * a.num_kv_heads + h) * TILE;
      const int64_t to = (tok * a.num_kv_heads + h) * D + seg * kRun;
      float x[kRun], y[kRun];
      load_vals<D, BS, FP4>(a.k_cache + at, off, seg, x);
      load_vals<D, BS, FP4>(a.v_cache + at, off, seg, y);
      store_vals(reinterpret_cast<Out*>(a.k_out) + to, x);
      store_vals(reinterpret_cast<Out*>(a.v_out) + to, y);
    }
  }
}

// The instance for a cache geometry.
template <class Fn>
void with_geometry(const pkv_quant_desc* c, Fn&& fn) {
  auto by_bs = [&](auto d, auto fp4) {
    if (c->block_size == 8) fn(d, std::integral_constant<int, 8>{}, fp4);
    else if (c->block_size == 16) fn(d, std::integral_constant<int, 16>{}, fp4);
    else fn(d, std::integral_constant<int, 32>{}, fp4);
  };
  auto by_d = [&](auto fp4) {
    if (c->head_dim == 64) by_bs(std::integral_constant<int, 64>{}, fp4);
    else by_bs(std::integral_constant<int, 128>{}, fp4);
  };
  if (c->format == PKV_QUANT_FP4) by_d(std::true_type{});
  else by_d(std::false_type{});
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

unsigned int* current_error_word() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess ? device_error_word(dev) : nullptr;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_quant_tile_bytes(int32_t head_dim, int32_t block_size, pkv_quant_format format) {
  const pkv_quant_desc c{1, block_size, 1, head_dim, format};
  return valid_quant_desc(&c) ? (size_t)quant_tile_bytes(head_dim, block_size, format == PKV_QUANT_FP4) : 0;
}

pkv_status pkv_kv_quantize_and_cache(const void* k, const void* v, pkv_dtype src_dtype, int32_t num_tokens,
                                     void* k_cache, void* v_cache, const pkv_quant_desc* cache,
                                     const int64_t* slot_mapping, pkv_stream_t stream) {
  if (num_tokens < 0 || !valid_quant_desc(cache)) return PKV_ERR_INVALID_ARG;
  if (src_dtype != PKV_F32 && src_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
    return PKV_ERR_INVALID_ARG;
  const int64_t threads =
      ((int64_t)num_tokens + kTokens - 1) / kTokens * kTokens * cache->num_kv_heads * (cache->head_dim / kRun);
  const int64_t ctas = (threads + kThreads - 1) / kThreads;
  if (ctas > 0x7FFFFFFF) return PKV_ERR_UNSUPPORTED;
  unsigned int* err = current_error_word();
  if (!err) return PKV_ERR_CUDA;
  const QuantWriteArgs a{err, k, v, num_tokens, cache->num_kv_heads, static_cast<uint8_t*>(k_cache),
                         static_cast<uint8_t*>(v_cache), (int64_t)cache->num_blocks * cache->block_size, slot_mapping};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  with_geometry(cache, [&](auto d, auto bs, auto fp4) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    constexpr bool F = decltype(fp4)::value;
    if (src_dtype == PKV_BF16) kv_quantize_kernel<__nv_bfloat16, D, BS, F><<<(unsigned)ctas, kThreads, 0, st>>>(a);
    else kv_quantize_kernel<float, D, BS, F><<<(unsigned)ctas, kThreads, 0, st>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_gather_kv_quant(void* k_out, void* v_out, pkv_dtype out_dtype, const void* k_cache,
                               const void* v_cache, const pkv_quant_desc* cache, const int32_t* block_tables,
                               int32_t max_blocks_per_seq, const int32_t* seq_lens, const int64_t* cu_seq_lens,
                               int32_t num_seqs, int64_t total_tokens, int32_t max_seq_len, pkv_stream_t stream) {
  if (num_seqs < 0 || max_seq_len < 0 || max_blocks_per_seq <= 0 || total_tokens < 0 || !valid_quant_desc(cache))
    return PKV_ERR_INVALID_ARG;
  if (out_dtype != PKV_F32 && out_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_seq_len == 0 || total_tokens == 0) return PKV_OK;
  if (num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
  if (!k_out || !v_out || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out) || !aligned16(k_cache) || !aligned16(v_cache) ||
      (reinterpret_cast<uintptr_t>(cu_seq_lens) & 7u) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return PKV_ERR_INVALID_ARG;
  unsigned int* err = current_error_word();
  if (!err) return PKV_ERR_CUDA;
  const int64_t table_tokens = (int64_t)max_blocks_per_seq * cache->block_size;
  const int len_clip = (int)(table_tokens < max_seq_len ? table_tokens : max_seq_len);
  const QuantGatherArgs a{err, k_out, v_out, static_cast<const uint8_t*>(k_cache),
                          static_cast<const uint8_t*>(v_cache), cache->num_blocks, cache->num_kv_heads, block_tables,
                          max_blocks_per_seq, seq_lens, cu_seq_lens, total_tokens, len_clip};
  const dim3 grid((unsigned)((len_clip + cache->block_size - 1) / cache->block_size), (unsigned)num_seqs);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  with_geometry(cache, [&](auto d, auto bs, auto fp4) {
    constexpr int D = decltype(d)::value, BS = decltype(bs)::value;
    constexpr bool F = decltype(fp4)::value;
    if (out_dtype == PKV_BF16) gather_quant_kernel<__nv_bfloat16, D, BS, F><<<grid, kThreads, 0, st>>>(a);
    else gather_quant_kernel<float, D, BS, F><<<grid, kThreads, 0, st>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
