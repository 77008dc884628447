// quant_cache.cu -- the quantised paged cache: tokens quantised as they are
// written into their slots, and the cache read back as contiguous values.
// Formats and tile layout: quant_layout.cuh, pkv.h.
//
// Both are bound by HBM: one pass over the data, each thread a run of 16
// elements of one row (so that an fp4 group and its scale belong to one
// thread), the 4 or 8 threads of a row joined by shuffles for its maximum.
#include <cmath>

#include "kernels.h"
#include "pkv_device.cuh"
#include "quant_layout.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 16;  // elements per thread

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

// 16 consecutive elements as binary32, from 16-byte aligned memory read once.
__device__ __forceinline__ void load_run(const float* p, float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load_run(const __nv_bfloat16* p, float (&x)[kRun]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = bf16x2_to_f2(w[k]);
      x[8 * i + 2 * k] = f.x;
      x[8 * i + 2 * k + 1] = f.y;
    }
  }
}

// The largest magnitude as its bits: the bits of magnitudes order as the
// magnitudes do, infinity and then NaN above every finite one.
__device__ __forceinline__ uint32_t run_max(const float (&x)[kRun]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// Two binary32 values -> two e2m1 codes (lo in bits 0..3), to nearest even,
// saturating.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// Four codes of 8 bits from four whole numbers -128..127 held as
// 0x4B400000 + n (a float whose unit is 1): the low bytes, plus 128.
__device__ __forceinline__ uint32_t pack4(const float* n) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= ((__float_as_uint(n[i]) + 128u) & 0xFFu) << (8 * i);
  return w;
}

// One run of a row, quantised into its tile: codes, group scale, row scale.
template <int D, int BS, bool FP4>
__device__ __forceinline__ void store_run(const float (&x)[kRun], uint32_t row_max, uint32_t run_m, int seg, int off,
                                          uint8_t* tile) {
  constexpr int ROW = quant_row_bytes(D, FP4);
  const bool bad = row_max >= 0x7F800000u;  // an infinity or a NaN in the row
  const float amax = __uint_as_float(row_max);
  const bool zero = bad || amax < kQuantTiny;
  float* scales = reinterpret_cast<float*>(tile + BS * (ROW + quant_group_bytes(D, FP4)));
  if constexpr (!FP4) {
    const float s = zero ? 0.f : __fdiv_rn(amax, 127.f);
    uint32_t w[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
    if (!zero) {
      float n[kRun];
#pragma unroll
      for (int i = 0; i < kRun; ++i) n[i] = __fadd_rn(rintf(__fdiv_rn(x[i], s)), 12582912.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack4(n + 4 * i);
    }
    *reinterpret_cast<uint4*>(tile + off * ROW + 16 * quant_chunk(off, seg, ROW)) = make_uint4(w[0], w[1], w[2], w[3]);
    if (seg == 0) scales[off] = bad ? __uint_as_float(0x7FC00000u) : s;
  } else {
    const float s = zero ? 0.f : __fdiv_rn(amax, 2688.f);
    uint32_t w[2] = {0u, 0u}, t = 0;
    if (!zero) {
      t = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(run_m), __fmul_rn(6.f, s)), __NV_SATFINITE, __NV_E4M3);
      __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)t, __NV_E4M3);
      const float step = __fmul_rn(__half2float(*reinterpret_cast<__half*>(&hr)), s);
      if (step > 0.f) {
#pragma unroll
        for (int i = 0; i < kRun / 2; ++i)
          w[i / 4] |= e2m1x2(__fdiv_rn(x[2 * i], step), __fdiv_rn(x[2 * i + 1], step)) << (8 * (i % 4));
      }
    }
    *reinterpret_cast<uint2*>(tile + off * ROW + 16 * quant_chunk(off, seg / 2, ROW) + 8 * (seg % 2)) =
        make_uint2(w[0], w[1]);
    tile[BS * ROW + off * (D / 16) + seg] = (uint8_t)t;
    if (seg == 0) scales[off] = bad ? __uint_as_float(0x7FC00000u) : s;
  }
}

// One thread per run: the K and the V run of the same (token, head, segment).
template <class Src, int D, int BS, bool FP4>
__global__ void __launch_bounds__(kThreads) kv_quantize_kernel(const __grid_constant__ QuantWriteArgs a) {
  constexpr int SEGS = D / kRun, TILE = quant_tile_bytes(D, BS, FP4);
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / SEGS;
  const int seg = (int)(i % SEGS);
  const int64_t rows = (int64_t)a.num_tokens * a.num_kv_heads;
  // a row's threads are SEGS consecutive lanes and end together; lanes past
  // the last row stay for the shuffles
  int64_t slot = -1;
  int h = 0;
  if (row < rows) {
    const int t = (int)(row / a.num_kv_heads);
    h = (int)(row % a.num_kv_heads);
    slot = __ldg(a.slot_mapping + t);
    if (slot >= a.num_slots) {
      raise_error(a.err, PKV_DEVERR_BAD_SLOT);
      slot = -1;
    }
  }
  float x[2][kRun];
  uint32_t m[2], rm[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (slot >= 0) {
      load_run(reinterpret_cast<const Src*>(c ? a.v : a.k) + row * D + seg * kRun, x[c]);
    } else {
#pragma unroll
      for (int e = 0; e < kRun; ++e) x[c][e] = 0.f;
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    m[c] = run_max(x[c]);
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
  for (int i = 0; i < 4; ++i)
    __stcs(reinterpret_cast<float4*>(p) + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
}
__device__ __forceinline__ void store_vals(__nv_bfloat16* p, const float (&x)[kRun]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
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
    for (int i = 0; i < kRun; ++i) x[i] = __fmul_rn((float)((int)(w[i / 4] >> (8 * (i % 4)) & 0xFFu) - 128), s);
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(tile + off * ROW + 16 * quant_chunk(off, seg / 2, ROW) + 8 * (seg % 2)));
    const uint32_t tc = __ldg(tile + BS * ROW + off * (D / 16) + seg);
    __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)tc, __NV_E4M3);
    const float t = __half2float(*reinterpret_cast<__half*>(&hr));
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const uint32_t c = w[i / 8] >> (4 * (i % 8));
      // e2m1 bits as the top bits of a binary16 exponent and mantissa: the
      // value times 2^-14, subnormals included
      const __half_raw raw{(unsigned short)((c & 7u) << 9 | (c & 8u) << 12)};
      x[i] = __fmul_rn(__half2float(*reinterpret_cast<const __half*>(&raw)) * 16384.f * t, s);
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
  const int64_t threads = (int64_t)num_tokens * cache->num_kv_heads * (cache->head_dim / kRun);
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
