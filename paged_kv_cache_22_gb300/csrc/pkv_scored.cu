// pkv_scored.cu -- host side of pkv_paged_attention_scored and
// pkv_paged_attention_quant: argument validation, the choice of kernel,
// workspace and launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <map>
#include <mutex>
#include <utility>

#include "attn_cols.cuh"
#include "attn_tiles.cuh"
#include "decode_launch.cuh"
#include "kernels.h"

namespace pkv {
namespace {

constexpr size_t kCounters = size_t(1) << 20;  // the other calls' merge counters: left alone

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Column tiles of a call: 8 query rows of a (sequence, kv head) or fewer take
// the 8-column instance, more the 16-column one.
int column_tiles(int64_t rows) { return rows <= 8 ? 1 : 2; }

// Whether a call takes the 128-row tiles: `rows` query rows per (sequence, kv
// head) at most.  The columns read K and V once per 16 rows but cut long
// sequences between all SMs; the tiles read them once per 256 rows and leave
// SMs idle when there are few (sequence, kv head) pairs.  So tiles when there
// are enough 16-row chunks in all.  Times in us, columns / tiles, 8 kv heads, D
// 128, for 64 sequences of 1024-2048 tokens and 4 of 2048-4096 (3 chunks per SM
// are 456 on 152 SMs; 4 x 8 x 192 rows are 384):
//   rows       32       48       64       128      192    | 4 seqs: 128  192
//   bf16     132/96   183/97   235/98   414/101  591/132  |    55/50   73/71
//   int8      98/117  133/118  170/119  313/122  455/162  |    52/68   70/93
//   fp4       97/119  132/120  168/120  309/123  448/162  |    51/69   68/93
// (fp8, D 64: 69/87, 95/88, 120/88, 218/89, 316/115; 38/49, 50/65).  Codes gain
// from 48 rows on; bf16 keeps the columns below 128, as
// pkv_paged_attention_multi does: they hold a weight in 16 bits, the tiles in 8.
bool takes_tiles(bool bf16, bool several, int64_t rows, int num_seqs, int num_kv_heads, int sms) {
  const int64_t chunks = (rows + 15) / 16 * num_seqs * num_kv_heads;
  return several && rows >= (bf16 ? 128 : 48) && chunks >= 3 * sms && num_seqs <= 65535 &&
         (rows + 2 * tiles::kTile - 1) / (2 * tiles::kTile) * num_kv_heads <= INT_MAX;
}

// CTAs per SM the workspace is sized for.
int max_ctas_per_sm(int nt) { return nt == 1 ? 16 : 8; }

// Opt a kernel into its dynamic shared memory once per device; its CTAs per SM.
int prepare(const void* fn, int threads, int smem, int dev) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> known;
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_pair(fn, dev);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  int occ = 0;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem) != cudaSuccess)
    return 0;
  known[key] = occ;
  return occ;
}

cols::Kernel pick_kernel(int kind, int D, int bs, int nt) {
  switch (kind) {
    case cols::kBf16: return D == 64 ? cols::pick_bf16_64(bs, nt) : cols::pick_bf16_128(bs, nt);
    case cols::kFp8: return D == 64 ? cols::pick_fp8_64(bs, nt) : cols::pick_fp8_128(bs, nt);
    case cols::kInt8: return D == 64 ? cols::pick_int8_64(bs, nt) : cols::pick_int8_128(bs, nt);
    default: return D == 64 ? cols::pick_fp4_64(bs, nt) : cols::pick_fp4_128(bs, nt);
  }
}

tiles::Kernel pick_tile_kernel(int kind, int D, int bs) {
  switch (kind) {
    case cols::kBf16: return tiles::pick_bf16(D, bs);
    case cols::kFp8: return tiles::pick_fp8(D, bs);
    case cols::kInt8: return tiles::pick_int8(D, bs);
    default: return tiles::pick_fp4(D, bs);
  }
}

// One call over a cache of any kind; `desc` carries the geometry (its dtype is
// read for the bf16 and fp8 kinds only).
pkv_status attend(int kind, const pkv_cache_desc& desc, void* out, const void* q, pkv_dtype q_dtype,
                  const int32_t* q_start, int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_q_heads,
                  const void* k_cache, const void* v_cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                  const int32_t* seq_lens, int32_t max_seq_len, float scale, float kv_scale,
                  const pkv_score_opts* opts, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  if (num_seqs < 0 || total_q < 0 || (q_start && max_q < 0)) return PKV_ERR_INVALID_ARG;
  if (num_q_heads <= 0 || num_q_heads % desc.num_kv_heads) return PKV_ERR_INVALID_ARG;
  if (max_blocks_per_seq <= 0 || max_seq_len < 0 || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (!(kv_scale > 0.f && std::isfinite(kv_scale))) return PKV_ERR_INVALID_ARG;
  const pkv_score_opts o = opts ? *opts : pkv_score_opts{};
  if (!(o.softcap >= 0.f && std::isfinite(o.softcap)) || o.window_tokens < 0 || o.sink_tokens < 0)
    return PKV_ERR_INVALID_ARG;
  if (q_dtype != PKV_BF16) return PKV_ERR_UNSUPPORTED;
  if (!q_start && total_q != num_seqs) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0) return PKV_OK;
  if (q_start && max_q == 0) return PKV_ERR_INVALID_ARG;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens) return PKV_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(q_start, 4) || !aligned(o.alibi_slopes, 4) ||
      !aligned(o.prefix_lens, 4))
    return PKV_ERR_INVALID_ARG;
  const int D = desc.head_dim, bs = desc.block_size, group = num_q_heads / desc.num_kv_heads;
  const int64_t rows = (int64_t)(q_start ? max_q : 1) * group;
  const int nt = column_tiles(rows), nc = 8 * nt;
  const int64_t chunks = (rows + nc - 1) / nc;
  if (rows > (1 << 30) || num_seqs * chunks > (1 << 30)) return PKV_ERR_UNSUPPORTED;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  unsigned int* err = device_error_word(dev);
  const int sms = pkv_device_sm_count();
  if (!err || sms <= 0) return PKV_ERR_CUDA;
  const size_t need = pkv_scored_workspace_bytes(num_seqs, q_start ? max_q : 1, num_q_heads, desc.num_kv_heads, D);
  if (!workspace || workspace_bytes < need) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PKV_ERR_INVALID_ARG;

  cols::Args a{};
  a.err = err;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_start = q_start;
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.block_tables = block_tables;
  a.table_stride = max_blocks_per_seq;
  a.seq_lens = seq_lens;
  a.num_seqs = num_seqs;
  a.total_q = total_q;
  a.max_q = max_q;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = desc.num_kv_heads;
  a.group = group;
  a.num_blocks = desc.num_blocks;
  const int64_t table_tokens = (int64_t)max_blocks_per_seq * bs;
  a.len_clip = (int)std::min<int64_t>(table_tokens, max_seq_len);
  a.chunks = (int)chunks;
  const float log2e = 1.4426950408889634f;
  a.qk_scale = scale * log2e * kv_scale;
  a.out_scale = kv_scale;
  a.cap = o.softcap * log2e;
  a.inv_cap = o.softcap > 0.f ? 1.f / a.cap : 0.f;
  a.slopes = o.alibi_slopes;
  a.prefix_lens = o.prefix_lens;
  a.window = o.window_tokens;
  a.sinks = o.window_tokens > 0 ? o.sink_tokens : 0;
  a.cuts = reinterpret_cast<cols::Cut*>(static_cast<char*>(workspace) + kCounters);
  a.partials = reinterpret_cast<float*>(a.cuts + (size_t)sms * max_ctas_per_sm(nt));

  TmaMaps maps{};
  if (takes_tiles(kind == cols::kBf16, q_start && max_q > 1, rows, num_seqs, desc.num_kv_heads, sms)) {
    const tiles::Kernel t = pick_tile_kernel(kind, D, bs);
    if (prepare(t.fn, t.threads, t.smem, dev) <= 0) return PKV_ERR_CUDA;
    if ((kind == cols::kBf16 || kind == cols::kFp8) && !encode_operand_maps(&desc, k_cache, v_cache, &maps))
      return PKV_ERR_CUDA;
    const int64_t pairs = (rows + 2 * tiles::kTile - 1) / (2 * tiles::kTile) * desc.num_kv_heads;
    const dim3 grid((unsigned)pairs, 1, (unsigned)num_seqs);
    // more than one wave: longest first, or a long sequence that starts late is
    // what the call ends on
    a.by_length = num_seqs > 1 && num_seqs <= 256 && pairs * num_seqs > sms;
    void* args[] = {&a, &maps};
    return cudaLaunchKernel(t.fn, grid, dim3(t.threads), args, t.smem, st) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  }
  const cols::Kernel k = pick_kernel(kind, D, bs, nt);
  const int occ = prepare(k.fn, 32, k.smem, dev);
  if (occ <= 0) return PKV_ERR_CUDA;
  if (kind == cols::kBf16 || kind == cols::kFp8) {
    DecodeKernel dk;
    dk.tensor_maps = true;
    if (!encode_cache_maps(dk, &desc, k_cache, v_cache, &maps)) return PKV_ERR_CUDA;
  }
  // one wave of warps, no more than there are tiles.  bf16 tiles: 7 warps per
  // SM (128 sequences of up to 8192 tokens in 251 us; 11, as many as fit, 256:
  // fewer copies queue at once); codes: as many as fit (8 x 32768 fp4 tokens:
  // 88 us with 8 warps per SM, 76 with 16)
  const int most = kind == cols::kBf16 && nt == 1 ? 7 : max_ctas_per_sm(nt);
  int64_t grid = (int64_t)sms * std::min(occ, most);
  const int64_t units = num_seqs * chunks * desc.num_kv_heads, each = (a.len_clip + (int64_t)k.tok - 1) / k.tok;  // (below 2^61)
  if (units >= INT_MAX || units * each >= INT_MAX) return PKV_ERR_UNSUPPORTED;  // the kernels count tiles in 32 bits
  const int64_t tiles = units * each;
  grid = std::max<int64_t>(1, std::min(grid, tiles));
  void* args[] = {&a, &maps};
  if (cudaLaunchKernel(k.fn, dim3((unsigned)grid), dim3(32), args, k.smem, st) != cudaSuccess) return PKV_ERR_CUDA;
  // segments cut between warps are merged by a programmatic dependent grid
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(32 * cols::merge_warps((int)std::min<int64_t>(rows, nc)));
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* margs[] = {&a};
  return cudaLaunchKernelExC(&cfg, k.merge, margs) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

size_t pkv_scored_workspace_bytes(int32_t num_seqs, int32_t max_q, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim) {
  if (num_seqs < 0 || max_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  const int sms = pkv_device_sm_count();
  if (sms <= 0) return 0;
  const int64_t rows = (int64_t)max_q * (num_q_heads / num_kv_heads);
  if (takes_tiles(true, max_q > 1, rows, num_seqs, num_kv_heads, sms) && takes_tiles(false, max_q > 1, rows, num_seqs, num_kv_heads, sms))
    return kCounters;  // nothing is cut, whatever the cache
  const int nt = column_tiles(rows);
  const size_t ctas = (size_t)sms * max_ctas_per_sm(nt);
  return kCounters + ctas * sizeof(cols::Cut) + 2 * ctas * cols::slot_floats(8 * nt, head_dim) * sizeof(float);
}

pkv_status pkv_paged_attention_scored(void* out, const void* q, pkv_dtype q_dtype, const int32_t* q_start,
                                      int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_q_heads,
                                      const void* k_cache, const void* v_cache, const pkv_cache_desc* cache,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* seq_lens, int32_t max_seq_len, float scale, float kv_scale,
                                      const pkv_score_opts* opts, void* workspace, size_t workspace_bytes,
                                      pkv_stream_t stream) {
  if (!cache || cache->num_blocks <= 0 || cache->num_kv_heads <= 0 ||
      (cache->head_dim != 64 && cache->head_dim != 128) ||
      (cache->block_size != 8 && cache->block_size != 16 && cache->block_size != 32))
    return PKV_ERR_INVALID_ARG;
  if (cache->dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;  // the products run on the tensor cores
  if (cache->dtype != PKV_BF16 && cache->dtype != PKV_FP8_E4M3) return PKV_ERR_INVALID_ARG;
  const bool fp8 = cache->dtype == PKV_FP8_E4M3;
  return attend(fp8 ? cols::kFp8 : cols::kBf16, *cache, out, q, q_dtype, q_start, num_seqs, total_q, max_q,
                num_q_heads, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens, max_seq_len, scale,
                fp8 ? kv_scale : 1.f, opts, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

pkv_status pkv_paged_attention_quant(void* out, const void* q, pkv_dtype q_dtype, const int32_t* q_start,
                                     int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_q_heads,
                                     const void* k_cache, const void* v_cache, const pkv_quant_desc* cache,
                                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                                     const int32_t* seq_lens, int32_t max_seq_len, float scale,
                                     const pkv_score_opts* opts, void* workspace, size_t workspace_bytes,
                                     pkv_stream_t stream) {
  if (!valid_quant_desc(cache)) return PKV_ERR_INVALID_ARG;
  const pkv_cache_desc geo{cache->num_blocks, cache->block_size, cache->num_kv_heads, cache->head_dim, PKV_BF16};
  return attend(cache->format == PKV_QUANT_FP4 ? cols::kFp4 : cols::kInt8, geo, out, q, q_dtype, q_start, num_seqs,
                total_q, max_q, num_q_heads, k_cache, v_cache, block_tables, max_blocks_per_seq, seq_lens,
                max_seq_len, scale, 1.f, opts, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
