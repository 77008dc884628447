// Column-attention instances (attn_cols.cuh): bf16 caches, head_dim 128.
#include "attn_cols.cuh"

namespace pkv {
namespace cols {
Kernel pick_bf16_128(int bs, int nt) { return pick<kBf16, 128>(bs, nt); }
}  // namespace cols
}  // namespace pkv
