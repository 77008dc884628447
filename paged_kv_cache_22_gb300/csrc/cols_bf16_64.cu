// Column-attention instances (attn_cols.cuh): bf16 caches, head_dim 64.
#include "attn_cols.cuh"

namespace pkv {
namespace cols {
Kernel pick_bf16_64(int bs, int nt) { return pick<kBf16, 64>(bs, nt); }
}  // namespace cols
}  // namespace pkv
