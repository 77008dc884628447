// Column-attention instances (attn_cols.cuh): int8 caches, head_dim 64.
#include "attn_cols.cuh"

namespace pkv {
namespace cols {
Kernel pick_int8_64(int bs, int nt) { return pick<kInt8, 64>(bs, nt); }
}  // namespace cols
}  // namespace pkv
