// Column-attention instances (attn_cols.cuh): int8 caches, head_dim 128.
#include "attn_cols.cuh"

namespace pkv {
namespace cols {
Kernel pick_int8_128(int bs, int nt) { return pick<kInt8, 128>(bs, nt); }
}  // namespace cols
}  // namespace pkv
