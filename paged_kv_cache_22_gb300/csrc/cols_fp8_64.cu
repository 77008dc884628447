// Column-attention instances (attn_cols.cuh): fp8 caches, head_dim 64.
#include "attn_cols.cuh"

namespace pkv {
namespace cols {
Kernel pick_fp8_64(int bs, int nt) { return pick<kFp8, 64>(bs, nt); }
}  // namespace cols
}  // namespace pkv
