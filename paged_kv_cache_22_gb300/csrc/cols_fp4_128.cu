// Column-attention instances (attn_cols.cuh): fp4 caches, head_dim 128.
#include "attn_cols.cuh"

namespace pkv {
namespace cols {
Kernel pick_fp4_128(int bs, int nt) { return pick<kFp4, 128>(bs, nt); }
}  // namespace cols
}  // namespace pkv
