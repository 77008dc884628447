// Tile-attention instances (attn_tiles.cuh): fp4 caches.
#include "attn_tiles.cuh"

namespace pkv {
namespace tiles {
Kernel pick_fp4(int D, int bs) { return pick<kFp4>(D, bs); }
}  // namespace tiles
}  // namespace pkv
