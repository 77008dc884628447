// Tile-attention instances (attn_tiles.cuh): fp8 caches.
#include "attn_tiles.cuh"

namespace pkv {
namespace tiles {
Kernel pick_fp8(int D, int bs) { return pick<kFp8>(D, bs); }
}  // namespace tiles
}  // namespace pkv
