// Tile-attention instances (attn_tiles.cuh): int8 caches.
#include "attn_tiles.cuh"

namespace pkv {
namespace tiles {
Kernel pick_int8(int D, int bs) { return pick<kInt8>(D, bs); }
}  // namespace tiles
}  // namespace pkv
