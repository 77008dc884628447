// Tile-attention instances (attn_tiles.cuh): bf16 caches.
#include "attn_tiles.cuh"

namespace pkv {
namespace tiles {
Kernel pick_bf16(int D, int bs) { return pick<kBf16>(D, bs); }
}  // namespace tiles
}  // namespace pkv
