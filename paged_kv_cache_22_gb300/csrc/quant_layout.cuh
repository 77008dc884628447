// quant_layout.cuh -- the layout of a quantised (block, kv head) tile, shared
// by the kernels that write it, read it back and attend over it, and by the
// host code that sizes it.
//
// A quantised cache is [num_blocks, Hkv, tile], tile a run of bytes:
//   codes         [bs][row bytes]   int8: one byte per element, code + 128;
//                                   fp4: two e2m1 codes per byte, the even
//                                   element in the low half
//   group scales  [bs][D / 16]      fp4 only: e4m3, one per 16 elements
//   row scales    [bs]              binary32, one per token
// so that one bulk copy brings everything a kernel needs of a tile.  The
// 16-byte chunks of a code row are permuted within the row by the row's
// 128-byte line, chunk c of row r at c ^ ((r * row / 128) mod (row / 16)):
// eight lanes that read the same chunk of eight consecutive lines, or eight
// chunks of one line, then fall in eight different bank groups of shared
// memory (the pattern of the 128- and 64-byte tensor-copy swizzles, here
// written to global memory so that a plain copy keeps it).
#pragma once

#include <stdint.h>

#include "../../include/pkv.h"

namespace pkv {

// Rows whose largest magnitude is below this are stored as zeros (scale 0):
// every other scale is then at least 2^-80 / 2688 > 2^-92, so that quotients
// and base-2 logarithms of scales stay in range.
constexpr float kQuantTiny = 0x1p-80f;

__host__ __device__ constexpr int quant_row_bytes(int D, bool fp4) { return fp4 ? D / 2 : D; }
__host__ __device__ constexpr int quant_group_bytes(int D, bool fp4) { return fp4 ? D / 16 : 0; }
__host__ __device__ constexpr int quant_tile_bytes(int D, int bs, bool fp4) {
  return bs * (quant_row_bytes(D, fp4) + quant_group_bytes(D, fp4) + 4);
}
// Position, within its row, of 16-byte chunk c of row r.
__host__ __device__ constexpr int quant_chunk(int r, int c, int row_bytes) {
  return c ^ ((r * row_bytes / 128) & (row_bytes / 16 - 1));
}

inline bool valid_quant_desc(const pkv_quant_desc* c) {
  return c && c->num_blocks > 0 && c->num_kv_heads > 0 && (c->head_dim == 64 || c->head_dim == 128) &&
         (c->block_size == 8 || c->block_size == 16 || c->block_size == 32) &&
         (c->format == PKV_QUANT_INT8 || c->format == PKV_QUANT_FP4);
}

}  // namespace pkv
