// Microscaled 4-bit floating point: formats, the layout of the scales and the
// bit fields of the block-scaled tensor-core instructions, shared by the host
// code, the kernels and the tests.
//
// Values are e2m1 ({0, .5, 1, 1.5, 2, 3, 4, 6} with a sign), two a byte, the
// even column in the low half; a matrix [R, K] is stored row-major, K / 2
// bytes a row.  Each block of 16 (nvfp4) or 32 (mxfp4) columns of a row has
// one scale byte (e4m3 or e8m0).  Scales lie in tiles of 128 rows x 4 blocks,
// 512 bytes each, tiles along K first:
//   byte (r % 32) * 16 + (r / 32 % 4) * 4 + b % 4 of tile (r / 128, b / 4),
// which is how the tensor cores want them: one tcgen05.cp of a tile's 32 rows
// of 16 bytes puts the 4 scales of row 32 q + l into TMEM lane l, column q.
// Bytes of a tile past the last block are zero, so that K need not fill the
// tile: a zero scale against zero-filled values adds zero.
// The rows of a group (an expert's) start on a new tile.
#pragma once

#include <cstdint>

#include "layout.h"

namespace bwg {

constexpr int kNvfp4 = 0;
constexpr int kMxfp4 = 1;
constexpr int kScaleTileRows = 128;
constexpr int kScaleTileBytes = 512;

// Largest number of rows or columns: rounded up to tiles it is still an int.
constexpr int kFp4MaxSize = 0x7fffffff - 511;

BWG_HD int fp4_block(int format) { return format == kNvfp4 ? 16 : 32; }

BWG_HD int pad128(int rows) { return (rows + 127) & ~127; }

// Scale tiles along K.
BWG_HD int fp4_k_tiles(int K, int format) {
  const int cols = 4 * fp4_block(format);
  return (K + cols - 1) / cols;
}

// Byte of the scale of (scale row r, block b).
BWG_HD long long fp4_scale_offset(long long r, int b, int k_tiles) {
  return ((r >> 7) * k_tiles + (b >> 2)) * kScaleTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// Instruction descriptor of the block-scaled kinds (public PTX ISA, tcgen05
// "Instruction descriptor" for .kind::mxf4nvf4):
//   [4,6) scale-B id   [7,10) A format (1 = e2m1)   [10,12) B format
//   [17,23) N >> 3     23 scale format (0 = ue4m3, 1 = ue8m0)
//   [27,29) M >> 7     [29,31) scale-A id
// The ids pick the first of the 2 scales an instruction uses (K = 64, blocks
// of 32) among the 4 of a TMEM word; with blocks of 16 it uses all 4 (id 0).
BWG_HD uint32_t make_idesc_fp4(int format, uint32_t m, uint32_t n, uint32_t scale_id) {
  return (scale_id << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((format == kMxfp4 ? 1u : 0u) << 23) |
         ((m >> 7) << 27) | (scale_id << 29);
}

}  // namespace bwg
