// nbits.cuh -- MatMulNBits: how weights of 4 bits lie in memory.
//
// The matrix is kept as tiles of 16 outputs x 128 k, the tiles of 16 outputs
// one behind the other along k.  A tile is what a warp multiplies by mma.sync
// m16n8k16 in eight steps, and lies as its lanes hold it:
//   512 bytes  outputs 0..7:  lane 4 g + t has 16 bytes of output g,
//   512 bytes  outputs 8..15: the same of output g + 8;
//              word b of a lane holds k = 32 b + 16 s + 4 t + j (s 0..1, j
//              0..3) in nibble 2 s + (j / 2) + 4 (j % 2), so that one shift
//              and one mask give the two neighbouring codes of a register;
//   scales     [16][128 / block] in the caller's type;
//   zeros      [16][128 / block] bytes (matrices with zero points).
// A block of 256 is two of 128 with the same scale and zero point.
#pragma once

#include "kv.cuh"

namespace i8q {
namespace nbits {

constexpr int kTileN = 16, kTileK = 128, kCodeBytes = kTileN * kTileK / 2;

struct Shape {
  int64_t N, K;
  int block;       // the caller's
  int scale_size;  // bytes
  int has_zero;
  int64_t strips, chunks;  // tiles along N and K
  int per;                 // blocks of a tile's row
  int tile_bytes;
};

}  // namespace nbits
}  // namespace i8q
