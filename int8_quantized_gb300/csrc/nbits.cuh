// nbits.cuh -- MatMulNBits: how weights of 4 bits lie in memory.
//
// The matrix is kept as tiles of 16 outputs x 128 k, the tiles of 16 outputs
// one behind the other along k.  A tile:
//   codes      [4][16][16 bytes]: of each 32 k, each output's; word t of an
//              output's four holds k = 16 s + 4 t + j (s 0..1, j 0..3) in
//              nibble s + 2 (j / 2) + 4 (j % 2), so that a shift and a mask
//              give two neighbouring codes (nibbles i and i + 4) for a
//              register of two 16-bit numbers.  A thread of nbits_tc.cu reads
//              an output's 16 bytes; lane 4 g + t of nbits.cu's mma.sync the
//              words t of outputs g and g + 8, which are words `lane` and
//              32 + `lane` of the 32 k's 64;
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

// A call, for either product kernel.
struct Args {
  Shape s;
  const uint8_t* packed;
  const void* A;
  int64_t lda;
  int a_aligned;  // four neighbouring activations can be read at once
  const float* bias;
  void* Y;
  int64_t ldy;
  int M;
  int wk, wf;     // warps along k, strips at a time: wk * wf warps
  int clusters;   // of a tile of rows
};

constexpr int kWarps = 16, kMostCtas = 8;  // of a CTA, of a cluster
constexpr int kRound = 16;                 // groups of strips between two meetings of a cluster

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// N scales or zero points of a tile's row, read as few words.
template <class T, int N>
struct Row {
  static constexpr int kBytes = N * (int)sizeof(T), kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ Row() {  // zero points of 8
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0x08080808u;
  }
  __device__ __forceinline__ Row(const uint8_t* tile, int row) {
    const uint8_t* p = tile + row * kBytes;
    if constexpr (kBytes == 1) w[0] = *p;
    else if constexpr (kBytes == 2) w[0] = *reinterpret_cast<const uint16_t*>(p);
    else if constexpr (kBytes == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) *reinterpret_cast<uint4*>(w + i) = *reinterpret_cast<const uint4*>(p + 4 * i);
    }
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ uint32_t pair(int i) const {  // a zero point twice, as code_pair() takes it
    return __byte_perm(w[i / 4], 0x3d3d3d3du, 0x4040u + (i & 3) * 0x0101u);
  }
};

// Codes enter the products as bf16 numbers of 2^-12, and sums keep that unit:
// a block's products of the largest activations (128 of them, by up to 15)
// stay within fp32, however small its scale.
constexpr float kUnit = 4096.0f;

// Two codes at nibbles 0 and 4 of w as bf16 numbers less their zero point:
// 0x3d over a byte c < 128 is 2^-5 + c 2^-12, and the zero point's number is
// subtracted exactly.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t zero) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x3d003d00, 0xea;" : "=r"(v) : "r"(w));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(zero));
  return r;
}

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The products of several rows of bf16 activations on the tcgen05 pipe
// (nbits_tc.cu): whether TMA can read them, and the launch.
bool tc_takes(const Args& a);
int run_tc(Args& a, cudaStream_t stream);

}  // namespace nbits
}  // namespace i8q
