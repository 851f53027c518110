// nbits.cu -- MatMulNBits [NBITS]: products of a few rows of fp32 or bf16
// activations with weights of 4 bits that have a scale, and perhaps a zero
// point, per block of their row:
//   Y[m][n] = sum_k A[m][k] (q[n][k] - z[n][k / block]) s[n][k / block] + bias[n].
#include <cooperative_groups.h>

#include <string>

#include "nbits.cuh"

namespace i8q {
namespace {

namespace cg = cooperative_groups;
using namespace nbits;

constexpr int64_t kMost = INT32_MAX - 65536;  // of N, K and M: indices of 32 bits step past them by a tile or two

int check_shape(int64_t N, int64_t K, int64_t block, int scale_type, bool has_zero, const char* who, Shape& out) {
  const std::string w = who;
  if (N < 1 || K < 1 || N > kMost || K > kMost) return fail(I8Q_ERR_INVALID_ARG, w + ": N and K must be 1 .. 2^31 - 2^16");
  if (scale_type != I8Q_F32 && scale_type != I8Q_BF16)
    return fail(I8Q_ERR_INVALID_ARG, w + ": scales must be I8Q_F32 or I8Q_BF16");
  if (block != 16 && block != 32 && block != 64 && block != 128 && block != 256)
    return fail(I8Q_ERR_UNSUPPORTED, w + ": block_size must be 16, 32, 64, 128 or 256");
  out.N = N, out.K = K, out.block = (int)block;
  out.scale_size = scale_type == I8Q_F32 ? 4 : 2, out.has_zero = has_zero;
  out.strips = ceil_div(N, kTileN), out.chunks = ceil_div(K, kTileK);
  out.per = kTileK / (int)std::min<int64_t>(block, kTileK);
  out.tile_bytes = kCodeBytes + kTileN * out.per * (out.scale_size + (has_zero ? 1 : 0));
  return I8Q_OK;
}

// ---- layout -------------------------------------------------------------
// A CTA a tile: a thread writes one word of codes, then shares of the scales
// and zero points.  Once per matrix, when a model is loaded: 128000 x 4096 in
// 330 us, of which its bytes take 83; a thread waits for the few it reads.
__global__ void __launch_bounds__(256)
pack_kernel(Shape s, const uint8_t* __restrict__ B, const void* __restrict__ scales, const uint8_t* __restrict__ zeros,
            uint8_t* __restrict__ packed) {
  const int64_t blocks = (s.K + s.block - 1) / s.block;
  const int64_t row_bytes = blocks * (s.block / 2), zero_bytes = (blocks + 1) / 2;  // (rows of 8 bytes or more, all even)
  const bool even = reinterpret_cast<uintptr_t>(B) % 2 == 0;
  for (int64_t tile = blockIdx.x; tile < s.strips * s.chunks; tile += gridDim.x) {
    const int64_t strip = tile / s.chunks, chunk = tile - strip * s.chunks;
    uint8_t* to = packed + tile * s.tile_bytes;
    {
      const int b = threadIdx.x / 64, t = threadIdx.x % 4;
      const int64_t n = strip * kTileN + threadIdx.x / 4 % 16;
      uint32_t word = 0;
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int64_t k = chunk * kTileK + 32 * b + 16 * st + 4 * t;
        uint32_t four = 0;  // codes k .. k + 3; past the matrix 0, which no activation or a scale of 0 meets
        if (n < s.N && k + 4 <= s.K && even) {
          four = *reinterpret_cast<const uint16_t*>(B + n * row_bytes + k / 2);
        } else {
          for (int j = 0; j < 4; ++j)
            if (n < s.N && k + j < s.K) four |= (B[n * row_bytes + (k + j) / 2] >> (4 * (j & 1)) & 15u) << 4 * j;
        }
        word |= ((four & 15u) | (four >> 4 & 15u) << 16 | (four >> 8 & 15u) << 8 | (four >> 12) << 24) << 4 * st;
      }
      reinterpret_cast<uint32_t*>(to)[threadIdx.x] = word;
    }
    for (int i = threadIdx.x; i < kTileN * s.per; i += blockDim.x) {
      const int64_t n = strip * kTileN + i / s.per, block = (chunk * kTileK + i % s.per * (kTileK / s.per)) / s.block;
      const bool in = n < s.N && block < blocks;
      if (s.scale_size == 4)
        reinterpret_cast<float*>(to + kCodeBytes)[i] = in ? static_cast<const float*>(scales)[n * blocks + block] : 0.0f;
      else
        reinterpret_cast<uint16_t*>(to + kCodeBytes)[i] = in ? static_cast<const uint16_t*>(scales)[n * blocks + block] : 0;
      if (s.has_zero)
        to[kCodeBytes + kTileN * s.per * s.scale_size + i] =
            in ? zeros[n * zero_bytes + block / 2] >> (4 * (block & 1)) & 15u : 8u;
    }
  }
}

constexpr int kRows = 8, kOut = kRows * kTileN;  // of a product, and its outputs

// A warp's ring: stages of its tiles of one strip (or of one tile, where it
// has no fixed number of them), one of which is read while the others arrive.
constexpr int stage_tiles(int c) { return c ? c : 1; }
constexpr int stages(int c) { return c == 4 ? 2 : c == 2 ? 3 : 6; }

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// The same with a sum of 0 before it.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(0.0f));
}

// A fragment of activations: four neighbours of row m from k on, as bf16
// pairs; fp32 in three parts of 8 bits cut off one after the other, which are
// all of its 24 (an infinity or a NaN in the first part alone).
template <class T>
struct Fragment;
template <>
struct Fragment<__nv_bfloat16> {
  static constexpr int kParts = 1;
  uint32_t b[1][2];
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int k, int K, bool live, bool aligned) {
    b[0][0] = b[0][1] = 0;
    if (!live) return;
    if (aligned && k + 4 <= K) {
      const uint2 v = *reinterpret_cast<const uint2*>(row + k);
      b[0][0] = v.x, b[0][1] = v.y;
      return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j < K)
        b[0][j / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(row)[k + j] << (16 * (j & 1));
  }
};
template <>
struct Fragment<float> {
  static constexpr int kParts = 3;
  uint32_t b[3][2];
  __device__ __forceinline__ void load(const float* row, int k, int K, bool live, bool aligned) {
    float x[4] = {};
    if (live) {
      if (aligned && k + 4 <= K) {
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(row + k);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k + j < K) x[j] = row[k + j];
      }
    }
    uint32_t part[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = __float_as_uint(x[j]);
      const bool odd = (u & 0x7f800000u) == 0x7f800000u;
      // a NaN keeps a bit of its mantissa
      part[0][j] = (u >> 16) | (odd && (u & 0x7fffffu) ? 0x40u : 0u);
      const float r1 = odd ? 0.0f : __fsub_rn(x[j], __uint_as_float(u & 0xffff0000u));
      part[1][j] = __float_as_uint(r1) >> 16;
      const float r2 = __fsub_rn(r1, __uint_as_float(__float_as_uint(r1) & 0xffff0000u));
      part[2][j] = __float_as_uint(r2) >> 16;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) b[p][0] = part[p][0] | part[p][1] << 16, b[p][1] = part[p][2] | part[p][3] << 16;
  }
};

// A warp has the activations of its share of k (at most C chunks of 128; C 0:
// read again for each tile) in registers, as the fragments of the products,
// and streams the tiles of one strip of 16 outputs after the other through a
// ring of its own in shared memory, each lane copying what it will read.  The
// warps of a strip add their sums up in shared memory, those of a cluster's
// CTAs through it.  Rows: 8 at a time.  G: the block, at most 128.  ST: the
// scales' type.  The products of a block are summed by the tensor pipe from 0
// and enter the row's sum by a rounded fma with the block's scale (the pipe
// cuts sums instead of rounding them; for fp32 activations only one step's 16
// products are left to it).
// Measured: 1 x 4096 -> 128000 62 us, 4.5 TB/s (the bytes take 42), 1 x 4096 ->
// 14336 10 (4.5), 8 x 14336 -> 4096 15 (5.1).  178 instructions for the 2048
// weights of a tile, of which 88 turn codes into bf16, take 0.63 of the issue
// slots: four warps a scheduler do not hide the chains of those conversions (per
// issue 1.2 cycles of fixed latency and 1.2 of a busy ALU pipe are waited for).
// In short calls the start and the strips' meetings come on top.  More tiles of a
// strip for each meeting pay (C 4 instead of 2 with all 16 warps along k: 63
// and 75 us), more tiles on their way do not.
template <class T, int C, int G, class ST>
__global__ void __launch_bounds__(512, 1)
nbits_kernel(const __grid_constant__ Args a) {
  constexpr int kParts = Fragment<T>::kParts, kPer = kTileK / G;
  constexpr int kStages = stages(C), kTiles = stage_tiles(C);
  extern __shared__ __align__(16) uint8_t smem[];
  const int S = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane / 4, t = lane & 3;
  const int wk = warp % a.wk, wf = warp / a.wk;
  const int cluster = blockIdx.x / S, rows0 = cluster / a.clusters * kRows, c0 = cluster % a.clusters;
  const int rows = min(kRows, a.M - rows0);
  const int chunks = (int)a.s.chunks, strips = (int)a.s.strips, tile_bytes = a.s.tile_bytes;
  const int parts = a.wk * S, part = rank * a.wk + wk;
  const int c_begin = (int)((int64_t)part * chunks / parts), cw = (int)((int64_t)(part + 1) * chunks / parts) - c_begin;
  const int groups = (strips + a.wf - 1) / a.wf, ng = (groups - c0 + a.clusters - 1) / a.clusters;
  const int strip0 = c0 * a.wf + wf, strip_step = a.clusters * a.wf;
  const int live = cw && strip0 < strips ? (strips - strip0 + strip_step - 1) / strip_step : 0;  // groups with a strip for this warp
  uint8_t* const ring = smem + (size_t)warp * kStages * kTiles * tile_bytes;
  float* const partial = reinterpret_cast<float*>(smem + (size_t)a.wk * a.wf * kStages * kTiles * tile_bytes);
  float* const held = partial + 2 * a.wk * a.wf * kOut;

  kv::next_kernel_may_start();
  kv::wait_previous_kernel();

  // the next stage to send for
  const uint8_t* from = a.packed + ((int64_t)strip0 * chunks + c_begin) * tile_bytes + lane * 16;
  const int64_t jump = ((int64_t)strip_step * chunks - (C ? 0 : cw)) * tile_bytes;
  int left = C ? live : live * cw, in_group = 0;  // (tiles of 1 KB at least: their number fits)
  const uint32_t ring_begin = (uint32_t)__cvta_generic_to_shared(ring) + lane * 16;
  const uint32_t ring_end = ring_begin + kStages * kTiles * tile_bytes;
  uint32_t to = ring_begin;
  const int meta = (tile_bytes - kCodeBytes) / 16;  // at most 40
  const bool meta1 = lane < meta, meta2 = lane + 32 < meta;
  auto send = [&] {
    if (left > 0) {
#pragma unroll
      for (int c = 0; c < kTiles; ++c) {
        if (C && c >= cw) break;
        const uint8_t* p = from + c * tile_bytes;
        const uint32_t d = to + c * tile_bytes;
        copy16(d, p);
        copy16(d + 512, p + 512);
        if (meta1) copy16(d + kCodeBytes, p + kCodeBytes);
        if (meta2) copy16(d + kCodeBytes + 512, p + kCodeBytes + 512);
      }
      --left;
      if (C) from += jump;
      else if (from += tile_bytes; ++in_group == cw) in_group = 0, from += jump;
      to += kTiles * tile_bytes;
      if (to == ring_end) to = ring_begin;
    }
    commit();
  };
  for (int i = 0; i < kStages - 1; ++i) send();

  const T* const A = static_cast<const T*>(a.A);
  Fragment<T> x[C ? C : 1][8];
  auto load_x = [&](int slot, int c) {
#pragma unroll
    for (int st = 0; st < 8; ++st)
      x[slot][st].load(A + (int64_t)(rows0 + g) * a.lda, (c_begin + c) * kTileK + st * 16 + 4 * t, (int)a.s.K,
                       c < cw && g < rows, a.a_aligned);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) load_x(c, c);

  const uint8_t* at = ring;
  auto next = [&] {
    at += kTiles * tile_bytes;
    if (at == ring + kStages * kTiles * tile_bytes) at = ring;
  };
  auto arrived = [&] {
    wait_copies<kStages - 2>();
    __syncwarp();  // the scales and zero points were copied by other lanes, and all have read the stage before
    send();
  };
  auto tile = [&](const Fragment<T> (&xc)[8], const uint8_t* at, float (&y)[4]) {
    uint32_t w0[4], w1[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      w0[b] = reinterpret_cast<const uint32_t*>(at)[b * 64 + lane];
      w1[b] = reinterpret_cast<const uint32_t*>(at)[b * 64 + 32 + lane];
    }
    const Row<ST, kPer> s0(at + kCodeBytes, g), s1(at + kCodeBytes, g + 8);
    Row<uint8_t, kPer> z0, z1;
    if (a.s.has_zero) {
      z0 = Row<uint8_t, kPer>(at + kCodeBytes + kTileN * kPer * sizeof(ST), g);
      z1 = Row<uint8_t, kPer>(at + kCodeBytes + kTileN * kPer * sizeof(ST), g + 8);
    }
    float acc[4];
#pragma unroll
    for (int st = 0; st < 8; ++st) {
      const int i = st * 16 / G;
      const uint32_t v0 = w0[st / 2] >> (4 * (st & 1)), v1 = w1[st / 2] >> (4 * (st & 1));
      const uint32_t f[4] = {code_pair(v0, z0.pair(i)), code_pair(v1, z1.pair(i)), code_pair(v0 >> 8, z0.pair(i)),
                             code_pair(v1 >> 8, z1.pair(i))};
      const bool first = kParts > 1 || st * 16 % G == 0, last = kParts > 1 || (st + 1) * 16 % G == 0;
#pragma unroll
      for (int p = kParts - 1; p >= 0; --p) {
        if (first && p == kParts - 1) mma_first(acc, f, xc[st].b[p]);
        else mma(acc, f, xc[st].b[p]);
      }
      if (last) {
        const float u0 = s0.value(i), u1 = s1.value(i);
        y[0] = __fmaf_rn(acc[0], u0, y[0]), y[1] = __fmaf_rn(acc[1], u0, y[1]);
        y[2] = __fmaf_rn(acc[2], u1, y[2]), y[3] = __fmaf_rn(acc[3], u1, y[3]);
      }
    }
  };

  T* const Y = static_cast<T*>(a.Y);
  auto put = [&](int group, int strip, int e, float v) {  // e: row and output
    const int m = rows0 + e / 16;
    const int64_t n = ((int64_t)(c0 + group * a.clusters) * a.wf + strip) * kTileN + e % 16;
    if (n >= a.s.N) return;
    v = __fmul_rn(v, kUnit);
    if (a.bias) v = __fadd_rn(v, a.bias[n]);
    store(Y + (int64_t)m * a.ldy + n, v);
  };

  for (int gi = 0; gi < ng; ++gi) {
    float y[4] = {};
    if (gi < live) {
      arrived();
      if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (c < cw) tile(x[c], at + c * tile_bytes, y);
        next();
      } else {
        for (int c = 0; c < cw; ++c) {
          load_x(0, c);
          if (c) arrived();
          tile(x[0], at, y);
          next();
        }
      }
    }
    // the sums of a strip's warps, two buffers in turn
    float* const mine = partial + ((gi & 1) * a.wf + wf) * a.wk * kOut;
    if (2 * t < rows) *reinterpret_cast<float4*>(mine + wk * kOut + lane * 4) = make_float4(y[0], y[1], y[2], y[3]);
    asm volatile("bar.sync %0, %1;\n" ::"r"(wf), "r"(a.wk * 32) : "memory");
    for (int e = wk * 32 + lane; e < rows * 16; e += a.wk * 32) {
      const int m = e / 16, f = e % 16;
      const float* p = mine + ((f & 7) * 4 + m / 2) * 4 + (m & 1) + 2 * (f / 8);
      float v = 0.0f;
#pragma unroll 4
      for (int w = 0; w < a.wk; ++w) v = __fadd_rn(v, p[w * kOut]);
      if (S == 1) put(gi, wf, e, v);
      else held[((gi % kRound) * a.wf + wf) * kOut + e] = v;
    }
    if (S > 1 && (gi % kRound == kRound - 1 || gi == ng - 1)) {
      cg::this_cluster().sync();
      const int first = gi / kRound * kRound, n = (gi - first + 1) * a.wf * kOut;
      for (int e = rank * blockDim.x + threadIdx.x; e < n; e += S * blockDim.x) {
        if (e % kOut >= rows * 16) continue;
        float v = 0.0f;
        for (int r = 0; r < S; ++r) v = __fadd_rn(v, cg::this_cluster().map_shared_rank(held, r)[e]);
        put(first + e / (a.wf * kOut), e / kOut % a.wf, e % kOut, v);
      }
      cg::this_cluster().sync();
    }
  }
}

template <class T, int C>
int run_block(Args& a, int S, cudaStream_t s) {
  const int warps = a.wk * a.wf;
  const int64_t row_tiles = ceil_div(a.M, kRows), groups = ceil_div(a.s.strips, a.wf);
  a.clusters = (int)std::min<int64_t>(groups, std::max<int64_t>(1, sm_count() / S / row_tiles));
  const int smem = warps * stages(C) * stage_tiles(C) * a.s.tile_bytes + 2 * warps * kOut * 4 + (S > 1 ? kRound * a.wf * kOut * 4 : 0);
  if (row_tiles * a.clusters * S > INT32_MAX) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: too many rows");
  auto run = [&](auto kernel) {
    return kv::launch(kernel, (unsigned)(row_tiles * a.clusters * S), 32 * warps, smem, S, s, "matmul_nbits", a);
  };
  auto scaled = [&](auto scale) {
    using ST = decltype(scale);
    switch (a.s.per) {
      case 8: return run(nbits_kernel<T, C, 16, ST>);
      case 4: return run(nbits_kernel<T, C, 32, ST>);
      case 2: return run(nbits_kernel<T, C, 64, ST>);
      default: return run(nbits_kernel<T, C, 128, ST>);
    }
  };
  return a.s.scale_size == 4 ? scaled(float()) : scaled(__nv_bfloat16());
}

int run_product(Args& a, int type, cudaStream_t s) {
  const int64_t chunks = a.s.chunks;
  // chunks of the rows that a warp's registers hold (two stages of four of the largest tiles would not fit)
  const int room = type == I8Q_F32 ? 1 : a.s.tile_bytes > 1408 ? 2 : 4;
  // Warps along k: as many as there are chunks; where strips go round for
  // several at a time in a CTA, no more than hold k in their registers.
  a.wk = (int)std::min<int64_t>(kWarps, chunks);
  const int64_t fewest = ceil_div(chunks, room);
  if (fewest < a.wk && a.s.strips * fewest >= (int64_t)sm_count() * kWarps) a.wk = (int)fewest;
  a.wf = (int)std::max<int64_t>(1, std::min<int64_t>(kWarps / a.wk, ceil_div(a.s.strips, sm_count())));
  int S = 1;
  const auto share = [&] { return ceil_div(chunks, (int64_t)a.wk * S); };  // chunks of a warp
  while (S < kMostCtas && share() > room) S *= 2;
  while (S < kMostCtas && a.s.strips * S * 2 <= sm_count() && chunks >= (int64_t)kWarps * S * 2) S *= 2;
  if (S > 1) a.wf = 1;
  const bool held = share() <= room;
  if (type == I8Q_F32) return held ? run_block<float, 1>(a, S, s) : run_block<float, 0>(a, S, s);
  using B = __nv_bfloat16;
  if (!held) return run_block<B, 0>(a, S, s);
  return share() <= 2 ? run_block<B, 2>(a, S, s) : run_block<B, 4>(a, S, s);
}

}  // namespace
}  // namespace i8q

using namespace i8q;

extern "C" size_t i8q_matmul_nbits_packed_size(int64_t N, int64_t K, int64_t block_size, int scale_type, int has_zero) {
  Shape s;
  if (check_shape(N, K, block_size, scale_type, has_zero != 0, "matmul_nbits_packed_size", s) != I8Q_OK) return 0;
  return (size_t)s.strips * (size_t)s.chunks * (size_t)s.tile_bytes;
}

extern "C" int i8q_matmul_nbits_pack(int64_t N, int64_t K, int64_t block_size, const uint8_t* B, const void* scales,
                                     int scale_type, const uint8_t* zero_points, void* packed, size_t packed_bytes,
                                     void* stream) {
  Shape s;
  const int rc = check_shape(N, K, block_size, scale_type, zero_points != nullptr, "matmul_nbits_pack", s);
  if (rc != I8Q_OK) return rc;
  if (!B || !scales || !packed) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits_pack: B, scales or packed is NULL");
  if (reinterpret_cast<uintptr_t>(scales) % s.scale_size)
    return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits_pack: scales are not aligned to their type");
  if (reinterpret_cast<uintptr_t>(packed) % 16)
    return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits_pack: packed must be 16-byte aligned");
  if (packed_bytes < (size_t)s.strips * (size_t)s.chunks * (size_t)s.tile_bytes)
    return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits_pack: packed is smaller than matmul_nbits_packed_size");
  // (allocated here, so that the product's first call may be a captured one)
  if (!device_status_word()) return fail(I8Q_ERR_CUDA, "matmul_nbits_pack: no status word");
  I8Q_PROF("matmul_nbits_pack", as_stream(stream));
  const int64_t blocks = std::min<int64_t>(s.strips * s.chunks, 64 * (int64_t)sm_count());
  pack_kernel<<<(unsigned)blocks, 256, 0, as_stream(stream)>>>(s, B, scales, zero_points, static_cast<uint8_t*>(packed));
  I8Q_LAUNCH_CHECK("matmul_nbits_pack");
  return I8Q_OK;
}

extern "C" int i8q_matmul_nbits(const void* A, int type, int64_t M, int64_t lda, const void* packed, size_t packed_bytes,
                                int64_t N, int64_t K, int64_t block_size, int scale_type, int has_zero, const float* bias,
                                void* Y, int64_t ldy, void* stream) {
  Args a{};
  const int rc = check_shape(N, K, block_size, scale_type, has_zero != 0, "matmul_nbits", a.s);
  if (rc != I8Q_OK) return rc;
  if (type != I8Q_F32 && type != I8Q_BF16) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: type must be I8Q_F32 or I8Q_BF16");
  if (M < 0 || M > kMost) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: M must be 0 .. 2^31 - 2^16");
  if (M == 0) return I8Q_OK;
  if (!A || !packed || !Y) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: A, packed or Y is NULL");
  if (M > 1 && (lda < K || ldy < N)) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: rows overlap (lda below K or ldy below N)");
  const uintptr_t es = type == I8Q_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(A) % es || reinterpret_cast<uintptr_t>(Y) % es || reinterpret_cast<uintptr_t>(bias) % 4)
    return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: A, Y or bias is not aligned to its type");
  if (reinterpret_cast<uintptr_t>(packed) % 16) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: packed must be 16-byte aligned");
  if (packed_bytes < (size_t)a.s.strips * (size_t)a.s.chunks * (size_t)a.s.tile_bytes)
    return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: packed is smaller than matmul_nbits_packed_size");
  a.packed = static_cast<const uint8_t*>(packed);
  a.A = A, a.lda = lda, a.bias = bias, a.Y = Y, a.ldy = ldy, a.M = (int)M;
  a.a_aligned = reinterpret_cast<uintptr_t>(A) % (4 * es) == 0 && (M == 1 || lda % 4 == 0);
  cudaStream_t s = as_stream(stream);
  I8Q_PROF("matmul_nbits", s);
  // more than one tile of 8 rows: 4096 -> 14336 by 16 rows 15.6 us there, 20 here; by 8 rows 17 and 11
  return type == I8Q_BF16 && M > 8 && tc_takes(a) ? run_tc(a, s) : run_product(a, type, s);
}
