// nbits_tc.cu -- MatMulNBits of bf16 activations on the tcgen05 tensor pipe.
//
// A tile of the product is 128 outputs x up to 64 rows x 128 k.  The matrix
// is the instruction's A operand, in TMEM, where a warp puts it from its
// registers: a thread has one output, turns its 128 codes of 4 bits into bf16
// numbers less their zero points (exact) and stores them as its lane's 64
// columns.  The activations are the B operand, as TMA brings them.  A block's
// products are summed from 0 in TMEM and enter the row's sum by a rounded fma
// with the block's scale, in the registers of four other warps.
//
// The matrix's bytes take 4.8 us of 64 x 4096 -> 14336, this kernel 21 (32 rows
// 17, 16 rows 15), mma.sync (nbits.cu) 57, which for up to 8 rows is the faster
// (1 row 10 us and 14.4).  There 112 CTAs have a tile of outputs each and the
// whole k; by clock stamps of a CTA's summing warps, in cycles (blocks of 64; 16,
// 32 and 64 rows): start and first chunk 5000, 4900 and 5200, each of the 31 other
// chunks 650, 710 and 860, output 1420, 2710 and 5190, 27000, 29800 and 37500 in
// all.  A chunk is a line of waits between the roles, with a wait for each 16
// columns of sums in the summing warps (blocks of 128 of 64 rows 720, of 32
// 1620); the output writes a row's elements of two bytes one after the other; 40
// of the 152 SMs have no tile, and every split of k that uses them has the longer
// line (share_k).  Tried at the same rate: two chunks at a time, two groups of
// summing warps, blocks' sums twice in TMEM, twice the codes on their way.
#include <cooperative_groups.h>

#include <map>
#include <string>

#include "nbits.cuh"
#include "tcgen05.cuh"

namespace i8q {
namespace nbits {
namespace {

namespace cg = cooperative_groups;
using namespace tc;

constexpr uint32_t ST_TIMEOUT_NBITS = 1u << 14;

constexpr int kOutputs = 128, kStrips = kOutputs / kTileN;
// Warps: two groups of four that turn codes into bf16, chunks in turn, each
// with a warp that issues its products (one for both took 900 cycles a chunk,
// nearly all of it waits that need not wait); four that scale and sum; one
// that sends for activations.
constexpr int kTurn = 8, kSum = 4, kIssueWarp = kTurn + kSum, kLoadWarp = kIssueWarp + 2, kThreads = 32 * (kLoadWarp + 1);
// tiles of codes of a group of four warps, all but one on their way
constexpr int code_stages(int rows) { return rows == 16 ? 8 : rows == 32 ? 6 : 4; }
constexpr int kA = 2;                      // tiles of bf16 weights in TMEM, of each group, 64 columns each
constexpr int kSlot = 4 * 2048 + 4 * 32 * 8;  // of a group: codes, then zero points (8 blocks of a row at most)

constexpr int kScales = 4;                 // chunks' scales on their way, 32 outputs x 8 blocks x 4 bytes a warp at most
constexpr int kScaleSlot = 4 * 1024;

constexpr int x_stages(int rows) { return rows == 16 ? 8 : rows == 32 ? 6 : 4; }
constexpr int x_bytes(int rows) { return rows * 256; }
// blocks whose sums stand in TMEM at a time, of each group: 128 columns at most
constexpr int batch_of(int rows, int per) { return per < 128 / rows ? per : 128 / rows; }

struct TcArgs {
  Args a;
  int units;   // tiles of outputs x tiles of rows
  int tiles;   // of outputs
  uint32_t* status;
};

struct Bars {
  uint64_t x_full[8], x_empty[8], a_full[2][kA], a_empty[2][kA], d_full[2], d_empty[2], joined[2], taken[2];
  uint32_t tmem;
  int abort;
};

// activations, codes and zero points, parts of sums from the cluster's CTAs
constexpr int smem_bytes(int rows) {
  return 1024 + x_stages(rows) * x_bytes(rows) + 2 * code_stages(rows) * kSlot + kScales * kScaleSlot +
         2 * rows * kOutputs * 4 + (int)sizeof(Bars);
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// One lane of a warp that runs as one.  (The products of a loop that `lane == 0`
// guards were sent 45 cycles apart, these 10: their operands then stay in
// uniform registers.)
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// A cluster has a unit (a tile of outputs by a tile of rows) at a time, its
// CTAs a share of k each; their sums meet in shared memory, each CTA adding up
// and writing a share of the rows.
template <int ROWS, int G>
__global__ void __launch_bounds__(kThreads, 1)
tc_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TcArgs args) {
  const Args& a = args.a;
  constexpr int kPer = kTileK / G, kBatch = batch_of(ROWS, kPer), kBatches = kPer / kBatch;
  constexpr int kX = x_stages(ROWS), kXBytes = x_bytes(ROWS), kStages = code_stages(ROWS);
  constexpr uint32_t kIdesc = idesc_bf16(kOutputs, ROWS);
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* const x_buf = smem;
  uint8_t* const codes = x_buf + kX * kXBytes;
  uint8_t* const scales = codes + 2 * kStages * kSlot;
  float* const red = reinterpret_cast<float*>(scales + kScales * kScaleSlot);
  Bars& bars = *reinterpret_cast<Bars*>(red + 2 * ROWS * kOutputs);
  volatile int* const abort = &bars.abort;
  const int S = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, quarter = warp & 3;
  const int chunks = (int)a.s.chunks, strips = (int)a.s.strips, tile_bytes = a.s.tile_bytes;
  const int c_begin = (int)((int64_t)rank * chunks / S), cw = (int)((int64_t)(rank + 1) * chunks / S) - c_begin;
  const int first = blockIdx.x / S, clusters = gridDim.x / S;
  const int my_units = (args.units - first + clusters - 1) / clusters, total = my_units * cw;
  const bool resident = cw <= kX;  // the activations of this CTA's share of k stay (one tile of rows)
  const bool reload = !resident || args.units > args.tiles;
  auto bar = [](const uint64_t& b) { return smem_u32(&b); };
  auto wait = [&](const uint64_t& b, uint32_t parity) { return wait_bar(smem_u32(&b), parity, abort, args.status, ST_TIMEOUT_NBITS); };

  kv::next_kernel_may_start();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kX; ++i) mbar_init(bar(bars.x_full[i]), 1), mbar_init(bar(bars.x_empty[i]), 1);
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < kA; ++j) mbar_init(bar(bars.a_full[i][j]), 4), mbar_init(bar(bars.a_empty[i][j]), 1);
      mbar_init(bar(bars.d_full[i]), 1), mbar_init(bar(bars.d_empty[i]), 4);
      mbar_init(bar(bars.joined[i]), 4 * S), mbar_init(bar(bars.taken[i]), 4 * S);
    }
    bars.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == kIssueWarp) tmem_alloc(smem_u32(&bars.tmem), 512);
  tc_fence_before();
  if (S > 1) cg::this_cluster().sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem, tmem_a = tmem + 256;
  kv::wait_previous_kernel();

  // the unit and chunk of a role's place in the line of chunks
  const bool one = args.units == args.tiles;  // tile of rows
  auto tile_of = [&](int u) { return one ? first + u * clusters : (first + u * clusters) % args.tiles; };
  auto rows_at = [&](int u) { return one ? 0 : (first + u * clusters) / args.tiles * ROWS; };

  if (warp < kTurn) {
    // ---- codes to bf16, in TMEM ----
    const int group = warp / 4, row = quarter * 32 + lane;
    uint8_t* const ring = codes + group * kStages * kSlot;
    // the next chunk to send for, and where this lane's part of it lies: its
    // output's codes, and 16 bytes of the zero points of the warp's two strips
    int su = 0, sc = group, to = 0;
    const uint8_t *p = nullptr, *pz = nullptr;
    const uint32_t d = smem_u32(ring) + row * 16, dz = smem_u32(ring) + 8192 + quarter * 256 + lane * 16;
    auto place = [&] {
      while (su < my_units && sc >= cw) sc -= cw, ++su;
      p = pz = nullptr;
      if (su >= my_units) return;
      const int strip = tile_of(su) * kStrips + quarter * 2, s1 = strip + lane / 16, s2 = strip + lane / kPer;
      if (s1 < strips) p = a.packed + ((int64_t)s1 * chunks + c_begin + sc) * tile_bytes + lane % 16 * 16;
      if (a.s.has_zero && lane < 2 * kPer && s2 < strips)
        pz = a.packed + ((int64_t)s2 * chunks + c_begin + sc) * tile_bytes + kCodeBytes + kTileN * kPer * a.s.scale_size +
             lane % kPer * 16;
    };
    place();
    auto send = [&] {
      if (p) {
#pragma unroll
        for (int q = 0; q < 4; ++q) copy16(d + to * kSlot + q * 2048, p + q * 256);
        p += 2 * tile_bytes;
      }
      if (pz) copy16(dz + to * kSlot, pz), pz += 2 * tile_bytes;
      commit();
      to = to + 1 == kStages ? 0 : to + 1;
      if ((sc += 2) >= cw) place();
    };
    for (int i = 0; i < kStages - 1; ++i) send();
    const uint32_t tmem_mine = tmem_a + group * (kA * 64) + ((uint32_t)quarter << 21);
    int from = 0, n = 0;
    for (int i = group; i < total; i += 2, ++n) {
      wait_copies<kStages - 2>();
      __syncwarp();  // the zero points were copied by other lanes, and all have read the slot that is sent for
      send();
      const uint8_t* const slot = ring + from * kSlot;
      from = from + 1 == kStages ? 0 : from + 1;
      Row<uint8_t, kPer> z;
      if (a.s.has_zero) z = Row<uint8_t, kPer>(slot + 8192 + quarter * 256, lane);
      const int buf = n % kA;
      if (!wait(bars.a_empty[group][buf], (n / kA & 1) ^ 1)) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot + q * 2048 + row * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w}, z0 = z.pair(q * 32 / G), z1 = z.pair((q * 32 + 16) / G);
        uint32_t r[16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          r[2 * t] = code_pair(w[t], z0), r[2 * t + 1] = code_pair(w[t] >> 8, z0);
          r[8 + 2 * t] = code_pair(w[t] >> 4, z1), r[9 + 2 * t] = code_pair(w[t] >> 12, z1);
        }
        tmem_st16(tmem_mine + buf * 64 + q * 16, r);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars.a_full[group][buf]));
    }
  } else if (warp < kIssueWarp) {
    // ---- blocks' sums, scaled and added up ----
    // 16-byte pieces of the scales of the warp's two strips, two a lane at most
    const int row = quarter * 32 + lane, pieces = kPer * a.s.scale_size, s1 = lane / pieces, s2 = (lane + 32) / pieces;
    const int o1 = lane % pieces * 16, o2 = (lane + 32) % pieces * 16;
    int su = cw ? 0 : my_units, sc = 0, to = 0;
    const uint8_t *p1 = nullptr, *p2 = nullptr;
    const uint32_t d = smem_u32(scales) + quarter * 1024 + lane * 16;
    auto place = [&] {
      p1 = p2 = nullptr;
      if (su >= my_units) return;
      const int strip = tile_of(su) * kStrips + quarter * 2;
      if (s1 < 2 && strip + s1 < strips) p1 = a.packed + ((int64_t)(strip + s1) * chunks + c_begin) * tile_bytes + kCodeBytes + o1;
      if (s2 < 2 && strip + s2 < strips) p2 = a.packed + ((int64_t)(strip + s2) * chunks + c_begin) * tile_bytes + kCodeBytes + o2;
    };
    place();
    auto send = [&] {
      if (p1) copy16(d + to * kScaleSlot, p1), p1 += tile_bytes;
      if (p2) copy16(d + to * kScaleSlot + 512, p2), p2 += tile_bytes;
      commit();
      to = to + 1 == kScales ? 0 : to + 1;
      if (++sc == cw) sc = 0, ++su, place();
    };
    for (int i = 0; i < kScales - 1; ++i) send();
    int from = 0, group = 0, phase = 0;  // of the chunk
    bool ok = true;
    for (int u = 0; u < my_units && ok; ++u) {
      float y[ROWS] = {};
      for (int c = 0; c < cw && ok; ++c) {
        wait_copies<kScales - 2>();
        __syncwarp();
        send();
        const uint8_t* const at = scales + from * kScaleSlot + quarter * 1024;
        from = from + 1 == kScales ? 0 : from + 1;
        float scale[kPer];
        if (a.s.scale_size == 4) {
          const Row<float, kPer> v(at, lane);
#pragma unroll
          for (int i = 0; i < kPer; ++i) scale[i] = v.value(i);
        } else {
          const Row<__nv_bfloat16, kPer> v(at, lane);
#pragma unroll
          for (int i = 0; i < kPer; ++i) scale[i] = v.value(i);
        }
#pragma unroll
        for (int b = 0; b < kBatches; ++b) {
          if (!wait(bars.d_full[group], (phase * kBatches + b) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const uint32_t d = tmem + group * 128 + i * ROWS + ((uint32_t)quarter << 21);
#pragma unroll
            for (int m = 0; m < ROWS; m += 16) {
              uint32_t r[16];
              tmem_ld16(d + m, r);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) y[m + j] = __fmaf_rn(__uint_as_float(r[j]), scale[b * kBatch + i], y[m + j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bars.d_empty[group]));
        }
        phase += group, group ^= 1;
      }
      if (!ok) break;
      const int row0 = rows_at(u);
      const int64_t n = (int64_t)tile_of(u) * kOutputs + row;
      __nv_bfloat16* const Y = static_cast<__nv_bfloat16*>(a.Y) + n;
      const float bias = a.bias && n < a.s.N ? a.bias[n] : 0.0f;
      auto put = [&](int m, float v) {
        v = __fmul_rn(v, kUnit);
        if (row0 + m < a.M && n < a.s.N) store(Y + (int64_t)(row0 + m) * a.ldy, a.bias ? __fadd_rn(v, bias) : v);
      };
      if (S == 1) {
#pragma unroll
        for (int m = 0; m < ROWS; ++m) put(m, y[m]);
        continue;
      }
      const int buf = u & 1, own = ROWS / S;
      if (!wait_bar<true>(bar(bars.taken[buf]), (u >> 1 & 1) ^ 1, abort, args.status, ST_TIMEOUT_NBITS)) break;
      // [buffer][CTA of the cluster][row of the owner][output]
      const uint32_t mine = smem_u32(red) + (((buf * S + rank) * own) * kOutputs + row) * 4;
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        const int owner = m / own;
        asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(map_shared_rank(mine, owner) + (m - owner * own) * kOutputs * 4), "f"(y[m]) : "memory");
      }
      __syncwarp();
      if (lane < S) mbar_arrive_cluster(map_shared_rank(bar(bars.joined[buf]), lane));
      if (!wait_bar<true>(bar(bars.joined[buf]), u >> 1 & 1, abort, args.status, ST_TIMEOUT_NBITS)) break;
      for (int m = 0; m < own; ++m) {
        float v = 0.0f;
        for (int r = 0; r < S; ++r) v = __fadd_rn(v, red[((buf * S + r) * own + m) * kOutputs + row]);
        put(rank * own + m, v);
      }
      __syncwarp();
      if (lane < S) mbar_arrive_cluster(map_shared_rank(bar(bars.taken[buf]), lane));
    }
  } else if (warp < kLoadWarp) {
    // ---- products ----
    const int group = warp - kIssueWarp;
    const uint32_t tmem_d = tmem + group * 128, tmem_mine = tmem_a + group * (kA * 64);
    const uint64_t x0 = desc_sw128(smem_u32(x_buf));
    int n = 0, c = group, stage = group, x_phase = 0;
    while (c >= cw && cw) c -= cw;
    bool ok = true;
    for (int i = group; i < total && ok; i += 2, ++n) {
      const int buf = n % kA;
      if (reload) ok = wait(bars.x_full[stage], x_phase);
      else if (i < 2 * cw) ok = wait(bars.x_full[c], 0);  // (this warp's first use of each: an odd cw swaps the groups' chunks)
      ok = ok && wait(bars.a_full[group][buf], n / kA & 1);
      const uint64_t x = x0 + (reload ? stage : c) * (kXBytes / 16);
#pragma unroll
      for (int b = 0; b < kBatches; ++b) {
        ok = ok && wait(bars.d_empty[group], ((n * kBatches + b) & 1) ^ 1);
        if (__any_sync(0xffffffffu, !ok)) break;
        tc_fence_after();
        if (elected()) {
#pragma unroll
          for (int j = 0; j < kBatch * G / 16; ++j) {
            const int step = b * (kBatch * G / 16) + j;  // of the chunk's eight (addresses in units of 16 bytes)
            mma_ts(tmem_d + j * 16 / G * ROWS, tmem_mine + buf * 64 + step * 8, x + step / 4 * (ROWS * 8) + step % 4 * 2, kIdesc,
                   j * 16 % G != 0);
          }
          tc_commit(bar(bars.d_full[group]));
          if (b == kBatches - 1) {
            tc_commit(bar(bars.a_empty[group][buf]));
            if (reload) tc_commit(bar(bars.x_empty[stage]));
          }
        }
        __syncwarp();
      }
      ok = !__any_sync(0xffffffffu, !ok);
      if (reload) {
        if ((stage += 2) >= kX) stage -= kX, x_phase ^= 1;
      } else {
        for (c += 2; c >= cw;) c -= cw;
      }
    }
    // the last commits arrive while this CTA's memory is still its own
    if (n > 0 && ok) {
      wait(bars.a_empty[group][(n - 1) % kA], (n - 1) / kA & 1);
      if (reload) wait(bars.x_empty[stage >= 2 ? stage - 2 : stage - 2 + kX], stage >= 2 ? x_phase : x_phase ^ 1);
    }
    __syncwarp();
  } else {
    // ---- activations ----
    if (lane == 0) {
      const int sends = reload ? total : (total ? cw : 0);
      int u = 0, c = 0, i = 0;
      for (; i < sends; ++i) {
        const int stage = i % kX;
        if (!wait(bars.x_empty[stage], (i / kX & 1) ^ 1)) break;
        const uint32_t full = bar(bars.x_full[stage]), d = smem_u32(x_buf) + stage * kXBytes;
        mbar_arrive_expect_tx(full, kXBytes);
        tma_load_2d(d, &map, full, (c_begin + c) * kTileK, rows_at(u));
        tma_load_2d(d + ROWS * 128, &map, full, (c_begin + c) * kTileK + 64, rows_at(u));
        if (++c == cw) c = 0, ++u;
      }
      // given up: what is on its way still lands in this CTA's memory (bounded)
      if (i < sends)
        for (int j = max(0, i - kX); j < i; ++j)
          for (int tries = 0; tries < 100000 && !mbar_try_wait(bar(bars.x_full[j % kX]), j / kX & 1); ++tries) {
          }
    }
    __syncwarp();
  }
  wait_copies<0>();
  tc_fence_before();
  if (S > 1) cg::this_cluster().sync();  // (no CTA leaves while others write to it)
  else __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
}

// CTAs of a cluster: the number by which the longest line of chunks is the
// shortest; of those, the fewest.  `fits`: clusters of S CTAs that run at once.
template <class F>
int share_k(const Shape& s, int64_t units, F fits) {
  int best = 1;
  int64_t line = INT64_MAX;
  for (int S = 1; S <= kMostCtas && S <= s.chunks; S *= 2) {
    const int64_t at_once = std::max(1, fits(S));
    // a unit's fixed part (sums' way through the cluster, output) is worth about a chunk, twice that in a cluster
    const int64_t l = ceil_div(units, at_once) * (ceil_div(s.chunks, S) + (S > 1 ? 2 : 1));
    if (l < line) line = l, best = S;
  }
  return best;
}

template <int ROWS, int G>
int run_form(TcArgs& t, const CUtensorMap& map, cudaStream_t s) {
  const auto kernel = tc_kernel<ROWS, G>;
  const int smem = smem_bytes(ROWS);
  // clusters of 1, 2, 4 and 8 CTAs that the device runs at once
  struct Fit {
    const void* kernel;
    int smem;
    int n[4];
  };
  static thread_local std::map<int, Fit> known;  // by device
  int dev = 0;
  I8Q_CUDA_TRY(cudaGetDevice(&dev));
  auto it = known.find(dev);
  if (it == known.end()) {
    Fit f{reinterpret_cast<const void*>(kernel), smem, {}};
    const int rc = smem_attr(f.kernel, smem);
    if (rc != I8Q_OK) return rc;
    for (int i = 0; i < 4; ++i) {
      cudaLaunchConfig_t cfg{};
      cudaLaunchAttribute attr[1] = {};
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 1u << i, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(1u << i), cfg.blockDim = dim3(kThreads), cfg.dynamicSmemBytes = smem;
      cfg.attrs = attr, cfg.numAttrs = 1;
      I8Q_CUDA_TRY(cudaOccupancyMaxActiveClusters(&f.n[i], f.kernel, &cfg));
    }
    it = known.emplace(dev, f).first;
  }
  const Fit& fit = it->second;
  const auto fits = [&](int S) { return fit.n[S == 1 ? 0 : S == 2 ? 1 : S == 4 ? 2 : 3]; };
  const int S = share_k(t.a.s, t.units, fits);
  const int clusters = (int)std::min<int64_t>(t.units, std::max(1, fits(S)));
  return kv::launch(kernel, (unsigned)(clusters * S), kThreads, smem, S, s, "matmul_nbits", map, t);
}

}  // namespace

bool tc_takes(const Args& a) {
  return reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && a.lda % 8 == 0 && a.lda <= (1LL << 36);
}

int run_tc(Args& a, cudaStream_t s) {
  const int rows = a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
  TcArgs t{a, 0, 0, device_status_word()};
  if (!t.status) return fail(I8Q_ERR_CUDA, "matmul_nbits: no status word");
  const int64_t tiles = ceil_div(a.s.N, kOutputs), units = tiles * ceil_div(a.M, rows);
  if (units > INT32_MAX / 2 / a.s.chunks) return fail(I8Q_ERR_INVALID_ARG, "matmul_nbits: too many rows");
  t.units = (int)units, t.tiles = (int)tiles;
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)a.s.K, (cuuint64_t)a.M};
  const cuuint64_t strides[1] = {(cuuint64_t)a.lda * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)rows};
  const int rc = make_tensor_map(&map, a.A, 2, dims, strides, box, "matmul_nbits");
  if (rc != I8Q_OK) return rc;
  auto blocked = [&](auto r) {
    constexpr int R = decltype(r)::value;
    switch (a.s.per) {
      case 8: return run_form<R, 16>(t, map, s);
      case 4: return run_form<R, 32>(t, map, s);
      case 2: return run_form<R, 64>(t, map, s);
      default: return run_form<R, 128>(t, map, s);
    }
  };
  return rows == 16 ? blocked(std::integral_constant<int, 16>()) : rows == 32 ? blocked(std::integral_constant<int, 32>())
                                                                              : blocked(std::integral_constant<int, 64>());
}

}  // namespace nbits
}  // namespace i8q
