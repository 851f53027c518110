// kv_attention.cuh -- attention of one new token per sequence over a paged
// key/value cache of int8 codes or bf16 values.
//
// For a key/value head, its G query heads and the tokens t of a sequence:
//   s_t = (q . k_t) softmax_scale log2 e,  o = sum_t 2^(s_t - m) v_t / l,
//   l = sum_t 2^(s_t - m),
// in one pass with a running m.  Every key and value is used once for a
// few heads, so the bound is the memory that holds them: at G = 4, D = 128
// and int8 a token costs 264 bytes and 4 kFLOP, where the card does 280
// FLOP per byte.  What a kernel has to do is keep enough reads in flight and
// spend few instructions per byte:
//
//  - a warp takes tiles of 16 tokens.  It forms S^T = K Q^T (tokens as the
//    16 rows of mma.m16n8k16, heads as its 8 columns) and O^T = V^T P^T (head
//    elements as rows), so that 8 heads cost no padding of the 16-row side.
//    tcgen05 wants 128 rows of fp16 operands in shared memory: the codes would
//    have to be converted and written back there, several times the traffic
//    of the fragments, for a product that takes a tenth of the time;
//  - each warp copies its tiles asynchronously into slots of shared memory of
//    its own, so there is no barrier in the loop, and a 16-token tile is 4 KB
//    in flight.  Eight lanes read 128 bytes in a row (reading rows in pieces
//    of 32 bytes, as the fragments lie, held the kernel to 4.3 TB/s);
//  - the order of the summation index is free, so both operands use the one
//    in which 16-byte pieces hold a lane's fragments;
//  - a byte with its sign bit flipped, code + 128, is part of an fp16 or bf16
//    number as it lies: one LOP3 and one subtraction or fma make two exact
//    codes.  Keys become fp16, and the query is scaled by a power of two into
//    fp16's range; values become bf16, because the weights that multiply them need
//    its range.  (Keys entered as code + 128, the 128s taken from the sum, save
//    the subtraction and no time, but a row with one large channel has codes of
//    about 1 elsewhere, and their sum kept the rounding of the 128s: 2e-5 of it
//    at 128 elements.);
//  - the running maximum moves only when a score exceeds it by 2^8: p stays
//    below 2^8, and most tiles need no reduction over the lanes;
//  - value scales multiply p (in fp32) before it is split into bf16 parts.
//
// Work split.  Each row (sequence, key/value head, group of query heads) is
// as long as its number of tiles plus a constant for its start and end;
// the rows form one line, cut into equal parts, one per warp.  A row that
// lies in one part is finished by that warp.  Of the others the warps of a
// CTA join what they have in shared memory, leave m, l and o in the
// workspace, and a second kernel joins those.  Rows that cannot be long are not
// cut: a CTA has them whole, or a cluster one, and there is no second kernel.
// The split follows from the sizes and lengths alone, so results repeat.
//
// Measured: one sequence of 131072 tokens, 8 heads of 128, int8, 32 query
// heads: 62 us a call, 277 MB (each further 131072 tokens 48 us, 5.8 TB/s; of
// bf16 83 us, 6.5 TB/s); 64 sequences of 8192 with scores: 245 us, 1.14 GB.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "kv.cuh"

namespace i8q {
namespace kva {

using kv::Cache;
using kv::Table;
using kv::next_kernel_may_start;
using kv::wait_previous_kernel;

struct Heads {  // [sequences][heads][dim], strides in elements
  void* p;
  int64_t token, head;
};

constexpr int kMaxSequences = 2048;  // of one launch: their line positions lie in shared memory
constexpr int kRowCost = 4;          // of a row's start and end, in tiles
constexpr int kMinPart = 4;          // tiles of a part of a row that is cut
constexpr int kShort = 12;           // tiles a warp, up to which rows may stay whole
constexpr int kMostCtas = 8;         // of a cluster
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Args {
  Cache c;
  Table tab;
  const int32_t* lengths;
  Heads q, out;
  float* lse;
  float scale;
  int64_t page_bytes, head_bytes, token_bytes, step_bytes;  // the pools' strides; of the rows that 32 lanes copy at once
  int q_heads, group, chunks;  // group: query heads of a key/value head; chunks: rows that share one
  int window;
  int aligned_q, aligned_out;  // 16-byte loads of q rows, paired stores of out rows
  int heads_per_row;           // of a partial: 8 or 16
  int ctas, warps;             // of the first kernel
  int per_row;                 // warps that share a row, where rows are not cut; else 0
  int cluster;                 // CTAs that share one then
  int* line;                   // [sequences + 1] start of each sequence on the line
  float2* part_stats;          // [ctas * warps][2][heads_per_row] (m, l)
  float* part_out;             // [ctas * warps][2][heads_per_row][DP of the form]
  float* logits;               // [sequences][q_heads][logit_pitch], or null
  int64_t logit_pitch;
  float* stats;                // [sequences][q_heads] m + log2 l (with logits)
  int fours;                   // scores of four neighbouring tokens can be read at once
  int scores_here;             // the first kernel adds the scores: its rows are whole and have all heads that share a key
  uint32_t* status;
};

__device__ __forceinline__ int first_token(const Args& a, int len) {
  return a.window && len > a.window ? len - a.window : 0;
}
__device__ __forceinline__ int tile_count(const Args& a, int len) {
  return len > 0 ? (len + 15) / 16 - first_token(a, len) / 16 : 0;
}
// The line of n units cut into parts whose lengths differ by one at most,
// the longer ones first; each CTA takes `per_cta` neighbours.
struct Cut {
  int parts, per_cta, q, longer;  // `longer` parts of q + 1 units, then parts of q
  __device__ int begin(int w) const { return w * q + min(w, longer); }
  __device__ int of(int x) const {
    const int split = longer * (q + 1);
    return x < split ? x / (q + 1) : longer + (x - split) / q;
  }
};
__device__ __forceinline__ Cut cut_line(const Args& a, int n, int rows) {
  Cut c;
  // rows are cut where a row holds two parts of kMinPart tiles and more
  const int tiles = n - rows * kRowCost;
  c.parts = min(tiles / (2 * kMinPart) >= rows ? tiles / kMinPart : rows, a.ctas * a.warps);
  c.per_cta = (c.parts + a.ctas - 1) / a.ctas;
  c.q = n / c.parts;
  c.longer = n - c.q * c.parts;
  return c;
}

// Short rows: a CTA keeps whole rows, `per_row` warps (a divisor of its number)
// to each, or a cluster of CTAs has one and joins its parts through their
// shared memory, so that one launch does it all (one sequence of 4000 tokens, 4
// heads: 11.3 us instead of 14.4, and with scores 13.4 instead of 21.4; of
// 2000: 9.5 instead of 14.5).  A tile a warp takes 0.9 to 1.6 us with a CTA's
// warps all at work; what cut rows need more is worth 5 tiles (with scores 7;
// fp32 4 and 5), less one for a cluster's exchange, and each SM has its even
// share of tiles then.  So rows stay whole while they have no more tiles a warp
// than that, and no more than kShort: the table may be wider than its sequences
// are long, some SMs' rows longer than others'.  (At the edge: 10 x 3000 tokens
// of 4 heads 18.2 us whole, 18.4 cut.)
// per_row 0: a row may be too long for that, or there are too many rows.
struct Share {
  int per_row, cluster;
};
inline Share share_rows(int warps, int ctas, int64_t rows, int64_t longest, bool scores, bool wide) {
  int k = warps, cluster = 1;
  while (k > 1 && (warps % k || rows > (int64_t)ctas * (warps / k))) --k;
  // (5 / 6: clusters of 8 do not fill every group of SMs)
  while (k == warps && cluster < kMostCtas && rows * cluster * 2 <= ctas * 5 / 6 && longest > 2 * cluster * warps)
    cluster *= 2;
  const int64_t each = ceil_div(longest, (int64_t)k * cluster), even = rows * longest / ((int64_t)ctas * warps);
  const int64_t most = std::min<int64_t>(kShort, even + (wide ? 4 + scores : 5 + 2 * scores) - (cluster > 1));
  if (rows > (int64_t)ctas * (warps / k) || each > most) return {0, 1};
  return {k * cluster, cluster};
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

template <bool HALF>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (HALF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// a += x and b += y in one instruction.
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 s, d;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 d, {%2, %3};\n\tadd.rn.f32x2 s, s, d;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
// 8 x 8 transpose of 16-bit values over the warp (a lane holds two
// neighbours of row lane / 4).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}

// Two codes in bytes 0 and 2 of w.  A byte with its sign bit flipped is the
// unsigned number u = code + 128.
//  as fp16 numbers: under 0x64 u stands for 1024 + u, and 1152 is taken;
__device__ __forceinline__ uint32_t codes_fp16(uint32_t w) {
  const uint32_t u = (w & 0x00ff00ffu) ^ 0x64806480u;
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
  return r;
}
//  as bf16 numbers code 2^-6: u alone is u 2^-133 there (7 bits of mantissa,
//  the eighth the lowest of the exponent), times 2^127, minus 128 2^-6.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t u = (w & 0x00ff00ffu) ^ 0x00800080u;
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(u), "r"(0x7f007f00u), "r"(0xc000c000u));
  return r;
}

// x as the sum of `N` 16-bit floats, the largest first; two values a word.  A
// second fp16 part is held 2^11 times as large, so that it is a normal number
// where the first is.
constexpr float kPartGain = 2048.0f;
template <bool HALF, int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (HALF) {
      const __half2 h = __floats2half2_rn(x, y);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
      if (i + 1 < N) x = (x - __low2float(h)) * kPartGain, y = (y - __high2float(h)) * kPartGain;
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      r[i] = *reinterpret_cast<const uint32_t*>(&h);
      if (i + 1 < N) x -= __low2float(h), y -= __high2float(h);
    }
  }
}

// N consecutive elements of a q row as they lie in memory, and in fp32.
template <class T, int N>
struct Piece {
  uint4 w[N * sizeof(T) / 16];
  __device__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ void load_any(const T* p) {  // at any alignment
    alignas(16) T e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = p[i];
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(e)[i];
  }
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ void to_float(float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int word = i * (int)sizeof(T) / 4;
      const uint4 u = w[word / 4];
      const uint32_t v = word % 4 == 0 ? u.x : word % 4 == 1 ? u.y : word % 4 == 2 ? u.z : u.w;
      if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(v);
      else x[i] = __uint_as_float(i & 1 ? v & 0xffff0000u : v << 16);
    }
  }
};

template <class T>
__device__ __forceinline__ void store_pair(T* p, float x, float y, bool paired) {
  if constexpr (std::is_same<T, float>::value) {
    if (paired) *reinterpret_cast<float2*>(p) = make_float2(x, y);
    else p[0] = x, p[1] = y;
  } else {
    if (paired) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
    else p[0] = __float2bfloat16_rn(x), p[1] = __float2bfloat16_rn(y);
  }
}

// What a kernel is made for.  QT: type of q and out; S8: int8 cache, else
// bf16; DP: head_dim rounded up to 64, 128 or 256; NT: groups of 8 heads.
template <class QT_, bool S8_, int DP_, int NT_>
struct Form {
  using QT = QT_;
  static constexpr bool S8 = S8_;
  static constexpr int DP = DP_, NT = NT_;
  static constexpr bool WIDE = std::is_same<QT, float>::value;
  // 16-bit parts of q (fp16 of 11 bits and a sign, or bf16 of 8) and of the
  // weights (bf16): together the 24 bits of an fp32 number.  A bf16 query is
  // exact in one.  (Two parts of the weights lost 2^-18 of values that cancel;
  // 64 sequences of 8192 took 230 us with them, 240 with three, shorter calls
  // the same.)
  static constexpr int NQ = WIDE ? (S8 ? 2 : 3) : 1;
  static constexpr int NP = 3;
  static constexpr int ES = S8 ? 1 : 2;
  static constexpr int KS = DP / 16;           // steps of the first product
  static constexpr int MT = DP / 16;           // row blocks of the second
  static constexpr int ROW = DP * ES;          // bytes of a token's keys
  static constexpr int PK = ROW / 64;          // 16-byte pieces of a key row per lane
  static constexpr int VB = ROW == 64 ? 8 : 16;
  static constexpr int PV = ROW / 8 / VB;      // pieces of a value row per lane
  static constexpr int E = (DP + 127) / 128;   // four elements of a head's result a lane, so many times
  static constexpr int CR = ROW / 16;          // pieces of a row
  static constexpr int CT = ROW / 32;          // pieces of half a tile that a lane copies
  static constexpr int SLOT = 16 * ROW + 144;  // half a tile: pieces; keys: 32 scales, the mask of the tokens
  static constexpr int Q_WORDS = NQ * NT * KS * 2;
  static constexpr bool Q_REG = Q_WORDS <= 32;                 // q fragments in registers
  static constexpr int Q_BYTES = Q_REG ? 0 : Q_WORDS * 128;
  // Warps: 16 of 128 registers where they suffice (int8 heads of 64, 64 x
  // 8192 tokens: 143 us against 155 with 12 of 168; of 128 with scores: 301
  // against 249), else 12 (64 x 8192 of 4 heads: 8 query heads of 128 to each
  // 111 us against 132 with 8 warps, 16 of 64 107 against 126; but 16 of 128 283
  // against 154), 8 or 4 of 255.
  static constexpr int W = NT == 1 && S8 && DP == 64 && !WIDE                               ? 16
                           : (NT == 1 && (S8 ? DP <= 128 : DP == 64)) || (DP == 64 && !WIDE) ? 12
                           : 8 * (Q_BYTES + 3 * SLOT) <= 208 * 1024                          ? 8
                                                                                             : 4;
  static constexpr int ROOM = (208 * 1024 / W - Q_BYTES) / SLOT;
  static constexpr int AHEAD = ROOM >= 5 ? 2 : 1;  // tiles in flight
  static constexpr int SLOTS = 2 * AHEAD + 1;
  static constexpr int WARP_BYTES = SLOTS * SLOT + Q_BYTES;
  static constexpr int SMEM = W * WARP_BYTES + (kMaxSequences + 1) * 4 + 12 + W * (8 * NT * 8 + 16);
  static_assert(8 * NT * DP * 4 <= WARP_BYTES, "a part's result lies in its ring");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // Where piece p of token t lies in a slot.  Copies go by rows (8 lanes read
  // 128 bytes in a row of memory; four lanes a row of 64), and the exclusive
  // or spreads what 8 lanes read at once, be it 4 pieces of tokens t and t +
  // 1 (keys) or 2 pieces of tokens t, t + 2, t + 4 and t + 6 (values), over
  // all banks.
  __device__ static int place(int t, int p) {
    if constexpr (ROW == 64) return t / 2 * 128 + ((((t & 1) * 4 + p) ^ (t & 6)) * 16);
    else return t * ROW + ((p ^ (t & 6) ^ ((t & 1) * 4)) * 16);
  }
  // The same for the r-th piece that a lane copies, from place(lane / CR, lane % CR).
  __device__ static constexpr int copy_place(int at, int r) {
    const int t = r * 32 / CR;
    return ROW == 64 ? at + r * 512 : (at ^ (((t & 6) ^ ((t & 1) * 4)) * 16)) + r * 512;
  }
  // Head element that lane group g holds in row g of block mt (row g + 8: the next one).
  __device__ static int row_element(int mt, int g) {
    if constexpr (S8) return DP == 64 ? g * 8 + mt * 2 : mt / 8 * 128 + g * 16 + mt % 8 * 2;
    else return mt / 4 * 64 + g * 8 + mt % 4 * 2;
  }
};

// The result of query head h of sequence b from its m, l and o, four elements
// a lane.
template <class QT, int DP>
__device__ __forceinline__ void finish_row(const Args& a, int b, int h, int lane, float m, float l,
                                           const float4 (&o)[(DP + 127) / 128]) {
  const bool none = l == 0.0f;
  if (lane == 0) {
    const float z = none ? -INFINITY : m + log2f(l);
    const int64_t id = (int64_t)b * a.q_heads + h;
    if (a.lse) a.lse[id] = z * kLn2;
    if (a.stats) a.stats[id] = z;
  }
  const float inv = none ? 0.0f : 1.0f / l;
  QT* out = static_cast<QT*>(a.out.p) + b * a.out.token + (int64_t)h * a.out.head;
#pragma unroll
  for (int e = 0; e < (DP + 127) / 128; ++e) {
    const int d = e * 128 + lane * 4;
    if (d < a.c.dim) {
      store_pair(out + d, o[e].x * inv, o[e].y * inv, a.aligned_out);
      store_pair(out + d + 2, o[e].z * inv, o[e].w * inv, a.aligned_out);
    }
  }
}

// The same of a part of a row, to the workspace.
template <int DP>
__device__ __forceinline__ void put_part(const Args& a, int64_t part, int lane, float m, float l,
                                         const float4 (&o)[(DP + 127) / 128]) {
  if (lane == 0) a.part_stats[part] = make_float2(m, l);
#pragma unroll
  for (int e = 0; e < (DP + 127) / 128; ++e)
    if (e * 128 + lane * 4 < DP) *reinterpret_cast<float4*>(a.part_out + part * DP + e * 128 + lane * 4) = o[e];
}

// score of tokens begin .. end - 1 of sequence b, V at a time a lane, += their
// weights, summed over the query heads that share key/value head kvh; log_of(i):
// the log2 of the sum of exponentials of the i-th of them, infinite where there
// is no weight.
template <int V, class LogOf>
__device__ __forceinline__ void add_weights(const Args& a, int b, int kvh, int first, int len, int begin, int end,
                                            int lane, LogOf&& log_of) {
  const Cache& c = a.c;
  const int64_t h0 = (int64_t)b * a.q_heads + kvh * a.group;
  for (int t = begin + lane * V; t < end; t += 32 * V) {
    if (t + V <= first) continue;
    int page, off;
    if (!kv::find(c, a.tab, b, t, page, off, a.status)) continue;
    float* score = c.score + kv::scale_at(c, page, kvh, off);
    const float* logit = a.logits + h0 * a.logit_pitch + t;
    float p[V] = {};
    // a logit outside the sequence or its window is -infinity: no weight
    if constexpr (V == 4) {
      // (scores past the length or before the window are not this call's to write, even unchanged)
      const bool whole = t >= first && t + 4 <= len;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (whole) s = *reinterpret_cast<const float4*>(score);
#pragma unroll 4
      for (int i = 0; i < a.group; ++i) {
        const float r = log_of(i);
        const float4 l = __ldcs(reinterpret_cast<const float4*>(logit + i * a.logit_pitch));
        p[0] += ex2_approx(l.x - r), p[1] += ex2_approx(l.y - r);
        p[2] += ex2_approx(l.z - r), p[3] += ex2_approx(l.w - r);
      }
      if (whole) {
        s.x += p[0], s.y += p[1], s.z += p[2], s.w += p[3];
        *reinterpret_cast<float4*>(score) = s;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t + j >= first && t + j < len) score[j] += p[j];
      }
    } else {
#pragma unroll 4
      for (int i = 0; i < a.group; ++i) p[0] += ex2_approx(logit[i * a.logit_pitch] - log_of(i));
      *score += p[0];
    }
  }
}

// CUT: the rows follow the line; WHOLE: a CTA has whole rows, SHARED: a cluster
// has one (share_rows).  (One kernel for the last two cost every short call 0.4
// us.)
enum Split { CUT, WHOLE, SHARED };
template <class F, Split SPLIT>
__global__ void __launch_bounds__(F::W * 32, 1) attend_kernel(const __grid_constant__ Args a) {
  using QT = typename F::QT;
  constexpr bool S8 = F::S8;
  constexpr int NT = F::NT;
  constexpr bool LINE = SPLIT == CUT;
  extern __shared__ __align__(16) unsigned char smem[];
  int* line = reinterpret_cast<int*>(smem + F::W * F::WARP_BYTES);
  float2* open_stats = reinterpret_cast<float2*>(line + kMaxSequences + 4);  // [W][8 NT], 16-byte aligned
  int* open_row = reinterpret_cast<int*>(open_stats + F::W * 8 * NT);        // [W] row left open by a warp, or -1
  int* open_head = open_row + F::W;                                          // [W] that warp began the row
  int* sums = open_head + F::W;                                              // [W]
  const Cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, tig = lane & 3;
  const int B = a.tab.sequences, R = c.heads * a.chunks;

  next_kernel_may_start();
  wait_previous_kernel();

  // ---- the line: where each sequence starts ----
  if (lane == 0) open_row[warp] = -1;
  if (LINE || (a.logits && !a.scores_here && blockIdx.x == 0)) {  // (the scores' kernel follows it too)
    int run = 0;
    for (int b0 = 0; b0 < B; b0 += F::W * 32) {
      const int b = b0 + threadIdx.x;
      int v = 0;
      if (b < B) v = (tile_count(a, kv::cut_length(c, a.tab, a.lengths[b], a.status)) + kRowCost) * R;
      int x = v;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, i);
        if (lane >= i) x += u;
      }
      if (lane == 31) sums[warp] = x;
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll 4
      for (int w = 0; w < F::W; ++w) {
        const int u = sums[w];
        before += w < warp ? u : 0;
        all += u;
      }
      if (b < B) line[b] = run + before + x - v;
      run += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) line[B] = run;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= B; b += F::W * 32) a.line[b] = line[b];
  }
  // where this warp begins: units x .. x_end of the line, or its part of row `row_id`
  const int rank = SPLIT == SHARED ? blockIdx.x % a.cluster : 0;  // in the cluster
  const int row_id = LINE ? 0 : SPLIT == SHARED ? blockIdx.x / a.cluster : warp / a.per_row * a.ctas + blockIdx.x;
  const int row_part = LINE ? 0 : SPLIT == SHARED ? rank * F::W + warp : warp % a.per_row;
  Cut cut{};
  int w = 0, x = 0, x_end = 0, b = 0;
  if constexpr (!LINE) {
    x_end = row_id < B * R;
    b = row_id / R;
  } else {
    cut = cut_line(a, line[B], B * R);
    w = blockIdx.x * cut.per_cta + warp;
    if (warp < cut.per_cta && w < cut.parts) x = cut.begin(w), x_end = cut.begin(w + 1);
    for (int lo = 0, hi = B; lo < hi;) {  // last b with line[b] <= x
      const int mid = (lo + hi) / 2;
      if (line[mid] <= x) b = mid, lo = mid + 1;
      else hi = mid;
    }
  }

  unsigned char* ring = smem + warp * F::WARP_BYTES;
  const uint32_t ring_u = smem_u32(ring);
  uint2* q_smem = reinterpret_cast<uint2*>(ring + F::SLOTS * F::SLOT) + lane;
  const bool whole_pages = c.page_size % 16 == 0;  // a tile lies in one page
  const bool packed = a.token_bytes == F::ROW;     // and is one run of memory
  // places that do not change, kept in registers (the compiler would work them out again in every tile)
  int copy_at = F::place(lane / F::CR, lane % F::CR), k_at = F::place(g, tig);
  int v_at0 = F::VB == 16 ? F::place(2 * tig, g) : F::place(2 * tig, g / 2) + g % 2 * 8;
  int v_at1 = F::VB == 16 ? F::place(2 * tig + 1, g) : F::place(2 * tig + 1, g / 2) + g % 2 * 8;
  const int piece_bytes = lane % F::CR * 16 < c.dim * F::ES ? 16 : 0;  // a piece past head_dim is zeros
  asm volatile("" : "+r"(copy_at), "+r"(k_at), "+r"(v_at0), "+r"(v_at1));
  const int per_page = c.page_size / 16;
  const int D = c.dim;

  for (; x < x_end; ++b) {
    const int b_end = !LINE ? x_end : min(line[b + 1], x_end);
    const int len = kv::cut_length(c, a.tab, a.lengths[b], a.status);
    const int first = first_token(a, len), tile0 = first / 16;
    const int cost = tile_count(a, len) + kRowCost;
    const int32_t* pages = a.tab.page + (int64_t)b * a.tab.stride;
    while (x < b_end) {
      int row, begin, end, seg_end;
      bool starts, ends;
      if constexpr (!LINE) {
        const int tiles = cost - kRowCost;
        row = row_id - b * R;
        begin = tiles * row_part / a.per_row, end = tiles * (row_part + 1) / a.per_row;
        starts = ends = a.per_row == 1;
        seg_end = x_end;
      } else {
        row = (x - line[b]) / cost;
        const int row_at = line[b] + row * cost, in = x - row_at;
        seg_end = min(row_at + cost, x_end);
        begin = max(in - kRowCost, 0), end = max(seg_end - row_at - kRowCost, 0);
        starts = in == 0, ends = seg_end == row_at + cost;
      }
      const int kvh = row / a.chunks, h0 = kvh * a.group + (row % a.chunks) * (8 * NT);
      const int heads = min(8 * NT, (kvh + 1) * a.group - h0);
      x = seg_end;

      // ---- copies: a tile is located once, then its keys, then its values are sent for ----
      // Addresses are a lane's own: its piece of the key/value head's first
      // rows, and the scale of token lane % 16 (lanes from 16 on: of its value).
      // A tile adds where its first row lies.
      const int64_t head_at = kvh * a.head_bytes;
      const int64_t lane_at = head_at + lane / F::CR * a.token_bytes + lane % F::CR * 16;
      const char* const k_lane = static_cast<const char*>(c.k) + lane_at;
      const char* const v_lane = static_cast<const char*>(c.v) + lane_at;
      const float* const s_head = (lane < 16 ? c.ks : c.vs) + kvh * c.s_head;
      const float* const s_lane = s_head + (lane & 15) * c.s_token;
      int64_t at = 0, scale_at = 0;      // of the tile: bytes (-1: no such page), and elements of the scales
      int64_t at32 = 0, scale_at32 = 0;  // of the 32 tiles from the last multiple of 32 on, one a lane
      int page_next = 0, off_next = 0;   // of the 32 after those
      uint32_t mask = 0xffffu;           // tokens of the tile that take part
      bool plain = false;                // all of them, in one page
      uint32_t odd_tiles = 0;            // bit j: of the tile sent for j tiles ago, not all tokens take part
      const int last = tile_count(a, len) - 1;
      bool in_next = false;
      auto look_up = [&](int i) {  // ahead of their use: tiles i + lane, or token lane % 16 of tile i
        if (whole_pages) {
          if (i + lane < end) {
            const int t = tile0 + i + lane, p = t / per_page;
            off_next = (t - p * per_page) * 16;
            page_next = pages[p];
          }
        } else {
          const int t = (tile0 + i) * 16 + (lane & 15);
          in_next = i < end && t >= first && t < len;
          const int p = (int)((unsigned)t / (unsigned)c.page_size);
          off_next = t - p * c.page_size;
          page_next = in_next ? pages[p] : 0;
        }
      };
      auto locate = [&](int i) {
        const int t0 = (tile0 + i) * 16;
        plain = false;
        if (whole_pages) {
          const int l = (i - begin) & 31;
          if (l == 0) {
            const bool bad = (unsigned)page_next >= (unsigned)c.pages;
            if (bad) kv::report_index(a.status);
            at32 = bad ? -1 : page_next * a.page_bytes + off_next * a.token_bytes;
            scale_at32 = page_next * c.s_page + off_next * c.s_token;
            look_up(i + 32);
          }
          at = __shfl_sync(0xffffffffu, at32, l);
          if constexpr (S8) scale_at = __shfl_sync(0xffffffffu, scale_at32, l);
          mask = 0xffffu;
          if (i == 0 && t0 < first) mask = 0xffffu << (first - t0) & 0xffffu;
          if (i == last && len - t0 < 16) mask &= 0xffffu >> (16 - (len - t0));
          if (at < 0) mask = 0;
          plain = mask == 0xffffu;
        } else {  // at and scale_at: of token lane % 16
          const bool bad = (unsigned)page_next >= (unsigned)c.pages;
          if (bad) kv::report_index(a.status);
          at = page_next * a.page_bytes + off_next * a.token_bytes;
          scale_at = page_next * c.s_page + off_next * c.s_token;
          mask = __ballot_sync(0xffffffffu, in_next && !bad) & 0xffffu;
          look_up(i + 1);
        }
      };
      auto send = [&](int put, const char* from, const void* pool) {
        const uint32_t dst = ring_u + put;
        if (plain) {
          const char* src = from + at;
          if (packed) {
#pragma unroll
            for (int r = 0; r < F::CT; ++r) copy16(dst + F::copy_place(copy_at, r), src + r * 512, piece_bytes);
          } else {
#pragma unroll
            for (int r = 0; r < F::CT; ++r, src += a.step_bytes)
              copy16(dst + F::copy_place(copy_at, r), src, piece_bytes);
          }
        } else if (!whole_pages && mask == 0xffffu) {  // rows of several pages
          const char* src = from - lane / F::CR * a.token_bytes;
#pragma unroll
          for (int r = 0; r < F::CT; ++r)
            copy16(dst + F::copy_place(copy_at, r), src + __shfl_sync(0xffffffffu, at, (r * 32 + lane) / F::CR), piece_bytes);
        } else {  // some tokens are zeros
#pragma unroll 1
          for (int r = 0; r < F::CT; ++r) {
            const int t = (r * 32 + lane) / F::CR, p = lane % F::CR;
            const int64_t row = whole_pages ? at + t * a.token_bytes : __shfl_sync(0xffffffffu, at, t);
            const bool ok = (mask >> t & 1) && p * 16 < D * F::ES;
            copy16(dst + F::place(t, p), static_cast<const char*>(pool) + (ok ? head_at + row + p * 16 : 0), ok ? 16 : 0);
          }
        }
      };
      auto send_keys = [&](int i, int put) {
        odd_tiles <<= 1;
        if (i < end) {
          locate(i);
          send(put, k_lane, c.k);
          const uint32_t dst = ring_u + put + 16 * F::ROW + lane * 4;
          if (plain) {
            if constexpr (S8) copy4(dst, s_lane + scale_at, 4);
          } else {
            odd_tiles |= mask != 0xffffu;
            if constexpr (S8) {
              const bool ok = mask >> (lane & 15) & 1;
              const float* src = (whole_pages ? s_lane : s_head) + scale_at;
              copy4(dst, ok ? src : c.ks, ok ? 4 : 0);
            }
            if (lane == 0) *reinterpret_cast<uint32_t*>(ring + put + 16 * F::ROW + 128) = mask;
          }
        }
        copy_commit();
      };
      auto send_values = [&](int i, int put) {  // of the tile located last
        if (i < end) send(put, v_lane, c.v);
        copy_commit();
      };
      // The copy for AHEAD tiles on goes where the half used last lay.
      int use = 0, free_slot = (F::SLOTS - 1) * F::SLOT;
      auto advance = [&]() {
        free_slot = use;
        use = use == (F::SLOTS - 1) * F::SLOT ? 0 : use + F::SLOT;
      };
      __syncwarp();
      look_up(begin);
      // the query's elements are asked for ahead of the tiles (behind them they
      // came 3 us later where all SMs begin at once)
      constexpr int N = S8 ? 16 : 8;  // elements of a piece
      Piece<QT, N> q_raw[NT][F::PK];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const bool live = nt * 8 + g < heads;
        const QT* src = static_cast<const QT*>(a.q.p) + b * a.q.token + (int64_t)(h0 + nt * 8 + g) * a.q.head;
#pragma unroll
        for (int j = 0; j < F::PK; ++j) {
          const int d = (j * 4 + tig) * N;
          if (!live || d >= D) q_raw[nt][j].clear();
          else if (a.aligned_q) q_raw[nt][j].load(src + d);
          else q_raw[nt][j].load_any(src + d);
        }
      }
#pragma unroll 1
      for (int i = 0; i < F::AHEAD; ++i) {
        send_keys(begin + i, 2 * i * F::SLOT);
        send_values(begin + i, (2 * i + 1) * F::SLOT);
      }

      // ---- the query heads, as the columns of the first product ----
      uint2 q_reg[F::Q_REG ? F::NQ * NT * F::KS : 1];
      float factor[NT][2];  // of the scores of heads 2 tig and 2 tig + 1
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float v[F::PK][N];
#pragma unroll
        for (int j = 0; j < F::PK; ++j) q_raw[nt][j].to_float(v[j]);
        float f = a.scale * kLog2e;
        if constexpr (S8) {
          // the largest by a power of two to [2^13, 2^14): elements down to
          // 2^-27 of it are normal numbers of fp16, and two parts hold them to
          // 2^-24 of themselves (smaller ones: to 2^-49 of the largest)
          uint32_t most = 0;
#pragma unroll
          for (int j = 0; j < F::PK; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) most = max(most, __float_as_uint(fabsf(v[j][i])));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          most = min(max(most & 0x7f800000u, 0x10000000u), 0x7e800000u);  // 2^-95 to 2^126: both powers are normal
          const float down = __uint_as_float(0x7f000000u + (13u << 23) - most);
          f *= __uint_as_float(most) * 0x1p-13f;
#pragma unroll
          for (int j = 0; j < F::PK; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i) v[j][i] *= down;
        }
        factor[nt][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
        factor[nt][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
#pragma unroll
        for (int ks = 0; ks < F::KS; ++ks) {
          const float* e = S8 ? &v[ks / 4][ks % 4 * 4] : &v[ks / 2][ks % 2 * 4];
          uint32_t r0[F::NQ], r1[F::NQ];
          // int8 codes come as (0, 2) and (1, 3) of a word
          split2<S8, F::NQ>(e[0], S8 ? e[2] : e[1], r0);
          split2<S8, F::NQ>(S8 ? e[1] : e[2], e[3], r1);
#pragma unroll
          for (int i = 0; i < F::NQ; ++i) {
            const int at_q = (i * NT + nt) * F::KS + ks;
            if constexpr (F::Q_REG) q_reg[at_q] = make_uint2(r0[i], r1[i]);
            else q_smem[at_q * 32] = make_uint2(r0[i], r1[i]);
          }
        }
      }

      // ---- the tiles ----
      float o[F::MT][NT][4], m[NT][2], ref[NT][2], l[NT][2];  // ref: m, or 0 while m is -infinity
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < F::MT; ++mt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.0f;
        m[nt][0] = m[nt][1] = -INFINITY;
        ref[nt][0] = ref[nt][1] = 0.0f;
        l[nt][0] = l[nt][1] = 0.0f;
      }
      bool unset = true;  // some m is -infinity
#pragma unroll 1
      for (int i = begin; i < end; ++i) {
        send_keys(i + F::AHEAD, free_slot);
        copy_wait<2 * F::AHEAD>();
        __syncwarp();
        const unsigned char* slot = ring + use;
        advance();
        // fp32 queries: the products with q's first part are added up outside the
        // tensor pipe, whose sums are cut rather than rounded (bf16 queries leave
        // it their DP / 16 steps, 5e-6 of a log-sum of about 10), and apart from the
        // others: bf16 keys may be infinite, and infinity times a later part (0, or
        // of the other sign) is NaN
        float s[NT][4], rest[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nt][j] = 0.0f, rest[nt][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < F::PK; ++j) {
          const unsigned char* piece = slot + (k_at ^ (j & 1) * 64) + j / 2 * 128;  // place(g, j * 4 + tig)
          const uint4 r0 = *reinterpret_cast<const uint4*>(piece);
          const uint4 r1 = *reinterpret_cast<const uint4*>(piece + 8 * F::ROW);
          const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
          for (int k = 0; k < (S8 ? 4 : 2); ++k) {
            const int ks = j * (S8 ? 4 : 2) + k;
            uint32_t a0, a1, a2, a3;
            if constexpr (S8) {
              a0 = codes_fp16(w0[k]), a2 = codes_fp16(w0[k] >> 8);
              a1 = codes_fp16(w1[k]), a3 = codes_fp16(w1[k] >> 8);
            } else {
              a0 = w0[2 * k], a2 = w0[2 * k + 1];
              a1 = w1[2 * k], a3 = w1[2 * k + 1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int p = 0; p < F::NQ; ++p) {
                const int at_q = (p * NT + nt) * F::KS + ks;
                uint2 bq;
                if constexpr (F::Q_REG) bq = q_reg[at_q];
                else bq = q_smem[at_q * 32];
                if (F::WIDE && p == 0) {
                  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma<S8>(x, a0, a1, a2, a3, bq.x, bq.y);
                  s[nt][0] += x[0], s[nt][1] += x[1], s[nt][2] += x[2], s[nt][3] += x[3];
                } else {
                  mma<S8>(F::WIDE ? rest[nt] : s[nt], a0, a1, a2, a3, bq.x, bq.y);
                }
              }
          }
        }
        if constexpr (F::WIDE) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (fabsf(rest[nt][j]) < INFINITY) s[nt][j] = fmaf(rest[nt][j], S8 ? 1.0f / kPartGain : 1.0f, s[nt][j]);
        }
        const float* scales = reinterpret_cast<const float*>(slot + 16 * F::ROW);
        float k0 = 1.0f, k1 = 1.0f, f0 = 1.0f, f1 = 1.0f;  // scales of tokens g and g + 8, keys and values
        if constexpr (S8) {
          k0 = scales[g], k1 = scales[g + 8], f0 = scales[g + 16], f1 = scales[g + 24];
          // an infinite scale times a code of 0 is NaN, whatever the sum of the others
          k0 += k0 - k0, k1 += k1 - k1;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nt][j] = s[nt][j] * (j < 2 ? k0 : k1) * factor[nt][j & 1];
        if (odd_tiles >> F::AHEAD & 1) {
          const uint32_t taken = reinterpret_cast<const uint32_t*>(scales)[32];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!(taken >> (g + (j & 2) * 4) & 1)) s[nt][j] = -INFINITY;
        }
        if (a.logits) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (nt * 8 + 2 * tig + j < heads) {
                float* to = a.logits + ((int64_t)b * a.q_heads + h0 + nt * 8 + 2 * tig + j) * a.logit_pitch +
                            (int64_t)(tile0 + i) * 16 + g;
                to[0] = s[nt][j], to[8] = s[nt][2 + j];
              }
        }
        // a new reference where an exponent exceeds 8
        bool rise = unset;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) rise |= fmaxf(s[nt][j], s[nt][2 + j]) > ref[nt][j] + 8.0f;
        if (__any_sync(0xffffffffu, rise)) {
          unset = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float most = fmaxf(m[nt][j], fmaxf(s[nt][j], s[nt][2 + j]));
              most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 4));
              most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 8));
              most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
              // no score above -infinity so far: nothing to keep, and s - 0 = -infinity
              const float next = most == -INFINITY ? 0.0f : most;
              const float keep = m[nt][j] == -INFINITY ? 0.0f : ex2_approx(m[nt][j] - next);
              unset |= most == -INFINITY;
              m[nt][j] = most, ref[nt][j] = next;
              l[nt][j] *= keep;
#pragma unroll
              for (int mt = 0; mt < F::MT; ++mt) o[mt][nt][j] *= keep, o[mt][nt][2 + j] *= keep;
            }
          unset = __any_sync(0xffffffffu, unset);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            s[nt][j] = ex2_approx(s[nt][j] - ref[nt][j]);
            s[nt][2 + j] = ex2_approx(s[nt][2 + j] - ref[nt][j]);
            l[nt][j] += s[nt][j] + s[nt][2 + j];
          }

        // The next copies go where these keys lie: every lane has read its scales
        // and the mask by then (votes order no memory).
        __syncwarp();
        send_values(i + F::AHEAD, free_slot);
        copy_wait<2 * F::AHEAD>();
        __syncwarp();
        slot = ring + use;
        advance();
        uint32_t b0[NT][F::NP], b1[NT][F::NP];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          split2<false, F::NP>(s[nt][0] * f0, s[nt][1] * f0, b0[nt]);
          split2<false, F::NP>(s[nt][2] * f1, s[nt][3] * f1, b1[nt]);
#pragma unroll
          for (int p = 0; p < F::NP; ++p) b0[nt][p] = transpose8(b0[nt][p]), b1[nt][p] = transpose8(b1[nt][p]);
        }
        auto product = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // a tile's sum by itself, then rounded to the whole: the tensor pipe
            // cuts its sums, always downwards (a row's 860 tiles lost 10^-4 of
            // values of one sign that way; 64 x 8192 tokens with scores took 240
            // us so, and 249 with rounded sums)
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = F::NP - 1; p >= 0; --p) mma<false>(x, a0, a1, a2, a3, b0[nt][p], b1[nt][p]);
            add2(o[mt][nt][0], o[mt][nt][1], x[0], x[1]);
            add2(o[mt][nt][2], o[mt][nt][3], x[2], x[3]);
          }
        };
#pragma unroll
        for (int j = 0; j < F::PV; ++j) {
          constexpr int N = F::VB / 4;  // words of a piece
          uint32_t v[4][N];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // token 2 tig + (0, 1, 8, 9)
            const unsigned char* piece = slot + (r & 1 ? v_at1 : v_at0) + r / 2 * 8 * F::ROW + j * 128;
            if constexpr (F::VB == 16) {
              const uint4 u = *reinterpret_cast<const uint4*>(piece);
              v[r][0] = u.x, v[r][1] = u.y, v[r][N - 2] = u.z, v[r][N - 1] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(piece);
              v[r][0] = u.x, v[r][1] = u.y;
            }
          }
#pragma unroll
          for (int k = 0; k < N; ++k) {
            // elements of two neighbouring tokens side by side
            const uint32_t x0 = __byte_perm(v[0][k], v[1][k], 0x5410), x1 = __byte_perm(v[0][k], v[1][k], 0x7632);
            const uint32_t y0 = __byte_perm(v[2][k], v[3][k], 0x5410), y1 = __byte_perm(v[2][k], v[3][k], 0x7632);
            if constexpr (S8) {
              product((j * N + k) * 2, codes_bf16(x0), codes_bf16(x0 >> 8), codes_bf16(y0),
                      codes_bf16(y0 >> 8));
              product((j * N + k) * 2 + 1, codes_bf16(x1), codes_bf16(x1 >> 8), codes_bf16(y1),
                      codes_bf16(y1 >> 8));
            } else {
              product(j * N + k, x0, x1, y0, y1);
            }
          }
        }
        __syncwarp();
      }

      // ---- the row, or this part of it, into the ring: a warp's stores of
      // fragments to the workspace or the output touch 32 sectors each (16 warps'
      // took 4 us).  Four elements at a time are moved by the head's number, so
      // that the lanes of a quad of heads do not all write one bank. ----
      constexpr float unit = S8 ? 64.0f : 1.0f;  // of codes_bf16
      float* const result = reinterpret_cast<float*>(ring);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float sum = l[nt][j];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const int hh = nt * 8 + 2 * tig + j;
          if (g == 0) open_stats[warp * 8 * NT + hh] = make_float2(m[nt][j], sum);
#pragma unroll
          for (int mt = 0; mt < F::MT; ++mt)
            *reinterpret_cast<float2*>(result + hh * F::DP + (F::row_element(mt, g) ^ tig * 4)) =
                make_float2(o[mt][nt][j] * unit, o[mt][nt][2 + j] * unit);
        }
      __syncwarp();
      if (ends) {
#pragma unroll 1
        for (int hh = 0; hh < heads; ++hh) {
          const float2 st = open_stats[warp * 8 * NT + hh];
          float4 acc[F::E];
#pragma unroll
          for (int e = 0; e < F::E; ++e)
            if (e * 128 + lane * 4 < F::DP)
              acc[e] = *reinterpret_cast<const float4*>(result + hh * F::DP + ((e * 128 + lane * 4) ^ (hh / 2 % 4 * 4)));
          if (starts) finish_row<QT, F::DP>(a, b, h0 + hh, lane, st.x, st.y, acc);
          else put_part<F::DP>(a, ((int64_t)w * 2) * (8 * NT) + hh, lane, st.x, st.y, acc);
        }
        __syncwarp();
      } else if (lane == 0) {  // this warp's last: to be joined with its neighbours' there
        open_row[warp] = b * R + row, open_head[warp] = starts;
      }
    }
  }

  // ---- rows left open: neighbours of one row are joined, in the order of the line ----
  __syncthreads();
  const int mine = open_row[warp];
  if (mine >= 0) {
    int from = warp, to = warp;
    while (from > 0 && open_row[from - 1] == mine) --from;
    while (to + 1 < F::W && open_row[to + 1] == mine) ++to;
    const int heads = min(8 * NT, a.group - mine % R % a.chunks * (8 * NT));
#pragma unroll 1
    for (int hh = warp - from; hh < heads; hh += to - from + 1) {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll 1
      for (int i = from; i <= to; ++i) top = fmaxf(top, open_stats[i * 8 * NT + hh].x);
      const float ref = top == -INFINITY ? 0.0f : top;
      float4 acc[F::E];
#pragma unroll
      for (int e = 0; e < F::E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
      for (int i = from; i <= to; ++i) {
        const float2 st = open_stats[i * 8 * NT + hh];
        const float f = ex2_approx(st.x - ref);  // a part without weight: 2^-infinity, or o and l of 0
        sum = fmaf(st.y, f, sum);
        const float* part = reinterpret_cast<const float*>(smem + i * F::WARP_BYTES) + hh * F::DP;
#pragma unroll
        for (int e = 0; e < F::E; ++e)
          if (e * 128 + lane * 4 < F::DP) {
            const float4 v = *reinterpret_cast<const float4*>(part + ((e * 128 + lane * 4) ^ (hh / 2 % 4 * 4)));
            acc[e].x = fmaf(v.x, f, acc[e].x), acc[e].y = fmaf(v.y, f, acc[e].y);
            acc[e].z = fmaf(v.z, f, acc[e].z), acc[e].w = fmaf(v.w, f, acc[e].w);
          }
      }
      if constexpr (SPLIT == WHOLE) {  // that was the row
        const int in_b = mine % R;
        finish_row<QT, F::DP>(a, mine / R, in_b / a.chunks * a.group + in_b % a.chunks * (8 * NT) + hh, lane, top, sum, acc);
      } else if constexpr (SPLIT == SHARED) {  // the CTA's part of it, in the place of the first warp's
        __syncwarp();
        if (lane == 0) open_stats[hh] = make_float2(top, sum);
#pragma unroll
        for (int e = 0; e < F::E; ++e)
          if (e * 128 + lane * 4 < F::DP)
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + hh * F::DP +
                                       ((e * 128 + lane * 4) ^ (hh / 2 % 4 * 4))) = acc[e];
      } else {
        put_part<F::DP>(a, ((int64_t)(blockIdx.x * cut.per_cta + from) * 2 + open_head[from]) * (8 * NT) + hh, lane, top,
                        sum, acc);
      }
    }
  }

  // ---- the parts of a cluster's CTAs, a warp of any of them per head ----
  if constexpr (SPLIT == SHARED) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int seq = row_id / R, in_b = row_id - seq * R, chunk = in_b % a.chunks * (8 * NT);
    const int heads = min(8 * NT, a.group - chunk);
    cluster.sync();
#pragma unroll 1
    for (int hh = rank * F::W + warp; hh < heads; hh += a.cluster * F::W) {
      float2 st = make_float2(-INFINITY, 0.0f);
      if (lane < a.cluster) st = cluster.map_shared_rank(open_stats, lane)[hh];
      float top = st.x;
#pragma unroll
      for (int i = 1; i < kMostCtas; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      top = __shfl_sync(0xffffffffu, top, 0);
      const float ref = top == -INFINITY ? 0.0f : top;
      const float f = ex2_approx(st.x - ref);
      float sum = 0.0f;
      float4 acc[F::E];
#pragma unroll
      for (int e = 0; e < F::E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < kMostCtas; ++r) {
        if (r >= a.cluster) break;
        const float fr = __shfl_sync(0xffffffffu, f, r);
        sum = fmaf(__shfl_sync(0xffffffffu, st.y, r), fr, sum);
        const float* part = reinterpret_cast<const float*>(cluster.map_shared_rank(smem, r)) + hh * F::DP;
#pragma unroll
        for (int e = 0; e < F::E; ++e)
          if (e * 128 + lane * 4 < F::DP) {
            const float4 v = *reinterpret_cast<const float4*>(part + ((e * 128 + lane * 4) ^ (hh / 2 % 4 * 4)));
            acc[e].x = fmaf(v.x, fr, acc[e].x), acc[e].y = fmaf(v.y, fr, acc[e].y);
            acc[e].z = fmaf(v.z, fr, acc[e].z), acc[e].w = fmaf(v.w, fr, acc[e].w);
          }
      }
      finish_row<QT, F::DP>(a, seq, in_b / a.chunks * a.group + chunk + hh, lane, top, sum, acc);
    }
    cluster.sync();  // no CTA leaves while another reads its part; and the sums are there for the scores
  }

  // ---- the scores, where whole rows are here: a warp's share is the tokens that it has seen ----
  if constexpr (!LINE) {
    if (!a.scores_here) return;
    __syncthreads();  // the sums and logits of the CTA's warps
    if (row_id >= B * R) return;
    const int seq = row_id / R, kvh = row_id - seq * R;
    const int len = kv::cut_length(c, a.tab, a.lengths[seq], a.status);
    const int first = first_token(a, len), tiles = tile_count(a, len);
    const int t0 = (first / 16 + tiles * row_part / a.per_row) * 16;
    const int t1 = min((first / 16 + tiles * (row_part + 1) / a.per_row) * 16, len);
    const float* sum = a.stats + (int64_t)seq * a.q_heads + kvh * a.group;
    auto log_of = [&](int i) { return sum[i] == -INFINITY ? INFINITY : sum[i]; };
    if (a.fours) add_weights<4>(a, seq, kvh, first, len, t0, t1, lane, log_of);
    else add_weights<1>(a, seq, kvh, first, len, t0, t1, lane, log_of);
  }
}

template <class F>
int launch_attend(Args& a, cudaStream_t s) {
  a.ctas = sm_count(), a.warps = F::W;
  a.step_bytes = a.token_bytes * 32 / F::CR;
  // (no sequence can be longer than its row of the table, and a window may begin and end inside a tile)
  int64_t longest = ceil_div((int64_t)a.tab.max_pages * a.c.page_size, 16);
  if (a.window) longest = std::min<int64_t>(longest, a.window / 16 + 2);
  const int64_t rows = (int64_t)a.tab.sequences * a.c.heads * a.chunks;
  const Share share = share_rows(F::W, a.ctas, rows, longest, a.logits != nullptr, F::WIDE);
  a.per_row = share.per_row, a.cluster = share.cluster;
  a.scores_here = a.per_row && a.logits && a.chunks == 1;
  const unsigned blocks = a.cluster > 1 ? (unsigned)(rows * a.cluster) : (unsigned)a.ctas;
  I8Q_PROF("paged_attention", s);
  const auto kernel = !a.per_row ? attend_kernel<F, CUT> : a.cluster == 1 ? attend_kernel<F, WHOLE> : attend_kernel<F, SHARED>;
  return kv::launch(kernel, blocks, F::W * 32, F::SMEM, a.cluster, s, "paged_attention", a);
}

template <class QT, bool S8, int DP>
int launch_groups(Args& a, cudaStream_t s) {
  return a.heads_per_row == 8 ? launch_attend<Form<QT, S8, DP, 1>>(a, s) : launch_attend<Form<QT, S8, DP, 2>>(a, s);
}

template <int DP>
int attend(Args& a, int type, bool s8, cudaStream_t s) {
  if (type == I8Q_F32) return s8 ? launch_groups<float, true, DP>(a, s) : launch_groups<float, false, DP>(a, s);
  return s8 ? launch_groups<__nv_bfloat16, true, DP>(a, s) : launch_groups<__nv_bfloat16, false, DP>(a, s);
}

// One translation unit each, for the build's sake.
int attend_64(Args& a, int type, bool s8, cudaStream_t s);
int attend_128(Args& a, int type, bool s8, cudaStream_t s);
int attend_256(Args& a, int type, bool s8, cudaStream_t s);

}  // namespace kva
}  // namespace i8q
