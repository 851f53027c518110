// sample.cu -- the next token of each row of logits: temperature, top-k,
// top-p and min-p, then a choice by a given random number.
#include <cooperative_groups.h>

#include <cmath>
#include <string>

#include "kv.cuh"

namespace i8q {
namespace {

namespace cg = cooperative_groups;

// ---- weights --------------------------------------------------------------
// A token's weight exp((x - max) / T) as a whole number of steps of 2^-42: the
// sums that decide which tokens are kept and which one is taken are sums of
// integers, exact in any order (2^20 of them fit 62 bits).  fp32 sums would
// miss a token's border by 1e-7 of the whole, a width of several tokens of a
// large vocabulary; fp64 has 1/64 of the rate.
//
// With y = (max - x) log2(e) / T = n + f, |f| <= 1/2, and j = rint(-512 f),
// r = -f - j / 512:   2^-y = 2^-n 2^(j/512) 2^r.   2^(j/512) comes from a table
// in two fp32 parts, 2^r - 1 = r ln2 + (r ln2)^2 / 2 + (r ln2)^3 / 6 (the next
// term is below 2^-46); what must be known to more than 24 bits is carried as
// the sum of two fp32 numbers.  Off by less than 2^-42 for every argument.
constexpr int kWeightBits = 42;
constexpr uint64_t kWhole = 1ull << kWeightBits;

constexpr int kSteps = 512;
constexpr double kLn2 = 0.693147180559945309417;

constexpr double exp_series(double x) {
  double sum = 1.0, term = 1.0;
  for (int i = 1; i < 24; ++i) term *= x / i, sum += term;
  return sum;
}

struct PowerTable {  // 2^(j / 512), j = -256 .. 256, in two parts
  float hi[kSteps + 1], lo[kSteps + 1];
  constexpr PowerTable() : hi(), lo() {
    for (int j = 0; j <= kSteps; ++j) {
      const double v = exp_series(kLn2 * (j - kSteps / 2) / kSteps);
      hi[j] = (float)v, lo[j] = (float)(v - (double)hi[j]);
    }
  }
};
__device__ const PowerTable g_powers = PowerTable();

struct Scale {
  float max, part;  // the row's largest logit, and f times it
  float minus;      // -f
  float ch, cl;     // log2(e) / (f T) in two parts
};

// Differences are those of logits times f, a power of two: a half, so that
// they do not overflow, but for a T by which log2(e) / (f T) would leave the
// range in which fp32 holds both its parts, or the logits that T tells apart
// have no half.  (A product with 2^60 that overflows is of a logit whose
// neighbours lie many times T from it: they weigh nothing.  Products are
// rounded before the sum: infinities of opposite signs give NaN, an infinity
// of the wrong sign never comes.)
__device__ __forceinline__ Scale make_scale(float max, float temperature) {
  const float f = temperature > 0x1p60f ? 0x1p-61f : temperature < 0x1p-60f ? 0x1p60f : 0.5f;
  const double c = 1.0 / kLn2 / (double)temperature / (double)f;
  const float ch = (float)c;
  return Scale{max, f * max, -f, ch, (float)(c - (double)ch)};
}

// powers: the table in shared memory.  0 for -infinity and NaN.
__device__ __forceinline__ uint64_t weight(float x, const Scale& s, const float2* powers) {
  if (x == s.max) return kWhole;
  const float xh = __fmul_rn(s.minus, x);
  const float h = __fadd_rn(s.part, xh), hv = __fsub_rn(h, s.part);
  const float hl = __fadd_rn(__fsub_rn(s.part, __fsub_rn(h, hv)), __fsub_rn(xh, hv));
  const float p = __fmul_rn(h, s.ch);
  if (!(p >= 0.0f && p < 43.5f)) return 0;
  const float pl = __fmaf_rn(hl, s.ch, __fmaf_rn(h, s.cl, __fmaf_rn(h, s.ch, -p)));
  constexpr float kMagic = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer
  const float nm = __fadd_rn(p, kMagic);
  const int n = __float_as_int(nm) - 0x4B400000;
  const float v = __fsub_rn(__fsub_rn(nm, kMagic), p);
  const float vh = __fsub_rn(v, pl), vl = __fsub_rn(__fsub_rn(v, vh), pl);
  const float jm = __fmaf_rn(vh, (float)kSteps, kMagic);
  const int j = __float_as_int(jm) - 0x4B400000;
  const float r = __fmaf_rn(__fsub_rn(jm, kMagic), -1.0f / kSteps, vh);
  constexpr float kLh = (float)kLn2, kLl = (float)(kLn2 - (double)kLh);
  constexpr float kC2 = (float)(kLn2 * kLn2 / 2), kC3 = (float)(kLn2 * kLn2 * kLn2 / 6);
  const float p1 = __fmul_rn(r, kLh);
  const float e1 = __fmaf_rn(r, kLl, __fmaf_rn(r, kLh, -p1));
  // (2^(r + vl): vl, 2^-26 at most, meets 1 + r ln2)
  const float t2 = __fmaf_rn(vl, __fmaf_rn(p1, kLh, kLh), __fmaf_rn(__fmul_rn(r, r), __fmaf_rn(r, kC3, kC2), e1));
  const float2 pw = powers[j + kSteps / 2];
  const float m = __fmul_rn(pw.x, p1);
  const float low = __fadd_rn(__fmaf_rn(pw.x, t2, __fmaf_rn(pw.x, p1, -m)), __fmaf_rn(pw.y, p1, pw.y));
  const float sum = __fadd_rn(pw.x, m);
  const float rest = __fadd_rn(__fsub_rn(m, __fsub_rn(sum, pw.x)), low);
  constexpr float kHalfBits = 2097152.0f;  // 2^21
  const float am = __fmaf_rn(sum, kHalfBits, kMagic);
  const float d = __fmaf_rn(rest, kHalfBits, __fmaf_rn(sum, kHalfBits, -__fsub_rn(am, kMagic)));
  const int a = __float_as_int(am) - 0x4B400000, b = __float_as_int(__fmaf_rn(d, kHalfBits, kMagic)) - 0x4B400000;
  const uint64_t w = ((uint64_t)(uint32_t)a << 21) + (int64_t)b;
  return (w + ((1ull << n) >> 1)) >> n;
}

// The same, out of line: for the few tokens that a table leaves.
__device__ __noinline__ uint64_t weight_apart(float x, const Scale& s, const float2* powers) { return weight(x, s, powers); }

// floor(f * sum) and whether something was cut off, 0 <= f < 1, sum < 2^63.
__device__ __forceinline__ uint64_t share(float f, uint64_t sum, bool& cut) {
  const uint32_t u = __float_as_uint(f), e = u >> 23;
  const uint64_t mant = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (int)(e ? e : 1);  // f = mant 2^-shift, shift >= 24
  const uint64_t hi = __umul64hi(mant, sum), lo = mant * sum;
  uint64_t q, rest;
  if (shift < 64) q = hi << (64 - shift) | lo >> shift, rest = lo << (64 - shift);
  else if (shift == 64) q = hi, rest = lo;
  else if (shift < 128) q = hi >> (shift - 64), rest = (hi << (128 - shift)) | lo;
  else q = 0, rest = hi | lo;
  cut = rest != 0;
  return q;
}

// ---- keys -----------------------------------------------------------------
// A logit as an unsigned number of the same order: NaN as -infinity, -0 as 0.
// bf16 logits have 16 bits.
template <class T>
struct Key;
template <>
struct Key<float> {
  static constexpr int kBits = 32, kVec = 4;
  static __device__ __forceinline__ uint32_t of(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
  }
};
template <>
struct Key<__nv_bfloat16> {
  static constexpr int kBits = 16, kVec = 8;
  static __device__ __forceinline__ uint32_t of(float x) { return Key<float>::of(x) >> 16; }
  static __device__ __forceinline__ float value(uint32_t k) {
    return Key<float>::value(k << 16 | ((k >> 15) ? 0u : 0xffffu));
  }
};

// bf16 logits have so few values that a row's weights can stand in a table, of
// the numbers from 2^-16 to 2^7 of either sign; others are worked out as they come.
constexpr uint32_t kTableFrom = (127 - 16) << 7, kTableTo = (127 + 7) << 7, kTableSize = kTableTo - kTableFrom;

struct Args {
  const void* logits;
  int64_t stride;
  int V;
  const float* random;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logprobs;
  uint32_t* status;
};

// Tokens of a CTA from which the table pays (64000: 205 us for 128 x 128000
// without it, 148 with; 16000: 49 us for 8 x 128000 without, 51 with).
constexpr int kTableShare = 32768;
constexpr int kThreads = 512, kWarps = kThreads / 32, kBins = 2048, kDigit = 11, kMostCtas = 8;
constexpr int kList = 1024, kLists = 2048;  // keys of the border's bin: of a CTA, of all
constexpr int kSmall = 6;                   // bits of a digit of those
constexpr int kFine = 64, kGroups = kBins / kFine;  // bins of a group: one for each lane
static_assert(kGroups == 32 && kMostCtas * kFine == kThreads, "");

struct Shared {
  float2 powers[kSteps + 1];
  uint32_t lo[2][kBins], hi[2][kBins];        // of this CTA, two histograms in turn
  uint64_t group[2][kMostCtas][kGroups];      // sums of their groups, of all CTAs
  uint64_t fine[kMostCtas][kFine];            // one group's bins, of all CTAs
  uint64_t warp_sum[kWarps];
  uint32_t list[kList], keys[kLists];
  uint32_t count;
  uint64_t best[kMostCtas];              // of each CTA of the cluster
  uint64_t mass[kMostCtas][kWarps];      // kept weight of each warp's tokens, of all CTAs
  uint32_t ties[kMostCtas][kWarps];      // and its tokens of the border's key
  Scale scale;
};

__device__ __forceinline__ void add(Shared& sh, int which, uint32_t bin, uint64_t w) {
  const uint32_t low = (uint32_t)w, old = atomicAdd(&sh.lo[which][bin], low);
  const uint32_t high = (uint32_t)(w >> 32) + (old + low < old);
  if (high) atomicAdd(&sh.hi[which][bin], high);
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint64_t u = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += u;
  }
  return v;
}

// One row by a cluster of CTAs, a contiguous share of its tokens each, and of
// that a contiguous share each warp.  The row is read again (from the caches) by
// each pass: the largest; counts (top-k), then weights' sums (top-p) by steps
// of the exponent, and the keys of the bin in which the border lies; the kept
// weight of each warp; the warp in which the random number falls alone.  Bound
// by the chain of these where rows are few (1 x 32000 bf16 with top-p 26 us, 12
// without), by issue slots where they are many (128 x 128000: bf16 121 us, fp32
// 194; without top-p 65 for bf16).  Tokens kept in registers or shared memory
// between the passes were not tried.
template <class T, bool TABLE>
__global__ void __launch_bounds__(kThreads, 2)
sample_kernel(const __grid_constant__ Args a) {
  using K = Key<T>;
  constexpr int kVec = K::kVec;
  extern __shared__ __align__(16) uint8_t memory[];
  Shared& sh = *reinterpret_cast<Shared*>(memory);
  const auto cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / S, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const auto meet = [&] { S > 1 ? cluster.sync() : __syncthreads(); };
  kv::next_kernel_may_start();
  // another CTA's memory may be written once that CTA has started: waited for before the first exchange
  if (S > 1) cluster.barrier_arrive();
  for (int i = threadIdx.x; i <= kSteps; i += kThreads) sh.powers[i] = make_float2(g_powers.hi[i], g_powers.lo[i]);
  kv::wait_previous_kernel();

  const T* const x = static_cast<const T*>(a.logits) + row * a.stride;
  // vectors of 16 bytes: the first begins `skew` tokens before the row
  const int skew = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T) % kVec);
  const int vectors = (int)(((int64_t)a.V + skew + kVec - 1) / kVec);
  const int part = rank * kWarps + warp, parts = S * kWarps;
  const int v0 = (int)((int64_t)vectors * part / parts), v1 = (int)((int64_t)vectors * (part + 1) / parts);
  auto load = [&](int v, float (&y)[kVec]) {
    const int first = v * kVec - skew;
    if (v < v1 && first >= 0 && first + kVec <= a.V) {
      const uint4 u = *reinterpret_cast<const uint4*>(x + first);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        y[j] = kVec == 4 ? __uint_as_float(w[j & 3]) : __uint_as_float(j & 1 ? w[j / 2 & 3] & 0xffff0000u : w[j / 2 & 3] << 16);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        y[j] = v < v1 && first + j >= 0 && first + j < a.V ? (float)x[first + j] : -INFINITY;
    }
  };

  // f(first token, logits) of each of this lane's vectors, two on their way
  auto each = [&](auto f) {
    for (int v = v0 + lane; v < v1; v += 64) {
      float y[kVec], z[kVec];
      load(v, y), load(v + 32, z);
      f(v * kVec - skew, y);
      if (v + 32 < v1) f((v + 32) * kVec - skew, z);
    }
  };

  // ---- the largest logit, and its first place ----
  const float temperature = a.temperature ? a.temperature[row] : 1.0f, u = a.random[row];
  const float top_p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f;
  int top_k = a.top_k ? a.top_k[row] : 0;
  if (top_k <= 0 || top_k > a.V) top_k = a.V;
  float high = -INFINITY;
  int place = 0x7fffffff;
  each([&](int first, const float (&y)[kVec]) {
    float top = y[0];  // (fmaxf leaves NaN out; places outside the row are -infinity)
#pragma unroll
    for (int j = 1; j < kVec; ++j) top = fmaxf(top, y[j]);
    if (top > high) {
      high = top;
#pragma unroll
      for (int j = kVec - 1; j >= 0; --j)
        if (y[j] == top) place = first + j;
    }
  });
  uint64_t best = (uint64_t)K::of(high) << 32 | (uint32_t)~place;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, m));
  if (lane == 0) sh.warp_sum[warp] = best;
  __syncthreads();
  if (S > 1) cluster.barrier_wait();
  if (threadIdx.x < S) {
    for (int w = 0; w < kWarps; ++w) best = max(best, sh.warp_sum[w]);
    cluster.map_shared_rank(sh.best, threadIdx.x)[rank] = best;
  }
  meet();
  best = 0;
  for (int r = 0; r < S; ++r) best = max(best, sh.best[r]);
  const float largest = K::value((uint32_t)(best >> 32));
  const bool valid = temperature >= 0.0f && u >= 0.0f && u < 1.0f && top_p >= 0.0f && min_p >= 0.0f && min_p <= 1.0f;
  if (!valid || temperature == 0.0f || largest == -INFINITY) {  // (the same for the whole cluster)
    if (rank == 0 && threadIdx.x == 0) {
      if (!valid) atomicOr(a.status, ST_SAMPLE);
      const bool none = !valid || largest == -INFINITY;
      a.tokens[row] = none ? -1 : (int)~(uint32_t)best;
      if (a.logprobs) a.logprobs[row] = !valid ? NAN : none ? -INFINITY : 0.0f;
    }
    return;
  }
  // (fp64 has two lanes a cycle: one division, not 512)
  if (threadIdx.x == 0) sh.scale = make_scale(largest, temperature);
  __syncthreads();
  const Scale scale = sh.scale;

  // a token's weight
  uint64_t* const table = reinterpret_cast<uint64_t*>(memory + (sizeof(Shared) + 15) / 16 * 16);
  if constexpr (TABLE) {
    for (uint32_t i = threadIdx.x; i < 2 * kTableSize; i += kThreads) {
      const uint32_t bits = i < kTableSize ? kTableFrom + i : 0x8000u | (kTableFrom + i - kTableSize);
      table[i] = weight(__uint_as_float(bits << 16), scale, sh.powers);  // (of numbers above the largest: not read)
    }
    __syncthreads();
  }
  auto weigh = [&](float y) {
    if constexpr (TABLE) {
      const uint32_t bits = __float_as_uint(y) >> 16, at = (bits & 0x7fffu) - kTableFrom;
      if (at < kTableSize) return table[at + (bits >> 15) * kTableSize];
      return y == -INFINITY ? (uint64_t)0 : weight_apart(y, sh.scale, sh.powers);
    }
    return weight(y, scale, sh.powers);
  };

  // ---- the border: kept are the keys above it and the first `ties` of its own ----
  // (logits compare as their keys do, but for NaN, which weighs nothing)
  uint32_t border = 0, ties = UINT32_MAX;
  float border_y = -INFINITY;
  bool cut = false;
  int which = 1;
  // Counts (or weights) of the tokens within the border so far by their bins,
  // bin(logit) (negative: left out).  The CTAs exchange the sums of groups
  // of bins; `find` then reads one group's bins.
  auto histogram = [&](bool by_weight, auto bin) {
    which ^= 1;  // (the other one may still be read)
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[which][i] = sh.hi[which][i] = 0;
    __syncthreads();
    each([&](int first, const float (&y)[kVec]) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const int b = bin(y[j]);
        if (b < 0) continue;
        if (!by_weight) {
          if (first + j >= 0 && first + j < a.V) atomicAdd(&sh.lo[which][b], 1u);
        } else if (!cut || y[j] > border_y) {
          const uint64_t w = weigh(y[j]);
          if (w) add(sh, which, b, w);
        }
      }
    });
    if (by_weight && cut && rank == 0 && threadIdx.x == 0) {
      const int b = bin(border_y);
      if (b >= 0) add(sh, which, b, ties * weight(border_y, scale, sh.powers));
    }
    __syncthreads();
    for (int g = warp; g < kGroups; g += kWarps) {
      uint64_t sum = 0;
#pragma unroll
      for (int b = g * kFine + lane; b < (g + 1) * kFine; b += 32) sum += (uint64_t)sh.hi[which][b] << 32 | sh.lo[which][b];
      sum = warp_sum64(sum);
      if (lane < S) cluster.map_shared_rank(&sh, lane)->group[which][rank][g] = sum;
    }
    meet();
  };
  // The place, from the top, at which the running sum of a lane's two values
  // (each lane's second below its first) reaches target: 2 lane + 0 or 1, and
  // the sum before it.  All warps of the CTA work it out.
  auto reached = [&](uint64_t first, uint64_t second, uint64_t target, uint64_t& before) {
    const uint64_t upto = warp_scan64(first + second, lane), mine = upto - first - second;
    const int at = __ffs(__ballot_sync(0xffffffffu, upto >= target)) - 1;
    const bool later = mine + first < target;
    before = __shfl_sync(0xffffffffu, later ? mine + first : mine, at);
    return 2 * at + (int)__shfl_sync(0xffffffffu, (unsigned)later, at);
  };
  auto group_sum = [&](int g) {
    uint64_t sum = 0;
    for (int r = 0; r < S; ++r) sum += sh.group[which][r][g];
    return sum;
  };
  // The digit in whose bin the sum from the top reaches target (at most the
  // whole sum), and the sum before it.
  auto find = [&](uint64_t target, uint64_t& before) {
    uint64_t inside;
    const int group = kGroups - 1 - reached(group_sum(kGroups - 1 - lane), 0, target, before) / 2;
    if ((int)threadIdx.x < S * kFine) {
      const int r = threadIdx.x / kFine, b = threadIdx.x % kFine;
      const Shared* other = cluster.map_shared_rank(&sh, r);
      sh.fine[r][b] = (uint64_t)other->hi[which][group * kFine + b] << 32 | other->lo[which][group * kFine + b];
    }
    __syncthreads();
    uint64_t t[2] = {0, 0};
    for (int r = 0; r < S; ++r) t[0] += sh.fine[r][kFine - 1 - 2 * lane], t[1] += sh.fine[r][kFine - 2 - 2 * lane];
    const int bin = group * kFine + kFine - 1 - reached(t[0], t[1], target - before, inside);
    before += inside;
    return (uint32_t)bin;
  };
  // The first bins are even steps of the exponent, 32 to a factor of 2 of the
  // weight: logits spread over several hundred of them, where the keys' first
  // digit has four to an octave, and a handful of addresses took all the adds
  // (32000 tokens: 8 us a histogram).
  auto step = [&](float y) {
    const float d = y == scale.max ? 0.0f : __fmul_rn(__fadd_rn(scale.part, __fmul_rn(scale.minus, y)), scale.ch);
    return kBins - 1 - (d < 63.9f ? (int)(32.0f * d) : kBins - 1);  // (infinities and NaN: the last)
  };
  // After the first histogram: the key at which the sum from the top reaches target, and what is missing before it.
  auto descend = [&](bool by_weight, uint64_t target, uint32_t& key, uint64_t& missing) {
    uint64_t before;
    const int bin = (int)find(target, before);
    target -= before;
    // the keys of that bin, where they are few, brought together in each CTA
    // (a range that holds the bin, where T is not below what fp32 tells apart near the largest, spares most the step)
    const float wide = (float)kLn2 / 32.0f * temperature;
    const bool plain = wide > 0x1p-18f * fabsf(scale.max) && wide > 1e-30f && wide < 1e30f && bin > 1;
    const float least_y = plain ? scale.max - (float)(kBins + 1 - bin) * wide : -INFINITY;
    const float most_y = plain ? scale.max - (float)(kBins - 3 - bin) * wide : INFINITY;
    if (threadIdx.x == 0) sh.count = 0;  // (read by others before the last meeting, at the latest)
    __syncthreads();
    each([&](int first, const float (&y)[kVec]) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (y[j] < least_y || y[j] > most_y || step(y[j]) != bin || first + j < 0 || first + j >= a.V ||
            (by_weight && cut && !(y[j] > border_y)))
          continue;
        const uint32_t at = atomicAdd(&sh.count, 1u);
        if (at < kList) sh.list[at] = K::of(y[j]);
      }
    });
    meet();
    uint32_t all = 0;
    bool few = true;
    for (int r = 0; r < S; ++r) {
      const Shared* other = cluster.map_shared_rank(&sh, r);
      const uint32_t n = other->count;
      few = few && n <= kList && all + n <= kLists;
      if (few)
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) sh.keys[all + i] = other->list[i];
      all += n;
    }
    key = 0;
    if (few) {  // (the same in all CTAs)
      const bool extra = by_weight && cut && step(border_y) == bin;  // the border's ties, as one
      for (int shift = K::kBits; shift > 0;) {
        const int bits = min(kSmall, shift);
        shift -= bits;
        if (threadIdx.x < 1 << kSmall) sh.lo[which ^ 1][threadIdx.x] = sh.hi[which ^ 1][threadIdx.x] = 0;
        __syncthreads();
        auto count = [&](uint32_t k, uint32_t times) {
          if (shift + bits < 32 && k >> (shift + bits) != key) return;
          add(sh, which ^ 1, k >> shift & ((1u << bits) - 1), times * (by_weight ? weight(K::value(k), scale, sh.powers) : 1));
        };
        for (uint32_t i = threadIdx.x; i < all; i += kThreads) count(sh.keys[i], 1);
        if (extra && threadIdx.x == 0) count(border, ties);
        __syncthreads();
        const int top = (1 << kSmall) - 1 - 2 * lane;
        const uint32_t* lo = sh.lo[which ^ 1];
        const uint32_t* hi = sh.hi[which ^ 1];
        uint64_t inside;
        const int at = reached((uint64_t)hi[top] << 32 | lo[top], (uint64_t)hi[top - 1] << 32 | lo[top - 1], target, inside);
        key = key << bits | (uint32_t)((1 << kSmall) - 1 - at);
        target -= inside;
        __syncthreads();
      }
    } else {  // (many equal logits, say) digits of the keys, from the top
      for (int shift = K::kBits; shift > 0;) {
        const int bits = min(kDigit, shift);
        shift -= bits;
        const uint32_t prefix = key, mask = (1u << bits) - 1;
        const int above = shift + bits, low = shift;
        histogram(by_weight, [&](float y) {
          const uint32_t k = K::of(y);
          return step(y) != bin || (above < 32 && k >> above != prefix) ? -1 : (int)(k >> low & mask);
        });
        key = key << bits | find(target, before);
        target -= before;
      }
    }
    missing = target;
  };
  if (top_k < a.V) {
    uint64_t missing;
    histogram(false, step);
    descend(false, (uint64_t)top_k, border, missing);
    ties = (uint32_t)missing, border_y = K::value(border), cut = true;
  }
  if (top_p < 1.0f) {
    histogram(true, step);
    const uint64_t sum = warp_sum64(group_sum(lane));
    bool more;
    uint64_t target = share(top_p, sum, more), missing;
    target = max(target + more, (uint64_t)1);
    uint32_t key;
    descend(true, target, key, missing);
    const uint64_t w = weight(K::value(key), scale, sh.powers);
    border = key, ties = (uint32_t)((missing + w - 1) / w), border_y = K::value(key), cut = true;
  }

  // ---- the kept weight of each warp's tokens ----
  bool more;
  const uint64_t least = [&] {
    if (min_p >= 1.0f) return kWhole;
    const uint64_t q = share(min_p, kWhole, more);
    return max(q + more, (uint64_t)1);
  }();
  uint64_t mass = 0;
  uint32_t same = 0;
  each([&](int, const float (&y)[kVec]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (cut && y[j] <= border_y) {
        same += y[j] == border_y;
        continue;
      }
      const uint64_t w = weigh(y[j]);
      if (w >= least) mass += w;
    }
  });
  mass = warp_sum64(mass);
  same = __reduce_add_sync(0xffffffffu, same);
  if (lane < S) {
    Shared* other = cluster.map_shared_rank(&sh, lane);
    other->mass[rank][warp] = mass, other->ties[rank][warp] = same;
  }
  meet();
  uint64_t tie_weight = cut ? weight(K::value(border), scale, sh.powers) : 0;
  if (tie_weight < least) tie_weight = 0;
  // the running sums of the warps of the cluster, four to a lane (parts <= 128); each warp works them out
  uint64_t part_mass[4], lane_mass = 0;
  uint32_t part_ties[4], lane_ties = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = lane * 4 + i;
    part_mass[i] = p < parts ? sh.mass[p / kWarps][p % kWarps] : 0;
    part_ties[i] = p < parts && cut ? sh.ties[p / kWarps][p % kWarps] : 0;
    lane_ties += part_ties[i];
  }
  uint32_t seen = lane_ties;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint32_t w = __shfl_up_sync(0xffffffffu, seen, m);
    if (lane >= m) seen += w;
  }
  seen -= lane_ties;
  uint32_t part_seen[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    part_seen[i] = seen;
    const uint32_t here = seen < ties ? min(part_ties[i], ties - seen) : 0;
    seen += part_ties[i];
    part_mass[i] += here * tie_weight;
    lane_mass += part_mass[i];
  }
  const uint64_t upto = warp_scan64(lane_mass, lane), sum = __shfl_sync(0xffffffffu, upto, 31);
  uint64_t before = upto - lane_mass;
  uint32_t seen_before = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < (part & 3)) before += part_mass[i];
    if (i == (part & 3)) mass = before + part_mass[i], seen_before = part_seen[i];
  }
  before = __shfl_sync(0xffffffffu, before, part / 4), mass = __shfl_sync(0xffffffffu, mass, part / 4);
  seen_before = __shfl_sync(0xffffffffu, seen_before, part / 4);
  const uint64_t target = share(u, sum, more);  // taken: the first token up to which the sum is above it
  if (!(before <= target && target < mass)) return;

  // ---- the token, by the warp that has it ----
  uint64_t at = before;
  uint32_t left = cut && seen_before < ties ? ties - seen_before : 0;
  for (int vb = v0; vb < v1; vb += 32) {
    const int v = vb + lane;
    float y[kVec];
    load(v, y);
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) mine += cut && K::of(y[j]) == border;
    uint32_t earlier = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const uint32_t w = __shfl_up_sync(0xffffffffu, earlier, m);
      if (lane >= m) earlier += w;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, earlier, 31);
    earlier -= mine;
    uint64_t w[kVec], total = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const uint32_t k = K::of(y[j]);
      w[j] = 0;
      if (cut && k <= border) {
        if (k == border && earlier++ < left) w[j] = tie_weight;
      } else {
        w[j] = weigh(y[j]);
        if (w[j] < least) w[j] = 0;
      }
      total += w[j];
    }
    const uint64_t inclusive = warp_scan64(total, lane) + at;
    const uint32_t past = __ballot_sync(0xffffffffu, inclusive > target);
    if (past) {
      if (lane == __ffs(past) - 1) {
        uint64_t c = inclusive - total, chosen = 0;
        int token = 0;
#pragma unroll
        for (int j = kVec - 1; j >= 0; --j) {  // from the last on: the first one past the target stays
          uint64_t upto = c;
          for (int i = 0; i <= j; ++i) upto += w[i];
          if (upto > target) token = v * kVec - skew + j, chosen = w[j];
        }
        a.tokens[row] = token;
        if (a.logprobs) {
          // near 1 from what is missing to it
          const float ratio = __fdiv_rn((float)chosen, (float)sum);
          a.logprobs[row] = ratio > 0.5f ? log1pf(-__fdiv_rn((float)(sum - chosen), (float)sum)) : logf(ratio);
        }
      }
      return;
    }
    at = __shfl_sync(0xffffffffu, inclusive, 31);
    left -= min(left, all);
  }
}

}  // namespace
}  // namespace i8q

using namespace i8q;

extern "C" int i8q_sample(const void* logits, int type, int64_t rows, int64_t vocabulary, int64_t row_stride,
                          const float* random, const i8q_sampling* sampling, int32_t* tokens, float* logprobs,
                          void* stream) {
  if (type != I8Q_F32 && type != I8Q_BF16) return fail(I8Q_ERR_INVALID_ARG, "sample: type must be I8Q_F32 or I8Q_BF16");
  if (rows < 0 || rows > (1 << 24)) return fail(I8Q_ERR_INVALID_ARG, "sample: rows must be 0 .. 2^24");
  if (vocabulary < 1 || vocabulary > I8Q_SAMPLE_MAX_VOCABULARY)
    return fail(I8Q_ERR_INVALID_ARG, "sample: vocabulary must be 1 .. 2^20");
  if (rows == 0) return I8Q_OK;
  if (!logits || !random || !tokens) return fail(I8Q_ERR_INVALID_ARG, "sample: logits, random or tokens is NULL");
  if (rows > 1 && row_stride < vocabulary) return fail(I8Q_ERR_INVALID_ARG, "sample: rows overlap (row_stride below vocabulary)");
  const uintptr_t es = type == I8Q_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % es) return fail(I8Q_ERR_INVALID_ARG, "sample: logits are not aligned to their type");
  const i8q_sampling none{};
  const i8q_sampling& p = sampling ? *sampling : none;
  for (const void* of_rows : {(const void*)random, (const void*)p.temperature, (const void*)p.top_k, (const void*)p.top_p,
                              (const void*)p.min_p, (const void*)tokens, (const void*)logprobs})
    if (reinterpret_cast<uintptr_t>(of_rows) % 4)
      return fail(I8Q_ERR_INVALID_ARG, "sample: random, a setting, tokens or logprobs are not aligned to their type");
  uint32_t* status = device_status_word();
  if (!status) return fail(I8Q_ERR_CUDA, "sample: no status word");
  Args a{logits, row_stride, (int)vocabulary, random, p.temperature, p.top_k, p.top_p, p.min_p, tokens, logprobs, status};
  // CTAs of a row: what two on each SM leave room for, of 4096 tokens at least
  int S = 1;
  while (S < kMostCtas && rows * S * 2 <= 2 * sm_count() && vocabulary >= 4096 * S * 2) S *= 2;
  cudaStream_t s = as_stream(stream);
  I8Q_PROF("sample", s);
  auto run = [&](auto kernel, int table) {
    return kv::launch(kernel, (unsigned)(rows * S), kThreads, (int)((sizeof(Shared) + 15) / 16 * 16) + table, S, s, "sample", a);
  };
  if (type == I8Q_F32) return run(sample_kernel<float, false>, 0);
  if (vocabulary / S < kTableShare) return run(sample_kernel<__nv_bfloat16, false>, 0);
  return run(sample_kernel<__nv_bfloat16, true>, 2 * kTableSize * 8);
}
