// kv_attention.cu -- paged_attention: the joining kernels, the workspace and
// the entry points.  The attention kernel itself is in kv_attention.cuh.
#include "kv_attention.cuh"

namespace i8q {
namespace {

using namespace kva;

// The parts of a row that was cut.
struct Parts {
  int w0, w1, cta0, count, per_cta;  // count 1: it was not
  // part k: what CTA w0 / per_cta joined from w0 on, what the next ones joined, and part w1
  __device__ int64_t at(const Args& a, int k, int hh) const {
    const int w = k == 0 ? w0 : k == count - 1 ? w1 : (cta0 + k) * per_cta;
    return ((int64_t)w * 2 + (k == 0)) * a.heads_per_row + hh;
  }
};
__device__ __forceinline__ Parts parts_of(const Args& a, const Cut& cut, int row_at, int cost) {
  Parts p;
  p.w0 = cut.of(row_at), p.w1 = cut.of(row_at + cost - 1);
  p.per_cta = cut.per_cta;
  p.cta0 = p.w0 / cut.per_cta;
  p.count = p.w0 == p.w1 ? 1 : (p.w1 - 1) / cut.per_cta - p.cta0 + 2;
  return p;
}

// Rows that lie in several parts: S warps per sequence and query head, each
// reading four parts at once (a chain of four dependent loads: 4 us a call).
template <class QT, int DP, int S>
__device__ __forceinline__ void join_rows(const Args& a) {
  constexpr int E = (DP + 127) / 128;
  __shared__ float4 s_out[S > 1 ? 8 : 1][E][32];
  __shared__ float2 s_stats[8];
  const Cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp % S;
  const int id = blockIdx.x * (8 / S) + warp / S;
  if (id >= a.tab.sequences * a.q_heads) return;  // (whole CTAs where S is 8, as in the other returns)
  const int b = id / a.q_heads, h = id % a.q_heads;
  const int gi = h % a.group, row = h / a.group * a.chunks + gi / a.heads_per_row, hh = gi % a.heads_per_row;
  const int R = c.heads * a.chunks;
  const int n = a.line[a.tab.sequences], at = a.line[b], cost = (a.line[b + 1] - at) / R;
  const Cut cut = cut_line(a, n, a.tab.sequences * R);
  const Parts p = parts_of(a, cut, at + row * cost, cost);
  const int count = p.count;
  if (count == 1) return;
  float top = -INFINITY, sum = 0.0f;
  float4 acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int N = 4;  // parts read at once
  for (int k0 = slice * N; k0 < count; k0 += S * N) {
    float2 st[N];
    float4 v[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      st[i] = make_float2(-INFINITY, 0.0f);
      if (k0 + i < count) st[i] = a.part_stats[p.at(a, k0 + i, hh)];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[i][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k0 + i < count && e * 128 + lane * 4 < DP)
          v[i][e] = *reinterpret_cast<const float4*>(a.part_out + p.at(a, k0 + i, hh) * DP + e * 128 + lane * 4);
      }
    }
    float next = top;
#pragma unroll
    for (int i = 0; i < N; ++i) next = fmaxf(next, st[i].x);
    const float ref = next == -INFINITY ? 0.0f : next;
    const float keep = ex2_approx(top - ref);  // 2^-infinity (or sums of 0) at first
    top = next;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e].x *= keep, acc[e].y *= keep, acc[e].z *= keep, acc[e].w *= keep;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float f = ex2_approx(st[i].x - ref);  // a part without weight: 2^-infinity, or o and l of 0
      sum = fmaf(st[i].y, f, sum);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        acc[e].x = fmaf(v[i][e].x, f, acc[e].x), acc[e].y = fmaf(v[i][e].y, f, acc[e].y);
        acc[e].z = fmaf(v[i][e].z, f, acc[e].z), acc[e].w = fmaf(v[i][e].w, f, acc[e].w);
      }
    }
  }
  if constexpr (S > 1) {
    if (lane == 0) s_stats[warp] = make_float2(top, sum);
#pragma unroll
    for (int e = 0; e < E; ++e) s_out[warp][e][lane] = acc[e];
    __syncthreads();
    if (slice) return;
    top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) top = fmaxf(top, s_stats[warp + i].x);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float f = ex2_approx(s_stats[warp + i].x - ref);
      sum = fmaf(s_stats[warp + i].y, f, sum);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float4 v = s_out[warp + i][e][lane];
        acc[e].x = fmaf(v.x, f, acc[e].x), acc[e].y = fmaf(v.y, f, acc[e].y);
        acc[e].z = fmaf(v.z, f, acc[e].z), acc[e].w = fmaf(v.w, f, acc[e].w);
      }
    }
  }
  finish_row<QT, DP>(a, b, h, lane, top, sum, acc);
}

// score of each token += its weights, summed over the query heads that share
// its key/value head.  The line again, with one row per key/value head; a
// lane takes V tokens at a time: 4 neighbours in one page, or 1 (64 sequences
// of 8192, 32 and 8 heads, 101 MB: 23 us with 4, 70 with 1).
// HERE: the log of the sum of exponentials of rows that were cut is joined
// here too, a lane per query head (at most 32), from the parts' maxima and
// sums: the scores then need not wait for join_rows.
template <int V, bool HERE>
__device__ __forceinline__ void add_scores(const Args& a, int block, int blocks) {
  __shared__ float s_log[8][32];
  const Cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, B = a.tab.sequences;
  const int w = block * 8 + warp;
  // parts of 16 tiles at least; the other warps have none
  const int total = a.line[B], n = total / a.chunks, parts = max(1, min(blocks * 8, n / 16));
  if (w >= parts) return;
  const Cut cut = cut_line(a, total, B * c.heads * a.chunks);
  const int q = n / parts, longer = n - q * parts;
  int x = w * q + min(w, longer);
  const int x_end = x + q + (w < longer);
  // the last sequence that begins at or before x, by 32 of them at a time
  // (a binary search would read the line eleven times in turn)
  int b = 0;
  for (int step = B <= 32 ? 1 : B <= 1024 ? 32 : 1024; step; step /= 32) {
    const int i = b + lane * step;
    const bool before = i < B && a.line[i] / a.chunks <= x;
    b += (__popc(__ballot_sync(0xffffffffu, before)) - 1) * step;
  }
  for (; x < x_end; ++b) {
    const int at = a.line[b] / a.chunks, b_end = min(a.line[b + 1] / a.chunks, x_end);
    const int len = kv::cut_length(c, a.tab, a.lengths[b], a.status);
    const int first = first_token(a, len), tile0 = first / 16, cost = tile_count(a, len) + kRowCost;
    while (x < b_end) {
      const int kvh = (x - at) / cost, row_at = at + kvh * cost, seg_end = min(row_at + cost, x_end);
      const int begin = max(x - row_at - kRowCost, 0), end = max(seg_end - row_at - kRowCost, 0);
      x = seg_end;
      const int64_t h0 = (int64_t)b * a.q_heads + kvh * a.group;
      if constexpr (HERE) {
        if (lane < a.group) {
          const int hh = lane % a.heads_per_row;
          const Parts p = parts_of(a, cut, a.line[b] + (kvh * a.chunks + lane / a.heads_per_row) * cost, cost);
          float z;
          if (p.count == 1) {
            z = a.stats[h0 + lane];
          } else {
            float top = -INFINITY, sum = 0.0f;
            for (int k0 = 0; k0 < p.count; k0 += 4) {
              float2 st[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                st[i] = k0 + i < p.count ? a.part_stats[p.at(a, k0 + i, hh)] : make_float2(-INFINITY, 0.0f);
              const float next = fmaxf(fmaxf(top, fmaxf(st[0].x, st[1].x)), fmaxf(st[2].x, st[3].x));
              const float ref = next == -INFINITY ? 0.0f : next;
              sum *= ex2_approx(top - ref);
              top = next;
#pragma unroll
              for (int i = 0; i < 4; ++i) sum = fmaf(st[i].y, ex2_approx(st[i].x - ref), sum);
            }
            z = sum == 0.0f ? -INFINITY : top + log2f(sum);
          }
          s_log[warp][lane] = z == -INFINITY ? INFINITY : z;
        }
        __syncwarp();
      }
      auto log_of = [&](int i) {  // infinite where there is no weight
        if constexpr (HERE) return s_log[warp][i];
        const float z = a.stats[h0 + i];
        return z == -INFINITY ? INFINITY : z;
      };
      add_weights<V>(a, b, kvh, first, len, (tile0 + begin) * 16, min((tile0 + end) * 16, len), lane, log_of);
      if constexpr (HERE) __syncwarp();  // (the next row's logs go to the same place)
    }
  }
}

template <class QT, int DP, int S>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
  next_kernel_may_start();
  wait_previous_kernel();
  join_rows<QT, DP, S>(a);
}

template <int V>
__global__ void __launch_bounds__(256) score_kernel(const __grid_constant__ Args a) {
  wait_previous_kernel();
  add_scores<V, false>(a, blockIdx.x, gridDim.x);
}

// Both at once: the first `joins` CTAs join rows, the others add scores.
template <class QT, int DP, int S, int V>
__global__ void __launch_bounds__(256) join_and_score_kernel(const __grid_constant__ Args a, int joins) {
  wait_previous_kernel();
  if ((int)blockIdx.x < joins) join_rows<QT, DP, S>(a);
  else add_scores<V, true>(a, blockIdx.x - joins, gridDim.x - joins);
}

int width_of(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
int groups_of(int group) { return group <= 8 ? 1 : 2; }
int most_warps(bool s8, int dp, int nt) { return s8 && dp == 64 && nt == 1 ? 16 : dp <= 128 && (nt == 1 || dp == 64) ? 12 : 8; }

// Most that one sequence takes of the line.
int64_t line_length(const Cache& c, const Table& tab, int64_t q_heads) {
  const int64_t group = q_heads / c.heads;
  return (ceil_div((int64_t)tab.max_pages * c.page_size, 16) + kRowCost) * c.heads *
         ceil_div(group, 8 * groups_of((int)group));
}

using Kernel = void (*)(Args);
using KernelAt = void (*)(Args, int);
template <class QT, int S>
Kernel join_of(int dp) {
  return dp == 64 ? join_kernel<QT, 64, S> : dp == 128 ? join_kernel<QT, 128, S> : join_kernel<QT, 256, S>;
}
template <class QT, int S>
KernelAt join_and_score_of(int dp, bool fours) {
  if (dp == 64) return fours ? join_and_score_kernel<QT, 64, S, 4> : join_and_score_kernel<QT, 64, S, 1>;
  if (dp == 128) return fours ? join_and_score_kernel<QT, 128, S, 4> : join_and_score_kernel<QT, 128, S, 1>;
  return fours ? join_and_score_kernel<QT, 256, S, 4> : join_and_score_kernel<QT, 256, S, 1>;
}

struct Layout {
  int64_t line, part_stats, part_out, stats, logits, bytes, pitch;
  int heads_per_row, dp;
};

Layout layout_of(const Cache& c, const Table& tab, bool s8, int64_t q_heads, int accumulate) {
  Layout l{};
  const int nt = groups_of((int)(q_heads / c.heads));
  l.dp = width_of(c.dim);
  l.heads_per_row = 8 * nt;
  const int64_t B = std::min(tab.sequences, kMaxSequences);
  const int64_t slots = (int64_t)sm_count() * most_warps(s8, l.dp, nt) * 2 * l.heads_per_row;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t p = at;
    at += round_up(bytes, 256);
    return p;
  };
  l.line = take((B + 1) * 4);
  l.part_stats = take(slots * 8);
  l.part_out = take(slots * l.dp * 4);
  l.pitch = round_up((int64_t)tab.max_pages * c.page_size, 16);
  if (accumulate) {
    l.stats = take(B * q_heads * 4);
    l.logits = take(B * q_heads * l.pitch * 4);
  }
  l.bytes = at;
  return l;
}

// What the workspace's size and the call itself refuse alike, and the device forms of the structs.
int check_sizes(const i8q_kv_cache* cache, const i8q_page_table* table, int64_t q_heads, int accumulate, const char* who,
                Cache& c, Table& tab) {
  int rc = kv::check_cache(cache, who, c);
  if (rc == I8Q_OK) rc = kv::check_table(table, c, who, tab);
  if (rc != I8Q_OK) return rc;
  const std::string w = who;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads)
    return fail(I8Q_ERR_INVALID_ARG, w + ": q_heads must be a multiple of kv_heads, in range");
  if (tab.sequences * q_heads > INT32_MAX) return fail(I8Q_ERR_INVALID_ARG, w + ": sequences * q_heads out of range");
  if (accumulate && !c.score) return fail(I8Q_ERR_INVALID_ARG, w + ": accumulate needs a cache that keeps scores");
  if (line_length(c, tab, q_heads) > INT32_MAX)
    return fail(I8Q_ERR_UNSUPPORTED, w + ": max_pages * page_size * kv_heads out of range");
  return I8Q_OK;
}

}  // namespace
}  // namespace i8q

using namespace i8q;

extern "C" size_t i8q_paged_attention_workspace_size(const i8q_kv_cache* cache, const i8q_page_table* table,
                                                     int64_t q_heads, int accumulate) {
  Cache c;
  Table tab;
  if (check_sizes(cache, table, q_heads, accumulate, "paged_attention_workspace_size", c, tab) != I8Q_OK) return 0;
  return (size_t)layout_of(c, tab, cache->type == I8Q_S8, q_heads, accumulate).bytes;
}

extern "C" int i8q_paged_attention(const i8q_kv_cache* cache, const i8q_page_table* table, const int32_t* lengths,
                                   int type, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   int64_t q_heads, void* out, int64_t out_token_stride, int64_t out_head_stride,
                                   float* lse, float softmax_scale, int64_t window, int accumulate, void* workspace,
                                   size_t ws_bytes, void* stream) {
  Args a{};
  int rc = check_sizes(cache, table, q_heads, accumulate, "paged_attention", a.c, a.tab);
  if (rc != I8Q_OK) return rc;
  if (type != I8Q_F32 && type != I8Q_BF16)
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: type must be I8Q_F32 or I8Q_BF16");
  if (!lengths || !q || !out) return fail(I8Q_ERR_INVALID_ARG, "paged_attention: lengths, q or out is NULL");
  if (window < 0) return fail(I8Q_ERR_INVALID_ARG, "paged_attention: window must not be negative");
  if (!(softmax_scale == softmax_scale)) return fail(I8Q_ERR_INVALID_ARG, "paged_attention: softmax_scale is NaN");
  const bool s8 = cache->type == I8Q_S8;
  const int slice = (int)std::min<int64_t>(kMaxSequences, INT32_MAX / line_length(a.c, a.tab, q_heads));
  const Layout l = layout_of(a.c, a.tab, s8, q_heads, accumulate);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || ws_bytes < (size_t)l.bytes)
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: workspace is NULL, unaligned or too small");
  const int64_t ces = s8 ? 1 : 2;
  a.page_bytes = a.c.page_stride * ces, a.head_bytes = a.c.head_stride * ces;
  a.token_bytes = a.c.token_stride * ces;
  a.scale = softmax_scale;
  a.q_heads = (int)q_heads;
  a.group = a.q_heads / a.c.heads;
  a.window = (int)std::min<int64_t>(window, INT32_MAX);
  a.heads_per_row = l.heads_per_row;
  a.chunks = (int)ceil_div(a.group, a.heads_per_row);
  char* ws = static_cast<char*>(workspace);
  a.line = reinterpret_cast<int*>(ws + l.line);
  a.part_stats = reinterpret_cast<float2*>(ws + l.part_stats);
  a.part_out = reinterpret_cast<float*>(ws + l.part_out);
  if (accumulate) {
    a.stats = reinterpret_cast<float*>(ws + l.stats);
    a.logits = reinterpret_cast<float*>(ws + l.logits);
    a.logit_pitch = l.pitch;
  }
  const int64_t es = type == I8Q_F32 ? 4 : 2;
  a.aligned_q = reinterpret_cast<uintptr_t>(q) % 16 == 0 && q_token_stride * es % 16 == 0 && q_head_stride * es % 16 == 0;
  a.aligned_out = reinterpret_cast<uintptr_t>(out) % (2 * es) == 0 && out_token_stride % 2 == 0 && out_head_stride % 2 == 0;
  a.status = device_status_word();
  if (!a.status) return fail(I8Q_ERR_CUDA, "paged_attention: no status word");
  cudaStream_t s = as_stream(stream);
  const Table all = a.tab;
  a.fours = a.c.page_size % 4 == 0 && a.c.s_token == 1 && a.c.s_page % 4 == 0 && a.c.s_head % 4 == 0 &&
            reinterpret_cast<uintptr_t>(a.c.score) % 16 == 0;
  for (int b0 = 0; b0 < all.sequences; b0 += slice) {
    a.tab = Table{all.page + b0 * all.stride, all.stride, std::min(slice, all.sequences - b0), all.max_pages};
    a.lengths = lengths + b0;
    a.q = Heads{const_cast<char*>(static_cast<const char*>(q)) + b0 * q_token_stride * es, q_token_stride, q_head_stride};
    a.out = Heads{static_cast<char*>(out) + b0 * out_token_stride * es, out_token_stride, out_head_stride};
    a.lse = lse ? lse + b0 * q_heads : nullptr;
    rc = (l.dp == 64 ? attend_64 : l.dp == 128 ? attend_128 : attend_256)(a, type, s8, s);
    if (rc != I8Q_OK) return rc;
    // few rows mean many parts each: 8 warps a row then, where one would read all in turn (18 parts of each of
    // 32 heads: 5 us against 9)
    const int heads = a.tab.sequences * a.q_heads;
    const bool few = heads <= 2 * sm_count();
    const unsigned joins = (unsigned)(few ? heads : ceil_div(heads, 8)), scores = 16 * (unsigned)sm_count();
    // Both in one launch where there is not much to score: 24 x 2500 tokens of 16 heads take 35 us instead of 38;
    // with twice the registers of the scores alone 64 x 8192 of 8 heads would take 249 instead of 244.
    const int64_t tokens = (int64_t)a.tab.sequences * a.c.heads * a.tab.max_pages * a.c.page_size;
    if (!a.per_row && accumulate && a.group <= 32 && tokens <= 1 << 21) {
      I8Q_PROF("paged_attention_join_and_scores", s);
      const KernelAt kernel = type == I8Q_F32
                                  ? (few ? join_and_score_of<float, 8>(l.dp, a.fours) : join_and_score_of<float, 1>(l.dp, a.fours))
                                  : (few ? join_and_score_of<__nv_bfloat16, 8>(l.dp, a.fours)
                                         : join_and_score_of<__nv_bfloat16, 1>(l.dp, a.fours));
      rc = kv::launch(kernel, joins + scores, 256, 0, 1, s, "paged_attention_join_and_scores", a, (int)joins);
      if (rc != I8Q_OK) return rc;
      continue;
    }
    if (!a.per_row) {
      I8Q_PROF("paged_attention_join", s);
      const Kernel join = type == I8Q_F32 ? (few ? join_of<float, 8>(l.dp) : join_of<float, 1>(l.dp))
                                          : (few ? join_of<__nv_bfloat16, 8>(l.dp) : join_of<__nv_bfloat16, 1>(l.dp));
      rc = kv::launch(join, joins, 256, 0, 1, s, "paged_attention_join", a);
      if (rc != I8Q_OK) return rc;
    }
    if (accumulate && !a.scores_here) {
      I8Q_PROF("paged_attention_scores", s);
      rc = kv::launch(a.fours ? score_kernel<4> : score_kernel<1>, scores, 256, 0, 1, s, "paged_attention_scores", a);
      if (rc != I8Q_OK) return rc;
    }
  }
  return I8Q_OK;
}
