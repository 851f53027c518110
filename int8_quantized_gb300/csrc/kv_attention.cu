// kv_attention.cu -- attention of one new token per sequence over a paged
// key/value cache.
#include <math.h>

#include "kv.cuh"

namespace i8q {
namespace {

using kv::Cache;
using kv::Table;

struct Heads {  // [sequences][heads][dim], strides in elements
  void* p;
  int64_t token, head;
};

struct Args {
  Cache c;
  Table tab;
  const int32_t* lengths;
  Heads q, out;
  float* lse;
  float scale;
  int q_heads, window, accumulate;
  float* logits;  // [sequences][q_heads][max tokens], accumulate only
  float* stats;   // [sequences][q_heads] log sum of exponentials
  uint32_t* status;
};

// One CTA per sequence and query head; each warp takes every eighth token
// and keeps a running maximum, sum and weighted value, joined at the end.
template <class T, bool S8>
__global__ void __launch_bounds__(256) attend_kernel(Args a) {
  constexpr int E = I8Q_KV_MAX_HEAD_DIM / 32;
  __shared__ float sm[8], sl[8], so[8][I8Q_KV_MAX_HEAD_DIM];
  const Cache& c = a.c;
  const int b = blockIdx.x / a.q_heads, h = blockIdx.x % a.q_heads, kvh = h / (a.q_heads / c.heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int len = kv::cut_length(c, a.tab, a.lengths[b], a.status);
  const int first = a.window && len > a.window ? len - a.window : 0;
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.token + h * a.q.head;
  float x[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int d = lane + 32 * e;
    x[e] = d < c.dim ? (float)q[d] * a.scale : 0.0f;
    acc[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  float* logit = a.accumulate ? a.logits + (int64_t)blockIdx.x * a.tab.max_pages * c.page_size : nullptr;
  for (int t = first + warp; t < len; t += 8) {
    int page, off;
    if (!kv::find(c, a.tab, b, t, page, off, a.status)) {
      if (logit && lane == 0) logit[t] = -INFINITY;
      continue;
    }
    const int64_t row = kv::row_at(c, page, kvh, off), sc = S8 ? kv::scale_at(c, page, kvh, off) : 0;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      if (d < c.dim)
        s = fmaf(x[e], S8 ? (float)static_cast<const int8_t*>(c.k)[row + d]
                          : (float)static_cast<const __nv_bfloat16*>(c.k)[row + d], s);
    }
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    if (S8) s *= c.ks[sc];
    if (logit && lane == 0) logit[t] = s;
    const float mn = s > m ? s : m;
    const float ref = mn == -INFINITY ? 0.0f : mn;  // no finite score yet: no weight either
    const float keep = m == -INFINITY ? 0.0f : expf(m - ref), p = expf(s - ref);
    m = mn;
    l = l * keep + p;
    const float pv = S8 ? p * c.vs[sc] : p;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int d = lane + 32 * e;
      if (d < c.dim)
        acc[e] = fmaf(pv, S8 ? (float)static_cast<const int8_t*>(c.v)[row + d]
                             : (float)static_cast<const __nv_bfloat16*>(c.v)[row + d], acc[e] * keep);
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = acc[e];
  __syncthreads();
  float top = -INFINITY, sum = 0.0f, o = 0.0f;
  for (int w = 0; w < 8; ++w) top = fmaxf(top, sm[w]);
  const float ref = top == -INFINITY ? 0.0f : top;
  for (int w = 0; w < 8; ++w) {
    const float f = sm[w] == -INFINITY ? (sl[w] == sl[w] ? 0.0f : sl[w]) : expf(sm[w] - ref);
    sum += sl[w] * f;
    o += so[w][threadIdx.x] * f;
  }
  if ((int)threadIdx.x < c.dim) {
    T* out = static_cast<T*>(a.out.p) + b * a.out.token + h * a.out.head + threadIdx.x;
    const float y = len > first ? o / sum : 0.0f;
    if constexpr (std::is_same<T, float>::value) *out = y;
    else *out = __float2bfloat16_rn(y);
  }
  if (threadIdx.x == 0) {
    const float z = len > first ? ref + logf(sum) : -INFINITY;
    if (a.lse) a.lse[blockIdx.x] = z;
    if (a.stats) a.stats[blockIdx.x] = z;
  }
}

// score of each token += its weights, summed over the query heads that share
// its key/value head
__global__ void __launch_bounds__(256) score_kernel(Args a) {
  const Cache& c = a.c;
  const int b = blockIdx.x / c.heads, kvh = blockIdx.x % c.heads, group = a.q_heads / c.heads;
  const int len = kv::cut_length(c, a.tab, a.lengths[b], a.status);
  const int first = a.window && len > a.window ? len - a.window : 0;
  const int64_t most = (int64_t)a.tab.max_pages * c.page_size;
  for (int t = first + threadIdx.x; t < len; t += 256) {
    int page, off;
    if (!kv::find(c, a.tab, b, t, page, off, a.status)) continue;
    float p = 0.0f;
    for (int g = 0; g < group; ++g) {
      const int64_t r = (int64_t)b * a.q_heads + kvh * group + g;
      p += expf(a.logits[r * most + t] - a.stats[r]);
    }
    c.score[kv::scale_at(c, page, kvh, off)] += p;
  }
}

size_t workspace_bytes(const Cache& c, const Table& tab, int64_t q_heads, int accumulate) {
  if (!accumulate) return 256;
  const int64_t rows = (int64_t)tab.sequences * q_heads;
  return (size_t)round_up(rows * 4, 256) + (size_t)rows * tab.max_pages * c.page_size * 4;
}

}  // namespace
}  // namespace i8q

using namespace i8q;

extern "C" size_t i8q_paged_attention_workspace_size(const i8q_kv_cache* cache, const i8q_page_table* table,
                                                     int64_t q_heads, int accumulate) {
  Cache c;
  Table tab;
  if (kv::check_cache(cache, "paged_attention_workspace_size", c) != I8Q_OK ||
      kv::check_table(table, c, "paged_attention_workspace_size", tab) != I8Q_OK)
    return 0;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads || tab.sequences * q_heads > INT32_MAX) {
    fail(I8Q_ERR_INVALID_ARG, "paged_attention_workspace_size: q_heads must be a multiple of kv_heads, in range");
    return 0;
  }
  return workspace_bytes(c, tab, q_heads, accumulate);
}

extern "C" int i8q_paged_attention(const i8q_kv_cache* cache, const i8q_page_table* table, const int32_t* lengths,
                                   int type, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                   int64_t q_heads, void* out, int64_t out_token_stride, int64_t out_head_stride,
                                   float* lse, float softmax_scale, int64_t window, int accumulate, void* workspace,
                                   size_t ws_bytes, void* stream) {
  Args a{};
  int rc = kv::check_cache(cache, "paged_attention", a.c);
  if (rc == I8Q_OK) rc = kv::check_table(table, a.c, "paged_attention", a.tab);
  if (rc != I8Q_OK) return rc;
  if (type != I8Q_F32 && type != I8Q_BF16)
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: type must be I8Q_F32 or I8Q_BF16");
  if (!lengths || !q || !out) return fail(I8Q_ERR_INVALID_ARG, "paged_attention: lengths, q or out is NULL");
  if (q_heads < 1 || q_heads > 65535 || q_heads % a.c.heads)
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: q_heads must be a multiple of kv_heads");
  if (a.tab.sequences * q_heads > INT32_MAX)
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: sequences * q_heads out of range");
  if (window < 0) return fail(I8Q_ERR_INVALID_ARG, "paged_attention: window must not be negative");
  if (!(softmax_scale == softmax_scale)) return fail(I8Q_ERR_INVALID_ARG, "paged_attention: softmax_scale is NaN");
  if (accumulate && !a.c.score)
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: accumulate needs a cache that keeps scores");
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      ws_bytes < workspace_bytes(a.c, a.tab, q_heads, accumulate))
    return fail(I8Q_ERR_INVALID_ARG, "paged_attention: workspace is NULL, unaligned or too small");
  a.lengths = lengths;
  a.q = Heads{const_cast<void*>(q), q_token_stride, q_head_stride};
  a.out = Heads{out, out_token_stride, out_head_stride};
  a.lse = lse;
  a.scale = softmax_scale;
  a.q_heads = (int)q_heads;
  a.window = (int)std::min<int64_t>(window, INT32_MAX);
  a.accumulate = accumulate != 0;
  if (accumulate) {
    a.stats = static_cast<float*>(workspace);
    a.logits = a.stats + round_up((int64_t)a.tab.sequences * q_heads * 4, 256) / 4;
  }
  a.status = device_status_word();
  if (!a.status) return fail(I8Q_ERR_CUDA, "paged_attention: no status word");
  cudaStream_t s = as_stream(stream);
  const unsigned blocks = (unsigned)(a.tab.sequences * q_heads);
  {
    I8Q_PROF("paged_attention", s);
    if (type == I8Q_F32) {
      if (cache->type == I8Q_S8) attend_kernel<float, true><<<blocks, 256, 0, s>>>(a);
      else attend_kernel<float, false><<<blocks, 256, 0, s>>>(a);
    } else {
      if (cache->type == I8Q_S8) attend_kernel<__nv_bfloat16, true><<<blocks, 256, 0, s>>>(a);
      else attend_kernel<__nv_bfloat16, false><<<blocks, 256, 0, s>>>(a);
    }
    I8Q_LAUNCH_CHECK("paged_attention");
  }
  if (accumulate) {
    I8Q_PROF("paged_attention_scores", s);
    score_kernel<<<(unsigned)a.tab.sequences * (unsigned)a.c.heads, 256, 0, s>>>(a);
    I8Q_LAUNCH_CHECK("paged_attention_scores");
  }
  return I8Q_OK;
}
