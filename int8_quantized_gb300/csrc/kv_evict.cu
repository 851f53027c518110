// kv_evict.cu -- eviction from a paged key/value cache by accumulated
// attention weight.
#include "kv.cuh"

namespace i8q {
namespace {

using kv::Cache;
using kv::Table;

struct Args {
  Cache c;
  Table tab, to;
  const int32_t* lengths;
  int32_t* kept;
  int32_t* new_lengths;
  int budget, sink, recent;
  uint32_t* status;
};

// A score as an unsigned number of the same order: NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ uint32_t key_of(const Args& a, int b, int h, int t) {
  int page, off;
  if (!kv::find(a.c, a.tab, b, t, page, off, a.status)) return 0;
  return order_key(a.c.score[kv::scale_at(a.c, page, h, off)]);
}

constexpr int kThreads = 1024;

// Inclusive sum over the block of v, and its total.
__device__ int block_scan(int v, int* total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int i = 1; i < 32; i <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, i);
    if (lane >= i) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    before += w < warp ? warp_sums[w] : 0;
    all += warp_sums[w];
  }
  *total = all;
  return v + before;
}

// One CTA per sequence and head: the key of the last kept candidate, found
// one 8-bit digit at a time from counts, then the kept indices in order.
__global__ void __launch_bounds__(kThreads) select_kernel(Args a) {
  __shared__ int count[256], warp_sums[kThreads / 32], s_digit, s_need;
  const int b = blockIdx.x / a.c.heads, h = blockIdx.x % a.c.heads;
  const int len = kv::cut_length(a.c, a.tab, a.lengths[b], a.status);
  const int n = min(len, a.budget);
  int32_t* kept = a.kept + (int64_t)blockIdx.x * a.budget;
  for (int j = n + threadIdx.x; j < a.budget; j += kThreads) kept[j] = -1;
  if (h == 0 && threadIdx.x == 0 && a.new_lengths) a.new_lengths[b] = n;
  if (n == len) {
    for (int j = threadIdx.x; j < n; j += kThreads) kept[j] = j;
    return;
  }
  const int lo = a.sink, hi = len - a.recent;
  int need = a.budget - a.sink - a.recent;  // of the hi - lo candidates, which are more
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; need && shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) count[threadIdx.x] = 0;
    __syncthreads();
    for (int t = lo + threadIdx.x; t < hi; t += kThreads) {
      const uint32_t key = key_of(a, b, h, t);
      if ((key & mask) == prefix) atomicAdd(&count[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int d = 255, left = need;
      while (d > 0 && count[d] < left) left -= count[d--];
      s_digit = d, s_need = left;
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    mask |= 255u << shift;
    need = s_need;
    __syncthreads();
  }
  // candidates above the key are kept, and the first `need` that equal it
  int at = 0, equal = 0;
  const bool none = a.budget == a.sink + a.recent;
  for (int t0 = 0; t0 < len; t0 += kThreads) {
    const int t = t0 + threadIdx.x;
    bool keep = t < len && (t < lo || t >= hi), eq = false;
    if (!none && t >= lo && t < hi) {
      const uint32_t key = key_of(a, b, h, t);
      keep = key > prefix;
      eq = key == prefix;
    }
    int total;
    const int rank = block_scan(eq, &total, warp_sums) + equal;
    if (eq && rank <= need) keep = true;
    equal += total;
    const int pos = block_scan(keep, &total, warp_sums) + at;
    if (keep) kept[pos - 1] = t;
    at += total;
  }
}

// One warp per kept token and head.
template <int BYTES>
__global__ void __launch_bounds__(256) move_kernel(Args a, int64_t rows) {
  const Cache& c = a.c;
  const int lane = threadIdx.x & 31;
  for (int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; w < rows; w += (int64_t)gridDim.x * 8) {
    const int64_t bh = w / a.budget;
    const int j = (int)(w - bh * a.budget);
    const int b = (int)(bh / c.heads), h = (int)(bh % c.heads);
    const int t = a.kept[w];
    if (t < 0) continue;
    int p0, o0, p1, o1;
    if (!kv::find(c, a.tab, b, t, p0, o0, a.status) || !kv::find(c, a.to, b, j, p1, o1, a.status)) continue;
    const int64_t src = kv::row_at(c, p0, h, o0) * BYTES, dst = kv::row_at(c, p1, h, o1) * BYTES;
    for (int e = lane * 16; e < c.dim * BYTES; e += 512) {
      *reinterpret_cast<uint4*>(static_cast<char*>(c.k) + dst + e) =
          *reinterpret_cast<const uint4*>(static_cast<const char*>(c.k) + src + e);
      *reinterpret_cast<uint4*>(static_cast<char*>(c.v) + dst + e) =
          *reinterpret_cast<const uint4*>(static_cast<const char*>(c.v) + src + e);
    }
    const int64_t s0 = kv::scale_at(c, p0, h, o0), s1 = kv::scale_at(c, p1, h, o1);
    if (lane == 0) c.score[s1] = c.score[s0];
    if (lane == 1 && c.ks) c.ks[s1] = c.ks[s0];
    if (lane == 2 && c.ks) c.vs[s1] = c.vs[s0];
  }
}

}  // namespace
}  // namespace i8q

using namespace i8q;

extern "C" int i8q_kv_evict(const i8q_kv_cache* cache, const i8q_page_table* table, const int32_t* lengths,
                            const i8q_page_table* new_table, int32_t* kept, int64_t budget, int64_t sink,
                            int64_t recent, int32_t* new_lengths, void* stream) {
  Args a{};
  int rc = kv::check_cache(cache, "kv_evict", a.c);
  if (rc == I8Q_OK) rc = kv::check_table(table, a.c, "kv_evict", a.tab);
  if (rc == I8Q_OK) rc = kv::check_table(new_table, a.c, "kv_evict", a.to);
  if (rc != I8Q_OK) return rc;
  if (!a.c.score) return fail(I8Q_ERR_INVALID_ARG, "kv_evict: the cache keeps no scores");
  if (!lengths || !kept) return fail(I8Q_ERR_INVALID_ARG, "kv_evict: lengths or kept is NULL");
  if (a.to.sequences != a.tab.sequences)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: table and new_table differ in sequences");
  if ((int64_t)a.tab.sequences * a.c.heads > INT32_MAX)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: sequences * kv_heads out of range");
  if (budget < 1 || budget > (int64_t)a.to.max_pages * a.c.page_size)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: budget must be 1 .. new_table's max_pages * page_size");
  if (sink < 0 || recent < 0 || sink > budget || recent > budget - sink)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: sink + recent must be within 0 .. budget");
  a.lengths = lengths, a.kept = kept, a.new_lengths = new_lengths;
  a.budget = (int)budget, a.sink = (int)sink, a.recent = (int)recent;
  a.status = device_status_word();
  if (!a.status) return fail(I8Q_ERR_CUDA, "kv_evict: no status word");
  cudaStream_t s = as_stream(stream);
  const int64_t heads = (int64_t)a.tab.sequences * a.c.heads;
  {
    I8Q_PROF("kv_evict_select", s);
    select_kernel<<<(unsigned)heads, kThreads, 0, s>>>(a);
    I8Q_LAUNCH_CHECK("kv_evict_select");
  }
  I8Q_PROF("kv_evict_move", s);
  const int64_t rows = heads * budget;
  const unsigned blocks = (unsigned)std::min<int64_t>(ceil_div(rows, 8), (int64_t)sm_count() * 64);
  if (cache->type == I8Q_S8) move_kernel<1><<<blocks, 256, 0, s>>>(a, rows);
  else move_kernel<2><<<blocks, 256, 0, s>>>(a, rows);
  I8Q_LAUNCH_CHECK("kv_evict_move");
  return I8Q_OK;
}
