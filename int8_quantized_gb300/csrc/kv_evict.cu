// kv_evict.cu -- eviction from a paged key/value cache by accumulated
// attention weight: which tokens of a sequence and head stay, then their
// copies into fewer pages.
#include <cooperative_groups.h>

#include "kv.cuh"

namespace i8q {
namespace {

namespace cg = cooperative_groups;

using kv::Cache;
using kv::Table;

struct Args {
  Cache c;
  Table tab, to;
  const int32_t* lengths;
  int32_t* kept;
  int32_t* new_lengths;
  int budget, sink, recent;
  int room;    // keys of a CTA's share that its shared memory holds
  int blocks;  // of a row in the second kernel
  int fours;   // four neighbouring tokens' scores can be read at once
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
  if (!kv::find(a.c, a.tab, b, t, page, off, a.status)) return order_key(-INFINITY);
  return order_key(a.c.score[kv::scale_at(a.c, page, h, off)]);
}

constexpr int kBins = 2048, kMostCtas = 8;  // CTAs of a cluster

// Inclusive sum of v over the block; total: of all.
template <int THREADS>
__device__ __forceinline__ int block_scan(int v, int* total, int* warp_sums) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, i);
    if (lane >= i) v += u;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int x = lane < kWarps ? warp_sums[lane] : 0;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += u;
  }
  *total = __shfl_sync(0xffffffffu, x, 31);
  const int before = __shfl_sync(0xffffffffu, x, warp ? warp - 1 : 0);
  return v + (warp ? before : 0);
}

// The keys of tokens t0 .. t0 + n - 1, V neighbours of a page at a time; those
// of tokens lo .. hi - 1 are counted by their first digit on the way.
constexpr int kFirstShift = 21;
template <int V, int THREADS>
__device__ __forceinline__ void hold(const Args& a, const int32_t* pages, const float* scores, int t0, int n,
                                     uint32_t* keys, int* count, int lo, int hi) {
  constexpr int N = 8;
  for (int i0 = threadIdx.x * V; i0 < n; i0 += N * V * THREADS) {
    int page[N], off[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + j * V * THREADS;
      if (i >= n) break;
      const int p = (int)((unsigned)(t0 + i) / (unsigned)a.c.page_size);
      page[j] = pages[p];
      off[j] = t0 + i - p * a.c.page_size;
    }
    float x[N][V];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (i0 + j * V * THREADS >= n) break;
      const float* at = scores + page[j] * a.c.s_page + off[j] * a.c.s_token;
      if ((unsigned)page[j] >= (unsigned)a.c.pages) {
        kv::report_index(a.status);
#pragma unroll
        for (int v = 0; v < V; ++v) x[j][v] = -INFINITY;
      } else if constexpr (V == 4) {
        *reinterpret_cast<float4*>(x[j]) = *reinterpret_cast<const float4*>(at);
      } else {
        x[j][0] = *at;
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + j * V * THREADS;
      if (i >= n) break;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t key = order_key(x[j][v]);
        keys[i + v] = key;
        if (i + v >= lo && i + v < hi) atomicAdd(&count[key >> kFirstShift], 1);
      }
    }
  }
}

// A cluster per sequence and head, each CTA an equal share of its tokens, so
// that a long sequence is read by several SMs and its keys are read once,
// into shared memory.  The key of the last kept candidate is found by digits
// of 11, 11 and 10 bits: each CTA counts its keys by digit, all add up the
// cluster's counts and pick the digit in which the wanted rank falls.  The
// kept indices then follow from counts of the tokens before, in order.  A
// pass whose digit is taken whole is the last: two passes mostly do.
// 512 threads of 64 registers, two CTAs to an SM (256 rows of 8192 tokens: 14
// us, of which 4 until the keys are there; 1024 threads took a quarter longer);
// 128 threads where the rows are short and more than that.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_kernel(const __grid_constant__ Args a) {
  constexpr int kThreads = THREADS, kWarps = kThreads / 32, kDigits = kBins / kThreads;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int count[kBins], total_count[kBins];
  __shared__ int warp_sums[kWarps], warp_more[kWarps], warp_equal[kWarps], s_digit, s_need, s_whole, s_more, s_equal;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / C, b = row / a.c.heads, h = row % a.c.heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  kv::next_kernel_may_start();
  for (int i = threadIdx.x; i < kBins; i += kThreads) count[i] = 0;
  __syncthreads();
  kv::wait_previous_kernel();
  const int len = kv::cut_length(a.c, a.tab, a.lengths[b], a.status);
  const int n = min(len, a.budget);
  int32_t* kept = a.kept + (int64_t)row * a.budget;
  const int all = C * kThreads, me = rank * kThreads + threadIdx.x;
  for (int j = n + me; j < a.budget; j += all) kept[j] = -1;
  if (h == 0 && me == 0 && a.new_lengths) a.new_lengths[b] = n;
  if (n == len) {  // (all CTAs of the cluster leave here)
    for (int j = me; j < n; j += all) kept[j] = j;
    return;
  }
  const int share = ((len + C - 1) / C + 3) / 4 * 4, t0 = min(rank * share, len), mine = min(share, len - t0);  // shares begin on multiples of 4
  const bool held = share <= a.room;
  // candidates: neither the first `sink` nor the last `recent`
  const int lo = a.sink - t0, hi = len - a.recent - t0, c0 = max(lo, 0), c1 = min(hi, mine);
  if (held) {
    // four neighbouring scores of a page at once where they lie so, and eight
    // places looked up before the first of them is read
    const int32_t* pages = a.tab.page + (int64_t)b * a.tab.stride;
    const float* scores = a.c.score + h * a.c.s_head;
    if (a.fours) hold<4, THREADS>(a, pages, scores, t0, mine, keys, count, c0, c1);
    else hold<1, THREADS>(a, pages, scores, t0, mine, keys, count, c0, c1);
  }
  int need = a.budget - a.sink - a.recent;
  const bool none = need == 0;
  if (none) __syncthreads();  // (else after the counts)
  uint32_t prefix = 0, mask = 0;
  bool whole = false;  // all keys that begin with prefix stay
  for (int shift = kFirstShift; !none && !whole && shift >= 0; shift -= shift == kFirstShift ? 11 : 10) {
    // digits at bits 21 to 31, 10 to 20 and 0 to 9
    const uint32_t digits = shift ? 0x7ffu : 0x3ffu;
    if (shift != kFirstShift) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) count[i] = 0;
      __syncthreads();
    }
    auto add = [&](uint32_t key) {
      if ((key & mask) == prefix) atomicAdd(&count[key >> shift & digits], 1);
    };
    if (!held) {
      for (int i = c0 + threadIdx.x; i < c1; i += kThreads) add(key_of(a, b, h, t0 + i));
    } else if (shift != kFirstShift) {  // four keys at a time between the ends
      const int q0 = (c0 + 3) / 4 * 4, q1 = max(q0, c1 / 4 * 4);
      for (int i = q0 + threadIdx.x * 4; i < q1; i += kThreads * 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
        add(k.x), add(k.y), add(k.z), add(k.w);
      }
      if (c0 + (int)threadIdx.x < min(q0, c1)) add(keys[c0 + threadIdx.x]);
      if (q1 + (int)threadIdx.x < c1) add(keys[q1 + threadIdx.x]);
    }
    // each CTA adds up a share of the digits and hands the sums to all
    const int* sums = count;
    if (C > 1) {
      cluster.sync();
      const int part = kBins / C;
      for (int i = rank * part + threadIdx.x; i < (rank + 1) * part; i += kThreads) {
        int y[kMostCtas], x = 0;
#pragma unroll
        for (int r = 0; r < kMostCtas; ++r) y[r] = r < C ? cluster.map_shared_rank(count, r)[i] : 0;
#pragma unroll
        for (int r = 0; r < kMostCtas; ++r) x += y[r];
#pragma unroll
        for (int r = 0; r < kMostCtas; ++r)
          if (r < C) cluster.map_shared_rank(total_count, r)[i] = x;
      }
      cluster.sync();
      sums = total_count;
    } else {
      __syncthreads();
    }
    // kDigits digits a thread, from the highest down
    const int d = kBins - kDigits * (threadIdx.x + 1);
    int sum[kDigits], mine_count = 0, total;
#pragma unroll
    for (int i = 0; i < kDigits; i += 4) *reinterpret_cast<int4*>(sum + i) = *reinterpret_cast<const int4*>(sums + d + i);
#pragma unroll
    for (int i = 0; i < kDigits; ++i) mine_count += sum[i];
    const int through = block_scan<THREADS>(mine_count, &total, warp_sums);
    int before = through - mine_count;
    if (before < need && need <= through) {
      bool found = false;
#pragma unroll
      for (int i = kDigits - 1; i >= 0; --i) {
        if (!found && need <= before + sum[i]) {
          found = true;
          s_digit = d + i;
          s_need = need - before;
          s_whole = need - before == sum[i];
        }
        before += sum[i];
      }
    }
    __syncthreads();
    prefix |= (uint32_t)s_digit << shift;
    mask |= digits << shift;
    need = s_need;
    whole = s_whole;
    // (a CTA that clears its counts has passed the second cluster.sync, after which none reads them; the
    // sums are written anew after the next pass's first)
    __syncthreads();
  }
  // Candidates above the key stay, and the first `need` that equal it (or all
  // from the prefix on).  Each warp has a run of the share.
  const int run = (mine + kWarps * 128 - 1) / (kWarps * 128) * 128, i0 = warp * run, i1 = min(i0 + run, mine);
  // no key has the value of all ones
  const uint32_t from = none ? ~0u : whole ? prefix : prefix + 1, same = none || whole ? ~0u : prefix;
  // of four neighbours: bit j of more: kept; of equal: kept by rank
  auto classes = [&](int i, uint32_t& more, uint32_t& equal) {
    more = equal = 0;
    if (i >= i1) return;
    uint32_t key[4] = {};
    if (held) {  // (the last four may reach past the share, within the room)
      const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
      key[0] = k.x, key[1] = k.y, key[2] = k.z, key[3] = k.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < i1) key[j] = key_of(a, b, h, t0 + i + j);
    }
    if (i >= lo && i + 4 <= min(hi, i1)) {  // candidates all
#pragma unroll
      for (int j = 0; j < 4; ++j) more |= (uint32_t)(key[j] >= from) << j, equal |= (uint32_t)(key[j] == same) << j;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j >= i1) break;
        const bool sure = i + j < lo || i + j >= hi;
        more |= (uint32_t)(sure || key[j] >= from) << j;
        equal |= (uint32_t)(!sure && key[j] == same) << j;
      }
    }
  };
  int mores = 0, equals = 0;
  for (int i = i0; i < i1; i += 128) {
    uint32_t more, equal;
    classes(i + 4 * lane, more, equal);
    if (held && i + 4 * lane < i1) keys[i + 4 * lane] = more | equal << 4;  // in place of the keys
    mores += __popc(more), equals += __popc(equal);
  }
  mores = __reduce_add_sync(0xffffffffu, mores), equals = __reduce_add_sync(0xffffffffu, equals);
  if (lane == 0) warp_more[warp] = mores, warp_equal[warp] = equals;
  __syncthreads();
  // of the share, then of the warps and CTAs before this one
  const int lane_more = lane < kWarps ? warp_more[lane] : 0, lane_equal = lane < kWarps ? warp_equal[lane] : 0;
  if (warp == 0) {
    const int m = __reduce_add_sync(0xffffffffu, lane_more), e = __reduce_add_sync(0xffffffffu, lane_equal);
    if (lane == 0) s_more = m, s_equal = e;
  }
  if (C > 1) cluster.sync();
  int more_before = lane < warp ? lane_more : 0, equal_before = lane < warp ? lane_equal : 0;
  if (lane < rank) more_before += *cluster.map_shared_rank(&s_more, lane), equal_before += *cluster.map_shared_rank(&s_equal, lane);
  more_before = __reduce_add_sync(0xffffffffu, more_before), equal_before = __reduce_add_sync(0xffffffffu, equal_before);
  const uint32_t lanes_before = (1u << lane) - 1;
  int at = more_before + min(equal_before, need);  // what a warp keeps is one run of `kept`
  for (int i = i0; i < i1; i += 128) {
    uint32_t more, equal;
    if (held) {
      const uint32_t both = i + 4 * lane < i1 ? keys[i + 4 * lane] : 0;
      more = both & 15, equal = both >> 4;
    } else {
      classes(i + 4 * lane, more, equal);
    }
    const int t = t0 + i + 4 * lane;
    if (__any_sync(0xffffffffu, equal)) {  // the first `need` of them stay
      int e = equal_before;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t of_all = __ballot_sync(0xffffffffu, equal >> j & 1);
        e += __popc(of_all & lanes_before), equal_before += __popc(of_all);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (equal >> j & 1) more |= (uint32_t)(e++ < need) << j;
    }
    const int own = __popc(more);  // 0 to 4: three votes add them up
    int m = at;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const uint32_t of_all = __ballot_sync(0xffffffffu, own >> j & 1);
      m += __popc(of_all & lanes_before) << j, at += __popc(of_all) << j;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (more >> j & 1) kept[m++] = t + j;
  }
  if (C > 1) cluster.sync();  // no CTA leaves while another reads its counts
}

// A CTA copies kRows kept tokens of a row (sequence and head): first a
// thread per token finds both places and moves its scales and score, then
// groups of lanes move the rows, 16 bytes a lane, four in flight.  Bound by
// its bytes, in scattered rows: 262144 rows of 128 bf16, 268 MB, in 51 us (5.2
// TB/s); with eight in flight a third longer.  The heads of the same tokens
// are neighbours in the grid, since they are in a page (1 us less).  Stores
// that give way in L2 took 3 us less here, and 4 more in the next read.
constexpr int kRows = 64;
template <int BYTES>
__global__ void __launch_bounds__(256) move_kernel(const __grid_constant__ Args a) {
  __shared__ int64_t from[kRows], to[kRows];  // bytes; from -1: nothing to move
  const Cache& c = a.c;
  const int cell = blockIdx.x / c.heads, h = blockIdx.x - cell * c.heads, b = cell / a.blocks;
  const int row = b * c.heads + h, j0 = (cell - b * a.blocks) * kRows;
  kv::next_kernel_may_start();
  kv::wait_previous_kernel();
  const int32_t* kept = a.kept + (int64_t)row * a.budget;
  if (kept[j0] < 0) return;  // past the last kept token
  if (threadIdx.x < kRows) {
    const int j = j0 + threadIdx.x;
    const int t = j < a.budget ? kept[j] : -1;
    int64_t src = -1, dst = 0;
    int p0, o0, p1, o1;
    if (t >= 0) {
      const bool room = j < a.to.max_pages * c.page_size;
      if (!room) kv::report_index(a.status);
      const bool ok0 = kv::find(c, a.tab, b, t, p0, o0, a.status);
      const bool ok1 = room && kv::find(c, a.to, b, j, p1, o1, a.status);
      if (ok0 && ok1) {
        src = kv::row_at(c, p0, h, o0) * BYTES, dst = kv::row_at(c, p1, h, o1) * BYTES;
        const int64_t s0 = kv::scale_at(c, p0, h, o0), s1 = kv::scale_at(c, p1, h, o1);
        const float score = c.score[s0];
        if (BYTES == 1) {
          const float ks = c.ks[s0], vs = c.vs[s0];
          c.ks[s1] = ks, c.vs[s1] = vs;
        }
        c.score[s1] = score;
      }
    }
    from[threadIdx.x] = src, to[threadIdx.x] = dst;
  }
  __syncthreads();
  const int pieces = c.dim * BYTES / 16;  // of a row, a lane each
  const int groups = 256 / pieces, group = threadIdx.x / pieces, e = threadIdx.x % pieces * 16;
  if (group >= groups) return;
  for (int r0 = group; r0 < 2 * kRows; r0 += 4 * groups) {
    uint4 x[4];
    char* dst[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i * groups;
      const int64_t src = r < 2 * kRows ? from[r % kRows] : -1;
      char* const pool = static_cast<char*>(r < kRows ? c.k : c.v);
      dst[i] = src < 0 ? nullptr : pool + to[r % kRows] + e;
      if (src >= 0) x[i] = __ldcs(reinterpret_cast<const uint4*>(pool + src + e));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = x[i];
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
  const int64_t heads = (int64_t)a.tab.sequences * a.c.heads;
  if (budget < 1 || budget > kv::kMostTokens)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: budget must be 1 .. 2^31 - 2^16");
  if (heads > INT32_MAX / 16 || heads * ceil_div(budget, kRows) > INT32_MAX)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: sequences * kv_heads * budget out of range");
  if (sink < 0 || recent < 0 || sink > budget || recent > budget - sink)
    return fail(I8Q_ERR_INVALID_ARG, "kv_evict: sink + recent must be within 0 .. budget");
  a.lengths = lengths, a.kept = kept, a.new_lengths = new_lengths;
  a.budget = (int)budget, a.sink = (int)sink, a.recent = (int)recent;
  a.status = device_status_word();
  if (!a.status) return fail(I8Q_ERR_CUDA, "kv_evict: no status word");
  cudaStream_t s = as_stream(stream);
  // Long rows have as many CTAs, up to the portable 8, as fit the SMs twice
  // over (8 rows of 131072 tokens took three times as long in clusters of 16):
  // a CTA takes 0.6 us per 1000 tokens, a cluster 4 us of its own.  So rows up
  // to 12288 tokens have one CTA, and many rows too, while two CTAs' keys fit
  // an SM (24K each): 256 rows of 18000 tokens 31 us, in clusters of two 42.  A
  // share whose keys shared memory cannot hold is read again in each pass.
  const int64_t most = (int64_t)a.tab.max_pages * a.c.page_size;
  int cluster = 1;
  while (most > 12288 && cluster < kMostCtas &&
         (heads * cluster * 2 <= sm_count() || ceil_div(most, cluster) > 24 * 1024))
    cluster *= 2;
  a.room = (int)std::min<int64_t>(round_up(ceil_div(most, cluster), 4), 48 * 1024);
  a.fours = a.c.page_size % 4 == 0 && a.c.s_token == 1 && a.c.s_page % 4 == 0 && a.c.s_head % 4 == 0 &&
            reinterpret_cast<uintptr_t>(a.c.score) % 16 == 0;
  {
    I8Q_PROF("kv_evict_select", s);
    rc = most <= 1024 && heads > 2 * sm_count() ? kv::launch(select_kernel<128>, (unsigned)(heads * cluster), 128, a.room * 4, cluster, s,
                                   "kv_evict_select", a)
                      : kv::launch(select_kernel<512>, (unsigned)(heads * cluster), 512, a.room * 4, cluster, s,
                                   "kv_evict_select", a);
    if (rc != I8Q_OK) return rc;
  }
  I8Q_PROF("kv_evict_move", s);
  a.blocks = (int)ceil_div(budget, kRows);
  const unsigned blocks = (unsigned)(heads * a.blocks);
  return cache->type == I8Q_S8 ? kv::launch(move_kernel<1>, blocks, 256, 0, 1, s, "kv_evict_move", a)
                               : kv::launch(move_kernel<2>, blocks, 256, 0, 1, s, "kv_evict_move", a);
}
