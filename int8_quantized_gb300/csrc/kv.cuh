// kv.cuh -- the paged key/value cache as the kernels see it, and the host
// checks that its entry points share.
#pragma once

#include <tuple>

#include "common.cuh"

namespace i8q {

// The device status word's bit for an index out of range in a key/value
// cache call's device data (the bits below belong to the bounded waits).
constexpr uint32_t ST_KV_INDEX = 1u << 31;
// ... and for a row's sampling parameters out of range.
constexpr uint32_t ST_SAMPLE = 1u << 30;

namespace kv {

// The most tokens that a row of a page table names, and that an eviction
// keeps: counters of 32 bits step past the end by up to 2^15 of them.
constexpr int64_t kMostTokens = (1LL << 31) - (1 << 16);

struct Cache {
  void* k;
  void* v;
  float* ks;  // scales (int8 pools)
  float* vs;
  float* score;
  int64_t page_stride, head_stride, token_stride;  // elements of k, v
  int64_t s_page, s_head, s_token;                 // elements of ks, vs, score
  int pages, heads, page_size, dim;
};

struct Table {
  const int32_t* page;
  int64_t stride;
  int sequences, max_pages;
};

__device__ __forceinline__ void report_index(uint32_t* status) { atomicOr(status, ST_KV_INDEX); }

// Page and offset of token t of sequence b; false (and reported) when the
// table names no page of the pools.
__device__ __forceinline__ bool find(const Cache& c, const Table& tab, int b, int t, int& page, int& off,
                                     uint32_t* status) {
  const int p = (int)((unsigned)t / (unsigned)c.page_size);
  off = t - p * c.page_size;
  page = tab.page[(int64_t)b * tab.stride + p];
  if ((unsigned)page < (unsigned)c.pages) return true;
  report_index(status);
  return false;
}

// A sequence's length, cut to what its row of the table can name.
__device__ __forceinline__ int cut_length(const Cache& c, const Table& tab, int len, uint32_t* status) {
  const int most = tab.max_pages * c.page_size;
  if (len >= 0 && len <= most) return len;
  report_index(status);
  return len < 0 ? 0 : most;
}

__device__ __forceinline__ int64_t row_at(const Cache& c, int page, int head, int off) {
  return page * c.page_stride + head * c.head_stride + off * c.token_stride;
}
__device__ __forceinline__ int64_t scale_at(const Cache& c, int page, int head, int off) {
  return page * c.s_page + head * c.s_head + off * c.s_token;
}

// A kernel launched by launch() may begin while the one before it ends: it
// waits for that one's results before it reads anything, and lets the next
// one begin.
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
__device__ __forceinline__ void wait_previous_kernel() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// Host side.
// Launch with the stream's order relaxed as above, in clusters of `cluster`
// CTAs.  All these kernels ask for the same division of the SM's memory, so
// that it is not changed between them.
int launch(const void* kernel, unsigned blocks, unsigned threads, int smem, int cluster, cudaStream_t s,
           const char* what, void** args);
template <class... P, class... V>
int launch(void (*kernel)(P...), unsigned blocks, unsigned threads, int smem, int cluster, cudaStream_t s,
           const char* what, const V&... v) {
  std::tuple<P...> p(v...);  // the parameters in the kernel's own types
  return std::apply([&](auto&... x) {
    void* args[] = {const_cast<void*>(static_cast<const void*>(&x))...};
    return launch(reinterpret_cast<const void*>(kernel), blocks, threads, smem, cluster, s, what, args);
  }, p);
}

// The arguments checked, and the device forms of the structs.
int check_cache(const i8q_kv_cache* c, const char* who, Cache& out);
int check_table(const i8q_page_table* t, const Cache& c, const char* who, Table& out);

}  // namespace kv
}  // namespace i8q
