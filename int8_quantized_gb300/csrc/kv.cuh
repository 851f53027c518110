// kv.cuh -- the paged key/value cache as the kernels see it, and the host
// checks that its entry points share.
#pragma once

#include "common.cuh"

namespace i8q {
namespace kv {

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

// Host side: the arguments checked, and the device forms of the structs.
int check_cache(const i8q_kv_cache* c, const char* who, Cache& out);
int check_table(const i8q_page_table* t, const Cache& c, const char* who, Table& out);

}  // namespace kv
}  // namespace i8q
