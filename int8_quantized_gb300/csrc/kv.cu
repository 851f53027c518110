// kv.cu -- writing a paged key/value cache (rotary positions, int8 rows) and
// reading it back, and the argument checks of all cache entry points.
#include <string>

#include "kv.cuh"

namespace i8q {
namespace kv {

int check_cache(const i8q_kv_cache* c, const char* who, Cache& out) {
  const std::string w = who;
  if (!c) return fail(I8Q_ERR_INVALID_ARG, w + ": cache is NULL");
  if (c->type != I8Q_S8 && c->type != I8Q_BF16)
    return fail(I8Q_ERR_INVALID_ARG, w + ": cache type must be I8Q_S8 or I8Q_BF16");
  if (!c->k || !c->v) return fail(I8Q_ERR_INVALID_ARG, w + ": cache pools are NULL");
  if (c->type == I8Q_S8 && (!c->k_scale || !c->v_scale))
    return fail(I8Q_ERR_INVALID_ARG, w + ": an int8 cache needs k_scale and v_scale");
  if (c->type == I8Q_BF16 && (c->k_scale || c->v_scale))
    return fail(I8Q_ERR_INVALID_ARG, w + ": a bf16 cache has no scales");
  if (c->pages < 1 || c->pages > INT32_MAX || c->kv_heads < 1 || c->kv_heads > 65535 || c->page_size < 1 ||
      c->page_size > (1 << 24))
    return fail(I8Q_ERR_INVALID_ARG, w + ": pages, kv_heads or page_size out of range");
  if (c->head_dim < 1) return fail(I8Q_ERR_INVALID_ARG, w + ": head_dim must be positive");
  if (c->head_dim % 16 != 0 || c->head_dim > I8Q_KV_MAX_HEAD_DIM)
    return fail(I8Q_ERR_UNSUPPORTED, w + ": head_dim must be a multiple of 16, at most 256");
  const int64_t unit = c->type == I8Q_S8 ? 16 : 8;  // elements in 16 bytes
  const int64_t ext[3] = {c->pages, c->kv_heads, c->page_size};
  const int64_t st[3] = {c->page_stride, c->head_stride, c->token_stride};
  const int64_t ss[3] = {c->scale_page_stride, c->scale_head_stride, c->scale_token_stride};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] > 1 && st[i] < c->head_dim)
      return fail(I8Q_ERR_INVALID_ARG, w + ": cache rows overlap (a stride is below head_dim)");
    if (st[i] % unit != 0) return fail(I8Q_ERR_INVALID_ARG, w + ": cache strides must be multiples of 16 bytes");
    if ((c->k_scale || c->score) && ext[i] > 1 && ss[i] < 1)
      return fail(I8Q_ERR_INVALID_ARG, w + ": scale strides must be positive");
  }
  if (reinterpret_cast<uintptr_t>(c->k) % 16 || reinterpret_cast<uintptr_t>(c->v) % 16)
    return fail(I8Q_ERR_INVALID_ARG, w + ": cache pools must be 16-byte aligned");
  out = Cache{c->k,
              c->v,
              c->k_scale,
              c->v_scale,
              c->score,
              c->page_stride,
              c->head_stride,
              c->token_stride,
              c->scale_page_stride,
              c->scale_head_stride,
              c->scale_token_stride,
              (int)c->pages,
              (int)c->kv_heads,
              (int)c->page_size,
              (int)c->head_dim};
  return I8Q_OK;
}

int check_table(const i8q_page_table* t, const Cache& c, const char* who, Table& out) {
  const std::string w = who;
  if (!t || !t->table) return fail(I8Q_ERR_INVALID_ARG, w + ": page table is NULL");
  if (t->sequences < 1 || t->sequences > 65536 || t->max_pages < 1)
    return fail(I8Q_ERR_INVALID_ARG, w + ": page table has no rows or columns, or too many");
  if (t->max_pages > INT32_MAX / c.page_size)
    return fail(I8Q_ERR_INVALID_ARG, w + ": max_pages * page_size must be below 2^31");
  if (t->sequences > 1 && t->stride < t->max_pages)
    return fail(I8Q_ERR_INVALID_ARG, w + ": page table rows overlap");
  out = Table{t->table, t->stride, (int)t->sequences, (int)t->max_pages};
  return I8Q_OK;
}

}  // namespace kv

namespace {

using kv::Cache;
using kv::Table;

struct Rows {  // [tokens][heads][dim], strides in elements
  void* p;
  int64_t token, head;
  int heads;
};

struct Rotary {
  const int32_t* positions;
  int64_t position_stride;
  const float* cos;
  const float* sin;
  int rows, pairs, axes, interleaved;
  uint32_t axis[I8Q_KV_MAX_HEAD_DIM / 2 / 16];  // two bits a pair
};

template <class T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (std::is_same<T, float>::value) return *p;
  else return __bfloat162float(*p);
}
template <class T>
__device__ __forceinline__ void store1(T* p, float v) {
  if constexpr (std::is_same<T, float>::value) *p = v;
  else *p = __float2bfloat16_rn(v);
}

// One warp per row of q, k or v: lane l turns pairs l, l + 32, ...
template <class T, bool S8>
__global__ void __launch_bounds__(256)
append_kernel(Cache c, Table tab, const int32_t* __restrict__ seq, const int32_t* __restrict__ index, int64_t tokens,
              Rows q, Rows qo, Rows k, Rows v, Rotary r, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int per = q.heads + 2 * c.heads;
  const int half = c.dim / 2;
  for (int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; w < tokens * per; w += (int64_t)gridDim.x * 8) {
    const int64_t t = w / per;
    const int row = (int)(w - t * per);
    const int b = seq[t];
    if (b < 0) continue;
    const int i = index[t];
    int page, off;
    if (b >= tab.sequences || i < 0 || i >= tab.max_pages * c.page_size) {
      kv::report_index(status);
      continue;
    }
    if (!kv::find(c, tab, b, i, page, off, status)) continue;
    bool turn_ok = true;
    for (int a = 0; a < r.axes; ++a) turn_ok &= (unsigned)r.positions[a * r.position_stride + t] < (unsigned)r.rows;
    if (!turn_ok) {
      kv::report_index(status);
      continue;
    }
    const int which = row < q.heads ? 0 : (row < q.heads + c.heads ? 1 : 2);
    const int head = which == 0 ? row : (row - q.heads) % c.heads;
    const Rows& in = which == 0 ? q : (which == 1 ? k : v);
    const T* src = static_cast<const T*>(in.p) + t * in.token + head * in.head;
    const int turned = which == 2 ? 0 : r.pairs;
    float y[I8Q_KV_MAX_HEAD_DIM / 32];
    int at[I8Q_KV_MAX_HEAD_DIM / 32];
    uint32_t most = 0;
#pragma unroll
    for (int u = 0; u < I8Q_KV_MAX_HEAD_DIM / 64; ++u) {
      const int j = lane + 32 * u;
      if (j < half) {
        const bool rot = j < turned;
        const bool split = rot && !r.interleaved;
        const int e1 = split ? j : 2 * j, e2 = split ? j + r.pairs : 2 * j + 1;
        float x1 = load1(src + e1), x2 = load1(src + e2);
        if (rot) {
          const int a = (r.axis[j >> 4] >> ((j & 15) * 2)) & 3;
          const int64_t g = (int64_t)r.positions[a * r.position_stride + t] * r.pairs + j;
          const float cs = r.cos[g], sn = r.sin[g];
          const float y1 = __fsub_rn(__fmul_rn(x1, cs), __fmul_rn(x2, sn));
          x2 = __fadd_rn(__fmul_rn(x2, cs), __fmul_rn(x1, sn));
          x1 = y1;
        }
        y[2 * u] = x1, y[2 * u + 1] = x2;
        at[2 * u] = e1, at[2 * u + 1] = e2;
        most = max(most, max(__float_as_uint(fabsf(x1)), __float_as_uint(fabsf(x2))));
      }
    }
    const int64_t dst = kv::row_at(c, page, head, off);
    if (which == 0) {
      T* o = static_cast<T*>(qo.p) + t * qo.token + head * qo.head;
      __syncwarp();  // qo may be q: every lane has read its pairs
#pragma unroll
      for (int u = 0; u < I8Q_KV_MAX_HEAD_DIM / 32; ++u)
        if (lane + 32 * (u / 2) < half) store1(o + at[u], y[u]);
    } else if (!S8) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(which == 1 ? c.k : c.v) + dst;
#pragma unroll
      for (int u = 0; u < I8Q_KV_MAX_HEAD_DIM / 32; ++u)
        if (lane + 32 * (u / 2) < half) store1(o + at[u], y[u]);
    } else {
      // largest magnitude as its bit pattern: a NaN is above infinity
      most = __reduce_max_sync(0xffffffffu, most);
      float s = __fdiv_rn(__uint_as_float(most), 127.0f);
      if (s == 0.0f) s = 1.0f;
      int8_t* o = static_cast<int8_t*>(which == 1 ? c.k : c.v) + dst;
#pragma unroll
      for (int u = 0; u < I8Q_KV_MAX_HEAD_DIM / 32; ++u)
        if (lane + 32 * (u / 2) < half) o[at[u]] = (int8_t)sat_rint(__fdiv_rn(y[u], s), -128.0f, 127.0f);
      if (lane == 0) (which == 1 ? c.ks : c.vs)[kv::scale_at(c, page, head, off)] = s;
    }
    if (which == 1 && c.score && lane == 0) c.score[kv::scale_at(c, page, head, off)] = 0.0f;
  }
}

template <class T, bool S8>
__global__ void __launch_bounds__(256)
gather_kernel(Cache c, Table tab, const int32_t* __restrict__ seq, const int32_t* __restrict__ index, int64_t tokens,
              Rows k, Rows v, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int per = 2 * c.heads;
  for (int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; w < tokens * per; w += (int64_t)gridDim.x * 8) {
    const int64_t t = w / per;
    const int row = (int)(w - t * per);
    const int b = seq[t];
    if (b < 0) continue;
    const int i = index[t];
    int page, off;
    if (b >= tab.sequences || i < 0 || i >= tab.max_pages * c.page_size) {
      kv::report_index(status);
      continue;
    }
    if (!kv::find(c, tab, b, i, page, off, status)) continue;
    const bool is_k = row < c.heads;
    const int head = is_k ? row : row - c.heads;
    const int64_t src = kv::row_at(c, page, head, off);
    T* o = is_k ? static_cast<T*>(k.p) + t * k.token + head * k.head : static_cast<T*>(v.p) + t * v.token + head * v.head;
    float s = 1.0f;
    if (S8) s = (is_k ? c.ks : c.vs)[kv::scale_at(c, page, head, off)];
    for (int e = lane; e < c.dim; e += 32) {
      float x;
      if (S8) x = __fmul_rn((float)static_cast<const int8_t*>(is_k ? c.k : c.v)[src + e], s);
      else x = __bfloat162float(static_cast<const __nv_bfloat16*>(is_k ? c.k : c.v)[src + e]);
      store1(o + e, x);
    }
  }
}

int check_tokens(const char* who, const int32_t* seq, const int32_t* index, int64_t tokens, int type) {
  const std::string w = who;
  if (tokens < 0 || tokens > INT32_MAX) return fail(I8Q_ERR_INVALID_ARG, w + ": tokens out of range");
  if (type != I8Q_F32 && type != I8Q_BF16) return fail(I8Q_ERR_INVALID_ARG, w + ": type must be I8Q_F32 or I8Q_BF16");
  if (tokens && (!seq || !index)) return fail(I8Q_ERR_INVALID_ARG, w + ": seq or index is NULL");
  return I8Q_OK;
}

template <class F>
int with_types(int type, int cache_type, F f) {
  if (type == I8Q_F32) return cache_type == I8Q_S8 ? f(float(), std::true_type()) : f(float(), std::false_type());
  return cache_type == I8Q_S8 ? f(__nv_bfloat16(), std::true_type()) : f(__nv_bfloat16(), std::false_type());
}

}  // namespace
}  // namespace i8q

using namespace i8q;

extern "C" int i8q_kv_append(const i8q_kv_cache* cache, const i8q_page_table* table, const int32_t* seq,
                             const int32_t* index, int64_t tokens, int type, const void* k, int64_t k_token_stride,
                             int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                             const void* q, int64_t q_token_stride, int64_t q_head_stride, int64_t q_heads,
                             void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                             const i8q_rotary* rotary, void* stream) {
  Cache c;
  Table tab;
  int rc = kv::check_cache(cache, "kv_append", c);
  if (rc == I8Q_OK) rc = kv::check_table(table, c, "kv_append", tab);
  if (rc == I8Q_OK) rc = check_tokens("kv_append", seq, index, tokens, type);
  if (rc != I8Q_OK) return rc;
  if (q_heads < 0 || q_heads > 65535) return fail(I8Q_ERR_INVALID_ARG, "kv_append: q_heads out of range");
  if (tokens && (!k || !v)) return fail(I8Q_ERR_INVALID_ARG, "kv_append: k or v is NULL");
  if (tokens && q_heads && (!q || !q_out)) return fail(I8Q_ERR_INVALID_ARG, "kv_append: q or q_out is NULL");
  Rotary r{};
  if (rotary) {
    if (rotary->pairs < 1 || 2 * rotary->pairs > c.dim)
      return fail(I8Q_ERR_INVALID_ARG, "kv_append: rotary pairs must be 1 .. head_dim / 2");
    if (rotary->axes < 1 || rotary->axes > I8Q_ROTARY_MAX_AXES)
      return fail(I8Q_ERR_INVALID_ARG, "kv_append: rotary axes must be 1 .. 4");
    if (!rotary->positions || !rotary->cos || !rotary->sin)
      return fail(I8Q_ERR_INVALID_ARG, "kv_append: rotary positions, cos or sin is NULL");
    if (rotary->rows < 1 || rotary->rows > INT32_MAX)
      return fail(I8Q_ERR_INVALID_ARG, "kv_append: rotary rows out of range");
    if (rotary->axes > 1 && rotary->position_stride < tokens)
      return fail(I8Q_ERR_INVALID_ARG, "kv_append: rotary positions' rows overlap");
    for (int64_t j = 0; j < rotary->pairs; ++j) {
      const int a = rotary->pair_axis ? rotary->pair_axis[j] : 0;
      if (a >= rotary->axes) return fail(I8Q_ERR_INVALID_ARG, "kv_append: pair_axis names an axis that is not given");
      r.axis[j >> 4] |= (uint32_t)a << ((j & 15) * 2);
    }
    r.positions = rotary->positions, r.position_stride = rotary->position_stride;
    r.cos = rotary->cos, r.sin = rotary->sin;
    r.rows = (int)rotary->rows, r.pairs = (int)rotary->pairs, r.axes = (int)rotary->axes;
    r.interleaved = rotary->interleaved != 0;
  }
  if (tokens == 0) return I8Q_OK;
  uint32_t* status = device_status_word();
  if (!status) return fail(I8Q_ERR_CUDA, "kv_append: no status word");
  const Rows rq{const_cast<void*>(q), q_token_stride, q_head_stride, (int)q_heads};
  const Rows ro{q_out, q_out_token_stride, q_out_head_stride, (int)q_heads};
  const Rows rk{const_cast<void*>(k), k_token_stride, k_head_stride, c.heads};
  const Rows rv{const_cast<void*>(v), v_token_stride, v_head_stride, c.heads};
  cudaStream_t s = as_stream(stream);
  return with_types(type, cache->type, [&](auto t, auto s8) -> int {
    using T = decltype(t);
    const int64_t blocks = std::min<int64_t>(ceil_div(tokens * (q_heads + 2 * c.heads), 8), (int64_t)sm_count() * 64);
    I8Q_PROF("kv_append", s);
    append_kernel<T, decltype(s8)::value>
        <<<(unsigned)blocks, 256, 0, s>>>(c, tab, seq, index, tokens, rq, ro, rk, rv, r, status);
    I8Q_LAUNCH_CHECK("kv_append");
    return I8Q_OK;
  });
}

extern "C" int i8q_kv_gather(const i8q_kv_cache* cache, const i8q_page_table* table, const int32_t* seq,
                             const int32_t* index, int64_t tokens, int type, void* k_out, int64_t k_token_stride,
                             int64_t k_head_stride, void* v_out, int64_t v_token_stride, int64_t v_head_stride,
                             void* stream) {
  Cache c;
  Table tab;
  int rc = kv::check_cache(cache, "kv_gather", c);
  if (rc == I8Q_OK) rc = kv::check_table(table, c, "kv_gather", tab);
  if (rc == I8Q_OK) rc = check_tokens("kv_gather", seq, index, tokens, type);
  if (rc != I8Q_OK) return rc;
  if (tokens == 0) return I8Q_OK;
  if (!k_out || !v_out) return fail(I8Q_ERR_INVALID_ARG, "kv_gather: k_out or v_out is NULL");
  uint32_t* status = device_status_word();
  if (!status) return fail(I8Q_ERR_CUDA, "kv_gather: no status word");
  const Rows rk{k_out, k_token_stride, k_head_stride, c.heads};
  const Rows rv{v_out, v_token_stride, v_head_stride, c.heads};
  cudaStream_t s = as_stream(stream);
  return with_types(type, cache->type, [&](auto t, auto s8) -> int {
    using T = decltype(t);
    const int64_t blocks = std::min<int64_t>(ceil_div(tokens * 2 * c.heads, 8), (int64_t)sm_count() * 64);
    I8Q_PROF("kv_gather", s);
    gather_kernel<T, decltype(s8)::value><<<(unsigned)blocks, 256, 0, s>>>(c, tab, seq, index, tokens, rk, rv, status);
    I8Q_LAUNCH_CHECK("kv_gather");
    return I8Q_OK;
  });
}
