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
    if (ext[i] == 1) continue;  // never multiplied
    if (st[i] < c->head_dim)
      return fail(I8Q_ERR_INVALID_ARG, w + ": cache rows overlap (a stride is below head_dim)");
    if (st[i] % unit != 0) return fail(I8Q_ERR_INVALID_ARG, w + ": cache strides must be multiples of 16 bytes");
    if ((c->k_scale || c->score) && ss[i] < 1)
      return fail(I8Q_ERR_INVALID_ARG, w + ": scale strides must be positive");
  }
  if (reinterpret_cast<uintptr_t>(c->k) % 16 || reinterpret_cast<uintptr_t>(c->v) % 16)
    return fail(I8Q_ERR_INVALID_ARG, w + ": cache pools must be 16-byte aligned");
  // (an axis of one place has the stride 0, and the kernels' rules on alignment need not look at it)
  const auto stride = [&](int i, const int64_t* s) { return ext[i] == 1 ? 0 : s[i]; };
  out = Cache{c->k,
              c->v,
              c->k_scale,
              c->v_scale,
              c->score,
              stride(0, st),
              stride(1, st),
              stride(2, st),
              stride(0, ss),
              stride(1, ss),
              stride(2, ss),
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
  if (t->max_pages > kMostTokens / c.page_size)
    return fail(I8Q_ERR_INVALID_ARG, w + ": max_pages * page_size must be at most 2^31 - 2^16");
  if (t->sequences > 1 && t->stride < t->max_pages)
    return fail(I8Q_ERR_INVALID_ARG, w + ": page table rows overlap");
  out = Table{t->table, t->stride, (int)t->sequences, (int)t->max_pages};
  return I8Q_OK;
}

int launch(const void* kernel, unsigned blocks, unsigned threads, int smem, int cluster, cudaStream_t s,
           const char* what, void** args) {
  struct Want {
    const void* kernel;
    int smem;
  } want{kernel, smem};
  const int rc = once_per_device(kernel, [](void* p) -> int {
    const Want* w = static_cast<const Want*>(p);
    I8Q_CUDA_TRY(cudaFuncSetAttribute(w->kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      cudaSharedmemCarveoutMaxShared));
    cudaFuncAttributes attr;
    I8Q_CUDA_TRY(cudaFuncGetAttributes(&attr, w->kernel));
    if (w->smem)
      I8Q_CUDA_TRY(cudaFuncSetAttribute(w->kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        227 * 1024 - (int)attr.sharedSizeBytes));
    return I8Q_OK;
  }, &want);
  if (rc != I8Q_OK) return rc;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = (size_t)smem, cfg.stream = s;
  cfg.attrs = attr, cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  return e == cudaSuccess ? I8Q_OK : cuda_fail(e, what);
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

// Rows of any alignment: one warp per row of q, k or v, lane l turns pairs
// l, l + 32, ...  (16384 tokens of 48 rows of 128: 484 us, where rows that can
// be read four elements at a time take 76 below.)
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

__device__ __forceinline__ void turn(float& x1, float& x2, float cs, float sn) {
  const float y1 = __fsub_rn(__fmul_rn(x1, cs), __fmul_rn(x2, sn));
  x2 = __fadd_rn(__fmul_rn(x2, cs), __fmul_rn(x1, sn));
  x1 = y1;
}

// The larger magnitude, or NaN where either is one.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// rint of the quotients y / s, |y| <= 127 s, as low bytes.  With r = fl(1 /
// s), the products y r (1 - 2^-20) and y r (1 + 2^-20) enclose the rounded
// quotient; one fma with 1.5 2^23 rounds each to an integer (its low bits).
// Where both round to the same integer so does the quotient; where they do
// not, or 1 / s is not a normal number, the eight quotients are formed.
__device__ __forceinline__ void quotient_codes(const float (&y)[8], float s, uint32_t (&code)[8]) {
  const float r = quot_rcp(s), hi = __fmul_rn(r, 1.0f + 0x1p-20f), lo = __fmul_rn(r, 1.0f - 0x1p-20f);
  const float2 magic = make_float2(12582912.0f, 12582912.0f);
  uint32_t differ = r != r;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float2 v = make_float2(y[j], y[j + 1]);
    const float2 h = fma2_rn(v, make_float2(hi, hi), magic), l = fma2_rn(v, make_float2(lo, lo), magic);
    code[j] = __float_as_uint(h.x), code[j + 1] = __float_as_uint(h.y);
    differ |= (code[j] ^ __float_as_uint(l.x)) | (code[j + 1] ^ __float_as_uint(l.y));
  }
  if (differ) {
#pragma unroll
    for (int j = 0; j < 8; ++j) code[j] = rint_code_bits(__fdiv_rn(y[j], s), -128.0f, 127.0f, 0);
  }
}

// Four neighbouring elements.
template <class T>
struct Four;
template <>
struct Four<float> {
  float4 v;
  __device__ float at(int i) const { return (&v.x)[i]; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 v;
  __device__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <class T>
__device__ __forceinline__ Four<T> load4(const T* p) {
  return Four<T>{__ldcs(reinterpret_cast<const decltype(Four<T>::v)*>(p))};
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The same on rows that can be read four elements at a time.  L lanes (8, 16
// or 32) hold a row, each the four pairs of its unit: elements 4u and pairs +
// 4u on, or 8u and 8u + 4 on.  A CTA has one token (or one of `splits` shares
// of its rows, for calls of few tokens); a lane keeps its unit, so its four
// cosines and sines serve all heads, and its first rows are sent for before
// the token's place and positions are known.  64 threads a token: what a
// thread does once is then a tenth of its work (16384 tokens of 48 rows of
// 128: 76 us, against 82 with 128 threads and 130 with 256).  The sums of two
// products are scalar: the compiler fuses a paired sum with its products.
constexpr int kUnitThreads = 64;
template <class T, bool S8, int L>
__global__ void __launch_bounds__(kUnitThreads)
append_units_kernel(Cache c, Table tab, const int32_t* __restrict__ seq, const int32_t* __restrict__ index, int splits,
                    Rows q, Rows qo, Rows k, Rows v, const __grid_constant__ Rotary r, uint32_t* status) {
  constexpr int G = kUnitThreads / L, NQ = 2;  // rows of q that a lane has in flight, beside one of k and one of v
  kv::next_kernel_may_start();
  kv::wait_previous_kernel();
  const int64_t t = splits == 1 ? blockIdx.x : blockIdx.x / splits;
  const int slot = threadIdx.x / L + (splits == 1 ? 0 : blockIdx.x % splits * G), u = threadIdx.x % L;
  const int step = G * splits;
  const bool in_row = u < c.dim / 8, turns = u < r.pairs / 4, split = turns && !r.interleaved;
  // a unit's two places in a row that is turned by halves, and in any other
  const int h1 = split ? 4 * u : 8 * u, h2 = split ? r.pairs + 4 * u : 8 * u + 4, e1 = 8 * u, e2 = 8 * u + 4;
  const T* q_row = static_cast<const T*>(q.p) + t * q.token;
  const T* k_row = static_cast<const T*>(k.p) + t * k.token;
  const T* v_row = static_cast<const T*>(v.p) + t * v.token;
  Four<T> xq[NQ][2], xk[2], xv[2];
  auto send_q = [&](int head) {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
      if (head + n * step < q.heads && in_row) {
        const T* src = q_row + (head + n * step) * q.head;
        xq[n][0] = load4(src + h1), xq[n][1] = load4(src + h2);
      }
  };
  auto send_kv = [&](int head) {
    if (head < c.heads && in_row) {
      const T *src = k_row + head * k.head, *from = v_row + head * v.head;
      xk[0] = load4(src + h1), xk[1] = load4(src + h2);
      xv[0] = load4(from + e1), xv[1] = load4(from + e2);
    }
  };
  send_kv(slot);
  send_q(slot);
  const int b = seq[t], i = index[t];
  const uint32_t axis = r.axis[u >> 2 & 7] >> ((u & 3) * 8) & 0xffu;  // two bits a pair
  int pos[4] = {0, 0, 0, 0};
  bool turn_ok = true;
  for (int a = 0; a < r.axes; ++a) {
    const int at = r.positions[a * r.position_stride + t];
    turn_ok &= (unsigned)at < (unsigned)r.rows;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((int)(axis >> 2 * j & 3) == a) pos[j] = at;
  }
  float cs[4] = {}, sn[4] = {};
  if (turns && turn_ok) {
    if (pos[0] == pos[1] && pos[0] == pos[2] && pos[0] == pos[3]) {
      const int64_t g = (int64_t)pos[0] * r.pairs + 4 * u;
      const float4 y = *reinterpret_cast<const float4*>(r.cos + g), z = *reinterpret_cast<const float4*>(r.sin + g);
      cs[0] = y.x, cs[1] = y.y, cs[2] = y.z, cs[3] = y.w;
      sn[0] = z.x, sn[1] = z.y, sn[2] = z.z, sn[3] = z.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t g = (int64_t)pos[j] * r.pairs + 4 * u + j;
        cs[j] = r.cos[g], sn[j] = r.sin[g];
      }
    }
  }
  if (b < 0) return;
  int page = 0, off = 0;
  bool ok = b < tab.sequences && i >= 0 && i < tab.max_pages * c.page_size && turn_ok;
  if (!ok && threadIdx.x == 0) kv::report_index(status);
  if (ok) ok = kv::find(c, tab, b, i, page, off, status);
  if (!ok) return;
  auto turned = [&](const Four<T> (&x)[2], float (&y)[8], bool really) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = x[0].at(j), y[4 + j] = x[1].at(j);
    if (!really) return;
    // pair j: elements j of the two halves, or two neighbours
    if (r.interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(y[2 * j], y[2 * j + 1], cs[j], sn[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn(y[j], y[4 + j], cs[j], sn[j]);
    }
  };
  T* const o_row = static_cast<T*>(qo.p) + t * qo.token;
  for (int head = slot; head < q.heads;) {
#pragma unroll
    for (int n = 0; n < NQ; ++n)
      if (head + n * step < q.heads && in_row) {
        float y[8];
        turned(xq[n], y, turns);
        T* o = o_row + (head + n * step) * qo.head;
        store4(o + h1, y), store4(o + h2, y + 4);
      }
    head += NQ * step;
    send_q(head);
  }
  const int64_t at = kv::row_at(c, page, 0, off), scale_at = kv::scale_at(c, page, 0, off);
  const uint32_t lanes = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1) << (threadIdx.x & 31 & ~(L - 1));
  auto put = [&](void* pool, float* scale, const float (&y)[8], int p1, int p2, int64_t dst, int64_t sc) {
    if constexpr (!S8) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(pool) + dst;
      if (in_row) store4(o + p1, y), store4(o + p2, y + 4);
    } else {
      float most = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) most = larger(most, y[e]);
#pragma unroll
      for (int m = 1; m < L; m <<= 1) most = larger(most, __shfl_xor_sync(lanes, most, m));
      float s = __fdiv_rn(most, 127.0f);
      if (s == 0.0f) s = 1.0f;
      if (in_row) {
        int8_t* o = static_cast<int8_t*>(pool) + dst;
        uint32_t code[8];
        quotient_codes(y, s, code);
        *reinterpret_cast<uint32_t*>(o + p1) = pack_low_bytes(code[0], code[1], code[2], code[3]);
        *reinterpret_cast<uint32_t*>(o + p2) = pack_low_bytes(code[4], code[5], code[6], code[7]);
      }
      if (u == 0) scale[sc] = s;
    }
  };
  for (int head = slot; head < c.heads;) {  // (the same for the L lanes of a row)
    const int64_t dst = at + head * c.head_stride, sc = scale_at + head * c.s_head;
    float y[8] = {};
    if (in_row) turned(xk, y, turns);
    put(c.k, c.ks, y, h1, h2, dst, sc);
    if (in_row) turned(xv, y, false);
    put(c.v, c.vs, y, e1, e2, dst, sc);
    if (c.score && u == 0) c.score[sc] = 0.0f;
    head += step;
    send_kv(head);
  }
}

// A CTA has kTokens tokens (or a share of their rows): a thread per token
// finds its place, then head_dim / 8 lanes hold a row, eight elements each,
// four rows in flight.  Bound by its bytes: 524288 rows of 128 to bf16, 407
// MB, in 66 us (6.2 TB/s); with every lane finding its own place 99 us.
constexpr int kTokens = 16;
template <class T, bool S8, int LANES>
__global__ void __launch_bounds__(256)
gather_kernel(Cache c, Table tab, const int32_t* __restrict__ seq, const int32_t* __restrict__ index, int64_t tokens,
              int splits, Rows k, Rows v, int aligned, uint32_t* status) {
  constexpr int N = 4;
  const int L = LANES ? LANES : c.dim / 8, G = 256 / L;  // (a constant for 64, 128 and 256: 32 registers, not 48)
  __shared__ int64_t at[kTokens], scale_at[kTokens];  // at -1: left out
  kv::next_kernel_may_start();
  kv::wait_previous_kernel();
  const int64_t t0 = blockIdx.x / splits * (int64_t)kTokens;
  if (threadIdx.x < kTokens) {
    int64_t src = -1;
    const int64_t t = t0 + threadIdx.x;
    if (t < tokens) {
      const int b = seq[t], i = index[t];
      int page = 0, off = 0;
      bool ok = b >= 0;
      if (ok) {
        ok = b < tab.sequences && i >= 0 && i < tab.max_pages * c.page_size;
        if (!ok) kv::report_index(status);
        if (ok) ok = kv::find(c, tab, b, i, page, off, status);
      }
      if (ok) src = kv::row_at(c, page, 0, off);
      scale_at[threadIdx.x] = kv::scale_at(c, page, 0, off);
    }
    at[threadIdx.x] = src;
  }
  __syncthreads();
  const int d = threadIdx.x % L * 8;
  if ((int)threadIdx.x >= L * G) return;
  // rows of the CTA: token by token within a head, so that neighbours of a page are read together
  const int rows = 2 * c.heads * kTokens, step = G * splits;
  for (int r0 = (blockIdx.x % splits) * G + threadIdx.x / L; r0 < rows; r0 += N * step) {
    uint4 w[N];
    float s[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = r0 + n * step, row = r / kTokens, t = r % kTokens;
      if (r < rows && at[t] >= 0) {
        const bool is_v = row >= c.heads;
        const int head = is_v ? row - c.heads : row;
        const int64_t src = at[t] + head * c.head_stride + d;
        if constexpr (S8) {
          const uint2 x = __ldcs(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(is_v ? c.v : c.k) + src));
          w[n].x = x.x, w[n].y = x.y;
          s[n] = (is_v ? c.vs : c.ks)[scale_at[t] + head * c.s_head];
        } else {
          w[n] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_v ? c.v : c.k) + src));
        }
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = r0 + n * step, row = r / kTokens, t = r % kTokens;
      if (r >= rows || at[t] < 0) continue;
      const uint32_t u[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (S8) y[j] = __fmul_rn((float)(int8_t)(u[j / 4] >> (8 * (j & 3))), s[n]);
        else y[j] = __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
      }
      const bool is_v = row >= c.heads;
      const int head = is_v ? row - c.heads : row;
      const Rows& to = is_v ? v : k;
      T* o = static_cast<T*>(to.p) + (t0 + t) * to.token + head * to.head + d;
      if (aligned) {
        if constexpr (std::is_same<T, float>::value) {
          __stcs(reinterpret_cast<float4*>(o), make_float4(y[0], y[1], y[2], y[3]));
          __stcs(reinterpret_cast<float4*>(o + 4), make_float4(y[4], y[5], y[6], y[7]));
        } else {
          uint32_t z[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            z[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          __stcs(reinterpret_cast<uint4*>(o), make_uint4(z[0], z[1], z[2], z[3]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) store1(o + j, y[j]);
      }
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

// Whether every row begins on a multiple of n elements.
bool rows_aligned(const Rows& r, int64_t es, int n) {
  return reinterpret_cast<uintptr_t>(r.p) % (size_t)(es * n) == 0 && r.token % n == 0 && r.head % n == 0;
}

// Lanes of a row at eight elements a lane, as a power of two.
int lanes_of(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

template <class F>
int with_lanes(int dim, F f) {
  const int l = lanes_of(dim);
  return l == 8 ? f(std::integral_constant<int, 8>()) : l == 16 ? f(std::integral_constant<int, 16>())
                                                                : f(std::integral_constant<int, 32>());
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
    I8Q_PROF("kv_append", s);
    const bool units = r.pairs % 4 == 0 && rows_aligned(rk, sizeof(T), 4) && rows_aligned(rv, sizeof(T), 4) &&
                       (!q_heads || (rows_aligned(rq, sizeof(T), 4) && rows_aligned(ro, sizeof(T), 4))) &&
                       reinterpret_cast<uintptr_t>(r.cos) % 16 == 0 && reinterpret_cast<uintptr_t>(r.sin) % 16 == 0;
    if (units)
      return with_lanes(c.dim, [&](auto lanes) -> int {
        constexpr int L = decltype(lanes)::value;
        // few tokens: their rows over as many CTAs as 16 for each SM (what fits), each with a row per L lanes
        // at least
        const int64_t most = ceil_div(std::max<int64_t>(q_heads, c.heads), kUnitThreads / L);
        const int splits = (int)std::max<int64_t>(1, std::min(most, 16 * sm_count() / tokens));
        return kv::launch(append_units_kernel<T, decltype(s8)::value, L>, (unsigned)(tokens * splits), kUnitThreads, 0, 1, s,
                          "kv_append", c, tab, seq, index, splits, rq, ro, rk, rv, r, status);
      });
    const int64_t blocks = std::min<int64_t>(ceil_div(tokens * (q_heads + 2 * c.heads), 8), (int64_t)sm_count() * 64);
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
    I8Q_PROF("kv_gather", s);
    const int aligned = rows_aligned(rk, sizeof(T), 16 / sizeof(T)) && rows_aligned(rv, sizeof(T), 16 / sizeof(T));
    const int64_t groups = ceil_div(tokens, kTokens), most = ceil_div(2 * c.heads * kTokens, 256 / (c.dim / 8));
    const int splits = (int)std::max<int64_t>(1, std::min(most, 2 * sm_count() / groups));
    constexpr bool S8 = decltype(s8)::value;
    auto run = [&](auto kernel) {
      return kv::launch(kernel, (unsigned)(groups * splits), 256, 0, 1, s, "kv_gather", c, tab, seq, index, tokens, splits,
                        rk, rv, aligned, status);
    };
    return c.dim == 64 ? run(gather_kernel<T, S8, 8>) : c.dim == 128 ? run(gather_kernel<T, S8, 16>)
           : c.dim == 256 ? run(gather_kernel<T, S8, 32>) : run(gather_kernel<T, S8, 0>);
  });
}
