// bcq_kv4.cu -- the key/value cache in 4 bits: rows into the cache, rows out
// of it, and attention over it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "bcq.h"
#include "bcq_device.cuh"
#include "bcq_launch.h"

namespace bcq {
namespace {

__device__ int g_kv4_error = 0;

constexpr int kKvGroup = BCQ_KV4_GROUP;
constexpr float kKvRange = 60000.f;  // beyond it a group becomes NaN: a c + z stays below fp16's 65504

// ------------------------------------------------------------------ types

template <typename T>
__device__ __forceinline__ float bits_to_float(uint32_t b);
template <>
__device__ __forceinline__ float bits_to_float<__half>(uint32_t b) { return h2f((uint16_t)b); }
template <>
__device__ __forceinline__ float bits_to_float<__nv_bfloat16>(uint32_t b) {
  return __uint_as_float(b << 16);
}

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// What a call knows of the cache's places.
struct Places {
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;
  int table_width, B, pages, page_size, heads;
};

// The sequence that row t belongs to: the last b with cu[b] <= t, or -1 when
// t is outside cu[0]..cu[B]-1.  Without cu, row t is sequence t's.
__device__ __forceinline__ int sequence_of(const Places& p, int t) {
  if (!p.cu) return t < p.B ? t : -1;
  if (t < p.cu[0] || t >= p.cu[p.B]) return -1;
  int lo = 0, hi = p.B;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// First row and number of rows of sequence b.
__device__ __forceinline__ int2 rows_of(const Places& p, int b) {
  return p.cu ? make_int2(p.cu[b], p.cu[b + 1] - p.cu[b]) : make_int2(b, 1);
}

// The slot (page * page_size + offset) of position j of sequence b, or -1.
__device__ __forceinline__ int64_t slot_of(const Places& p, int b, int j) {
  if (j < 0 || j / p.page_size >= p.table_width) return -1;
  const int page = p.table[(int64_t)b * p.table_width + j / p.page_size];
  if (page < 0 || page >= p.pages) return -1;
  return (int64_t)page * p.page_size + j % p.page_size;
}

// The vector (token slot, head) as an index into [pages][heads][page_size].
__device__ __forceinline__ int64_t vector_of(const Places& p, int64_t slot, int h) {
  return (slot / p.page_size * p.heads + h) * p.page_size + slot % p.page_size;
}

// ------------------------------------------------------------------ append

struct AppendParams {
  Places at;
  const uint16_t* x[2];  // K, V
  int64_t ld[2], hd[2];
  uint8_t* code[2];
  __half2* param[2];
  int T, D;
};

// Eight lanes a group of 64: eight values a lane, one 32-bit word of codes.
// The codes' quotient is taken in fp32 with a rounded reciprocal; where it
// lies within 1e-4 of a half (its error is below 16 * 4 * 2^-24 < 4e-6, and
// the difference's rounding adds less) the half decides in fp64, where x - z
// and (c + 1/2) a are exact.
template <typename T>
__global__ void __launch_bounds__(256) kv4_append_kernel(AppendParams p) {
  const int G = p.D / kKvGroup;
  const int64_t units = (int64_t)p.T * p.at.heads * G * 2;
  const int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 3;
  const int sub = threadIdx.x & 7;
  if (u >= units) return;  // whole groups of eight lanes leave
  const uint32_t mask = 0xFFu << (threadIdx.x & 24);
  const int g = (int)(u % G);
  const int h = (int)(u / G % p.at.heads);
  const int kv = (int)(u / G / p.at.heads % 2);
  const int t = (int)(u / G / p.at.heads / 2);
  const int b = sequence_of(p.at, t);
  if (b < 0) return;
  const int2 rows = rows_of(p.at, b);
  const int j = p.at.kv_len[b] - rows.y + (t - rows.x);
  const int64_t slot = slot_of(p.at, b, j);
  if (slot < 0) {
    if (sub == 0) record_error(&g_kv4_error, BCQ_ERR_PAGE);
    return;
  }
  const uint4 raw = *reinterpret_cast<const uint4*>(p.x[kv] + (int64_t)t * p.ld[kv] +
                                                    (int64_t)h * p.hd[kv] + g * kKvGroup + sub * 8);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float f[8];
  float lo = INFINITY, hi = -INFINITY;
  bool ok = true;
  for (int i = 0; i < 8; ++i) {
    f[i] = bits_to_float<T>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    ok = ok && fabsf(f[i]) <= kKvRange;  // false for a NaN
    lo = fminf(lo, f[i]);
    hi = fmaxf(hi, f[i]);
  }
  for (int o = 1; o < 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
  }
  ok = __all_sync(mask, ok);
  const __half a16 = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f));
  const __half z16 = __float2half_rn(lo);
  const float a = __half2float(a16), z = __half2float(z16);
  uint32_t word = 0;
  if (ok && a > 0.f) {
    const float inv = __fdiv_rn(1.f, a);
    for (int i = 0; i < 8; ++i) {
      const float v = (f[i] - z) * inv;
      float r = rintf(v);
      if (fabsf(v - r) > 0.4999f) {
        const float c = floorf(v);  // the half in question is c + 1/2
        const double d = (double)f[i] - (double)z, edge = ((double)c + 0.5) * (double)a;
        r = d > edge ? c + 1.f : d < edge ? c : 2.f * rintf(0.5f * c + 0.25f);
      }
      word |= (uint32_t)fminf(fmaxf(r, 0.f), 15.f) << (4 * i);
    }
  }
  const int64_t vec = vector_of(p.at, slot, h);
  *reinterpret_cast<uint32_t*>(p.code[kv] + vec * (p.D / 2) + g * (kKvGroup / 2) + sub * 4) = word;
  if (sub == 0) {
    const __half nan = __ushort_as_half(0x7E00);
    p.param[kv][vec * G + g] = ok ? __halves2half2(a16, z16) : __halves2half2(nan, nan);
  }
}

// -------------------------------------------------------------------- read

struct ReadParams {
  Places at;
  const uint8_t* code[2];
  const __half2* param[2];
  void* y[2];
  int T, D;
};

// Eight values (one word of codes) a thread.
template <typename TO>
__global__ void __launch_bounds__(256) kv4_read_kernel(ReadParams p) {
  const int W = p.D / 8;
  const int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= (int64_t)p.T * p.at.heads * W * 2) return;
  const int i = (int)(u % W);
  const int h = (int)(u / W % p.at.heads);
  const int kv = (int)(u / W / p.at.heads % 2);
  const int t = (int)(u / W / p.at.heads / 2);
  const int b = sequence_of(p.at, t);
  if (b < 0) return;
  const int2 rows = rows_of(p.at, b);
  const int64_t slot = slot_of(p.at, b, p.at.kv_len[b] - rows.y + (t - rows.x));
  float f[8] = {};
  if (slot >= 0) {
    const int64_t vec = vector_of(p.at, slot, h);
    const uint32_t word = *reinterpret_cast<const uint32_t*>(p.code[kv] + vec * (p.D / 2) + 4 * i);
    const float2 az = __half22float2(p.param[kv][vec * (p.D / kKvGroup) + i / 8]);
    for (int e = 0; e < 8; ++e) f[e] = fmaf((float)((word >> (4 * e)) & 15u), az.x, az.y);
  } else if (i == 0) {
    record_error(&g_kv4_error, BCQ_ERR_PAGE);
  }
  TO out[8];
  for (int e = 0; e < 8; ++e) out[e] = from_float<TO>(f[e]);
  TO* y = static_cast<TO*>(p.y[kv]) + ((int64_t)t * p.at.heads + h) * p.D + 8 * i;
  const uint4* src = reinterpret_cast<const uint4*>(out);
  for (int e = 0; e < (int)(8 * sizeof(TO) / 16); ++e) reinterpret_cast<uint4*>(y)[e] = src[e];
}

// --------------------------------------------------------------- attention

struct AttentionParams {
  Places at;
  const uint8_t* k;
  const __half2* k_param;
  const uint8_t* v;
  const __half2* v_param;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int64_t ld_q, hd_q, ld_o, hd_o;
  int T, q_heads, D, max_q, causal, window;
  float scale;
};

// One block a (row, query head), 128 positions at a time: a thread a
// position's score, then a thread two values of the output.
template <typename T>
__global__ void __launch_bounds__(128) kv4_attention_kernel(AttentionParams p) {
  __shared__ float qs[256], ps[128], red[4];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, D = p.D;
  const int b = sequence_of(p.at, t);
  if (b < 0) return;
  const int2 rows = rows_of(p.at, b);
  if (t - rows.x >= p.max_q) {
    if (tid == 0) record_error(&g_kv4_error, BCQ_ERR_SHAPE);
    return;
  }
  int len = p.at.kv_len[b];
  if (len < 0 || len > (int64_t)p.at.table_width * p.at.page_size) {
    if (tid == 0) record_error(&g_kv4_error, BCQ_ERR_PAGE);
    len = len < 0 ? 0 : p.at.table_width * p.at.page_size;
  }
  const int pos = p.at.kv_len[b] - rows.y + (t - rows.x);
  const int hi = p.causal ? min(len, pos + 1) : len;
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const int kvh = h / (p.q_heads / p.at.heads);
  for (int d = tid; d < D; d += 128)
    qs[d] = bits_to_float<T>(p.q[(int64_t)t * p.ld_q + (int64_t)h * p.hd_q + d]) * p.scale;
  float top = -INFINITY, sum = 0.f, acc[2] = {0.f, 0.f};
  for (int j0 = lo; j0 < hi; j0 += 128) {
    __syncthreads();
    const int j = j0 + tid;
    const int64_t slot = j < hi ? slot_of(p.at, b, j) : -1;
    if (j < hi && slot < 0) record_error(&g_kv4_error, BCQ_ERR_PAGE);
    float s = -INFINITY;
    if (slot >= 0) {
      const int64_t vec = vector_of(p.at, slot, kvh);
      s = 0.f;
      for (int d = 0; d < D; ++d) {
        const float2 az = __half22float2(p.k_param[vec * (D / kKvGroup) + d / kKvGroup]);
        const uint32_t c = p.k[vec * (D / 2) + d / 2] >> (4 * (d & 1)) & 15u;
        s = fmaf(qs[d], fmaf((float)c, az.x, az.y), s);
      }
    }
    float m = s;
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(top, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = m == -INFINITY ? 0.f : m;
    const float fix = expf(top - base);
    ps[tid] = expf(s - base);
    __syncthreads();
    sum *= fix;
    acc[0] *= fix;
    acc[1] *= fix;
    for (int i = 0; i < 128 && j0 + i < hi; ++i) {
      const float w = ps[i];
      sum += w;
      const int64_t sl = slot_of(p.at, b, j0 + i);
      if (sl < 0) continue;
      const int64_t vec = vector_of(p.at, sl, kvh);
      for (int e = 0; e < 2; ++e) {
        const int d = tid + 128 * e;
        if (d >= D) continue;
        const float2 az = __half22float2(p.v_param[vec * (D / kKvGroup) + d / kKvGroup]);
        const uint32_t c = p.v[vec * (D / 2) + d / 2] >> (4 * (d & 1)) & 15u;
        acc[e] = fmaf(w, fmaf((float)c, az.x, az.y), acc[e]);
      }
    }
    top = m;
  }
  for (int e = 0; e < 2; ++e) {
    const int d = tid + 128 * e;
    if (d < D) {
      const T r = from_float<T>(sum > 0.f || sum != sum ? acc[e] / sum : 0.f);
      p.out[(int64_t)t * p.ld_o + (int64_t)h * p.hd_o + d] = *reinterpret_cast<const uint16_t*>(&r);
    }
  }
  if (p.lse && tid == 0) p.lse[(int64_t)t * p.q_heads + h] = sum > 0.f || sum != sum ? top + logf(sum) : -INFINITY;
}

// -------------------------------------------------------------------- host

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is16(int dtype) { return dtype == BCQ_F16 || dtype == BCQ_BF16; }

bool cache_sizes_ok(const bcq_kv4* c) {
  return c->pages >= 1 && c->heads >= 1 && c->page_size >= 16 && c->page_size % 16 == 0;
}

bool head_dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

bcq_status check_cache(const bcq_kv4* c, int T, const int32_t* table, int table_width,
                       const int32_t* kv_len, const int32_t* cu, int B) {
  if (!c || !c->k || !c->k_param || !c->v || !c->v_param || !table || !kv_len)
    return BCQ_ERR_NULL;
  if (!cache_sizes_ok(c) || T < 0 || B < 1 || table_width < 1 ||
      (int64_t)table_width * c->page_size > INT32_MAX || (!cu && T != B))
    return BCQ_ERR_SHAPE;
  if (!head_dim_ok(c->head_dim)) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->k_param, 16) || !aligned(c->v, 16) ||
      !aligned(c->v_param, 16) || !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(cu, 4))
    return BCQ_ERR_ALIGN;
  return BCQ_OK;
}

// Rows [T][heads][D] of a 16-bit type, strided.
bcq_status check_rows(const void* x, int64_t ld, int64_t hd, int dtype) {
  if (!x) return BCQ_ERR_NULL;
  if (!is16(dtype)) return BCQ_ERR_UNSUPPORTED;
  if (ld < 0 || hd < 0) return BCQ_ERR_SHAPE;
  return !aligned(x, 16) || ld % 8 || hd % 8 ? BCQ_ERR_ALIGN : BCQ_OK;
}

Places places_of(const bcq_kv4* c, const int32_t* table, int table_width, const int32_t* kv_len,
                 const int32_t* cu, int B) {
  return {table, kv_len, cu, table_width, B, c->pages, c->page_size, c->heads};
}

bcq_status launched() { return cudaGetLastError() == cudaSuccess ? BCQ_OK : BCQ_ERR_CUDA; }

}  // namespace

cudaError_t read_and_clear_kv4_error(int* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_kv4_error, sizeof(int));
  if (e == cudaSuccess && *code != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_kv4_error, &zero, sizeof(int));
  }
  return e;
}

}  // namespace bcq

using namespace bcq;

extern "C" {

bcq_status bcq_kv4_append(const bcq_kv4* cache, const void* k, int64_t ld_k, int64_t hd_k,
                          const void* v, int64_t ld_v, int64_t hd_v, int dtype, int T,
                          const int32_t* table, int table_width, const int32_t* kv_len,
                          const int32_t* cu, int B, void* stream) {
  bcq_status s = check_cache(cache, T, table, table_width, kv_len, cu, B);
  if (s != BCQ_OK || T == 0) return s;
  if ((s = check_rows(k, ld_k, hd_k, dtype)) != BCQ_OK) return s;
  if ((s = check_rows(v, ld_v, hd_v, dtype)) != BCQ_OK) return s;
  AppendParams p = {places_of(cache, table, table_width, kv_len, cu, B),
                    {static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v)},
                    {ld_k, ld_v},
                    {hd_k, hd_v},
                    {cache->k, cache->v},
                    {reinterpret_cast<__half2*>(cache->k_param), reinterpret_cast<__half2*>(cache->v_param)},
                    T,
                    cache->head_dim};
  const int64_t blocks = ((int64_t)T * cache->heads * (cache->head_dim / kKvGroup) * 2 + 31) / 32;
  if (blocks > INT32_MAX) return BCQ_ERR_SHAPE;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == BCQ_F16) kv4_append_kernel<__half><<<(unsigned)blocks, 256, 0, st>>>(p);
  else kv4_append_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, st>>>(p);
  return launched();
}

bcq_status bcq_kv4_read(const bcq_kv4* cache, void* k, void* v, int dtype, int T,
                        const int32_t* table, int table_width, const int32_t* kv_len,
                        const int32_t* cu, int B, void* stream) {
  const bcq_status s = check_cache(cache, T, table, table_width, kv_len, cu, B);
  if (s != BCQ_OK || T == 0) return s;
  if (!k || !v) return BCQ_ERR_NULL;
  if (!is16(dtype) && dtype != BCQ_F32) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16)) return BCQ_ERR_ALIGN;
  ReadParams p = {places_of(cache, table, table_width, kv_len, cu, B),
                  {cache->k, cache->v},
                  {reinterpret_cast<const __half2*>(cache->k_param),
                   reinterpret_cast<const __half2*>(cache->v_param)},
                  {k, v},
                  T,
                  cache->head_dim};
  const int64_t blocks = ((int64_t)T * cache->heads * (cache->head_dim / 8) * 2 + 255) / 256;
  if (blocks > INT32_MAX) return BCQ_ERR_SHAPE;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == BCQ_F16) kv4_read_kernel<__half><<<(unsigned)blocks, 256, 0, st>>>(p);
  else if (dtype == BCQ_BF16) kv4_read_kernel<__nv_bfloat16><<<(unsigned)blocks, 256, 0, st>>>(p);
  else kv4_read_kernel<float><<<(unsigned)blocks, 256, 0, st>>>(p);
  return launched();
}

size_t bcq_kv4_attention_workspace_bytes(const bcq_kv4* cache, int T, int q_heads, int B,
                                         int max_q, int max_kv) {
  if (!cache || !cache_sizes_ok(cache) || !head_dim_ok(cache->head_dim) || T < 0 || B < 1 ||
      max_q < 1 || max_kv < 1 || q_heads < 1)
    return 0;
  return 0;
}

bcq_status bcq_kv4_attention(const bcq_kv4* cache, const void* q, int64_t ld_q, int64_t hd_q,
                             int dtype, int T, int q_heads, const int32_t* table,
                             int table_width, const int32_t* kv_len, const int32_t* cu, int B,
                             int max_q, int max_kv, int causal, int window, float scale,
                             void* out, int64_t ld_o, int64_t hd_o, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  bcq_status s = check_cache(cache, T, table, table_width, kv_len, cu, B);
  if (s != BCQ_OK) return s;
  if (q_heads < 1 || q_heads % cache->heads || q_heads / cache->heads > 128 || max_q < 1 ||
      max_kv < 1 || window < 0 || !std::isfinite(scale))
    return BCQ_ERR_SHAPE;
  if (T == 0) return BCQ_OK;
  if ((s = check_rows(q, ld_q, hd_q, dtype)) != BCQ_OK) return s;
  if ((s = check_rows(out, ld_o, hd_o, dtype)) != BCQ_OK) return s;
  if (lse && !aligned(lse, 4)) return BCQ_ERR_ALIGN;
  const size_t need = bcq_kv4_attention_workspace_bytes(cache, T, q_heads, B, max_q, max_kv);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return BCQ_ERR_NULL;
    if (!aligned(workspace, 16)) return BCQ_ERR_ALIGN;
  }
  AttentionParams p = {places_of(cache, table, table_width, kv_len, cu, B),
                       cache->k,
                       reinterpret_cast<const __half2*>(cache->k_param),
                       cache->v,
                       reinterpret_cast<const __half2*>(cache->v_param),
                       static_cast<const uint16_t*>(q),
                       static_cast<uint16_t*>(out),
                       lse,
                       ld_q,
                       hd_q,
                       ld_o,
                       hd_o,
                       T,
                       q_heads,
                       cache->head_dim,
                       max_q,
                       causal,
                       window,
                       scale};
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)T, (unsigned)q_heads);
  if (dtype == BCQ_F16) kv4_attention_kernel<__half><<<grid, 128, 0, st>>>(p);
  else kv4_attention_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(p);
  return launched();
}

}  // extern "C"
