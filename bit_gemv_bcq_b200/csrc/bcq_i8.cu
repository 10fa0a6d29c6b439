// bcq_i8.cu -- the 8-bit integer product: rows to codes, and
//   y[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k]   (the sum exact in int32).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "bcq.h"
#include "bcq_device.cuh"
#include "bcq_launch.h"

namespace bcq {
namespace {

__device__ int g_i8_error = 0;

// ------------------------------------------------------------------ types

template <typename T>
struct Bits16;  // 16-bit floating types by their bits
template <>
struct Bits16<__half> {
  static constexpr uint32_t kInf = 0x7C00u;
  static __device__ __forceinline__ float to_float(uint32_t b) { return h2f((uint16_t)b); }
};
template <>
struct Bits16<__nv_bfloat16> {
  static constexpr uint32_t kInf = 0x7F80u;
  static __device__ __forceinline__ float to_float(uint32_t b) { return __uint_as_float(b << 16); }
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// ----------------------------------------------------------- rows to codes

// One block a row.  |x| is compared by its bits, which order like the values
// (an infinity or a NaN is the largest of all).  The code is 127 x / a to the
// nearest integer: x times 127 / a first; where that lies within 1e-4 of a
// half (its error is below 127 * 3 * 2^-24 < 3e-5) the quotient itself
// decides.  With the mantissas X and A (at most 11 bits) the quotient is 127 X
// / A times a power of two that is at most 1, so one that is no half is at
// least 1 / (254 X) > 2^-19 of itself away from it, more than the division's
// rounding (2^-24): the rounded quotient is on the right side of the half.
// 127 X is exact, and so is a quotient that is a half.
// Rows of very large or very small values are scaled by a power of two first,
// exactly, so that neither 127 x nor 127 / a leaves fp32.
template <typename T>
__global__ void __launch_bounds__(256) quantize_i8_kernel(const uint16_t* __restrict__ x,
                                                          int64_t ldx, int K, int8_t* q,
                                                          int64_t ldq, float* scale) {
  __shared__ uint32_t s_max[8];
  const int64_t m = blockIdx.x;
  const uint16_t* row = x + m * ldx;
  uint32_t top = 0;
  for (int k = threadIdx.x; k < K; k += blockDim.x) top = max(top, (uint32_t)row[k] & 0x7FFFu);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
  __syncthreads();
  top = 0;
  for (int i = 0; i < 8; ++i) top = max(top, s_max[i]);
  const bool finite = top < Bits16<T>::kInf;
  const float a = Bits16<T>::to_float(top);
  if (threadIdx.x == 0) scale[m] = finite ? __fdiv_rn(a, 127.f) : __uint_as_float(0x7FC00000u);
  const float pre = a > 0x1p64f ? 0x1p-64f : a < 0x1p-64f ? 0x1p64f : 1.f;
  const float as = a * pre;
  const float inv = __fdiv_rn(127.f, as);
  for (int k = threadIdx.x; k < K; k += blockDim.x) {
    int c = 0;
    if (finite && top) {
      const float xs = Bits16<T>::to_float(row[k]) * pre;
      const float v = xs * inv;
      float r = rintf(v);
      if (fabsf(v - r) > 0.4999f) r = rintf(__fdiv_rn(xs * 127.f, as));
      c = (int)r;
    }
    q[m * ldq + k] = (int8_t)c;
  }
}

// ------------------------------------------------------------- the product

// 64 x 64 outputs a block, 64 columns of K at a time through shared memory.
template <typename TO>
__global__ void __launch_bounds__(256) gemm_i8_kernel(const int8_t* __restrict__ x, int64_t ldx,
                                                      const float* __restrict__ sx,
                                                      const int8_t* __restrict__ w, int64_t ldw,
                                                      const float* __restrict__ sw, int M, int N,
                                                      int K, TO* y, int64_t ldy) {
  __shared__ int xs[64][17], ws[64][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 64) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i >> 4, c = i & 15;
      int a = 0, b = 0;
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 4 * c + j;
        if (k < K && m0 + r < M) a |= (int)(uint8_t)x[(m0 + r) * ldx + k] << (8 * j);
        if (k < K && n0 + r < N) b |= (int)(uint8_t)w[(n0 + r) * ldw + k] << (8 * j);
      }
      xs[r][c] = a;
      ws[r][c] = b;
    }
    __syncthreads();
    for (int c = 0; c < 16; ++c)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[ty + 16 * i][c], ws[tx + 16 * j][c], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m < M && n < N) store_out(y + m * ldy + n, (float)acc[i][j] * sx[m] * sw[n]);
    }
}

// -------------------------------------------------------------------- host

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int64_t padded_k(int K) { return ((int64_t)K + 15) / 16 * 16; }

bool sizes_ok(int M, int K) { return M >= 0 && K >= 1 && K <= BCQ_I8_MAX_K; }

bool is16(int dtype) { return dtype == BCQ_F16 || dtype == BCQ_BF16; }

cudaError_t launch_quantize(const void* x, int dtype, int M, int K, int64_t ldx, int8_t* q,
                            int64_t ldq, float* scale, cudaStream_t st) {
  const uint16_t* p = static_cast<const uint16_t*>(x);
  if (dtype == BCQ_F16)
    quantize_i8_kernel<__half><<<M, 256, 0, st>>>(p, ldx, K, q, ldq, scale);
  else
    quantize_i8_kernel<__nv_bfloat16><<<M, 256, 0, st>>>(p, ldx, K, q, ldq, scale);
  return cudaGetLastError();
}

cudaError_t launch_gemm(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w,
                        int64_t ldw, const float* sw, int M, int N, int K, void* y, int dtype,
                        int64_t ldy, cudaStream_t st) {
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64));
  if (dtype == BCQ_F32)
    gemm_i8_kernel<<<grid, 256, 0, st>>>(x, ldx, sx, w, ldw, sw, M, N, K, (float*)y, ldy);
  else if (dtype == BCQ_F16)
    gemm_i8_kernel<<<grid, 256, 0, st>>>(x, ldx, sx, w, ldw, sw, M, N, K, (__half*)y, ldy);
  else
    gemm_i8_kernel<<<grid, 256, 0, st>>>(x, ldx, sx, w, ldw, sw, M, N, K, (__nv_bfloat16*)y, ldy);
  return cudaGetLastError();
}

// The weight's and the output's arguments, shared by bcq_gemm_i8 and bcq_linear_i8.
bcq_status check_product(const int8_t* w, int64_t ldw, const float* sw, int M, int N, int K,
                         const void* y, int dtype, int64_t ldy) {
  if (!w || !sw || !y) return BCQ_ERR_NULL;
  if (!sizes_ok(M, K) || N < 1 || ldw < K || ldy < N) return BCQ_ERR_SHAPE;
  if (!is16(dtype) && dtype != BCQ_F32) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(w, 16) || ldw % 16 || !aligned(sw, 4) || !aligned(y, dtype == BCQ_F32 ? 4 : 2))
    return BCQ_ERR_ALIGN;
  return BCQ_OK;
}

}  // namespace

cudaError_t read_and_clear_i8_error(int* code) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_i8_error, sizeof(int));
  if (e == cudaSuccess && *code != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_i8_error, &zero, sizeof(int));
  }
  return e;
}

}  // namespace bcq

using namespace bcq;

extern "C" {

bcq_status bcq_quantize_i8(const void* x, int dtype, int M, int K, int64_t ldx, int8_t* q,
                           int64_t ldq, float* scale, void* stream) {
  if (M == 0 && sizes_ok(M, K)) return BCQ_OK;
  if (!x || !q || !scale) return BCQ_ERR_NULL;
  if (!sizes_ok(M, K) || ldx < K || ldq < K) return BCQ_ERR_SHAPE;
  if (!is16(dtype)) return BCQ_ERR_UNSUPPORTED;
  if (!aligned(x, 2) || !aligned(q, 16) || ldq % 16 || !aligned(scale, 4)) return BCQ_ERR_ALIGN;
  return launch_quantize(x, dtype, M, K, ldx, q, ldq, scale, (cudaStream_t)stream) == cudaSuccess
             ? BCQ_OK
             : BCQ_ERR_CUDA;
}

bcq_status bcq_gemm_i8(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w,
                       int64_t ldw, const float* sw, int M, int N, int K, void* y, int dtype,
                       int64_t ldy, void* stream) {
  if (M == 0 && sizes_ok(M, K) && N >= 1) return BCQ_OK;
  if (!x || !sx) return BCQ_ERR_NULL;
  const bcq_status s = check_product(w, ldw, sw, M, N, K, y, dtype, ldy);
  if (s != BCQ_OK) return s;
  if (ldx < K) return BCQ_ERR_SHAPE;
  if (!aligned(x, 16) || ldx % 16 || !aligned(sx, 4)) return BCQ_ERR_ALIGN;
  return launch_gemm(x, ldx, sx, w, ldw, sw, M, N, K, y, dtype, ldy, (cudaStream_t)stream) ==
                 cudaSuccess
             ? BCQ_OK
             : BCQ_ERR_CUDA;
}

size_t bcq_linear_i8_workspace_bytes(int M, int K) {
  if (!sizes_ok(M, K)) return 0;
  return (size_t)M * (size_t)padded_k(K) + ((size_t)M * 4 + 15) / 16 * 16;
}

bcq_status bcq_linear_i8(const void* x, int dtype, int64_t ldx, const int8_t* w, int64_t ldw,
                         const float* sw, int M, int N, int K, void* y, int64_t ldy,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (M == 0 && sizes_ok(M, K) && N >= 1) return BCQ_OK;
  if (!x || !workspace) return BCQ_ERR_NULL;
  if (!is16(dtype)) return BCQ_ERR_UNSUPPORTED;
  const bcq_status s = check_product(w, ldw, sw, M, N, K, y, dtype, ldy);
  if (s != BCQ_OK) return s;
  if (ldx < K) return BCQ_ERR_SHAPE;
  if (!aligned(x, 2) || !aligned(workspace, 16)) return BCQ_ERR_ALIGN;
  if (workspace_bytes < bcq_linear_i8_workspace_bytes(M, K)) return BCQ_ERR_NULL;
  const int64_t ldq = padded_k(K);
  int8_t* q = static_cast<int8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(q + (size_t)M * (size_t)ldq);
  cudaStream_t st = (cudaStream_t)stream;
  if (launch_quantize(x, dtype, M, K, ldx, q, ldq, sx, st) != cudaSuccess) return BCQ_ERR_CUDA;
  return launch_gemm(q, ldq, sx, w, ldw, sw, M, N, K, y, dtype, ldy, st) == cudaSuccess
             ? BCQ_OK
             : BCQ_ERR_CUDA;
}

}  // extern "C"
