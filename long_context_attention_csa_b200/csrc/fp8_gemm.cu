// Matrix product of E4M3 operands with a power-of-two scale per 128 columns
// (one row of X; 128 rows of W): y[m, n] = sum_b 2^(ex[m,b] + ew[n/128,b])
// sum_{k in b} x[m,k] w[n,k].  The block's products are summed in float32
// (they are exact there up to 2^24 steps of the smallest product), the scale
// applied once per block and the blocks summed in float32.
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8.h"
#include "internal.h"

namespace csa {

namespace {

constexpr int kT = 64;    // tile rows and columns
constexpr int kTK = 32;   // K per step

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__device__ __forceinline__ float pow2(uint8_t byte) {
  return byte == 255 ? __int_as_float(0x7fffffff) : exp2f((float)byte - 127.f);
}

__global__ void __launch_bounds__(256) fp8_gemm_kernel(Fp8GemmParams p) {
  __shared__ float xs[kTK][kT + 1], ws[kTK][kT + 1];
  pdl_wait();
  const int64_t m0 = (int64_t)blockIdx.x * kT;
  const int n0 = blockIdx.y * kT, z = blockIdx.z;
  const int xb = (p.x_cols + 127) / 128, wb = (p.K + 127) / 128, wrb = (p.N + 127) / 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kTK) {
    for (int i = threadIdx.x; i < kT * kTK; i += 256) {
      const int r = i / kTK, k = i % kTK;
      const int64_t m = m0 + r;
      const int n = n0 + r;
      xs[k][r] = m < p.M && k0 + k < p.K
                     ? e4m3(p.x[m * p.x_cols + (int64_t)z * p.x_koff + k0 + k]) : 0.f;
      ws[k][r] = n < p.N && k0 + k < p.K
                     ? e4m3(p.w[((int64_t)z * p.N + n) * p.K + k0 + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          part[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx * 4 + j], part[i][j]);
    __syncthreads();
    if ((k0 + kTK) % 128 == 0 || k0 + kTK >= p.K) {
      const int kb = k0 / 128;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + ty * 4 + i;
          const int n = n0 + tx * 4 + j;
          if (m < p.M && n < p.N) {
            const float sx = pow2(p.x_sf[m * xb + z * (p.x_koff / 128) + kb]);
            const float sw = pow2(p.w_sf[((int64_t)z * wrb + n / 128) * wb + kb]);
            acc[i][j] += part[i][j] * sx * sw;
          }
          part[i][j] = 0.f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i;
      const int n = n0 + tx * 4 + j;
      if (m < p.M && n < p.N) {
        const int64_t at = m * p.y_ld + (int64_t)z * p.y_noff + n;
        if (p.out_dtype == CSA_BF16)
          static_cast<bf16*>(p.y)[at] = __float2bfloat16_rn(acc[i][j]);
        else
          static_cast<float*>(p.y)[at] = acc[i][j];
      }
    }
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, cudaStream_t stream) {
  if (p.M == 0 || p.N == 0) return cudaSuccess;
  const dim3 grid((unsigned)((p.M + kT - 1) / kT), (unsigned)((p.N + kT - 1) / kT), (unsigned)p.Z);
  return launch_pdl(fp8_gemm_kernel, grid, dim3(256), 0, stream, p);
}

}  // namespace csa
