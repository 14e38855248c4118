// The 8-bit activations of the projection path: RMSNorm with the residual
// addition, and plain quantization of rows or weights, both to E4M3 codes with
// one power-of-two scale per block of 128 columns.
//
// Format: block amax a (over the finite elements) gives the smallest e >= -127
// with a <= 448 2^e; the scale byte is e + 127 (UE8M0) and the codes are
// x 2^-e rounded to nearest even, so no finite element saturates and a normal
// code's relative error is at most 2^-4 whatever the scale.  NaN and infinity
// become the NaN code and do not touch the scale.
#include "common.cuh"
#include "fp8.h"
#include "fp8_codes.cuh"
#include "internal.h"

namespace csa {

namespace {

constexpr int kVec = 8;   // elements a thread holds per step; 16 lanes are one block

// Eight consecutive elements as float, read once.
__device__ __forceinline__ void load8(const bf16* p, float* v) { load_vec_stream(p, v); }
__device__ __forceinline__ void load8(const float* p, float* v) {
  load_vec_stream(p, v);
  load_vec_stream(p + 4, v + 4);
}
__device__ __forceinline__ void store8(bf16* p, const float* v) { store_vec(p, v); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  store_vec(p, v);
  store_vec(p + 4, v + 4);
}

__device__ __forceinline__ float amax8(const float* v) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) a = fmaxf(a, fabsf(v[i]));   // fmaxf skips NaN
  return a;
}

// The larger of the 16 lanes that hold one 128-column block.
__device__ __forceinline__ float half_warp_max(float a) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// Infinities become NaN, so that the codes say so and the scale does not.
__device__ __forceinline__ void drop_inf8(float* v) {
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (isinf(v[i])) v[i] = __int_as_float(0x7fffffff);
}

// Block scale and codes of this lane's eight elements.  Every lane of the warp
// calls it.
__device__ __forceinline__ uint32_t quantize8(float* v, uint2* codes) {
  float a = half_warp_max(amax8(v));
  if (__any_sync(0xffffffffu, isinf(a))) {   // rare: the scale from the finite elements
    drop_inf8(v);
    a = half_warp_max(amax8(v));
  }
  const uint32_t byte = scale_byte(a);
  *codes = codes8(v, byte);
  return byte;
}

// ---- RMSNorm with the residual addition ------------------------------------

struct NormArgs {
  int64_t T;
  int d, nb;              // columns, 128-column blocks (the last may be short)
  int64_t x_ld, r_ld, s_ld;
  const void* x;
  const void* res;        // or null
  const float* gain;      // or null
  float eps;
  void* sum_out;          // or null
  uint8_t* codes;
  uint8_t* scales;
};

// blockDim = (threads per row, rows per block); a thread holds VPT vectors of
// eight columns, tpr apart, in registers, so that x is read once: the sum of
// squares over the row's threads, then scale and codes from the registers.
template <typename T, int VPT>
__global__ void __launch_bounds__(512) rmsnorm_fp8_kernel(NormArgs a) {
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int tpr = blockDim.x;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.T;
  const int nvec = a.d / kVec;
  const int wpr = tpr >> 5, warp0 = threadIdx.y * wpr;
  float h[VPT][kVec];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * tpr;
#pragma unroll
    for (int j = 0; j < kVec; ++j) h[i][j] = 0.f;
    if (live && c < nvec)
      load8(static_cast<const T*>(a.x) + row * a.x_ld + (int64_t)c * kVec, h[i]);
  }
  if (a.res != nullptr) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = threadIdx.x + i * tpr;
      if (live && c < nvec) {
        float r[kVec];
        load8(static_cast<const T*>(a.res) + row * a.r_ld + (int64_t)c * kVec, r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[i][j] += r[j];
        if (a.sum_out != nullptr)
          store8(static_cast<T*>(a.sum_out) + row * a.s_ld + (int64_t)c * kVec, h[i]);
      }
    }
  }
  // mean of squares over the row, in a fixed order
  auto row_sum = [&](float s, int slot) {
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) red[slot][warp0 + (threadIdx.x >> 5)] = s;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < wpr; ++w) t += red[slot][warp0 + w];
    return t;
  };
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) s = fmaf(h[i][j], h[i][j], s);
  const float n = 1.f / (float)a.d;
  float ms = row_sum(s, 0);
  float rstd = rsqrtf(fmaf(ms, n, a.eps));
  // squares beyond float32 (|h| > 1e19): the sum again on 2^-80 h, where eps
  // counts for nothing; a row that holds an infinity ends with 1/inf = 0
  if (__syncthreads_or(isinf(ms))) {
    constexpr float kDown = 8.271806125530277e-25f;   // 2^-80
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float t = h[i][j] * kDown;
        s2 = fmaf(t, t, s2);
      }
    s2 = row_sum(s2, 1);
    if (isinf(ms)) rstd = rsqrtf(s2 * n) * kDown;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = threadIdx.x + i * tpr;
    const bool in = live && c < nvec;
#pragma unroll
    for (int j = 0; j < kVec; ++j) h[i][j] *= rstd;
    if (a.gain != nullptr && in) {
      const float4 g0 = __ldg(reinterpret_cast<const float4*>(a.gain + (int64_t)c * kVec));
      const float4 g1 = __ldg(reinterpret_cast<const float4*>(a.gain + (int64_t)c * kVec + 4));
      h[i][0] *= g0.x; h[i][1] *= g0.y; h[i][2] *= g0.z; h[i][3] *= g0.w;
      h[i][4] *= g1.x; h[i][5] *= g1.y; h[i][6] *= g1.z; h[i][7] *= g1.w;
    }
    if (!in) {   // columns past the row: no part of the last block's scale
#pragma unroll
      for (int j = 0; j < kVec; ++j) h[i][j] = 0.f;
    }
    uint2 q;
    const uint32_t byte = quantize8(h[i], &q);
    if (in) {
      *reinterpret_cast<uint2*>(a.codes + row * a.d + (int64_t)c * kVec) = q;
      if ((c & 15) == 0) a.scales[row * a.nb + (c >> 4)] = (uint8_t)byte;
    }
  }
}

template <typename T>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t stream) {
  const int nvec = a.d / kVec;
  int vpt = nvec >= 128 ? 4 : nvec >= 64 ? 2 : 1;
  while ((nvec + vpt - 1) / vpt > 512) vpt *= 2;
  const int tpr = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
  const int rpb = tpr >= 128 ? 1 : 128 / tpr;
  const dim3 block(tpr, rpb);
  const int64_t grid = (a.T + rpb - 1) / rpb;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  switch (vpt) {
    case 1: return launch_pdl(rmsnorm_fp8_kernel<T, 1>, dim3((unsigned)grid), block, 0, stream, a);
    case 2: return launch_pdl(rmsnorm_fp8_kernel<T, 2>, dim3((unsigned)grid), block, 0, stream, a);
    case 4: return launch_pdl(rmsnorm_fp8_kernel<T, 4>, dim3((unsigned)grid), block, 0, stream, a);
    default: return launch_pdl(rmsnorm_fp8_kernel<T, 8>, dim3((unsigned)grid), block, 0, stream, a);
  }
}

// ---- quantization ------------------------------------------------------------

constexpr int kQUnroll = 4;

// One block of 128 columns of a row per half-warp, four blocks in flight.
template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const T* x, int64_t ld, int d,
                                                                int nb, int64_t blocks,
                                                                uint8_t* codes, uint8_t* scales) {
  pdl_wait();
  pdl_trigger();
  const int lane16 = threadIdx.x & 15;
  const int64_t first = (int64_t)blockIdx.x * (16 * kQUnroll) + (threadIdx.x >> 4);
  float v[kQUnroll][kVec];
  int64_t at[kQUnroll];   // element offset of this thread's codes, -1 past the end
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const int64_t b = first + 16 * u;
    const int64_t row = b / nb;
    const int c = (int)(b - row * nb) * 128 + lane16 * kVec;
    const bool in = b < blocks && c < d;
    at[u] = in ? row * d + c : -1;
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[u][j] = 0.f;
    if (in) load8(x + row * ld + c, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    uint2 q;
    const uint32_t byte = quantize8(v[u], &q);
    if (at[u] >= 0) {
      *reinterpret_cast<uint2*>(codes + at[u]) = q;
      if (lane16 == 0) scales[first + 16 * u] = (uint8_t)byte;
    }
  }
}

// One 128 x 128 block per CTA: a half-warp holds eight of its rows.
template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_block_kernel(const T* x, int64_t ld,
                                                                 int64_t rows, int d, int nb,
                                                                 uint8_t* codes,
                                                                 uint8_t* scales) {
  __shared__ float red[8];
  pdl_wait();
  pdl_trigger();
  const int64_t br = blockIdx.x / nb;
  const int bc = (int)(blockIdx.x - br * nb);
  const int c = bc * 128 + (threadIdx.x & 15) * kVec;
  const int64_t r0 = br * 128 + (threadIdx.x >> 4);
  float v[8][kVec];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] = 0.f;
    if (r < rows && c < d) load8(x + r * ld + c, v[i]);
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, amax8(v[i]));
  if (__syncthreads_or(isinf(a))) {
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      drop_inf8(v[i]);
      a = fmaxf(a, amax8(v[i]));
    }
  }
  a = half_warp_max(a);
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, red[w]);
  const uint32_t byte = scale_byte(a);
  if (threadIdx.x == 0) scales[(int64_t)blockIdx.x] = (uint8_t)byte;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < rows && c < d) *reinterpret_cast<uint2*>(codes + r * d + c) = codes8(v[i], byte);
  }
}

template <typename T>
cudaError_t quantize_launch(const T* x, int64_t ld, int64_t rows, int d, int block_rows,
                            uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  const int nb = (d + 127) / 128;
  if (block_rows == 1) {
    const int64_t blocks = rows * nb;
    const int64_t grid = (blocks + 16 * kQUnroll - 1) / (16 * kQUnroll);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(fp8_quantize_rows_kernel<T>, dim3((unsigned)grid), dim3(256), 0, stream, x,
                      ld, d, nb, blocks, codes, scales);
  }
  const int64_t grid = (rows + 127) / 128 * nb;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(fp8_quantize_block_kernel<T>, dim3((unsigned)grid), dim3(256), 0, stream, x,
                    ld, rows, d, nb, codes, scales);
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(int dtype, const NormParams& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  NormArgs a{p.T, p.d, (p.d + 127) / 128, p.x_ld, p.res_ld, p.sum_ld, p.x, p.residual,
             p.gain, p.eps, p.sum_out, static_cast<uint8_t*>(p.codes),
             static_cast<uint8_t*>(p.scales)};
  return dtype == CSA_BF16 ? norm_launch<bf16>(a, stream) : norm_launch<float>(a, stream);
}

cudaError_t launch_fp8_quantize(int dtype, const void* x, int64_t ld, int64_t rows, int d,
                                int block_rows, void* codes, void* scales, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  uint8_t* c = static_cast<uint8_t*>(codes);
  uint8_t* s = static_cast<uint8_t*>(scales);
  return dtype == CSA_BF16
             ? quantize_launch(static_cast<const bf16*>(x), ld, rows, d, block_rows, c, s, stream)
             : quantize_launch(static_cast<const float*>(x), ld, rows, d, block_rows, c, s, stream);
}

}  // namespace csa
