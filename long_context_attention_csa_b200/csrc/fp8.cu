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

// Eight consecutive elements as they lie in memory, and as float.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) {
    u = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
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

// Block scale and codes of this lane's eight elements.  Every lane of the warp
// calls it.
__device__ __forceinline__ uint32_t quantize8(float* v, uint2* codes) {
  float a = half_warp_max(amax8(v));
  if (__any_sync(0xffffffffu, isinf(a))) {   // rare: the scale from the finite elements
    drop_infinities<kVec>(v);
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

// A row's tpr threads hold VPT vectors of eight columns each, tpr apart, in
// registers, so that x is read once: the sum of squares over the row, then scale
// and codes from the registers.  CTAs walk the rows with the next row's loads in
// flight and the gain in registers; a row of one warp takes no block
// barrier, and a CTA then walks four rows at a time.
template <typename T, int VPT>
__global__ void __launch_bounds__(512) rmsnorm_fp8_kernel(NormArgs a) {
  constexpr bool kAhead = VPT * sizeof(T) <= 8;   // registers for it
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int tpr = blockDim.x, tid = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int nvec = a.d / kVec;
  const int wpr = tpr >> 5;
  const float n = 1.f / (float)a.d;
  Raw8<T> xr[VPT], rr[kAhead ? VPT : 1];
  float g[kAhead ? VPT : 1][kVec];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * tpr;
      if (at < a.T && c < nvec) {
        xr[i].load(static_cast<const T*>(a.x) + at * a.x_ld + (int64_t)c * kVec);
        if (kAhead && a.res != nullptr)
          rr[kAhead ? i : 0].load(static_cast<const T*>(a.res) + at * a.r_ld + (int64_t)c * kVec);
      } else {
        xr[i].clear();
        if (kAhead) rr[kAhead ? i : 0].clear();
      }
    }
  };
  auto gain8 = [&](int c, float* w) {
    const float4 lo = __ldg(reinterpret_cast<const float4*>(a.gain) + 2 * c);
    const float4 hi = __ldg(reinterpret_cast<const float4*>(a.gain) + 2 * c + 1);
    w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
    w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
  };
  load(row);
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[i][j] = 1.f;
      if (a.gain != nullptr && tid + i * tpr < nvec) gain8(tid + i * tpr, g[i]);
    }
  }
  // sum over the row's threads, in a fixed order
  auto row_sum = [&](float s, int slot) {
    s = warp_sum(s);
    if (wpr == 1) return s;
    if ((tid & 31) == 0) red[slot][tid >> 5] = s;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < wpr; ++w) t += red[slot][w];
    return t;
  };
  // rows of one warp: the block's rows end apart; else the whole block goes on
  for (int it = 0; row < a.T; row += step, it ^= 1) {
    float h[VPT][kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      xr[i].get(h[i]);
      if (a.res != nullptr) {
        float r[kVec];
        const int c = tid + i * tpr;
        if (!kAhead) {
          rr[0].clear();
          if (c < nvec)
            rr[0].load(static_cast<const T*>(a.res) + row * a.r_ld + (int64_t)c * kVec);
        }
        rr[kAhead ? i : 0].get(r);
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) s = fmaf(h[i][j], h[i][j], s);
    }
    if (kAhead) load(row + step);
    if (a.sum_out != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        if (c < nvec)
          store8(static_cast<T*>(a.sum_out) + row * a.s_ld + (int64_t)c * kVec, h[i]);
      }
    }
    const float ms = row_sum(s, it);
    float rstd = rsqrtf(fmaf(ms, n, a.eps));
    // squares beyond float32 (|h| > 1e19): the sum again on 2^-80 h, where eps
    // counts for nothing; a row that holds an infinity ends with 1/inf = 0
    if (isinf(ms)) {   // uniform over the row's threads, which are a warp or the block
      constexpr float kDown = 8.271806125530277e-25f;   // 2^-80
      float s2 = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float t = h[i][j] * kDown;
          s2 = fmaf(t, t, s2);
        }
      if (wpr > 1) __syncthreads();   // the slot has been read
      rstd = rsqrtf(row_sum(s2, it) * n) * kDown;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * tpr;
      if constexpr (kAhead) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[i][j] = h[i][j] * rstd * g[i][j];
      } else {
        float w[kVec] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
        if (a.gain != nullptr && c < nvec) gain8(c, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[i][j] = h[i][j] * rstd * w[j];
      }
      if (c >= nvec) {   // past the row: no part of the last block's scale
#pragma unroll
        for (int j = 0; j < kVec; ++j) h[i][j] = 0.f;
      }
      uint2 q;
      const uint32_t byte = quantize8(h[i], &q);
      if (c < nvec) {
        *reinterpret_cast<uint2*>(a.codes + row * a.d + (int64_t)c * kVec) = q;
        if ((c & 15) == 0) a.scales[row * a.nb + (c >> 4)] = (uint8_t)byte;
      }
    }
    if (!kAhead) load(row + step);
  }
}

template <typename T>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t stream) {
  const int nvec = a.d / kVec;
  const int64_t sms = sm_count();
  // few rows: one vector a thread, for latency (a row of 4096 bf16 columns, 9.5
  // -> TODO us); many: four, for bytes in flight
  int vpt = a.T <= 2 * sms ? 1 : nvec > 64 && sizeof(T) == 2 ? 4 : nvec > 32 ? 2 : 1;
  while ((nvec + vpt - 1) / vpt > 512) vpt *= 2;
  const int tpr = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
  const int rpb = tpr == 32 ? 4 : 1;
  const dim3 block(tpr, rpb);
  const int64_t blocks = (a.T + rpb - 1) / rpb;
  // 128 registers a thread: what fits at once, each walking its share of the rows
  const int64_t room = sms * (512 / (tpr * rpb) > 0 ? 512 / (tpr * rpb) : 1);
  const dim3 grid((unsigned)(blocks < room ? blocks : room));
  switch (vpt) {
    case 1: return launch_pdl(rmsnorm_fp8_kernel<T, 1>, grid, block, 0, stream, a);
    case 2: return launch_pdl(rmsnorm_fp8_kernel<T, 2>, grid, block, 0, stream, a);
    case 4: return launch_pdl(rmsnorm_fp8_kernel<T, 4>, grid, block, 0, stream, a);
    default: return launch_pdl(rmsnorm_fp8_kernel<T, 8>, grid, block, 0, stream, a);
  }
}

// ---- quantization ------------------------------------------------------------

constexpr int kQUnroll = 4;

// One block of 128 columns of a row per half-warp, four blocks in flight.
// blockIdx.x counts groups of 64 blocks in row order; the division by the
// blocks of a row is taken in 32 bits from the group's own first row and block.
template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const T* x, int64_t ld, int d,
                                                                int nb, int64_t blocks,
                                                                uint8_t* codes, uint8_t* scales) {
  pdl_wait();
  pdl_trigger();
  const int lane16 = threadIdx.x & 15;
  const int64_t first = (int64_t)blockIdx.x * (16 * kQUnroll);
  const int64_t row0 = first / nb;
  const uint32_t blk0 = (uint32_t)(first - row0 * nb);
  Raw8<T> raw[kQUnroll];
  int64_t at[kQUnroll];   // element offset of this thread's codes, -1 past the end
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint32_t b = (threadIdx.x >> 4) + 16 * u;
    const uint32_t r = (blk0 + b) / (uint32_t)nb;
    const int c = (int)(blk0 + b - r * nb) * 128 + lane16 * kVec;
    const bool in = first + b < blocks && c < d;
    at[u] = in ? (row0 + r) * d + c : -1;
    if (in) raw[u].load(x + (row0 + r) * ld + c);
    else raw[u].clear();
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    float v[kVec];
    raw[u].get(v);
    uint2 q;
    const uint32_t byte = quantize8(v, &q);
    if (at[u] >= 0) {
      *reinterpret_cast<uint2*>(codes + at[u]) = q;
      if (lane16 == 0) scales[first + (threadIdx.x >> 4) + 16 * u] = (uint8_t)byte;
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
  Raw8<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < rows && c < d) raw[i].load(x + r * ld + c);
    else raw[i].clear();
  }
  float v[8][kVec];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    raw[i].get(v[i]);
    a = fmaxf(a, amax8(v[i]));
  }
  if (__syncthreads_or(isinf(a))) {   // rare: the scale from the finite elements
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      drop_infinities<kVec>(v[i]);
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
