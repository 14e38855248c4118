// The 8-bit projection path: E4M3 codes with a power-of-two scale per 128
// columns (activations: of one row; weights: of 128 rows).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace csa {

constexpr int kFp8MaxNormDim = 32768;   // columns rmsnorm_fp8 holds in registers

constexpr int64_t kFp8MaxDim = 1 << 30;  // rows and columns of a product: tile ends fit 32 bits
constexpr int64_t kFp8MaxK = 1 << 26;    // a tile's sum ends well within a bounded wait
// Columns of one tensor-core sum.  Each MMA cuts off up to 2^-23 of the sum so far,
// every 32 columns: at most 2^-11 over 2^17 columns, an eighth of bf16's half step
// (operands of one sign, 2^17 columns: 1.6e-4).  bf16 and E4M3 results, which no
// float32 buffer adds up from parts, take no more; over 2^20 columns the cut would
// reach bf16's rounding itself.
constexpr int64_t kFp8MaxOneSum = 1 << 17;

struct NormParams {
  int64_t T;
  int d;
  const void* x;          // [T, d], row stride x_ld elements
  int64_t x_ld;
  const void* residual;   // or null
  int64_t res_ld;
  const float* gain;      // [d] or null
  float eps;
  void* sum_out;          // [T, d] or null
  int64_t sum_ld;
  void* codes;            // [T, d]
  void* scales;           // [T, ceil(d / 128)]
};
constexpr int kMaxDevices = 64;

// The current device, or -1.
inline int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev < kMaxDevices ? dev : -1;
}

// SMs of the current device (asked once per device).
inline int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = current_device();
  int n = dev >= 0 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (dev < 0 ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_rmsnorm_fp8(int dtype, const NormParams& p, cudaStream_t stream);

cudaError_t launch_fp8_quantize(int dtype, const void* x, int64_t ld, int64_t rows, int d,
                                int block_rows, void* codes, void* scales, cudaStream_t stream);

constexpr int kFp8Out = 2;   // Y as E4M3 codes with their own scales

// Y[m, z y_noff + n] = sum_k X[m, z x_koff + k] W[z][n, k], n < N, k < K.
struct Fp8GemmParams {
  int64_t M;
  int N, K, Z;
  const uint8_t* x;        // [M, x_cols] codes
  const uint8_t* x_sf;     // [M, ceil(x_cols / 128)]
  int x_cols;
  int x_koff;              // per z, a multiple of 128
  const uint8_t* w;        // [Z, N, K] codes
  const uint8_t* w_sf;     // [Z, ceil(N / 128), ceil(K / 128)]
  int out;                 // CSA_F32, CSA_BF16, or kFp8Out
  void* y;                 // kFp8Out: codes (N, y_ld and y_noff multiples of 128)
  uint8_t* y_sf;           // kFp8Out: their scales [M, y_ld / 128]
  int64_t y_ld;
  int y_noff;              // per z
  unsigned* status;
  unsigned long long* launches;   // counted up
};
cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, cudaStream_t stream);

}  // namespace csa
