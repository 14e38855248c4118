// The 8-bit activations of the projection path: RMSNorm with the residual
// addition, and plain quantization of rows or weights, both to E4M3 codes with
// one power-of-two scale per block of 128 columns.
//
// Format: block amax a (over the finite elements) gives the smallest e >= -127
// with a <= 448 2^e; the scale byte is e + 127 (UE8M0) and the codes are
// x 2^-e rounded to nearest even, so no finite element saturates and a normal
// code's relative error is at most 2^-4 whatever the scale.  NaN and infinity
// become the NaN code and do not touch the scale.
//
// A lane holds sixteen consecutive columns (one 32-byte load of bf16, one 16-byte
// store of codes), eight lanes a block.  With eight columns a lane and scalar
// arithmetic the norm was bound by its instructions (155 for eight columns, 64% of
// the issue slots): 8192 x 4096 bf16 without a residual took 30.5 us, 19.3 now.
// Measured (B200, copy rate 6.55 TB/s): 65536 x 4096 bf16 with residual 277 us
// (6.8 TB/s), 8192 x 4096 38.3 us (6.1), rows of 8192 x 32768 quantized in 118 us
// (6.8), weights of 4096 x 8192 float32 in 27 us (6.2); one row 2.2 us between
// captured launches.
#include "common.cuh"
#include "fp8.h"
#include "fp8_codes.cuh"
#include "internal.h"

namespace csa {

namespace {

constexpr int kUnit = 16;          // columns a lane holds
constexpr int kUnitLanes = 8;      // lanes of one block

// ---- pairs of floats in one 64-bit register -----------------------------------
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(f2 p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 32 bytes, read once; `wide`: on a 32-byte boundary (else on a 16-byte one).
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = __ldcs(static_cast<const uint4*>(p));
    const uint4 b = __ldcs(static_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t* w) {
  if (wide) {
    store_sector(p, w);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Sixteen columns as they lie in memory, and as eight pairs of floats.
template <typename T> struct Raw;
template <> struct Raw<bf16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const bf16* p, bool wide) { load32(p, wide, w); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void forget() {   // what the compiler knows of the words
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(w[i]));
  }
  __device__ __forceinline__ void get(f2* v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <> struct Raw<float> {
  uint32_t w[16];
  __device__ __forceinline__ void load(const float* p, bool wide) {
    load32(p, wide, w);
    load32(p + 8, wide, w + 8);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void forget() {}
  __device__ __forceinline__ void get(f2* v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
};
__device__ __forceinline__ void store16(bf16* p, bool wide, const f2* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    split(v[i], a, b);
    w[i] = pack_bf16x2(a, b);
  }
  store32(p, wide, w);
}
__device__ __forceinline__ void store16(float* p, bool wide, const f2* v) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    split(v[i], a, b);
    w[2 * i] = __float_as_uint(a);
    w[2 * i + 1] = __float_as_uint(b);
  }
  store32(p, wide, w);
  store32(p + 8, wide, w + 8);
}

__device__ __forceinline__ float amax16(const f2* v) {
  float m = 0.f;   // fmaxf skips NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    split(v[i], a, b);
    m = fmaxf(fmaxf(m, fabsf(a)), fabsf(b));
  }
  return m;
}

// The largest of the eight lanes that hold one block.
__device__ __forceinline__ float block_max(float a) {
#pragma unroll
  for (int o = 1; o < kUnitLanes; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

__device__ __forceinline__ void drop_infinities16(f2* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a[2];
    split(v[i], a[0], a[1]);
    drop_infinities<2>(a);
    v[i] = pair(a[0], a[1]);
  }
}

__device__ __forceinline__ float pow2_of(uint32_t e127) { return __uint_as_float(e127 << 23); }

// Codes of the sixteen v times `factor`; no product is infinite.
__device__ __forceinline__ uint4 codes16(const f2* v, float factor) {
  const f2 f = pair(factor, factor);
  uint32_t c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float a, b, d, e;
    split(mul2(v[2 * q], f), a, b);
    split(mul2(v[2 * q + 1], f), d, e);
    c[q] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(d, e), __NV_SATFINITE, __NV_E4M3)
            << 16);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

inline bool aligned32(const void* p, int64_t ld, int elem) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * elem)) & 31) == 0;
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
  bool x_wide, r_wide, s_wide;   // rows start on 32-byte boundaries
};

// A row's tpr threads hold U units of sixteen columns each, tpr apart, in
// registers, so that x is read once: the sum of squares over the row, then scale
// and codes from the registers.  CTAs walk the rows with the next row's loads in
// flight and the gain in registers, where they fit.  A row of a warp or less (8,
// 16 or 32 lanes) takes no block barrier, and a CTA then walks 128 / tpr rows at a
// time.  tpr and U follow from d alone, so a row's sum has one order whatever T is.
template <typename T, int U>
__global__ void __launch_bounds__(512) rmsnorm_fp8_kernel(NormArgs a) {
  constexpr bool kAhead = U * sizeof(T) <= 4;
  __shared__ float red[2][16];
  pdl_wait();
  pdl_trigger();
  const int tpr = blockDim.x, tid = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int units = a.d / kUnit;
  const int wpr = tpr >> 5;   // 0: less than a warp
  const float n = 1.f / (float)a.d;
  const T* xp = static_cast<const T*>(a.x);
  const T* rp = static_cast<const T*>(a.res);
  Raw<T> xr[U], rr[kAhead ? U : 1];
  f2 g[kAhead ? U : 1][8];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = tid + i * tpr;
      xr[i].clear();
      if (at < a.T && c < units) xr[i].load(xp + at * a.x_ld + c * kUnit, a.x_wide);
      if (kAhead && rp != nullptr) {
        rr[kAhead ? i : 0].clear();
        if (at < a.T && c < units)
          rr[kAhead ? i : 0].load(rp + at * a.r_ld + c * kUnit, a.r_wide);
      }
    }
  };
  auto gain16 = [&](int c, f2* w) {
    const float4* p = reinterpret_cast<const float4*>(a.gain + c * kUnit);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = __ldg(p + q);
      w[2 * q] = pair(v.x, v.y);
      w[2 * q + 1] = pair(v.z, v.w);
    }
  };
  load(row);
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = 0;
      if (a.gain != nullptr && tid + i * tpr < units) gain16(tid + i * tpr, g[i]);
    }
  }
  auto row_sum = [&](float s, int slot) {
    if (wpr <= 1) {
      for (int o = tpr >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      return s;
    }
    s = warp_sum(s);
    if ((tid & 31) == 0) red[slot][tid >> 5] = s;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < wpr; ++w) t += red[slot][w];
    return t;
  };
  // the block goes on as long as its first row is one of T
  for (int it = 0; row - threadIdx.y < a.T; row += step, it ^= 1) {
    const bool live = row < a.T;
    f2 h[U][8];
    f2 s = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      xr[i].get(h[i]);
      if (rp != nullptr) {
        const int c = tid + i * tpr;
        if (!kAhead) {
          rr[0].clear();
          if (live && c < units) rr[0].load(rp + row * a.r_ld + c * kUnit, a.r_wide);
        }
        f2 r[8];
        rr[kAhead ? i : 0].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = add2(h[i][j], r[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fma2(h[i][j], h[i][j], s);
    }
    if (kAhead) {
      load(row + step);
    } else if (row + step < a.T) {   // at least into L2
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = tid + i * tpr;
        if (c < units) {
          prefetch_l2(xp + (row + step) * a.x_ld + c * kUnit);
          if (rp != nullptr) prefetch_l2(rp + (row + step) * a.r_ld + c * kUnit);
        }
      }
    }
    if (a.sum_out != nullptr) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = tid + i * tpr;
        if (live && c < units)
          store16(static_cast<T*>(a.sum_out) + row * a.s_ld + c * kUnit, a.s_wide, h[i]);
      }
    }
    float s0, s1;
    split(s, s0, s1);
    const float ms = row_sum(s0 + s1, it);
    float rstd = rsqrtf(fmaf(ms, n, a.eps));
    // squares beyond float32 (|h| > 1e19), or near its smallest where eps does not
    // hide them: the same on 2^-80 h or 2^80 h, eps times that twice; a row that
    // holds an infinity ends with 1/inf = 0
    const bool tiny = a.eps < 0x1p-100f && ms < 0x1p-100f;
    if (__any_sync(0xffffffffu, isinf(ms) || tiny)) {   // alike in a row's warps
      const float by = isinf(ms) ? 0x1p-80f : tiny ? 0x1p80f : 1.f;
      const f2 down = pair(by, by);
      f2 q = 0;
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i][j] = mul2(h[i][j], down);
          q = fma2(h[i][j], h[i][j], q);
        }
      split(q, s0, s1);
      if (wpr > 1) __syncthreads();   // the slot has been read
      const float ms2 = row_sum(s0 + s1, it);
      if (by != 1.f) rstd = rsqrtf(fmaf(ms2, n, a.eps * by * by));
    }
    // y = h gain rstd: the largest |h gain| of a block, times rstd, gives its
    // scale, and one product per element, by rstd 2^-e, its code
    float top[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (a.gain != nullptr) {
        f2 w[8];
        if constexpr (!kAhead) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = 0;
          if (tid + i * tpr < units) gain16(tid + i * tpr, w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = mul2(h[i][j], kAhead ? g[kAhead ? i : 0][j] : w[j]);
      }
      top[i] = amax16(h[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) top[i] = block_max(top[i]);
    uint32_t byte[U];
    float f[U];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float most = top[i] * rstd;   // the block's largest |y|
      byte[i] = scale_byte(fmaxf(most, 0.f));
      // an infinite most: |h gain|, or y alone, is beyond float32; rstd 2^-e stays
      // finite for e >= -63; a block of zeros takes any factor
      odd = odd || !(most < INFINITY) || !(rstd < 1e18f) || (byte[i] < 64u && top[i] != 0.f);
      f[i] = rstd * pow2_of(254u - (byte[i] < 64u ? 64u : byte[i]));
    }
    if (__any_sync(0xffffffffu, odd)) {   // infinities, or values below 2^-54: step by step
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = mul2(h[i][j], pair(rstd, rstd));
        drop_infinities16(h[i]);
        byte[i] = scale_byte(block_max(amax16(h[i])));
        f[i] = pow2_of(254u - byte[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = tid + i * tpr;
      if (live && c < units) {
        *reinterpret_cast<uint4*>(a.codes + row * a.d + c * kUnit) = codes16(h[i], f[i]);
        if ((c & (kUnitLanes - 1)) == 0)
          a.scales[row * a.nb + c / kUnitLanes] = (uint8_t)byte[i];
      }
    }
    if (!kAhead) load(row + step);
  }
}

template <typename T>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t stream) {
  const int units = a.d / kUnit;
  const int64_t sms = sm_count();
  int u = units > 32 && sizeof(T) == 2 ? 2 : 1;
  while ((units + u - 1) / u > 512) u *= 2;
  const int lanes = (units + u - 1) / u;
  const int tpr = lanes <= 8 ? 8 : lanes <= 16 ? 16 : (lanes + 31) / 32 * 32;
  const int rpb = tpr <= 32 ? 128 / tpr : 1;
  const dim3 block(tpr, rpb);
  const int64_t blocks = (a.T + rpb - 1) / rpb;
  // what fits at once (128 registers a thread), each CTA walking its rows
  const int64_t room = sms * (512 / (tpr * rpb) > 0 ? 512 / (tpr * rpb) : 1);
  // Three streams of wide rows: CTAs that walk many rows drift apart and spread
  // their rows over too many DRAM pages (65536 x 4096 bf16: 315 us), so there each
  // walks eight and the next ones take their place in order (277 us).  Where they
  // walk 24 or fewer, or one stream in or narrow rows, the drift costs less than
  // the starts (8192 x 4096: 38.3 us, eight rows each 42).
  const bool short_walks =
      a.res != nullptr && u * sizeof(T) <= 4 && tpr >= 128 && blocks > 24 * room;
  const int64_t want = short_walks ? (blocks + 7) / 8 : room;
  const dim3 grid((unsigned)(blocks < want ? blocks : want));
  switch (u) {
    case 1: return launch_pdl(rmsnorm_fp8_kernel<T, 1>, grid, block, 0, stream, a);
    case 2: return launch_pdl(rmsnorm_fp8_kernel<T, 2>, grid, block, 0, stream, a);
    default: return launch_pdl(rmsnorm_fp8_kernel<T, 4>, grid, block, 0, stream, a);
  }
}

// ---- quantization ------------------------------------------------------------

// Scale byte and codes of one block's eight lanes.  Every lane of the warp calls it.
__device__ __forceinline__ uint32_t quantize16(f2* v, uint4* codes) {
  float a = block_max(amax16(v));
  if (__any_sync(0xffffffffu, isinf(a))) {   // rare: the scale from the finite elements
    drop_infinities16(v);
    a = block_max(amax16(v));
  }
  const uint32_t byte = scale_byte(a);
  *codes = codes16(v, pow2_of(254u - byte));
  return byte;
}

constexpr int kQUnroll = 2;
constexpr int kQBlocks = 256 / kUnitLanes;   // blocks of a CTA per step

// One block of 128 columns of a row per eight lanes, two blocks in flight.
// blockIdx.x counts groups of 64 blocks in row order; the division by the
// blocks of a row is taken in 32 bits from the group's own first row and block.
template <typename T>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const T* x, int64_t ld, bool wide,
                                                                int d, int nb, int64_t blocks,
                                                                uint8_t* codes, uint8_t* scales) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (kUnitLanes - 1);
  const int64_t first = (int64_t)blockIdx.x * (kQBlocks * kQUnroll);
  const int64_t row0 = first / nb;
  const uint32_t blk0 = (uint32_t)(first - row0 * nb);
  Raw<T> raw[kQUnroll];
  int64_t at[kQUnroll];   // element offset of this thread's codes, -1 past the end
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint32_t b = threadIdx.x / kUnitLanes + kQBlocks * u;
    const uint32_t r = (blk0 + b) / (uint32_t)nb;
    const int c = (int)(blk0 + b - r * nb) * 128 + lane * kUnit;
    const bool in = first + b < blocks && c < d;
    at[u] = in ? (row0 + r) * d + c : -1;
    if (in) raw[u].load(x + (row0 + r) * ld + c, wide);
    else raw[u].clear();
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    f2 v[8];
    raw[u].get(v);
    uint4 q;
    const uint32_t byte = quantize16(v, &q);
    if (at[u] >= 0) {
      *reinterpret_cast<uint4*>(codes + at[u]) = q;
      if (lane == 0) scales[first + threadIdx.x / kUnitLanes + kQBlocks * u] = (uint8_t)byte;
    }
  }
}

// One 128 x 128 block per CTA: eight lanes hold four of its rows.
template <typename T>
__global__ void __launch_bounds__(256, 2) fp8_quantize_block_kernel(const T* x, int64_t ld,
                                                                    bool wide, int64_t rows,
                                                                    int d, int nb, uint8_t* codes,
                                                                    uint8_t* scales) {
  __shared__ float red[2][8];
  pdl_wait();
  pdl_trigger();
  const int64_t br = blockIdx.x / nb;
  const int bc = (int)(blockIdx.x - br * nb);
  const int c = bc * 128 + (threadIdx.x & (kUnitLanes - 1)) * kUnit;
  const int64_t r0 = br * 128 + threadIdx.x / kUnitLanes;
  Raw<T> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + kQBlocks * i;
    if (r < rows && c < d) raw[i].load(x + r * ld + c, wide);
    else raw[i].clear();
  }
  f2 v[8];
  auto block_amax = [&](bool finite, float* slot) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      raw[i].get(v);
      if (finite) drop_infinities16(v);
      a = fmaxf(a, amax16(v));
    }
    a = warp_max(a);
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) a = fmaxf(a, slot[w]);
    return a;
  };
  float a = block_amax(false, red[0]);
  // the columns are unpacked again below: held as floats, they spill
#pragma unroll
  for (int i = 0; i < 4; ++i) raw[i].forget();
  const bool infinite = isinf(a);                  // rare, the same in every thread:
  if (infinite) a = block_amax(true, red[1]);      // the scale from the finite elements
  const uint32_t byte = scale_byte(a);
  if (threadIdx.x == 0) scales[(int64_t)blockIdx.x] = (uint8_t)byte;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + kQBlocks * i;
    raw[i].get(v);
    if (infinite) drop_infinities16(v);
    if (r < rows && c < d)
      *reinterpret_cast<uint4*>(codes + r * d + c) = codes16(v, pow2_of(254u - byte));
  }
}

template <typename T>
cudaError_t quantize_launch(const T* x, int64_t ld, int64_t rows, int d, int block_rows,
                            uint8_t* codes, uint8_t* scales, cudaStream_t stream) {
  const int nb = (d + 127) / 128;
  const bool wide = aligned32(x, ld, sizeof(T));
  if (block_rows == 1) {
    const int64_t blocks = rows * nb;
    const int64_t grid = (blocks + kQBlocks * kQUnroll - 1) / (kQBlocks * kQUnroll);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(fp8_quantize_rows_kernel<T>, dim3((unsigned)grid), dim3(256), 0, stream, x,
                      ld, wide, d, nb, blocks, codes, scales);
  }
  const int64_t grid = (rows + 127) / 128 * nb;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(fp8_quantize_block_kernel<T>, dim3((unsigned)grid), dim3(256), 0, stream, x,
                    ld, wide, rows, d, nb, codes, scales);
}

}  // namespace

cudaError_t launch_rmsnorm_fp8(int dtype, const NormParams& p, cudaStream_t stream) {
  if (p.T == 0) return cudaSuccess;
  const int e = dtype == CSA_BF16 ? 2 : 4;
  NormArgs a{p.T, p.d, (p.d + 127) / 128, p.x_ld, p.res_ld, p.sum_ld, p.x, p.residual,
             p.gain, p.eps, p.sum_out, static_cast<uint8_t*>(p.codes),
             static_cast<uint8_t*>(p.scales), aligned32(p.x, p.x_ld, e),
             aligned32(p.residual, p.res_ld, e), aligned32(p.sum_out, p.sum_ld, e)};
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
