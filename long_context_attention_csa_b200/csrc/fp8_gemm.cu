// Matrix product of E4M3 operands with a power-of-two scale per 128 columns
// (of one row of X, of 128 rows of W) on the block-scaled 5th-generation
// tensor cores:
//   Y[m, n] = sum_b 2^(ex[m,b] + ew[n/128,b]) sum_{k in block b} X[m,k] W[n,k],
// products and sums in float32 (kind::mxf8f6f4.block_scale; accumulators in
// TMEM), rounded once on the way out: bf16, float32, or E4M3 again with its own
// scales (the grouped projection's intermediate).
//
// Scales.  The MMA takes one scale byte per row and 32 columns; a block of 128
// columns is four MMAs (K = 32 each) that use the same byte.  So one TMEM word
// per row holds the bytes of four consecutive blocks (512 columns, a "chunk"),
// and the MMA descriptor's scale index picks block kb mod 4.  The scales stay
// in their natural layout in memory; one warp turns a chunk's words into the
// 512-byte tile of the tensor cores (row r's word at byte 16 (r mod 32) + 4
// (r div 32)) and tcgen05.cp brings it into TMEM, two chunks deep.
//
// Two kernels.  fp8_gemm_kernel: many rows, X rows on the MMA's M, 256 columns
// on N, persistent.  Bound by the tensor cores and, back to back, by the chip's
// power: 8192 x 8192 x 4096 to bf16 in 190 us alone (2.9 PFLOP/s), back to back in
// 215 to 231, by the card (2.4 to 2.5 PFLOP/s at 1.3 GHz).
// fp8_gemm_few_kernel: few rows, where the bytes of W are the bound: W rows on M,
// the few X rows on N, K split over a cluster.  1 x 8192 x 4096 in 8.5 us, 32 rows
// in 9.5 (W's 33.6 MB take 5 us of it, at the copy rate).
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "fp8.h"
#include "fp8_codes.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace csa {

namespace {

using namespace sm100;

constexpr int kBK = 128;          // columns per stage: one 128-byte swizzled row, one scale block
constexpr int kChunk = 4;         // scale blocks per TMEM word
constexpr int kTileM = 128;       // MMA M
constexpr int kTileA = kTileM * kBK;

// Rows of scale bytes [rows][blocks], read four bytes at a time.  `align`: rows
// start, and the first blocks asked for lie, on multiples of that many bytes (16,
// 4 or 1).
struct ScaleRows {
  const uint8_t *begin, *end;   // the whole tensor
  int blocks, align;

  // Scales b0 .. b0 + 4 N - 1 of a row, block b0 + i's in byte i: in rows that
  // start anywhere the aligned words around them, shifted.  Bytes of blocks past
  // the row's last hold no scale of the row.
  template <int N>
  __device__ __forceinline__ void get(int64_t row, int b0, uint32_t* w) const {
    const uint8_t* p = begin + row * blocks + b0;
    if (N == 4 && align >= 16) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (b0 < blocks) q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x; w[N > 1 ? 1 : 0] = q.y; w[N > 2 ? 2 : 0] = q.z; w[N > 3 ? 3 : 0] = q.w;
      return;
    }
    if (align >= 4) {
#pragma unroll
      for (int c = 0; c < N; ++c)
        w[c] = b0 + 4 * c < blocks ? reinterpret_cast<const uint32_t*>(p)[c] : 0u;
      return;
    }
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint8_t* lo = p - off;
    if (lo >= begin && lo + 4 * (N + 1) <= end) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(lo);
      uint32_t v[N + 1];
#pragma unroll
      for (int c = 0; c <= N; ++c) v[c] = q[c];
#pragma unroll
      for (int c = 0; c < N; ++c) w[c] = __funnelshift_r(v[c], v[c + 1], 8 * off);
    } else {   // at the tensor's ends
#pragma unroll
      for (int c = 0; c < N; ++c) {
        w[c] = 0;
#pragma unroll
        for (int i = 4 * c; i < 4 * c + 4; ++i)
          if (b0 + i < blocks) w[c] |= (uint32_t)p[i] << (8 * (i & 3));
      }
    }
  }
};

struct GemmArgs {
  Fp8GemmParams p;
  int kb_first, kb_n;    // scale blocks (stages) of K that the launch takes (many rows: all)
  int run;               // many rows, float32: blocks that one accumulator takes
  bool add;              // few rows: onto what Y holds (float32)
  ScaleRows xs, ws;      // scales of X and of all W
  int w_rblocks;         // scale block rows of one W
  int y_align;           // 32, 16 or 1: the boundaries that rows of Y start on
  int64_t tiles;
  int m_tiles, n_tiles;
};

// 2^e of the block and codes of 128 consecutive values of one row.
__device__ __forceinline__ void store_codes128(float* v, uint8_t* codes, uint8_t* scale) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 128; ++i) a = fmaxf(a, fabsf(v[i]));
  if (isinf(a)) {   // rare: the scale from the finite elements
    drop_infinities<128>(v);
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 128; ++i) a = fmaxf(a, fabsf(v[i]));
  }
  const uint32_t byte = scale_byte(a);
  *scale = (uint8_t)byte;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = codes4(v + 32 * q + 4 * i, byte);
    store_sector(codes + 32 * q, w);
  }
}

// N consecutive words of a row that starts on a 32-byte or a 16-byte boundary.
template <int N>
__device__ __forceinline__ void store_words(void* dst, const uint32_t* w, bool sectors) {
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    if (sectors) {
      store_sector(static_cast<uint32_t*>(dst) + 8 * q, w + 8 * q);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        static_cast<uint4*>(dst)[2 * q + i] = make_uint4(
            w[8 * q + 4 * i], w[8 * q + 4 * i + 1], w[8 * q + 4 * i + 2], w[8 * q + 4 * i + 3]);
    }
  }
}

// Thirty-two consecutive values of one row that starts on a 16-byte boundary (32
// with `sectors`), `n` of them inside Y.
template <int OUT, bool ADD>
__device__ __forceinline__ void store_row32(void* y, int64_t at, uint32_t* r, int n,
                                            bool sectors) {
  if constexpr (OUT == CSA_BF16) {
    bf16* dst = static_cast<bf16*>(y) + at;
    if (n >= 32) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      store_words<16>(dst, w, sectors);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n) dst[i] = __float2bfloat16_rn(__uint_as_float(r[i]));
    }
  } else {
    float* dst = static_cast<float*>(y) + at;
    if (n >= 32) {
      if constexpr (ADD) {
        float4 q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = reinterpret_cast<const float4*>(dst)[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[4 * i] = __float_as_uint(q[i].x + __uint_as_float(r[4 * i]));
          r[4 * i + 1] = __float_as_uint(q[i].y + __uint_as_float(r[4 * i + 1]));
          r[4 * i + 2] = __float_as_uint(q[i].z + __uint_as_float(r[4 * i + 2]));
          r[4 * i + 3] = __float_as_uint(q[i].w + __uint_as_float(r[4 * i + 3]));
        }
      }
      store_words<32>(dst, r, sectors);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < n) dst[i] = ADD ? dst[i] + __uint_as_float(r[i]) : __uint_as_float(r[i]);
    }
  }
}

// ---- many rows ----------------------------------------------------------------
//
// Persistent CTA pairs walk 256 x 256 tiles, n fastest (the pairs that run at
// once share their X tiles and all of W through L2).  One MMA spans the pair
// (cta_group::2): each CTA holds 128 rows of X and of the accumulator and half
// of the tile's W, so an SM reads 32 KB per K block instead of the 48 KB of a
// 128 x 256 tile of its own.
//   warp 0     TMA producer, a six-slot ring of K blocks (16 + 16 KB); both CTAs'
//              loads complete on rank 0's barrier
//   warp 1     TMEM owner; rank 0: single-thread MMA issuer for the pair
//   warps 2-3  scale tiles in shared memory, by turns
//   warps 4-7  epilogue, thread = row
// The two 256-column accumulators and the scales' 24 columns do not fit 512, so
// the accumulators share 24 columns: the epilogue reads those first and only
// then lets the next tile's MMAs begin.
constexpr int kN = 256;
constexpr int kStages = 6;
constexpr int kStage = kTileA + kN / 2 * kBK;   // bytes of one CTA
constexpr int kSfSlot = 512 + kN / 128 * 512;
constexpr int kOffSf = kStages * kStage;
constexpr int kGroup = 4;                       // chunks whose scales are handed over together
constexpr int kSfSlots = 3;                     // such groups in shared memory
constexpr int kOffBar = kOffSf + kSfSlots * kGroup * kSfSlot;
constexpr int kEpiWarps = 4;   // eight: 2.5% slower, their stores come in bursts
constexpr int kOffStage = kOffBar + 256;        // per epilogue warp: 32 rows of 16 words, padded
constexpr int kStagePitch = 17;
constexpr int kSmem = kOffStage + kEpiWarps * 32 * kStagePitch * 4;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kAcc1 = 232;               // second accumulator: columns 232 .. 487
constexpr uint32_t kSfCol = 488;              // scales: 2 x (4 + 8) columns
static_assert(kSmem + 1024 <= 232448, "shared memory budget");
static_assert(kGroup * kChunk == 16, "a group is what aligned rows load at once");

// Thirty-two columns of a warp's `rows` rows (lane = row), `n` of them inside Y,
// whose rows start anywhere: through shared memory, so that a store's lanes lie
// side by side, a row a store (two rows of bf16 pairs, where rows start on 4-byte
// boundaries: 4097 x 4098 x 1024 35.6 us, this way 28.7).  One warp a scheduler
// runs this, so its instructions count: sixteen a row were 52 us of a 3412 x 5471
// x 944 product.
template <bool WHOLE, typename E>
__device__ __forceinline__ void store_rows32(E* dst, int64_t ld, const uint32_t* stage, int rows,
                                             bool in, int shift) {
#pragma unroll
  for (int q = 0; q < 32; ++q, dst += ld) {
    const uint32_t w = stage[q * kStagePitch] >> shift;
    if (in && (WHOLE || q < rows)) *dst = (E)w;
  }
}

template <int OUT, bool ADD>
__device__ __forceinline__ void store_tile32(void* y, int64_t at, int64_t ld, const uint32_t* r,
                                             int rows, int n, uint32_t* stage, int lane) {
  __syncwarp();
  if constexpr (OUT == CSA_BF16) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      stage[lane * kStagePitch + i] =
          pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    __syncwarp();
    uint16_t* dst = static_cast<uint16_t*>(y) + at + lane;
    const uint32_t* src = stage + (lane >> 1);
    const int shift = (lane & 1) * 16;
    if (rows >= 32) store_rows32<true>(dst, ld, src, rows, lane < n, shift);
    else store_rows32<false>(dst, ld, src, rows, lane < n, shift);
  } else {
    // sixteen columns at a time: the warp's halves take even and odd rows
    const int half = lane >> 4, c = lane & 15;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h) __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) stage[lane * kStagePitch + i] = r[16 * h + i];
      __syncwarp();
      float* dst = static_cast<float*>(y) + at + half * ld + 16 * h + c;
      const uint32_t* src = stage + half * kStagePitch + c;
      const bool in = 16 * h + c < n;
      if constexpr (ADD) {
        float old[16];
#pragma unroll
        for (int q = 0; q < 16; ++q)
          old[q] = in && 2 * q + half < rows ? dst[2 * q * ld] : 0.f;
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (in && 2 * q + half < rows)
            dst[2 * q * ld] = old[q] + __uint_as_float(src[2 * q * kStagePitch]);
      } else {
#pragma unroll
        for (int q = 0; q < 32; q += 2, dst += 2 * ld) {
          const uint32_t w = src[q * kStagePitch];
          if (in && q + half < rows) *dst = __uint_as_float(w);
        }
      }
    }
  }
}

template <int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_w, GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kOffBar);   // [stages] operands landed (rank 0)
  uint64_t* empty = full + kStages;         // [stages] operands consumed
  uint64_t* sfull = empty + kStages;        // [slots] both CTAs' scale tiles written (rank 0)
  uint64_t* sempty = sfull + kSfSlots;      // [slots] the group's MMAs are done
  uint64_t* cdone = sempty + kSfSlots;      // [2] the chunk's MMAs are done (rank 0)
  uint64_t* tfull = cdone + 2;              // accumulator complete
  uint64_t* tfree = tfull + 1;              // the shared columns have been read (rank 0)
  uint64_t* drain = tfree + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t first = blockIdx.x >> 1, step = gridDim.x >> 1, tiles = (uint32_t)a.tiles;
  const Fp8GemmParams& p = a.p;
  const int run = OUT == CSA_F32 ? a.run : a.kb_n;   // a multiple of a group, or all

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&sfull[s], 2);
      mbar_init(&sempty[s], 1);
    }
    mbar_init(&cdone[0], 1);
    mbar_init(&cdone[1], 1);
    mbar_init(tfull, 1);
    mbar_init(tfree, 2 * kEpiWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  auto tile_of = [&](uint32_t u, int& z, int64_t& m0, int& n0) {
    const uint32_t r = u / (uint32_t)a.n_tiles, q = r / (uint32_t)a.m_tiles;
    m0 = (int64_t)(r - q * a.m_tiles) * (2 * kTileM) + rank * kTileM;   // this CTA's rows
    z = (int)q;
    n0 = (int)(u - r * a.n_tiles) * kN;
  };
  auto give_up = [&](unsigned where) {
    *abort_flag = 1;
    report(p.status, CSA_DEV_TIMEOUT, where);
  };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t u = first; u < tiles && ok; u += step) {
        int z, n0;
        int64_t m0;
        tile_of(u, z, m0, n0);
        for (int kb = 0; kb < a.kb_n; ++kb) {
          const uint32_t s = it % kStages;
          ok = !*abort_flag && mbar_wait(&empty[s], ((it / kStages) & 1u) ^ 1u);
          if (!ok) {
            give_up(0x801u);
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStage);
          const uint32_t bar = cluster_addr(&full[s], 0);
          uint8_t* dst = sm + s * kStage;
          tma_load_3d_pair(dst, &map_x, bar, z * p.x_koff + kb * kBK, (int32_t)m0, 0);
          tma_load_3d_pair(dst + kTileA, &map_w, bar, kb * kBK,
                           n0 + (int)rank * (kN / 2), z);
          ++it;
        }
      }
      // rank 0's commits have all arrived here before this CTA may exit, which
      // also says that every load has landed; after a timeout the loads in
      // flight are given a millisecond
      for (uint32_t i = it > kStages ? it - kStages : 0; i < it && ok; ++i)
        ok = mbar_wait(&empty[i % kStages], (i / kStages) & 1u);
      if (!ok)
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000ull;) {
        }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      uint32_t it = 0, ch = 0, gr = 0, n = 0;   // stages, chunks, groups, sums
      bool landed = false;                      // stage `it` is known to have landed
      int kr = 0;                               // the sum's first block
      for (uint32_t u = first; u < tiles; ++n) {
        if (*abort_flag || (n > 0 && !mbar_wait(tfree, (n - 1) & 1u))) {
          give_up(0x802u);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ((n & 1u) ? kAcc1 : 0u);
        const int end = min(kr + run, a.kb_n);
        bool ok = true;
        for (int kb = kr; kb < end; ++kb, ++it) {
          const uint32_t s = it % kStages, slot = gr % kSfSlots;
          const uint32_t sfa = tmem + kSfCol + (ch & 1u) * 12u, sfb = sfa + 4u;
          const int c = kb / kChunk % kGroup;   // chunk of its group
          ok = !*abort_flag;
          if (ok && kb % kChunk == 0) {
            // the MMAs of the chunk before last are done with these columns
            ok = (ch < 2 || mbar_wait(&cdone[ch & 1u], ((ch >> 1) - 1) & 1u)) &&
                 (c != 0 || mbar_wait_cluster(&sfull[slot], (gr / kSfSlots) & 1u));
            if (ok) {
              tc_fence_after();
              const uint32_t ss = smem_u32(sm + kOffSf + (slot * kGroup + c) * kSfSlot);
              tmem_cp_32x128b_x4_pair(sfa, smem_desc(ss, 16, 128, 0));
              tmem_cp_32x128b_x4_pair(sfb, smem_desc(ss + 512, 16, 128, 0));
              tmem_cp_32x128b_x4_pair(sfb + 4, smem_desc(ss + 1024, 16, 128, 0));
            }
          }
          ok = ok && (landed || mbar_wait(&full[s], (it / kStages) & 1u));
          if (!ok) {
            give_up(0x803u);
            break;
          }
          tc_fence_after();
          // Issuing four MMAs takes this thread about 340 of the 512 cycles that
          // they run for, so it looks at the next stage's barrier before it does.
          landed = mbar_test(&full[(it + 1) % kStages], ((it + 1) / kStages) & 1u);
          const uint32_t sa = smem_u32(sm + s * kStage);
          const uint32_t id = (uint32_t)kb & 3u;
          const uint32_t idesc = idesc_mxf8_e4m3(2 * kTileM, kN, id, id);
#pragma unroll
          for (int kk = 0; kk < kBK / 32; ++kk)
            mma_mxf8_ss_pair(d, smem_desc(sa + kk * 32, 16, 1024, 2),
                             smem_desc(sa + kTileA + kk * 32, 16, 1024, 2), idesc,
                             sfa | (id << 30), sfb | (id << 30), (kb > kr || kk > 0) ? 1u : 0u);
          mma_commit_pair(&empty[s]);
          const bool last = kb == end - 1;
          if (kb % kChunk == kChunk - 1 || last) {
            mma_commit_one_of_pair(&cdone[ch & 1u]);
            ++ch;
            if (c == kGroup - 1 || last) {
              mma_commit_pair(&sempty[slot]);
              ++gr;
            }
          }
        }
        if (!ok) break;
        mma_commit_pair(tfull);
        kr = end;
        if (OUT != CSA_F32 || end == a.kb_n) {
          kr = 0;
          u += step;
        }
      }
      mma_commit_one_of_pair(drain);
      mbar_wait(drain, 0);
    }
  } else if (warp < 4) {
    // scale tiles: a lane holds rows lane, lane + 32, ... of X; W's rows all
    // carry their 128-row block's word.  The loads, and the fence and arrival at
    // rank 0 (2400 cycles), each take longer than a chunk's MMAs (2048), so four
    // chunks go together (9472 x 2048 x 16384: one at a time 281 us, loads by fours
    // 253, both 225) and two warps take turns.
    uint32_t gr = 0;
    bool ok = true;
    for (uint32_t u = first; u < tiles && ok; u += step) {
      int z, n0;
      int64_t m0;
      tile_of(u, z, m0, n0);
      const int xb0 = z * (p.x_koff / 128);
      const int64_t wr = (int64_t)z * a.w_rblocks + n0 / 128;
      const bool second = n0 / 128 + 1 < a.w_rblocks;
      for (int kb = 0; kb < a.kb_n; kb += kGroup * kChunk, ++gr) {
        if ((gr & 1u) != (uint32_t)(warp & 1)) continue;   // the other warp's
        uint32_t x[4][kGroup], w[2][kGroup];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t m = m0 + 32 * i + lane;   // rows past the last: any row's scales
          a.xs.get<kGroup>(m < p.M ? m : p.M - 1, xb0 + kb, x[i]);
        }
        a.ws.get<kGroup>(wr, kb, w[0]);
        a.ws.get<kGroup>(second ? wr + 1 : wr, kb, w[1]);
        const uint32_t slot = gr % kSfSlots;
        ok = __all_sync(0xffffffffu, !*abort_flag && mbar_wait(&sempty[slot],
                                                               ((gr / kSfSlots) & 1u) ^ 1u));
        if (!ok) {
          give_up(0x804u);
          break;
        }
#pragma unroll
        for (int c = 0; c < kGroup; ++c) {
          uint4* dst =
              reinterpret_cast<uint4*>(sm + kOffSf + (slot * kGroup + c) * kSfSlot) + lane;
          dst[0] = make_uint4(x[0][c], x[1][c], x[2][c], x[3][c]);
          dst[32] = make_uint4(w[0][c], w[0][c], w[0][c], w[0][c]);
          dst[64] = make_uint4(w[1][c], w[1][c], w[1][c], w[1][c]);
        }
        fence_proxy_async_all();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(cluster_addr(&sfull[slot], 0));
      }
    }
    for (uint32_t i = gr > kSfSlots ? gr - kSfSlots : 0; i < gr && ok; ++i)   // the last commits
      ok = mbar_wait(&sempty[i % kSfSlots], (i / kSfSlots) & 1u);
  } else if (warp >= 4) {
    const int quarter = warp & 3;
    const uint32_t free_bar = cluster_addr(tfree, 0);
    uint32_t* stage =
        reinterpret_cast<uint32_t*>(sm + kOffStage) + quarter * 32 * kStagePitch;
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_exec(free_bar);
    };
    uint32_t n = 0;
    int kr = 0;
    for (uint32_t u = first; u < tiles; ++n) {
      int z, n0;
      int64_t m0;
      tile_of(u, z, m0, n0);
      const bool add = OUT == CSA_F32 && kr > 0;
      kr += run;
      if (OUT != CSA_F32 || kr >= a.kb_n) {
        kr = 0;
        u += step;
      }
      // warp-uniform decision: the TMEM loads below are warp-collective
      if (!__all_sync(0xffffffffu, !*abort_flag && mbar_wait(tfull, n & 1u))) {
        give_up(0x805u);
        break;
      }
      tc_fence_after();
      const int64_t row = m0 + quarter * 32 + lane;
      const int64_t at = row * p.y_ld + (int64_t)z * p.y_noff + n0;
      const bool odd = (n & 1u) != 0;
      const uint32_t base = tmem_addr(tmem, (uint32_t)(quarter * 32), odd ? kAcc1 : 0u);
      const bool live = row < p.M;
      if constexpr (OUT == kFp8Out) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int c0 = 128 * (odd ? i : 1 - i);   // the half with the shared columns first
          uint32_t r[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(base + c0 + q * 32, r + q * 32);
          tmem_ld_wait();
          if (i == 0) release();
          if (live && n0 + c0 < p.N)   // N is a multiple of 128
            store_codes128(reinterpret_cast<float*>(r), static_cast<uint8_t*>(p.y) + at + c0,
                           p.y_sf + (at + c0) / 128);
        }
      } else {
        // thirty-two columns at a time, the shared ones first, the next ones on
        // their way from TMEM while these are stored
        const int64_t mw = m0 + quarter * 32;   // this warp's first row
        const int rows = (int)(p.M - mw < 32 ? p.M - mw : 32);
        auto col = [&](int i) { return odd ? 32 * i : kN - 32 - 32 * i; };
        uint32_t r[2][32];
        auto store = [&](int cc, uint32_t* r, auto adds) {
          constexpr bool kAdd = decltype(adds)::value;
          const int n_in = p.N - n0 - cc;
          if (n_in <= 0) return;
          if (a.y_align < 16)
            store_tile32<OUT, kAdd>(p.y, at - lane * p.y_ld + cc, p.y_ld, r, rows, n_in, stage,
                                    lane);
          else if (live)
            store_row32<OUT, kAdd>(p.y, at + cc, r, n_in, a.y_align >= 32);
        };
        auto store_all = [&](auto adds) {
#pragma unroll 1
          for (int i = 0; i < kN / 32; i += 2) {
            tmem_ld32(base + col(i + 1), r[1]);
            store(col(i), r[0], adds);
            tmem_ld_wait();
            if (i + 2 < kN / 32) tmem_ld32(base + col(i + 2), r[0]);
            store(col(i + 1), r[1], adds);
            tmem_ld_wait();
          }
        };
        tmem_ld32(base + col(0), r[0]);
        tmem_ld_wait();
        release();
        if (OUT == CSA_F32 && add) store_all(std::integral_constant<bool, OUT == CSA_F32>{});
        else store_all(std::false_type{});
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the pair's MMAs and arrivals are over
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---- few rows -------------------------------------------------------------------
//
// One CTA: 128 rows of W against up to NT rows of X over its share of K.  A
// cluster's CTAs hold the shares of one tile; each sends its float32 partials of
// X row t to CTA t mod SPLIT, which adds them in rank order (the sum's order does
// not depend on timing) and writes Y.  With one share, a bf16 or float32 tile
// goes from TMEM to Y, a lane for each column.
//   warp 0     TMA producer
//   warp 1     TMEM owner, single-thread MMA issuer
//   warp 2     scale tiles
//   all four   the accumulator, lane = row of W = column of Y
template <int NT, bool SUM>   // SUM: partials are gathered in shared memory
struct Few {
  static constexpr int stage = kTileA + NT * kBK;
  static constexpr int stages = NT <= 16 ? 5 : NT <= 32 ? 4 : NT <= 64 ? (SUM ? 3 : 4)
                                : SUM ? 4 : 3;
  static constexpr int off_sf = stages * stage;
  static constexpr int off_bar = off_sf + 2 * 1024;
  static constexpr int off_part = off_bar + 256;
  static constexpr int smem = off_part + (SUM ? NT * kTileM * 4 : 0);
  static constexpr uint32_t cols = NT <= 16 ? 32 : NT <= 32 ? 64 : NT <= 64 ? 128 : 256;
  static constexpr uint32_t sf_col = NT;   // after the accumulator: 2 x (4 + 4) columns
  static_assert(smem + 1024 <= 232448, "shared memory budget");
};

// Codes need the largest of 128 columns of a row, so where one CTA has the whole
// sum and 128 rows, X takes the MMA's M and a lane holds its row's columns (128
// rows gathered in shared memory and reduced a warp a row: 12 us a CTA).
template <int NT, int SPLIT, int OUT>
constexpr bool few_rows_on_m = NT == 128 && SPLIT == 1 && OUT == kFp8Out;

template <int NT, int SPLIT, int OUT>
__global__ void __launch_bounds__(128)
    fp8_gemm_few_kernel(const __grid_constant__ CUtensorMap map_x,
                        const __grid_constant__ CUtensorMap map_w, GemmArgs a) {
  constexpr bool kRows = few_rows_on_m<NT, SPLIT, OUT>;
  constexpr bool kSum = (SPLIT > 1 || OUT == kFp8Out) && !kRows;
  using L = Few<NT, kSum>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::off_bar);
  uint64_t* empty = full + L::stages;
  uint64_t* sfull = empty + L::stages;
  uint64_t* sempty = sfull + 2;
  uint64_t* done = sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Fp8GemmParams& p = a.p;
  const int rank = (int)(blockIdx.x % SPLIT);
  const int64_t u = blockIdx.x / SPLIT;
  const int nt = (int)(u % a.n_tiles);
  const int64_t m0 = (u / a.n_tiles) % a.m_tiles * NT;
  const int z = (int)(u / a.n_tiles / a.m_tiles);
  const int n0 = nt * kTileM;
  // this CTA's chunks of K
  const int chunks = (a.kb_n + kChunk - 1) / kChunk;
  const int c0 = (int)((int64_t)chunks * rank / SPLIT);
  const int c1 = (int)((int64_t)chunks * (rank + 1) / SPLIT);
  const int kb0 = c0 * kChunk, kb1 = min(c1 * kChunk, a.kb_n);

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&map_x);
    tma_prefetch_desc(&map_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (SPLIT > 1) cluster_arrive();   // this CTA runs: its shared memory may be written
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  auto give_up = [&](unsigned where) {
    *abort_flag = 1;
    report(p.status, CSA_DEV_TIMEOUT, where);
  };

  if (warp == 0) {
    if (elect_one()) {
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t s = it % L::stages;
        if (*abort_flag || !mbar_wait(&empty[s], ((it / L::stages) & 1u) ^ 1u)) {
          give_up(0x811u);
          break;
        }
        mbar_arrive_expect_tx(&full[s], L::stage);
        uint8_t* dst = sm + s * L::stage;
        const int k = (a.kb_first + kb) * kBK;
        tma_load_3d(dst, &map_w, &full[s], k, n0, z);
        tma_load_3d(dst + kTileA, &map_x, &full[s], z * p.x_koff + k, (int32_t)m0, 0);
        ++it;
      }
      for (uint32_t i = it > L::stages ? it - L::stages : 0; i < it; ++i)
        mbar_wait(&full[i % L::stages], (i / L::stages) & 1u);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      uint32_t it = 0, ch = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t s = it % L::stages, slot = ch & 1u;
        const uint32_t sfa = tmem + L::sf_col + slot * 8u, sfb = sfa + 4u;
        bool ok = !*abort_flag;
        if (ok && (kb & 3) == 0) {
          ok = mbar_wait(&sfull[slot], (ch >> 1) & 1u);
          if (ok) {
            tc_fence_after();
            const uint32_t ss = smem_u32(sm + L::off_sf + slot * 1024);
            tmem_cp_32x128b_x4(kRows ? sfb : sfa, smem_desc(ss, 16, 128, 0));
            tmem_cp_32x128b_x4(kRows ? sfa : sfb, smem_desc(ss + 512, 16, 128, 0));
          }
        }
        if (!ok || !mbar_wait(&full[s], (it / L::stages) & 1u)) {
          give_up(0x812u);
          break;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(sm + s * L::stage);
        const uint32_t id = (uint32_t)kb & 3u;
        const uint32_t idesc = idesc_mxf8_e4m3(kTileM, NT, id, id);
#pragma unroll
        for (int kk = 0; kk < kBK / 32; ++kk)
          mma_mxf8_ss(tmem, smem_desc(sa + (kRows ? kTileA : 0) + kk * 32, 16, 1024, 2),
                      smem_desc(sa + (kRows ? 0 : kTileA) + kk * 32, 16, 1024, 2), idesc,
                      sfa | (id << 30),
                      sfb | (id << 30), (kb > kb0 || kk > 0) ? 1u : 0u);
        mma_commit(&empty[s]);
        if ((kb & 3) == 3) {
          mma_commit(&sempty[slot]);
          ++ch;
        }
      }
      mma_commit(done);
    }
  } else if (warp == 2) {
    const int xb0 = z * (p.x_koff / 128) + a.kb_first;
    const int64_t wr = (int64_t)z * a.w_rblocks + nt;
    constexpr int kMine = NT < 32 ? 1 : NT / 32;   // rows of this lane
    uint32_t x[4] = {0u, 0u, 0u, 0u}, w;
    auto load = [&](int kb) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int64_t m = m0 + 32 * i + lane;   // rows past the last: any row's scales
        a.xs.get<1>(m < p.M ? m : p.M - 1, xb0 + kb, &x[i]);
      }
      a.ws.get<1>(wr, a.kb_first + kb, &w);
    };
    load(kb0);
    uint32_t ch = 0;
    for (int kb = kb0; kb < kb1; kb += kChunk, ++ch) {
      const uint32_t slot = ch & 1u;
      if (!__all_sync(0xffffffffu,
                      !*abort_flag && mbar_wait(&sempty[slot], ((ch >> 1) & 1u) ^ 1u))) {
        give_up(0x813u);
        break;
      }
      uint4* dst = reinterpret_cast<uint4*>(sm + L::off_sf + slot * 1024) + lane;
      dst[0] = make_uint4(w, w, w, w);
      dst[32] = make_uint4(x[0], x[1], x[2], x[3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sfull[slot]);
      if (kb + kChunk < kb1) load(kb + kChunk);   // the fence would wait for it
    }
  }
  __syncwarp();
  // `done` follows every MMA, so every landed stage has been read
  if (!__all_sync(0xffffffffu, mbar_wait(done, 0))) give_up(0x814u);
  if (SPLIT > 1) cluster_wait();
  else __syncthreads();
  tc_fence_after();
  const uint32_t base = tmem_addr(tmem, (uint32_t)(warp * 32), 0);
  constexpr int step = NT < 32 ? NT : 32;
  const int rows = (int)(p.M - m0 < NT ? p.M - m0 : NT);
  const int col = warp * 32 + lane;
  const int64_t y0 = m0 * p.y_ld + (int64_t)z * p.y_noff + n0;
  if constexpr (kRows) {
    uint32_t r[128];
#pragma unroll
    for (int q = 0; q < 4; ++q) tmem_ld32(base + q * 32, r + q * 32);
    tmem_ld_wait();
    const int64_t at = y0 + col * p.y_ld;   // col: this lane's row of X
    if (col < rows)   // N is a multiple of 128
      store_codes128(reinterpret_cast<float*>(r), static_cast<uint8_t*>(p.y) + at,
                     p.y_sf + at / 128);
  }
  float* part = reinterpret_cast<float*>(sm + L::off_part);   // [row t / SPLIT][rank][128]
  uint32_t to[SPLIT];
#pragma unroll
  for (int j = 0; j < SPLIT; ++j)
    to[j] = cluster_addr(part + rank * kTileM + col, (uint32_t)j);
  constexpr int kElem = OUT == CSA_BF16 ? 2 : 4;
  const bool inside = n0 + col < p.N;   // this lane's column, where it goes straight to Y
  const int64_t pitch = p.y_ld * kElem;
  char* dst = static_cast<char*>(p.y) + (y0 + col) * kElem;
#pragma unroll 1
  for (int t0 = 0; t0 < rows && !kRows; t0 += step) {
    uint32_t r[step];
    if constexpr (step == 32) tmem_ld32(base + t0, r);
    else tmem_ld16(base + t0, r);
    if (OUT == CSA_F32 && !kSum && a.add) {
      float old[step];
#pragma unroll
      for (int i = 0; i < step; ++i)
        old[i] = inside && t0 + i < rows ? *reinterpret_cast<const float*>(dst + i * pitch) : 0.f;
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < step; ++i) r[i] = __float_as_uint(old[i] + __uint_as_float(r[i]));
    }
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < step; ++i) {
      const int t = t0 + i;
      const float v = __uint_as_float(r[i]);
      if constexpr (kSum) {
        if (t >= rows) continue;
        // step is a multiple of SPLIT, so t mod SPLIT is i mod SPLIT
        dsmem_st_f32(to[i % SPLIT] + (uint32_t)(t - i % SPLIT) * (kTileM * 4), v);
      } else if constexpr (!kRows) {
        if (inside && t < rows) {
          if (OUT == CSA_BF16) *reinterpret_cast<bf16*>(dst) = __float2bfloat16_rn(v);
          else *reinterpret_cast<float*>(dst) = v;
        }
        dst += pitch;
      }
    }
  }
  tc_fence_before();
  if (SPLIT > 1) cluster_sync();   // every partial has arrived
  else __syncthreads();
  if constexpr (kSum) {
    // a warp adds one X row's partials, four columns a lane: side by side where
    // Y's rows take 8- or 16-byte stores, else 32 apart
    const bool vec = OUT == kFp8Out || a.y_align >= 16;
#pragma unroll 2
    for (int k = warp; k * SPLIT + rank < rows; k += 4) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < SPLIT; ++j) {
        const float* src = part + (k * SPLIT + j) * kTileM;
        if (vec) {
          const float4 q = *reinterpret_cast<const float4*>(src + 4 * lane);
          v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += src[lane + 32 * i];
        }
      }
      const int64_t row = y0 + (int64_t)(k * SPLIT + rank) * p.y_ld;
      if constexpr (OUT == kFp8Out) {   // N, and rows of Y, are multiples of 128
        drop_infinities<4>(v);
        const float am = warp_max(fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])),   // skips NaN
                                              fmaxf(fabsf(v[2]), fabsf(v[3]))), 0.f));
        const uint32_t byte = scale_byte(am);
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row + 4 * lane) =
            codes4(v, byte);
        if (lane == 0) p.y_sf[row / 128] = (uint8_t)byte;
      } else {
        const int n = p.N - n0;   // columns of Y from this tile's first on
        const bool whole = vec && 4 * lane + 4 <= n;
        if (OUT == CSA_BF16) {
          bf16* dst = static_cast<bf16*>(p.y) + row;
          if (whole)
            *reinterpret_cast<uint2*>(dst + 4 * lane) =
                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = vec ? 4 * lane + i : lane + 32 * i;
            if (!whole && c < n) dst[c] = __float2bfloat16_rn(v[i]);
          }
        } else {
          float* dst = static_cast<float*>(p.y) + row;
          if (a.add) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = vec ? 4 * lane + i : lane + 32 * i;
              if (c < n) v[i] += dst[c];
            }
          }
          if (whole) store_vec(dst + 4 * lane, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = vec ? 4 * lane + i : lane + 32 * i;
            if (!whole && c < n) dst[c] = v[i];
          }
        }
      }
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::cols);
  }
}

// Lets `kernel` take `smem` bytes on the current device; asked once per device.
template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...), int smem, std::atomic<bool>* done) {
  const int dev = current_device();
  if (dev >= 0 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev >= 0) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// A launch in clusters of `cluster` CTAs with programmatic stream serialization.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[2];
  ClusterLaunch(int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream) {
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
  }
};

// The tensor core cuts off what does not fit its accumulator at every MMA, always
// towards zero.  Relative to the result, 2048 x 1024 x K, operands of mean zero /
// of one sign (whose cuts all add up): K = 8192 4.9e-7 / 3.9e-6, 16384 1.2e-6 /
// 9.9e-6, 65536 7.7e-6 / 6.0e-5; a float32 product of the same K = 8192 operands on
// the CUDA cores 1.3e-7 / 4.3e-7.  So for float32 results no accumulator takes more
// than 8192 columns, and the parts are added in Y with rounding: many rows within a
// launch, a tile's sums one after the other (2048 x 2048 x 16384 55 us, a launch a
// part 77, in bf16 46), few rows a launch a part, where K outgrows the shares.
// Parts of 4096 columns would halve the cut and take a quarter longer (8192 x 4096 x
// 8192: 201 us, 254; of 2048, 372).
constexpr int kSumBlocks = 8192 / kBK;
constexpr int kEven = kGroup * kChunk;   // parts start where scales load by the group

// One launch, or one a part.  The parts are of even length: a short last one would
// leave shares without a chunk, and so without a sum.
template <typename Launch>
cudaError_t in_parts(GemmArgs& a, int split, Launch launch) {
  const int all = a.kb_n, groups = (all + kEven - 1) / kEven;
  const int parts =
      a.p.out == CSA_F32 ? (all + kSumBlocks * split - 1) / (kSumBlocks * split) : 1;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < parts && e == cudaSuccess; ++i) {
    const int end = (int)((int64_t)groups * (i + 1) / parts) * kEven;
    a.kb_first = (int)((int64_t)groups * i / parts) * kEven;
    a.kb_n = (end < all ? end : all) - a.kb_first;
    a.add = i > 0;
    e = launch(a);
    if (e == cudaSuccess) ++*a.p.launches;
  }
  a.kb_n = all;
  return e;
}

template <int OUT>
cudaError_t launch_many(GemmArgs& a, cudaStream_t stream) {
  const Fp8GemmParams& p = a.p;
  a.m_tiles = (int)((p.M + 2 * kTileM - 1) / (2 * kTileM));
  a.n_tiles = (p.N + kN - 1) / kN;
  a.tiles = (int64_t)p.Z * a.m_tiles * a.n_tiles;
  if (a.tiles > 0x7fffffffLL) return cudaErrorInvalidValue;   // no memory holds such a Y
  CUtensorMap mx, mw;
  if (!make_map_u8_3d(&mx, p.x, (uint64_t)p.x_cols, (uint64_t)p.M, 1, kBK, kTileM) ||
      !make_map_u8_3d(&mw, p.w, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.Z, kBK, kN / 2))
    return cudaErrorInvalidValue;
  const int smem = kSmem + 1024;
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = allow_smem(fp8_gemm_kernel<OUT>, smem, done);
  if (e != cudaSuccess) return e;
  const int64_t pairs = sm_count() / 2;
  ClusterLaunch l(2 * (a.tiles < pairs ? a.tiles : pairs), kThreads, smem, 2, stream);
  a.run = kSumBlocks;
  e = cudaLaunchKernelEx(&l.cfg, fp8_gemm_kernel<OUT>, mx, mw, a);
  if (e == cudaSuccess) ++*p.launches;
  return e;
}

template <int NT, int SPLIT, int OUT>
struct FewKernel {
  static constexpr bool sum = (SPLIT > 1 || OUT == kFp8Out) && !few_rows_on_m<NT, SPLIT, OUT>;
  static constexpr int smem = Few<NT, sum>::smem + 1024;

  static cudaError_t allow() {
    static std::atomic<bool> done[kMaxDevices];
    return allow_smem(fp8_gemm_few_kernel<NT, SPLIT, OUT>, smem, done);
  }
  // Clusters that run at once on the current device (asked once per device): a
  // cluster lies within a GPC, so there are fewer than the SMs would hold.  The
  // answer is for one CTA on an SM (74, 33 and 15 clusters of two, four and eight);
  // with two, odd SMs of a GPC pair up, which makes two more (32 x N x 4096 by
  // fours: 68 tiles 9.9 us, 72 14.3; by eights: 32 tiles 10.1, 34 14.3).
  static int clusters() {
    constexpr int per_sm = 2 * (smem + 1024) <= 233472 ? 2 : 1;
    static std::atomic<int> known[kMaxDevices];
    const int dev = current_device();
    int n = dev >= 0 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    ClusterLaunch l(SPLIT, 128, smem, SPLIT, nullptr);
    if (allow() != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fp8_gemm_few_kernel<NT, SPLIT, OUT>, &l.cfg) !=
            cudaSuccess ||
        n <= 0) {
      cudaGetLastError();
      return per_sm * sm_count() / SPLIT * 3 / 4;
    }
    if (per_sm == 2) n = 2 * n + 2;
    if (dev >= 0) known[dev].store(n, std::memory_order_relaxed);
    return n;
  }
  static cudaError_t launch(GemmArgs& a, cudaStream_t stream) {
    const Fp8GemmParams& p = a.p;
    CUtensorMap mx, mw;
    if (!make_map_u8_3d(&mx, p.x, (uint64_t)p.x_cols, (uint64_t)p.M, 1, kBK, NT) ||
        !make_map_u8_3d(&mw, p.w, (uint64_t)p.K, (uint64_t)p.N, (uint64_t)p.Z, kBK, kTileM))
      return cudaErrorInvalidValue;
    const cudaError_t e = allow();
    if (e != cudaSuccess) return e;
    ClusterLaunch l(a.tiles * SPLIT, 128, smem, SPLIT, stream);
    return in_parts(a, SPLIT, [&](const GemmArgs& part) {
      return cudaLaunchKernelEx(&l.cfg, fp8_gemm_few_kernel<NT, SPLIT, OUT>, mx, mw, part);
    });
  }
};

template <int NT, int OUT>
cudaError_t launch_few(GemmArgs& a, cudaStream_t stream) {
  const Fp8GemmParams& p = a.p;
  a.m_tiles = (int)((p.M + NT - 1) / NT);
  a.n_tiles = (p.N + kTileM - 1) / kTileM;
  a.tiles = (int64_t)p.Z * a.m_tiles * a.n_tiles;
  if (a.tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  // K shares: as many as run at once (57 x 9216 x 10752, 72 tiles: clusters of four
  // did not all, 30 us; of two 23), of two chunks or more unless fewer than
  // 48 CTAs would run (1 x 4096 x 4096: four shares 4.7 us, eight 5.2; 1 x 1024 x
  // 4096: four 4.4, eight 3.7)
  const int chunks = (a.kb_n + kChunk - 1) / kChunk;
  auto more = [&](int split) {
    return split * 2 <= chunks && (split * 4 <= chunks || a.tiles * split < 48);
  };
  if (!more(1) || a.tiles > FewKernel<NT, 2, OUT>::clusters())
    return FewKernel<NT, 1, OUT>::launch(a, stream);
  if (!more(2) || a.tiles > FewKernel<NT, 4, OUT>::clusters())
    return FewKernel<NT, 2, OUT>::launch(a, stream);
  if (!more(4) || a.tiles > FewKernel<NT, 8, OUT>::clusters())
    return FewKernel<NT, 4, OUT>::launch(a, stream);
  return FewKernel<NT, 8, OUT>::launch(a, stream);
}

template <int OUT>
cudaError_t launch(GemmArgs& a, cudaStream_t stream) {
  const Fp8GemmParams& p = a.p;
  const int64_t sms = sm_count();
  auto tiles = [&](int64_t rows, int64_t cols) {
    return (int64_t)p.Z * ((p.M + rows - 1) / rows) * ((p.N + cols - 1) / cols);
  };
  // Many rows: the pairs' 256 x 256 tiles pay from about two thirds of a wave of K =
  // 4096, or as much work in more waves.  Us between captured launches, the pairs /
  // 128-row / 64-row tiles of the few-row kernel (128 columns each):
  //    768 x 4096 x 4096   20.7 / 21.3 / 28.4
  //   4096 x 2048 x 1024   14.2 / 16.1 / 23.6
  //   2048 x 2048 x 2048   13.4 / 12.3 / 18.3
  //    512 x 4096 x 4096   16.0 / 15.5 / 13.8
  // Where 128 x 128 tiles would fit the SMs at once the few-row kernel, which then
  // takes 64 rows, uses more of them,
  //    300 x 5000 x 8192   27.1 / 27.1 / 23.4
  //    512 x 4096 x 8192   27.5 / 29.4 / 23.7
  //    700 x 3000 x 16384  46.1 / 51.5 / 45.6
  //    256 x 8192 x 8192   27.2 / 30.7 / 26.4
  // unless one row of pairs takes a longer K,
  //    256 x 8192 x 16384  45.3 / 55.8 / 50.3
  // or Y are codes (a projection of 36 pairs, K = 8192: pairs 42.0, few 43.6).
  const int64_t pairs = tiles(2 * kTileM, kN), t128 = tiles(128, kTileM);
  const bool one_wave = OUT != kFp8Out && t128 <= sms && (p.M > 2 * kTileM || a.kb_n <= 64);
  if (p.M > 128 && pairs >= 32 && pairs * a.kb_n >= (2 * pairs > sms ? 1024 : 1536) && !one_wave)
    return launch_many<OUT>(a, stream);
  if (p.M <= 16) return launch_few<16, OUT>(a, stream);
  // Few rows, smaller row tiles: more SMs share the epilogue, at the price of reading
  // W again.  32 rows where K <= 1024 and the tiles fit the SMs at once (100 x 256 x
  // 640: 4.4 us, 128-row tiles 6.5); 64 rows where K <= 2048 and they do (777 x 1111 x
  // 1040: 5.9, 7.9), where there are few at any K (300 x 300 x 8192: 6.0, 7.3), and
  // where 128-row tiles would run one to an SM on 60% of the SMs or more: the 64-row
  // ones run two, with twice the stages in flight (512 x 4096 x 4096: 13.8, 15.5).
  // Else 128 rows (96 x 4096 x 4096: 8.7, 64-row tiles 9.1).
  if (p.M <= 32 || (a.kb_n <= 8 && tiles(32, kTileM) <= sms))
    return launch_few<32, OUT>(a, stream);
  const int64_t t64 = tiles(64, kTileM);
  if (p.M > 64 && OUT == kFp8Out) return launch_few<128, OUT>(a, stream);
  if (p.M <= 64 || t64 <= 32 || (a.kb_n <= 16 && t64 <= sms) ||
      (5 * t128 > 3 * sms && t128 <= sms && t64 <= 2 * sms))
    return launch_few<64, OUT>(a, stream);
  return launch_few<128, OUT>(a, stream);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams& p, cudaStream_t stream) {
  if (p.M == 0 || p.N == 0) return cudaSuccess;
  GemmArgs a{};
  a.p = p;
  a.kb_n = (p.K + kBK - 1) / kBK;
  a.w_rblocks = (p.N + 127) / 128;
  auto align = [](uintptr_t bits) { return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1; };
  const int xb = (p.x_cols + 127) / 128;
  a.xs = {p.x_sf, p.x_sf + p.M * xb, xb,
          align(reinterpret_cast<uintptr_t>(p.x_sf) | (uintptr_t)xb |
                (uintptr_t)(p.x_koff / 128))};
  a.ws = {p.w_sf, p.w_sf + (int64_t)p.Z * a.w_rblocks * a.kb_n, a.kb_n,
          align(reinterpret_cast<uintptr_t>(p.w_sf) | (uintptr_t)a.kb_n)};
  const int64_t e = p.out == CSA_BF16 ? 2 : 4;
  const uintptr_t y = reinterpret_cast<uintptr_t>(p.y) | (uintptr_t)(p.y_ld * e);
  a.y_align = y % 32 == 0 ? 32 : y % 16 == 0 ? 16 : 1;
  switch (p.out) {
    case CSA_BF16: return launch<CSA_BF16>(a, stream);
    case CSA_F32: return launch<CSA_F32>(a, stream);
    default: return launch<kFp8Out>(a, stream);
  }
}

}  // namespace csa
