// lm_head_scaled.cuh -- LM-head logits in 8-bit floating point with a scale for each block
// of 128, and the quantisers that bring rows and weights into that form:
//     logits[r, v] = sum over blocks t of  hs[t, r] * ws[v / 128, t] * (sum of h[r, k] w[v, k], k in block t)
// with h, w in e4m3 and hs, ws in fp32.
//
// A product of two e4m3 values is exact in fp32, and the tensor core sums a block's 128 of
// them in fp32 (measured against fp64: relative error 1.3e-8 on normal data, as an fp32 FMA
// chain); the blocks are scaled and summed in fp32 registers.
//
// Two forms, by the number of tree rows (times of the product alone, without the quantiser):
//   up to 16 rows    swap-AB like lm_head.cuh: 128 vocabulary rows are the MMA's M, the tree
//                    rows its N; the weight streams once and bounds it (32000 x 4096: 1 row
//                    23.0 us, 5.7 TB/s, the other form 30.6; 16 rows 24.6 and 28.0).  A thread
//                    has 8 accumulators: 16 rows are all that it takes;
//   more             tree rows as M (128 a tile), one or two blocks of 128 vocabulary rows
//                    as N, so that a thread's accumulators all share one scale (32 rows 24.6).
// In both, per K block one 128-deep MMA chain goes into a fresh TMEM buffer and eight
// epilogue warps scale it into their register accumulators while the next blocks' MMAs run.
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace eagle {

constexpr int kScBlock = 128;        // elements that share a scale; vocabulary rows per CTA
constexpr int kScThreads = 32 * 10;  // TMA, MMA, 8 epilogue warps
constexpr int kScEpiWarps = 8;
constexpr int kScFewRows = 16;       // rows up to which the weight is the MMA's M

// 2^e and 2^-e for the smallest e >= -126 with amax <= 448 * 2^e: amax = m * 2^k with
// 1 <= m < 2, and 448 = 1.75 * 2^8, so e = k - 8 while m <= 1.75 and k - 7 above.  The
// scale is a power of two, so x * 2^-e is exact and the only rounding is the one to e4m3.
// A block that holds an infinity or a NaN gets a NaN scale: it stays visible.
__device__ __forceinline__ float2 block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = static_cast<int>(u >> 23) - 127;
  if (k == 128) return make_float2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
  int e = k - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : e;
  return make_float2(__uint_as_float(static_cast<uint32_t>(e + 127) << 23),
                     __uint_as_float(static_cast<uint32_t>(127 - e) << 23));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// |x| with NaN kept the largest: magnitudes compare as their bit patterns, and every NaN's
// is above infinity's.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&f)[4]);
template <>
__device__ __forceinline__ void load4<float>(const float* p, float (&f)[4]) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  f[0] = w.x;
  f[1] = w.y;
  f[2] = w.z;
  f[3] = w.w;
}
template <>
__device__ __forceinline__ void load4<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(w.x << 16);
  f[1] = __uint_as_float(w.x & 0xFFFF0000u);
  f[2] = __uint_as_float(w.y << 16);
  f[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// 1 x 128 blocks: one warp per block, four elements a lane.  Each element is read once.
// Latency-bound: a thread has one load in flight, then the block's maximum, then its store.
// 512 rows of 4096 in bf16: 5.1 us, 1.2 TB/s (6.8 from a cold cache, at 8 % of HBM); one row
// 1.4 us.
template <typename T>
__global__ void __launch_bounds__(128)
    quantize_rows_kernel(const T* __restrict__ x, uint8_t* __restrict__ x8, float* __restrict__ scales, int rows,
                         int cols, int kblocks, int ldm) {
  const int64_t blk = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  pdl_launch_dependents();  // the GEMM that reads this waits for the whole grid
  if (blk >= static_cast<int64_t>(rows) * kblocks) return;
  const int r = static_cast<int>(blk / kblocks), kb = static_cast<int>(blk % kblocks);
  const int c = kb * kScBlock + lane * 4;
  const bool in = c < cols;  // cols is a multiple of 16
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  if (in) load4(x + static_cast<size_t>(r) * cols + c, f);
  uint32_t m = max(max(abs_bits(f[0]), abs_bits(f[1])), max(abs_bits(f[2]), abs_bits(f[3])));
  m = __reduce_max_sync(0xffffffffu, m);
  const float2 s = block_scale(__uint_as_float(m));
  if (in)
    *reinterpret_cast<uint32_t*>(x8 + static_cast<size_t>(r) * cols + c) =
        pack_e4m3x4(f[0] * s.y, f[1] * s.y, f[2] * s.y, f[3] * s.y);
  if (lane == 0) scales[static_cast<size_t>(kb) * ldm + r] = s.x;
}

// 128 x 128 blocks: one CTA per block, a warp per 16 of its rows, the block kept in
// registers between its maximum and its rounding.  Run when a weight is loaded.  128256 x 4096:
// fp32 378 us, 6.9 TB/s, HBM-bound; bf16 321 us, 4.9 TB/s, with loads of 8 bytes a lane.
template <typename T>
__global__ void __launch_bounds__(256)
    quantize_blocks_kernel(const T* __restrict__ w, uint8_t* __restrict__ w8, float* __restrict__ scales, int rows,
                           int cols, int kblocks) {
  __shared__ uint32_t part[8];
  const int kb = static_cast<int>(blockIdx.x % kblocks), vb = static_cast<int>(blockIdx.x / kblocks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = kb * kScBlock + lane * 4;
  float f[16][4];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int r = vb * kScBlock + warp * 16 + j;
    f[j][0] = f[j][1] = f[j][2] = f[j][3] = 0.f;
    if (r < rows && c < cols) load4(w + static_cast<size_t>(r) * cols + c, f[j]);
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    m = max(m, max(max(abs_bits(f[j][0]), abs_bits(f[j][1])), max(abs_bits(f[j][2]), abs_bits(f[j][3]))));
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) part[warp] = m;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, part[j]);
  const float2 s = block_scale(__uint_as_float(m));
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int r = vb * kScBlock + warp * 16 + j;
    if (r < rows && c < cols)
      *reinterpret_cast<uint32_t*>(w8 + static_cast<size_t>(r) * cols + c) =
          pack_e4m3x4(f[j][0] * s.y, f[j][1] * s.y, f[j][2] * s.y, f[j][3] * s.y);
  }
  if (threadIdx.x == 0) scales[static_cast<size_t>(vb) * kblocks + kb] = s.x;
}

// ------------------------------------------------------------------ GEMM

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f8f6f4 (e4m3 inputs, fp32 accumulation), K = 32.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: fp32 D, e4m3 A and B (format 0), both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
struct ScaledParams {
  float* logits;
  const float* hs;  // [KB, ldm]
  const float* ws;  // [ceil(V / 128), KB]
  int32_t M, V, H, KB, ldm;
  int32_t bn;       // few rows: rows rounded up to 16; many: row tiles
  int32_t stages;   // few rows: slots of the ring; many: vocabulary tiles
  int32_t vec;      // many rows: rows of logits are 16-byte aligned
};

constexpr uint32_t kScTile = kScBlock * kScBlock;  // bytes of 128 rows of a K block

// ------------------------------------------------------------------ few rows

__host__ __device__ inline uint32_t scaled_stage_bytes(int bn) {
  return kScTile + static_cast<uint32_t>(bn) * kScBlock;
}
__host__ __device__ inline size_t scaled_smem_bytes(int bn, int stages) {
  return 1024 + static_cast<size_t>(stages) * scaled_stage_bytes(bn) + (2 * stages + 9) * 8 + 16;
}

constexpr int kScCW = 8;      // accumulator columns (tree rows) of an epilogue thread
constexpr int kScCols = 32;   // TMEM columns of a buffer (the least that can be allocated)
constexpr int kScBufs = 4;    // two CTAs of an SM fit TMEM's 512 columns together

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__global__ void __launch_bounds__(kScThreads, 2)
    lm_head_scaled_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h,
                          const ScaledParams prm) {
  extern __shared__ uint8_t sc_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sc_smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = prm.stages, bn = prm.bn, KB = prm.KB;
  uint8_t* w_tiles = smem;
  uint8_t* h_tiles = w_tiles + S * kScTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(h_tiles + S * bn * kScBlock);
  uint64_t* full = bars;
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 4;
  uint64_t* mma_done = acc_empty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int vb = blockIdx.x, v0 = vb * kScBlock;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_h);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int u = 0; u < kScBufs; ++u) {
      mbar_init(smem_u32(&acc_full[u]), 1);
      mbar_init(smem_u32(&acc_empty[u]), kScEpiWarps);
    }
    mbar_init(smem_u32(mma_done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kScCols * kScBufs);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      const uint32_t bytes = scaled_stage_bytes(bn);
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_h = l2_policy_evict_last();
      int issued = 0;
      for (int kb = 0; kb < KB; ++kb) {
        const int s = kb % S, n = kb / S;
        if (n > 0 && !mbar_wait(smem_u32(&empty[s]), (n - 1) & 1, kErrLmProducerWait)) break;
        const uint32_t fb = smem_u32(&full[s]);
        mbar_arrive_expect_tx(fb, bytes);
        tma_load_2d_hint(smem_u32(w_tiles + s * kScTile), &tm_w, fb, kb * kScBlock, v0, pol_w);
        tma_load_2d_hint(smem_u32(h_tiles + s * bn * kScBlock), &tm_h, fb, kb * kScBlock, 0, pol_h);
        issued = kb + 1;
      }
      // every issued load lands before this CTA's shared memory can be released
      for (int kb = (issued > S ? issued - S : 0); kb < issued; ++kb)
        mbar_wait(smem_u32(&full[kb % S]), (kb / S) & 1, kErrLmProducerWait);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------- MMA issuer
      const uint32_t idesc = idesc_e4m3_f32(kScBlock, bn);
      for (int kb = 0; kb < KB; ++kb) {
        const int s = kb % S, u = kb % kScBufs;
        bool ok = kb < kScBufs ||
                  mbar_wait(smem_u32(&acc_empty[u]), (kb / kScBufs - 1) & 1, kErrLmMmaWait);
        ok = ok && mbar_wait(smem_u32(&full[s]), (kb / S) & 1, kErrLmMmaWait);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = smem_desc_k_sw128(smem_u32(w_tiles + s * kScTile));
        const uint64_t b = smem_desc_k_sw128(smem_u32(h_tiles + s * bn * kScBlock));
#pragma unroll
        for (int k = 0; k < kScBlock / 32; ++k)
          tc_mma_f8(tmem + static_cast<uint32_t>(u * kScCols), a + 2 * k, b + 2 * k, idesc, k > 0 ? 1u : 0u);
        tc_commit(smem_u32(&empty[s]));
        tc_commit(smem_u32(&acc_full[u]));
      }
      // orders the TMEM release after every MMA issued
      tc_commit(smem_u32(mma_done));
      mbar_wait(smem_u32(mma_done), 0, kErrLmMmaWait);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: TMEM -> scaled sums in registers -> global
    const int quarter = warp & 3;         // TMEM lanes this warp may access
    const int grp = (warp - 2) >> 2;      // half of the tree rows
    const int col0 = grp * kScCW;
    const int v = v0 + quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(col0);
    const float* wsv = prm.ws + static_cast<size_t>(vb) * KB;
    // the row scales come through L1 (every lane reads the same ones); columns past the last
    // row take the scales of rows that exist, for sums that are not stored
    const int last4 = prm.ldm / 4 - 1;
    const bool any = col0 < prm.M;
    float2 acc[kScCW / 2];
#pragma unroll
    for (int j = 0; j < kScCW / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    float w_next = wsv[0];
    bool ok = true;
    for (int kb = 0; kb < KB; ++kb) {
      const int u = kb % kScBufs;
      const float w = w_next;
      if (kb + 1 < KB) w_next = wsv[kb + 1];
      const float4* hs = reinterpret_cast<const float4*>(prm.hs + static_cast<size_t>(kb) * prm.ldm);
      ok = ok && mbar_wait(smem_u32(&acc_full[u]), (kb / kScBufs) & 1, kErrLmEpilogueWait);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      uint32_t d[kScCW];
      if (any) {
        tmem_ld_32x32b_x8(lane_base + static_cast<uint32_t>(u * kScCols), d);
        tmem_ld_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[u]));
      if (any) {
#pragma unroll
        for (int j = 0; j < kScCW / 4; ++j) {
          const float4 h4 = hs[min(col0 / 4 + j, last4)];
          const float2 s0 = fmul2(make_float2(h4.x, h4.y), make_float2(w, w));
          const float2 s1 = fmul2(make_float2(h4.z, h4.w), make_float2(w, w));
          acc[2 * j] = ffma2(make_float2(__uint_as_float(d[4 * j]), __uint_as_float(d[4 * j + 1])), s0, acc[2 * j]);
          acc[2 * j + 1] =
              ffma2(make_float2(__uint_as_float(d[4 * j + 2]), __uint_as_float(d[4 * j + 3])), s1, acc[2 * j + 1]);
        }
      }
    }
    if (ok && v < prm.V) {
#pragma unroll
      for (int j = 0; j < kScCW; ++j) {
        if (col0 + j < prm.M)
          prm.logits[static_cast<size_t>(col0 + j) * prm.V + v] = (j & 1) ? acc[j / 2].y : acc[j / 2].x;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kScCols * kScBufs);
  }
}

// ------------------------------------------------------------------ many rows
// One CTA per SM walks the (vocabulary tile, row tile) pairs, row tiles fastest, so CTAs
// that need the same weight tile run side by side and it comes from HBM once.  A thread owns
// one tree row and half of the tile's columns: its scale is one number per K block (row
// scale x block scale), and nothing of the epilogue goes through shared memory, where per K
// block and two vocabulary blocks TMA writes 48 KB and the MMAs read 48 KB in 512 MMA
// clocks.  The logits leave through a 2 KB patch per warp, so that whole sectors are written
// (each thread writing its own row instead: 360 us against 318 on 512 rows of 128256 x 4096).
// That case runs at about 1,050 clocks per K block under the power cap, 296 to 304 us at first
// and 344 once the card is warm: 160 are the stores, 590 the MMAs and their operands alone, the
// rest the hand-offs of the two TMEM buffers.  Sixteen epilogue warps with a quarter of the
// columns each took the same time, swap-AB with 256 tree rows as N 747.  60 rows of 32000 x
// 8192: 46 us, 5.8 TB/s, HBM-bound.

// Warps 0-7 epilogue, 8 TMA, 9 MMA; 10 and 11 only complete a group of four, which is what
// registers are moved between.
constexpr int kScRowsThreads = 32 * 12;
constexpr int kScRowsTmaWarp = 8, kScRowsMmaWarp = 9;
constexpr int kScRowsEpiRegs = 208, kScRowsOtherRegs = 88;  // of the launch's 168 x 384 registers

// NV: vocabulary blocks of a tile; kRows: rows of hidden that are loaded, 128 or 64 (the MMA
// then reads the weight's bytes as rows 64-127, whose sums nobody takes).
template <int NV, int kRows>
struct ScaledRowsCfg {
  static constexpr int kN = kScBlock * NV;          // vocabulary rows of a tile
  static constexpr int kCW = kN / 2;                // accumulators of a thread
  // K blocks of a ring slot and of a hand-off: two where TMEM has room for two buffers of two
  static constexpr int kKB = NV == 2 ? 1 : 2;
  static constexpr int kHBytes = kRows * kScBlock;
  static constexpr int kBlock = kHBytes + NV * kScTile;  // one K block's operands
  static constexpr int kStage = kBlock * kKB;
  static constexpr int kStages = kRows == 64 ? 4 : (NV == 2 ? 4 : 3);
  static constexpr int kCols = kN * kKB;            // TMEM columns of a buffer
  static constexpr int kBufs = 512 / kCols;         // all of TMEM
  static constexpr int kPatch = 32 * 64;            // a warp's 32 rows x 16 columns
  static constexpr int kPatchOff = kStages * kStage;
  static constexpr int kBarOff = kPatchOff + kScEpiWarps * kPatch;
  static constexpr int kBytes = kBarOff + (2 * kStages + 2 * kBufs + 1) * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

template <int NV, int kRows>
__global__ void __launch_bounds__(kScRowsThreads, 1)
    lm_head_scaled_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h,
                               const ScaledParams prm) {
  using C = ScaledRowsCfg<NV, kRows>;
  constexpr int S = C::kStages, kBufs = C::kBufs, CW = C::kCW, KPS = C::kKB;
  extern __shared__ uint8_t scr_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(scr_smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t full = sbase + C::kBarOff, empty = full + 8 * S, acc_full = empty + 8 * S;
  const uint32_t acc_empty = acc_full + 8 * kBufs, mma_done = acc_empty + 8 * kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + (2 * S + 2 * kBufs + 1) * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int KB = prm.KB, KS = (KB + KPS - 1) / KPS, row_tiles = prm.bn;
  const int64_t tiles = static_cast<int64_t>(prm.stages) * row_tiles;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_h);
    for (int s = 0; s < S; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int u = 0; u < kBufs; ++u) {
      mbar_init(acc_full + 8 * u, 1);
      mbar_init(acc_empty + 8 * u, kScEpiWarps);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (warp == kScRowsMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // (registers: the epilogue of two blocks holds 128 sums a thread)
  if (warp >= kScEpiWarps) {
    if constexpr (NV == 2) reg_dec<kScRowsOtherRegs>();
    if (warp == kScRowsTmaWarp && elect_one()) {
      // ---------------- TMA producer
      const uint64_t pol_w = row_tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
      const uint64_t pol_h = l2_policy_evict_last();
      int s = 0;
      int64_t issued = 0;
      uint32_t phase = 1;  // parity of the slot's last release; the first round waits for none
      bool ok = true;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const int vt = static_cast<int>(t / row_tiles), rt = static_cast<int>(t % row_tiles);
        for (int ks = 0; ks < KS; ++ks) {
          if (issued >= S && !mbar_wait(empty + 8 * s, phase, kErrLmProducerWait)) {
            ok = false;
            break;
          }
          const uint32_t fb = full + 8 * s, dst = sbase + s * C::kStage;
          mbar_arrive_expect_tx(fb, C::kStage);
          // (a block past the last comes in as zeros)
#pragma unroll
          for (int j = 0; j < KPS; ++j) {
            const int x = (ks * KPS + j) * kScBlock;
            const uint32_t at = dst + j * C::kBlock;
            tma_load_2d_hint(at, &tm_h, fb, x, rt * kScBlock, pol_h);
#pragma unroll
            for (int b = 0; b < NV; ++b)
              tma_load_2d_hint(at + C::kHBytes + b * kScTile, &tm_w, fb, x, (vt * NV + b) * kScBlock, pol_w);
          }
          ++issued;
          if (++s == S) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // every issued load lands before this CTA's shared memory can be released
      for (int64_t i = issued > S ? issued - S : 0; i < issued; ++i)
        mbar_wait(full + 8 * static_cast<int>(i % S), static_cast<uint32_t>(i / S) & 1, kErrLmProducerWait);
    }
    if (warp == kScRowsMmaWarp && elect_one()) {
      // ---------------- MMA issuer
      constexpr uint32_t idesc = idesc_e4m3_f32(kScBlock, C::kN);
      int s = 0, u = 0;
      uint32_t ph = 0, pu = 1;
      int64_t n = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int ks = 0; ks < KS; ++ks) {
          ok = (n < kBufs || mbar_wait(acc_empty + 8 * u, pu, kErrLmMmaWait)) &&
               mbar_wait(full + 8 * s, ph, kErrLmMmaWait);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = smem_desc_k_sw128(sbase + s * C::kStage);
          const uint64_t b = smem_desc_k_sw128(sbase + s * C::kStage + C::kHBytes);
#pragma unroll
          for (int j = 0; j < KPS; ++j) {
#pragma unroll
            for (int k = 0; k < kScBlock / 32; ++k) {
              const uint32_t off = j * (C::kBlock / 16) + 2 * k;
              tc_mma_f8(tmem + static_cast<uint32_t>(u * C::kCols + j * C::kN), a + off, b + off, idesc,
                        k > 0 ? 1u : 0u);
            }
          }
          tc_commit(empty + 8 * s);
          tc_commit(acc_full + 8 * u);
          ++n;
          if (++s == S) {
            s = 0;
            ph ^= 1;
          }
          if (++u == kBufs) {
            u = 0;
            pu ^= 1;
          }
        }
      }
      // orders the TMEM release after every MMA issued
      tc_commit(mma_done);
      mbar_wait(mma_done, 0, kErrLmMmaWait);
    }
    __syncwarp();
  } else {
    if constexpr (NV == 2) reg_inc<kScRowsEpiRegs>();
    // ---------------- epilogue
    const int quarter = warp & 3;         // TMEM lanes this warp may access
    const int grp = warp >> 2;            // half of the tile's columns
    const uint32_t lane_base =
        tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(grp * CW);
    float* patch = reinterpret_cast<float*>(smem + C::kPatchOff + warp * C::kPatch);
    int u = 0;
    uint32_t pu = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const int vt = static_cast<int>(t / row_tiles), rt = static_cast<int>(t % row_tiles);
      const int row0 = rt * kScBlock + quarter * 32;      // the warp's first row
      const int col0 = vt * C::kN + grp * CW;             // ... and column
      const bool any = row0 < prm.M && col0 < prm.V;
      const float* wsv = prm.ws + static_cast<size_t>(any ? col0 / kScBlock : 0) * KB;
      const float* hsv = prm.hs + min(row0 + lane, prm.M - 1);
      float2 acc[CW / 2];
#pragma unroll
      for (int j = 0; j < CW / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      // scales are loaded three hand-offs ahead (about an L2 round trip); 0 past the last block
      float w1[KPS], h1[KPS], w2[KPS], h2[KPS], w3[KPS], h3[KPS];
      auto scales = [&](int ks, float (&w)[KPS], float (&h)[KPS]) {
#pragma unroll
        for (int j = 0; j < KPS; ++j) {
          const int kb = ks * KPS + j;
          w[j] = h[j] = 0.f;
          if (kb < KB) {
            w[j] = wsv[kb];
            h[j] = hsv[static_cast<size_t>(kb) * prm.ldm];
          }
        }
      };
      scales(0, w1, h1);
      scales(1, w2, h2);
      scales(2, w3, h3);
      for (int ks = 0; ks < KS; ++ks) {
        float sc[KPS];
#pragma unroll
        for (int j = 0; j < KPS; ++j) {
          sc[j] = w1[j] * h1[j];
          w1[j] = w2[j];
          h1[j] = h2[j];
          w2[j] = w3[j];
          h2[j] = h3[j];
        }
        scales(ks + 3, w3, h3);
        ok = ok && mbar_wait(acc_full + 8 * u, pu, kErrLmEpilogueWait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (any) {
#pragma unroll
          for (int j = 0; j < KPS; ++j) {
            const uint32_t at = lane_base + static_cast<uint32_t>(u * C::kCols + j * C::kN);
            const float2 s2 = make_float2(sc[j], sc[j]);
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
              uint32_t d[16];
              tmem_ld_cols<16>(at + c, d);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                acc[c / 2 + q] =
                    ffma2(make_float2(__uint_as_float(d[2 * q]), __uint_as_float(d[2 * q + 1])), s2, acc[c / 2 + q]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * u);
        if (++u == kBufs) {
          u = 0;
          pu ^= 1;
        }
      }
      if (!ok || !any) continue;
      // 16 columns at a time: thread = row into the patch (16-byte chunks, index XOR row / 2),
      // then 4 threads a row out of it
#pragma unroll
      for (int c = 0; c < CW; c += 16) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<float4*>(patch)[lane * 4 + (q ^ ((lane >> 1) & 3))] =
              make_float4(acc[c / 2 + 2 * q].x, acc[c / 2 + 2 * q].y, acc[c / 2 + 2 * q + 1].x, acc[c / 2 + 2 * q + 1].y);
        __syncwarp();
        const int q = lane & 3, col = col0 + c + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2);
          const float4 x = reinterpret_cast<const float4*>(patch)[r * 4 + (q ^ ((r >> 1) & 3))];
          if (row0 + r >= prm.M) continue;
          float* dst = prm.logits + static_cast<size_t>(row0 + r) * prm.V + col;
          if (prm.vec) {
            if (col < prm.V) *reinterpret_cast<float4*>(dst) = x;  // V is a multiple of 4
          } else {
            if (col < prm.V) dst[0] = x.x;
            if (col + 1 < prm.V) dst[1] = x.y;
            if (col + 2 < prm.V) dst[2] = x.z;
            if (col + 3 < prm.V) dst[3] = x.w;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScRowsMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace eagle
