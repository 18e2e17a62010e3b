// lm_head_scaled.cuh -- LM-head logits in 8-bit floating point with a scale for each block
// of 128, and the quantisers that bring rows and weights into that form:
//     logits[r, v] = sum over blocks t of  hs[t, r] * ws[v / 128, t] * (sum of h[r, k] w[v, k], k in block t)
// with h, w in e4m3 and hs, ws in fp32.
//
// A product of two e4m3 values is exact in fp32, and the tensor core sums a block's 128 of
// them in fp32 (measured against fp64: relative error 1.3e-8 on normal data, as an fp32 FMA
// chain); the blocks are scaled and summed in fp32 registers.
//
// The GEMM is swap-AB like lm_head.cuh: 128 vocabulary rows are the MMA's M, the few tree
// rows its N, so the weight streams once.  A vocabulary tile is one row of scale blocks, so
// every K block of a tile has a single ws.  Per K block one 128-deep MMA chain goes into a
// fresh TMEM buffer; two groups of four epilogue warps (thread = vocabulary row, group =
// half of the tree rows) scale it into their register accumulators while the next block's
// MMAs run.
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace eagle {

constexpr int kScBlock = 128;        // elements that share a scale; vocabulary rows per CTA
constexpr int kScThreads = 32 * 10;  // TMA, MMA, 8 epilogue warps
constexpr int kScEpiWarps = 8;

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

// 1 x 128 blocks: one warp per block, four elements a lane.  Streaming, HBM- or
// launch-bound: each element is read once.
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
// registers between its maximum and its rounding.
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
// Untiled bulk copy (addresses and size multiples of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

struct ScaledParams {
  float* logits;
  const float* hs;  // [KB, ldm]
  const float* ws;  // [ceil(V / 128), KB]
  int32_t M, V, H, KB, ldm;
  int32_t bn;       // tree rows per CTA (MMA N): a multiple of 16, <= 2 * CW
  int32_t stages;
};

constexpr uint32_t kScW = kScBlock * kScBlock;  // bytes of a W tile
constexpr uint32_t kScHs = 1024;                // bytes of a stage's row scales (256 rows)
__host__ __device__ inline uint32_t scaled_stage_bytes(int bn) {
  return kScW + static_cast<uint32_t>(bn) * kScBlock + kScHs;
}
__host__ __device__ inline size_t scaled_smem_bytes(int bn, int stages) {
  return 1024 + static_cast<size_t>(stages) * scaled_stage_bytes(bn) + (2 * stages + 9) * 8 + 16;
}

// CW: accumulator columns (tree rows) of an epilogue thread.
template <int CW>
struct ScaledCfg {
  // TMEM columns of a buffer (tcgen05.alloc takes powers of two from 32), and buffers:
  // four while two CTAs of an SM fit their 512 columns together
  static constexpr int kCols = 2 * CW < 32 ? 32 : 2 * CW;
  static constexpr int kBufs = CW <= 32 ? 4 : 2;
  static constexpr int kStep = CW < 16 ? CW : 16;  // columns per TMEM load
};

__device__ __forceinline__ void tmem_ld_step(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld_32x32b_x16(taddr, r); }
__device__ __forceinline__ void tmem_ld_step(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

template <int CW>
__global__ void __launch_bounds__(kScThreads)
    lm_head_scaled_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h,
                          const ScaledParams prm) {
  using C = ScaledCfg<CW>;
  extern __shared__ uint8_t sc_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sc_smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int S = prm.stages, bn = prm.bn, KB = prm.KB;
  uint8_t* w_tiles = smem;
  uint8_t* h_tiles = w_tiles + S * kScW;
  uint8_t* hs_tiles = h_tiles + S * bn * kScBlock;
  uint64_t* bars = reinterpret_cast<uint64_t*>(hs_tiles + S * kScHs);
  uint64_t* full = bars;
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 4;
  uint64_t* mma_done = acc_empty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * bn;
  const int vb = blockIdx.y, v0 = vb * kScBlock;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_h);
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1 + kScEpiWarps);  // the MMAs and the readers of the scales
    }
    for (int u = 0; u < C::kBufs; ++u) {
      mbar_init(smem_u32(&acc_full[u]), 1);
      mbar_init(smem_u32(&acc_empty[u]), kScEpiWarps);
    }
    mbar_init(smem_u32(mma_done), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::kCols * C::kBufs);
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
      const int hs_rows = min(bn, prm.ldm - r0);
      const uint32_t bytes = kScW + static_cast<uint32_t>(bn) * kScBlock + static_cast<uint32_t>(hs_rows) * 4;
      const uint64_t pol_w = l2_policy_evict_first();
      const uint64_t pol_h = l2_policy_evict_last();
      int issued = 0;
      for (int kb = 0; kb < KB; ++kb) {
        const int s = kb % S, n = kb / S;
        if (n > 0 && !mbar_wait(smem_u32(&empty[s]), (n - 1) & 1, kErrLmProducerWait)) break;
        const uint32_t fb = smem_u32(&full[s]);
        mbar_arrive_expect_tx(fb, bytes);
        tma_load_2d_hint(smem_u32(w_tiles + s * kScW), &tm_w, fb, kb * kScBlock, v0, pol_w);
        tma_load_2d_hint(smem_u32(h_tiles + s * bn * kScBlock), &tm_h, fb, kb * kScBlock, r0, pol_h);
        bulk_load(smem_u32(hs_tiles + s * kScHs), prm.hs + static_cast<size_t>(kb) * prm.ldm + r0,
                  static_cast<uint32_t>(hs_rows) * 4, fb);
        issued = kb + 1;
      }
      // every issued load lands before this CTA's shared memory can be released
      for (int kb = (issued > S ? issued - S : 0); kb < issued; ++kb)
        mbar_wait(smem_u32(&full[kb % S]), (kb / S) & 1, kErrLmProducerWait);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer
      const uint32_t idesc = idesc_e4m3_f32(kScBlock, bn);
      for (int kb = 0; kb < KB; ++kb) {
        const int s = kb % S, u = kb % C::kBufs;
        bool ok = kb < C::kBufs ||
                  mbar_wait(smem_u32(&acc_empty[u]), (kb / C::kBufs - 1) & 1, kErrLmMmaWait);
        ok = ok && mbar_wait(smem_u32(&full[s]), (kb / S) & 1, kErrLmMmaWait);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = smem_desc_k_sw128(smem_u32(w_tiles + s * kScW));
        const uint64_t b = smem_desc_k_sw128(smem_u32(h_tiles + s * bn * kScBlock));
#pragma unroll
        for (int k = 0; k < kScBlock / 32; ++k)
          tc_mma_f8(tmem + static_cast<uint32_t>(u * C::kCols), a + 2 * k, b + 2 * k, idesc, k > 0 ? 1u : 0u);
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
    const int col0 = grp * CW;
    const int v = v0 + quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(col0);
    const float* wsv = prm.ws + static_cast<size_t>(vb) * KB;
    float2 acc[CW / 2];
#pragma unroll
    for (int j = 0; j < CW / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    float w_next = wsv[0];
    bool ok = true;
    for (int kb = 0; kb < KB && ok; ++kb) {
      const int s = kb % S, u = kb % C::kBufs;
      const float w = w_next;
      if (kb + 1 < KB) w_next = wsv[kb + 1];
      ok = mbar_wait(smem_u32(&full[s]), (kb / S) & 1, kErrLmEpilogueWait) &&
           mbar_wait(smem_u32(&acc_full[u]), (kb / C::kBufs) & 1, kErrLmEpilogueWait);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const float4* hs = reinterpret_cast<const float4*>(hs_tiles + s * kScHs) + col0 / 4;
#pragma unroll
      for (int c = 0; c < CW; c += C::kStep) {
        if (col0 + c >= bn) continue;  // uniform over the warp
        uint32_t d[C::kStep];
        tmem_ld_step(lane_base + static_cast<uint32_t>(u * C::kCols + c), d);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < C::kStep; j += 4) {
          const float4 h4 = hs[(c + j) / 4];
          const float2 s0 = fmul2(make_float2(h4.x, h4.y), make_float2(w, w));
          const float2 s1 = fmul2(make_float2(h4.z, h4.w), make_float2(w, w));
          acc[(c + j) / 2] =
              ffma2(make_float2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])), s0, acc[(c + j) / 2]);
          acc[(c + j) / 2 + 1] =
              ffma2(make_float2(__uint_as_float(d[j + 2]), __uint_as_float(d[j + 3])), s1, acc[(c + j) / 2 + 1]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&acc_empty[u]));
        mbar_arrive(smem_u32(&empty[s]));
      }
    }
    if (ok && v < prm.V) {
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        const int row = r0 + col0 + j;
        if (col0 + j < bn && row < prm.M)
          prm.logits[static_cast<size_t>(row) * prm.V + v] = (j & 1) ? acc[j / 2].y : acc[j / 2].x;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kCols * C::kBufs);
  }
}

}  // namespace eagle
