// paged_attention.cuh -- tree attention over a paged K/V cache (layout: paged.cuh).
#pragma once

#include "paged.cuh"

namespace eagle {

struct PagedAttnParams {
  PageMap map;
  const int32_t* prefix_lens;  // [B]
  const int32_t* parents;      // [B, N]
  int32_t B, N, Hq, Hkv, G, Lmax, shared;
  float scale;
};

// fp32: one warp per output row: 32 keys at a time, one per lane for the scores, then D / 32
// output columns per lane.
template <int D>
__global__ void __launch_bounds__(128)
    tree_attn_paged_simple_kernel(const float* __restrict__ q, const float* __restrict__ kp,
                                  const float* __restrict__ vp, const float* __restrict__ kt,
                                  const float* __restrict__ vt, float* __restrict__ out,
                                  const PagedAttnParams p) {
  __shared__ float q_s[4][D];
  __shared__ int path_s[4][64];
  const int wid = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + wid;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<int64_t>(p.B) * p.N * p.Hq) return;
  const int b = static_cast<int>(row / (p.N * p.Hq));
  const int i = static_cast<int>((row / p.Hq) % p.N);
  const int g = static_cast<int>(row % p.Hq) / p.G;
  constexpr int kPer = D / 32;
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q_s[wid][lane + 32 * e] = q[row * D + lane + 32 * e];
    acc[e] = 0.f;
  }
  int np = 0;
  if (lane == 0) {
    int a = i;
    for (int guard = 0; guard < 64 && a >= 0; ++guard) {
      path_s[wid][np++] = a;
      const int up = p.parents[static_cast<size_t>(b) * p.N + a];
      a = (up >= 0 && up < a) ? up : -1;
    }
  }
  np = __shfl_sync(0xffffffffu, np, 0);
  __syncwarp();
  int L = p.prefix_lens[b];
  if ((L < 0 || L > p.Lmax) && lane == 0) record_error(kErrAttnPrefixLen);
  L = L < 0 ? 0 : (L > p.Lmax ? p.Lmax : L);
  auto key_row = [&](int j, const float* pool, const float* tree) -> const float* {
    if (j >= L) return tree + ((static_cast<size_t>(b) * p.N + path_s[wid][j - L]) * p.Hkv + g) * D;
    const int32_t pg = page_of(p.map, b, j);
    return pg < 0 ? nullptr : pool + page_row(p.map, pg, g, p.Hkv, j, D);
  };
  const int nk = L + np;
  float m = -INFINITY, l = 0.f;
  for (int c = 0; c < nk; c += 32) {
    const int j = c + lane;
    float s = -INFINITY;
    if (j < nk) {
      const float* kr = key_row(j, kp, kt);
      float dot = 0.f;
      if (kr != nullptr)
        for (int d = 0; d < D; ++d) dot = fmaf(q_s[wid][d], kr[d], dot);
      s = dot * p.scale;
    }
    float cm = s;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, off));
    const float mn = fmaxf(m, cm);
    const float corr = expf(m - mn);
    const float pr = j < nk ? expf(s - mn) : 0.f;
    float ps = pr;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
    l = l * corr + ps;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= corr;
    const int cnt = min(32, nk - c);
    for (int t = 0; t < cnt; ++t) {
      const float* vr = key_row(c + t, vp, vt);
      const float pt = __shfl_sync(0xffffffffu, pr, t);
      if (vr != nullptr) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(pt, vr[lane + 32 * e], acc[e]);
      }
    }
    m = mn;
  }
  const float inv = 1.0f / l;
#pragma unroll
  for (int e = 0; e < kPer; ++e) out[row * D + lane + 32 * e] = acc[e] * inv;
}

}  // namespace eagle
