// paged_attention.cuh -- tree attention over a paged, partly shared K/V cache (layout:
// paged.cuh): what both types share, and the fp32 kernels.  The bf16 ones are in
// paged_attention_tc.cuh.
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

// ------------------------------------------------------------------ fp32
// The exact path: all products and sums on the fp32 pipe.  An item is a tile of kRT rows of
// a kv head -- of one sequence (its own positions and its tree) or of the whole batch (the
// shared positions, whose K/V is so read once for kRT rows of any sequences) -- and its key
// tiles are divided among S CTAs, whose partials (m, l, acc) a second kernel merges.
//
// 128 threads: thread (ty, tx) has rows ty + kTY i and, of a tile, keys tx + kTX j in S = Q K^T
// and columns 4 tx + 4 kTX k in O += P V, so that operands come from shared memory 16 bytes at
// a time without bank conflicts.  64-row tiles feed 8 to 13 multiply-adds with each float4 (23
// to 25 TFLOP/s of the pipe's 74); 32 rows give small problems more CTAs (with heads of 128
// they spill 16 bytes a thread), 16 and 4 rows are for single tokens, whose cost is the cache's
// bytes and the latency of a tile (4 rows: one warp a row).  K and V tiles are double-buffered
// by asynchronous copies, which fill rows that are not there with zeros.

struct PagedF32Params {
  PagedAttnParams a;
  const float* q;
  const float* kp;
  const float* vp;
  const float* kt;
  const float* vt;
  float* out;
  float* part_acc;  // [item][S][kRT][D]
  float2* part_ml;  // [item][S][kRT]
  int32_t splits;
  int32_t tiles_own, tiles_sh;  // row tiles of a sequence's kv head, of the batch's (0: no shared part)
  int32_t direct;               // one split and no shared part: rows are complete
};

template <int D, int RT>
struct PagedF32Cfg {
  static constexpr int kKT = D == 128 ? 32 : 64;  // keys of a tile (16 KB of K)
  static constexpr int kTY = RT < 16 ? RT : 16;   // threads over the rows, over keys and columns
  static constexpr int kTX = 128 / kTY;
  static constexpr int kQS = D + 4;               // row strides in floats: 16 bytes past a multiple of 128
  static constexpr int kKS = D + 4;
  static constexpr int kPS = kKT + 4;
  static constexpr int kStage = kKT * kKS + kKT * D;
  static constexpr int kFloats = RT * kQS + 2 * kStage + RT * kPS;
  static constexpr int kBytes = kFloats * 4 + RT * 8 + 64 * 4 + 16;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

template <int D, int RT>
__global__ void __launch_bounds__(128) paged_attn_f32_kernel(const __grid_constant__ PagedF32Params p) {
  using C = PagedF32Cfg<D, RT>;
  constexpr int KT = C::kKT, TX = C::kTX, TY = C::kTY, RPT = RT / TY, KPT = KT / TX;
  constexpr int CPT = D >= 4 * TX ? D / (4 * TX) : 1;  // (D = 64 leaves half of 32 threads without columns)
  extern __shared__ __align__(16) float f32_smem[];
  float* q_s = f32_smem;
  float* kv_s = q_s + RT * C::kQS;
  float* p_s = kv_s + 2 * C::kStage;
  uint64_t* anc_s = reinterpret_cast<uint64_t*>(p_s + RT * C::kPS);
  int32_t* par_s = reinterpret_cast<int32_t*>(anc_s + RT);
  int32_t* live_s = par_s + 64;
  const PagedAttnParams& a = p.a;
  const int tid = threadIdx.x, ty = tid / TX, tx = tid % TX;
  const bool cols = 4 * tx < D;
  const int N = a.N, G = a.G, Hkv = a.Hkv;

  pdl_launch_dependents();  // the merge waits for this grid
  pdl_wait();

  // ---- the item and its keys
  int64_t it = blockIdx.x;
  const int64_t shared_items = static_cast<int64_t>(p.tiles_sh) * Hkv;
  const bool sh = it < shared_items;
  int b = 0, kvh;
  int64_t row0;                 // first row, in (node, head) order
  int64_t rows;                 // rows there are
  int begin = 0, L, trees = 0;  // key positions [begin, L), then the tree's tiles
  if (sh) {
    kvh = static_cast<int>(it / p.tiles_sh);
    row0 = (it % p.tiles_sh) * RT;
    rows = static_cast<int64_t>(a.B) * N * G;
    // a sequence that holds the whole shared part
    if (tid == 0) *live_s = INT32_MAX;
    __syncthreads();
    for (int i = tid; i < a.B; i += 128)
      if (min(a.prefix_lens[i], a.Lmax) >= a.shared) atomicMin(live_s, i);
    __syncthreads();
    b = *live_s;
    L = b < a.B ? a.shared : 0;
  } else {
    it -= shared_items;
    row0 = (it % p.tiles_own) * RT;
    const int64_t bk = it / p.tiles_own;
    kvh = static_cast<int>(bk % Hkv);
    b = static_cast<int>(bk / Hkv);
    rows = static_cast<int64_t>(N) * G;
    L = a.prefix_lens[b];
    if ((L < 0 || L > a.Lmax) && tid == 0) record_error(kErrAttnPrefixLen);
    L = L < 0 ? 0 : (L > a.Lmax ? a.Lmax : L);
    begin = L >= a.shared ? a.shared : 0;
    trees = (N + KT - 1) / KT;
  }
  const int prefix_tiles = (L - begin + KT - 1) / KT;
  const int64_t T = prefix_tiles + trees;
  const int t0 = static_cast<int>(T * blockIdx.y / p.splits), t1 = static_cast<int>(T * (blockIdx.y + 1) / p.splits);

  // element offset in q and out of a row (node, head) of this item
  auto row_at = [&](int64_t rr) -> int64_t {
    return ((static_cast<int64_t>(sh ? 0 : b) * N + rr / G) * a.Hq + kvh * G + rr % G) * D;
  };
  auto row_ok = [&](int64_t rr) {
    return rr < rows && (!sh || min(a.prefix_lens[rr / G / N], a.Lmax) >= a.shared);
  };

  auto load_tile = [&](int t) {
    float* ks = kv_s + (t & 1) * C::kStage;
    float* vs = ks + KT * C::kKS;
#pragma unroll 4
    for (int i = tid; i < KT * (D / 4); i += 128) {
      const int j = i / (D / 4), c = (i % (D / 4)) * 4;
      const float *ksrc = p.kt, *vsrc = p.vt;
      bool in;
      if (t < prefix_tiles) {
        const int pos = begin + t * KT + j;
        in = pos < L;
        if (in) {
          const int32_t pg = page_of(a.map, b, pos);
          in = pg >= 0;
          if (in) {
            const size_t at = page_row(a.map, pg, kvh, Hkv, pos, D) + c;
            ksrc = p.kp + at;
            vsrc = p.vp + at;
          }
        }
      } else {
        const int node = (t - prefix_tiles) * KT + j;
        in = node < N;
        if (in) {
          const size_t at = ((static_cast<size_t>(b) * N + node) * Hkv + kvh) * D + c;
          ksrc = p.kt + at;
          vsrc = p.vt + at;
        }
      }
      cp_async16(smem_u32(ks + j * C::kKS + c), ksrc, in);
      cp_async16(smem_u32(vs + j * D + c), vsrc, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  if (t0 < t1) load_tile(t0);
  for (int i = tid; i < RT * (D / 4); i += 128) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < rows) x = *reinterpret_cast<const float4*>(p.q + row_at(row0 + r) + c);
    *reinterpret_cast<float4*>(q_s + r * C::kQS + c) = x;
  }
  if (!sh && t1 > prefix_tiles) {
    // ancestor masks: a node and every node up its parent chain (a link that does not point
    // to an earlier node ends it)
    if (tid < N) par_s[tid] = a.parents[static_cast<size_t>(b) * N + tid];
    __syncthreads();
    if (tid < RT) {
      uint64_t m = 0;
      int i = row0 + tid < rows ? static_cast<int>((row0 + tid) / G) : -1;
      for (int guard = 0; guard < 64 && i >= 0; ++guard) {
        m |= 1ull << i;
        const int up = par_s[i];
        i = (up >= 0 && up < i) ? up : -1;
      }
      anc_s[tid] = m;
    }
  }
  float m[RPT], l[RPT];
  float4 o[RPT][CPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int k = 0; k < CPT; ++k) o[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int t = t0; t < t1; ++t) {
    if (t + 1 < t1) {
      load_tile(t + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const float* ks = kv_s + (t & 1) * C::kStage;
    const float* vs = ks + KT * C::kKS;
    float s[RPT][KPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < KPT; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 qv[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) qv[i] = *reinterpret_cast<const float4*>(q_s + (ty + TY * i) * C::kQS + d);
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const float4 kv = *reinterpret_cast<const float4*>(ks + (tx + TX * j) * C::kKS + d);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
          s[i][j] = fmaf(qv[i].w, kv.w, fmaf(qv[i].z, kv.z, fmaf(qv[i].y, kv.y, fmaf(qv[i].x, kv.x, s[i][j]))));
      }
    }
    const bool tree = t >= prefix_tiles;
    const int first = tree ? (t - prefix_tiles) * KT : begin + t * KT;  // node or position of key 0
    const int end = tree ? N : L;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const uint64_t see = tree ? anc_s[ty + TY * i] : 0ull;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const int key = first + tx + TX * j;
        const bool in = key < end && (!tree || ((see >> (key & 63)) & 1ull));
        s[i][j] = in ? s[i][j] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
#pragma unroll
      for (int off = 1; off < TX; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == -INFINITY ? 0.f : mn;  // every key so far is masked
      const float f = expf(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < KPT; ++j) {
        const float e = expf(s[i][j] - base);
        sum += e;
        p_s[(ty + TY * i) * C::kPS + tx + TX * j] = e;
      }
#pragma unroll
      for (int off = 1; off < TX; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[i] = l[i] * f + sum;
      m[i] = mn;
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        o[i][k] = make_float4(o[i][k].x * f, o[i][k].y * f, o[i][k].z * f, o[i][k].w * f);
    }
    __syncwarp();  // a row's weights come from the lanes of its ty, all in this warp
#pragma unroll 2
    for (int j = 0; j < KT && cols; j += 4) {
      float4 w[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i) w[i] = *reinterpret_cast<const float4*>(p_s + (ty + TY * i) * C::kPS + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int k = 0; k < CPT; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(vs + (j + jj) * D + 4 * tx + 4 * TX * k);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float e = jj == 0 ? w[i].x : (jj == 1 ? w[i].y : (jj == 2 ? w[i].z : w[i].w));
            o[i][k].x = fmaf(e, v.x, o[i][k].x);
            o[i][k].y = fmaf(e, v.y, o[i][k].y);
            o[i][k].z = fmaf(e, v.z, o[i][k].z);
            o[i][k].w = fmaf(e, v.w, o[i][k].w);
          }
        }
      }
    }
    __syncthreads();  // the tile's buffer and the weights are free
  }
  const int64_t part = (static_cast<int64_t>(blockIdx.x) * p.splits + blockIdx.y) * RT;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = ty + TY * i;
    if (!row_ok(row0 + r)) continue;
    if (p.direct) {
      const float inv = 1.0f / l[i];  // the node itself is always visible
      float* dst = p.out + row_at(row0 + r);
      if (!cols) continue;
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        *reinterpret_cast<float4*>(dst + 4 * tx + 4 * TX * k) =
            make_float4(o[i][k].x * inv, o[i][k].y * inv, o[i][k].z * inv, o[i][k].w * inv);
      continue;
    }
    if (t0 < t1 && cols) {
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        *reinterpret_cast<float4*>(p.part_acc + (part + r) * D + 4 * tx + 4 * TX * k) = o[i][k];
    }
    if (tx == 0) p.part_ml[part + r] = make_float2(m[i], l[i]);
  }
}

// Output row = the sum of its partials weighted by exp(m_p - m), over the sum of their l: a
// thread per four columns, the S own partials, then the S shared ones.
template <int D, int RT>
__global__ void __launch_bounds__(128) paged_attn_f32_merge_kernel(const __grid_constant__ PagedF32Params p) {
  const PagedAttnParams& a = p.a;
  const int64_t x = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) / (D / 4);
  const int c = (threadIdx.x % (D / 4)) * 4;
  pdl_launch_dependents();
  pdl_wait();
  if (x >= static_cast<int64_t>(a.B) * a.N * a.Hq) return;
  const int64_t fnode = x / a.Hq;
  const int h = static_cast<int>(x % a.Hq), kvh = h / a.G, hg = h % a.G;
  const int b = static_cast<int>(fnode / a.N), node = static_cast<int>(fnode % a.N);
  const int64_t shared_items = static_cast<int64_t>(p.tiles_sh) * a.Hkv;
  int64_t part[2];
  {
    const int64_t rr = static_cast<int64_t>(node) * a.G + hg;
    const int64_t item = shared_items + (static_cast<int64_t>(b) * a.Hkv + kvh) * p.tiles_own + rr / RT;
    part[0] = item * p.splits * RT + rr % RT;
    const int64_t rs = fnode * a.G + hg;
    part[1] = (static_cast<int64_t>(kvh) * p.tiles_sh + rs / RT) * p.splits * RT + rs % RT;
  }
  const int n = p.tiles_sh > 0 && min(a.prefix_lens[b], a.Lmax) >= a.shared ? 2 * p.splits : p.splits;
  auto at = [&](int i) { return i < p.splits ? part[0] + static_cast<int64_t>(i) * RT : part[1] + static_cast<int64_t>(i - p.splits) * RT; };
  float m = -INFINITY, den = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 8) {
    float2 ml[8];
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + k < n) {
        ml[k] = p.part_ml[at(i0 + k)];
        v[k] = *reinterpret_cast<const float4*>(p.part_acc + at(i0 + k) * D + c);
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = fmaxf(mn, ml[k].x);
    const float base = mn == -INFINITY ? 0.f : mn;  // (no maximum, but perhaps a NaN sum)
    const float f = expf(m - base);
    den *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (ml[k].y == 0.f) continue;  // an empty partial's accumulator was never written
      const float w = expf(ml[k].x - base);
      den += w * ml[k].y;
      o = make_float4(fmaf(w, v[k].x, o.x), fmaf(w, v[k].y, o.y), fmaf(w, v[k].z, o.z), fmaf(w, v[k].w, o.w));
    }
    m = mn;
  }
  const float inv = 1.0f / den;  // the node itself is always visible
  *reinterpret_cast<float4*>(p.out + x * D + c) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

}  // namespace eagle
