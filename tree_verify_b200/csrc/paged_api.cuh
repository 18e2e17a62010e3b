// paged_api.cuh -- C ABI of the paged-cache operators and of the e4m3 LM head (declared in
// include/eagle_verify.h): argument checks, launch plans and launches.  Included by
// eagle_verify.cu, whose helpers it uses.
#pragma once

#include <atomic>
#include <type_traits>

#include "lm_head_scaled.cuh"
#include "paged.cuh"
#include "paged_attention.cuh"
#include "paged_attention_tc.cuh"

namespace eagle {
namespace {

// ------------------------------------------------------------------ checks

eagle_status_t check_pages(const eagle_pages_t* pg) {
  if (pg == nullptr) return EAGLE_ERR_INVALID_ARGUMENT;
  if (pg->num_pages < 1 || pg->max_pages < 1) return EAGLE_ERR_INVALID_ARGUMENT;
  const int32_t ps = pg->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return EAGLE_ERR_INVALID_ARGUMENT;
  // positions are 32-bit
  if (static_cast<int64_t>(pg->max_pages) * ps > INT32_MAX) return EAGLE_ERR_INVALID_ARGUMENT;
  return EAGLE_OK;
}

PageMap page_map(const eagle_pages_t* pg, const int32_t* table) {
  int shift = 4;
  while ((1 << shift) < pg->page_size) ++shift;
  return PageMap{table, pg->num_pages, shift, pg->max_pages};
}

eagle_status_t check_paged_shape(const eagle_shape_t* s, const eagle_pages_t* pg, int32_t shared_len) {
  eagle_status_t rc = check_shape(s);
  if (rc == EAGLE_OK) rc = check_pages(pg);
  if (rc != EAGLE_OK) return rc;
  if (static_cast<int64_t>(pg->max_pages) * pg->page_size < s->max_prefix_len) return EAGLE_ERR_INVALID_ARGUMENT;
  if (shared_len < 0 || shared_len > s->max_prefix_len) return EAGLE_ERR_INVALID_ARGUMENT;
  // positions, rounded up to tiles, are 32-bit
  if (s->max_prefix_len > INT32_MAX - 512) return EAGLE_ERR_INVALID_ARGUMENT;
  return EAGLE_OK;
}

// [a, a + an) and [b, b + bn) share a byte
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bn && y < x + an;
}

// Bytes of a page pool.
size_t pool_bytes(const eagle_pages_t* pg, const eagle_shape_t* s, int esize) {
  return static_cast<size_t>(pg->num_pages) * pg->page_size * s->num_kv_heads * s->head_dim * esize;
}

int elem_size(const eagle_shape_t* s) { return s->dtype == EAGLE_DTYPE_BF16 ? 2 : 4; }

// ------------------------------------------------------------------ kernel attributes

// Set once for each device.
template <auto kKernel>
bool allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // bit per device (kMaxDevices of them)
  static_assert(kMaxDevices <= 64, "a bit per device");
  int dev;
  if (!current_device(&dev)) return false;
  if ((done.load(std::memory_order_relaxed) >> dev) & 1) return true;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return true;
}

// Kernels whose first warps take `inc` registers a thread out of what the CTA was launched
// with, the last four keeping `dec`: a build that was launched with fewer would wait for
// ever, so it is never launched.
template <auto kKernel>
bool register_shares_fit(int threads, int inc, int dec) {
  static std::atomic<bool> fit{false};  // (the same on every device; asked again after an error)
  if (fit.load(std::memory_order_relaxed)) return true;
  cudaFuncAttributes a{};
  if (cudaFuncGetAttributes(&a, kKernel) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (a.numRegs * threads < (threads - 128) * inc + 128 * dec) return false;
  fit.store(true, std::memory_order_relaxed);
  return true;
}

// ------------------------------------------------------------------ append

template <typename T, int D>
void launch_append(const AppendParams& p, bool interleaved, int rows, cudaStream_t st) {
  if (interleaved)
    rope_append_kernel<T, D, true><<<rows, kAppendThreads, 0, st>>>(p);
  else
    rope_append_kernel<T, D, false><<<rows, kAppendThreads, 0, st>>>(p);
}

// A strided operand: 16-byte aligned rows that do not overlap one another, all of them
// within 2^62 bytes.
bool rows_ok(const void* x, int64_t stride, int64_t width, int esize, int64_t rows) {
  return aligned16(x) && stride >= width && stride <= (static_cast<int64_t>(1) << 60) / rows &&
         (stride * esize) % 16 == 0;
}

// A strided operand of `rows` rows and its bytes, first to last.
struct RowSpan {
  const void* p;
  int64_t stride, width;
  size_t bytes(int64_t rows, int esize) const {
    return p == nullptr ? 0 : static_cast<size_t>(((rows - 1) * stride + width) * esize);
  }
};

// A rotated output (dense) either is its own dense input, in[own], or lies apart from every
// input; in place too it lies apart from the others, wherever they begin.
bool rotated_out_ok(const void* out, int64_t width, int own, const RowSpan (&in)[3], int64_t rows, int esize) {
  const bool in_place = out == in[own].p;
  if (in_place && in[own].stride != width) return false;
  for (int i = 0; i < 3; ++i) {
    if (in[i].p == nullptr || (i == own && in_place)) continue;
    if (overlap(in[i].p, in[i].bytes(rows, esize), out, static_cast<size_t>(rows * width * esize))) return false;
  }
  return true;
}

// ------------------------------------------------------------------ attention

// The fp32 form's row tiles: 4 or 16 rows where no more are in a sequence's kv head (32 tokens
// of 32/8 heads over 1000 shared + 0..3000 keys: 4 rows 261 us, 16 rows 391); else 64, or 32
// where 64 would leave most SMs with a tile or two (three 13-node trees of 8/2 heads of 64 over
// 333 shared + 0..300 keys: 32 rows 15.9 us, 64 rows 18.5; eight 64-node trees of 32/8 heads
// over 1000 shared + 0..500: 580 and 429).  Key tiles are
// divided so that there are about five CTAs for each SM.
struct PagedF32Plan {
  int rt, splits, tiles_own, tiles_sh;
  int64_t items;
  size_t ml_bytes, acc_bytes;
  bool direct() const { return splits == 1 && tiles_sh == 0; }
  size_t bytes() const { return direct() ? 0 : ml_bytes + acc_bytes; }
};

PagedF32Plan plan_paged_f32(const eagle_shape_t* s, int32_t shared_len) {
  PagedF32Plan p{};
  const int64_t G = s->num_q_heads / s->num_kv_heads, B = s->batch, N = s->num_nodes, Hkv = s->num_kv_heads;
  auto tile = [&](int rt) {
    p.rt = rt;
    p.tiles_own = static_cast<int>((N * G + rt - 1) / rt);
    p.tiles_sh = shared_len > 0 ? static_cast<int>((B * N * G + rt - 1) / rt) : 0;
    p.items = Hkv * (static_cast<int64_t>(B) * p.tiles_own + p.tiles_sh);
  };
  const int kt = s->head_dim == 128 ? PagedF32Cfg<128, 64>::kKT : PagedF32Cfg<64, 64>::kKT;
  const int64_t tiles = (static_cast<int64_t>(s->max_prefix_len) + kt - 1) / kt + (N + kt - 1) / kt;
  tile(N * G <= 4 ? 4 : (N * G <= 16 ? 16 : 64));
  if (p.rt == 64 && p.items * tiles < 4 * kNumSMs) tile(32);
  int64_t splits = (5 * kNumSMs + p.items - 1) / p.items;
  if (splits > tiles) splits = tiles;
  p.splits = static_cast<int>(splits);
  const size_t rows = static_cast<size_t>(p.items) * p.splits * p.rt;
  p.ml_bytes = align256(rows * sizeof(float2));
  p.acc_bytes = align256(rows * s->head_dim * sizeof(float));
  return p;
}

template <int D, int RT>
eagle_status_t launch_paged_f32(const PagedF32Plan& plan, const void* q, const void* kp, const void* vp,
                                const void* kt, const void* vt, void* out, void* ws, const PagedAttnParams& ap,
                                cudaStream_t st) {
  constexpr int bytes = PagedF32Cfg<D, RT>::kBytes;
  if (!allow_smem<paged_attn_f32_kernel<D, RT>>(bytes)) return EAGLE_ERR_CUDA;
  PagedF32Params p{};
  p.a = ap;
  p.q = static_cast<const float*>(q);
  p.kp = static_cast<const float*>(kp);
  p.vp = static_cast<const float*>(vp);
  p.kt = static_cast<const float*>(kt);
  p.vt = static_cast<const float*>(vt);
  p.out = static_cast<float*>(out);
  p.part_ml = static_cast<float2*>(ws);
  p.part_acc = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + plan.ml_bytes);
  p.splits = plan.splits;
  p.tiles_own = plan.tiles_own;
  p.tiles_sh = plan.tiles_sh;
  p.direct = plan.direct();
  // either kernel may be launched while the one before it on the stream ends, and waits for it
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.items), plan.splits);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_attn_f32_kernel<D, RT>, p) != cudaSuccess) {
    cudaGetLastError();
    return EAGLE_ERR_CUDA;
  }
  const eagle_status_t rc = launch_status();
  if (rc != EAGLE_OK || p.direct) return rc;
  const int64_t threads = static_cast<int64_t>(ap.B) * ap.N * ap.Hq * (D / 4);
  cfg.gridDim = dim3(static_cast<unsigned>((threads + 127) / 128));
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, paged_attn_f32_merge_kernel<D, RT>, p) != cudaSuccess) {
    cudaGetLastError();
    return EAGLE_ERR_CUDA;
  }
  return launch_status();
}

// Row tiles and partials of the tensor-core form, from what the host knows: the lengths may
// be anything up to Lmax, so every item may be cut, and each has a run more than it is cut.
struct PagedPlan {
  int nodes_per_tile, rb_own, rb_sh, rows_own, rows_sh;
  int64_t own_row0, part_rows;
  size_t plan_bytes, ml_bytes, acc_bytes;
  size_t bytes() const { return plan_bytes + ml_bytes + acc_bytes; }
};

PagedPlan plan_paged(const eagle_shape_t* s, int32_t shared_len) {
  PagedPlan p{};
  const int G = s->num_q_heads / s->num_kv_heads;
  const int64_t B = s->batch, N = s->num_nodes, Hkv = s->num_kv_heads;
  const int nb = G <= kTcRows ? kTcRows / G : 1;
  p.nodes_per_tile = nb;
  p.rb_own = static_cast<int>((N + nb - 1) / nb);
  p.rb_sh = shared_len > 0 ? static_cast<int>((B * N + nb - 1) / nb) : 0;
  p.rows_own = static_cast<int>(N < nb ? N : nb) * G;
  p.rows_sh = static_cast<int>(B * N < nb ? B * N : nb) * G;
  p.own_row0 = shared_len > 0 ? 2 * (Hkv * ((p.rb_sh + 1) / 2) + kNumSMs) * p.rows_sh : 0;
  p.part_rows = p.own_row0 + 2 * (B * Hkv * ((p.rb_own + 1) / 2) + kNumSMs) * p.rows_own;
  const int64_t items = Hkv * ((p.rb_sh + 1) / 2 + B * ((p.rb_own + 1) / 2));
  p.plan_bytes = 256 + align256(static_cast<size_t>(items) * sizeof(int2));  // run_shared, cuts
  p.ml_bytes = align256(static_cast<size_t>(p.part_rows) * sizeof(float2));
  p.acc_bytes = align256(static_cast<size_t>(p.part_rows) * s->head_dim * sizeof(float));
  return p;
}

template <int D>
eagle_status_t launch_paged_tc(const eagle_shape_t* s, const eagle_pages_t* pg, const PagedAttnParams& ap,
                               const void* q, const void* kp, const void* vp, const void* kt, const void* vt,
                               void* out, void* ws, cudaStream_t st) {
  if (!register_shares_fit<paged_attn_tc_kernel<D>>(kPgThreads, kPgSoftRegs, kPgOtherRegs) ||
      !allow_smem<paged_attn_tc_kernel<D>>(PgSmem<D>::kAlloc))
    return EAGLE_ERR_CUDA;
  const PagedPlan plan = plan_paged(s, ap.shared);
  PagedTcParams p{};
  p.a = ap;
  p.out = static_cast<__nv_bfloat16*>(out);
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.run_shared = reinterpret_cast<int32_t*>(w);
  p.cuts = reinterpret_cast<int2*>(w + 256);
  p.part_ml = reinterpret_cast<float2*>(w + plan.plan_bytes);
  p.part_acc = reinterpret_cast<float*>(w + plan.plan_bytes + plan.ml_bytes);
  p.NB = plan.nodes_per_tile;
  p.rb_own = plan.rb_own;
  p.rb_sh = plan.rb_sh;
  p.rows_own = plan.rows_own;
  p.rows_sh = plan.rows_sh;
  p.own_row0 = plan.own_row0;
  p.box = pg->page_size < kHalf ? pg->page_size : kHalf;
  p.scale_log2 = ap.scale * 1.4426950408889634f;
  CUtensorMap tq, tk, tv, tkt, tvt;
  using u64 = cuuint64_t;
  const u64 Dn = D, Hq = ap.Hq, Hkv = ap.Hkv, N = ap.N, B = ap.B, ps = pg->page_size;
  // pages viewed as [num_pages][Hkv][page_size][D]: a box is `box` rows of one page and head
  const u64 kdims[4] = {Dn, ps, Hkv, static_cast<u64>(pg->num_pages)};
  const u64 kstrides[3] = {Dn * 2, ps * Dn * 2, Hkv * ps * Dn * 2};
  const cuuint32_t kbox[4] = {64, static_cast<cuuint32_t>(p.box), 1, 1};
  // queries viewed as [B * N, Hq, D]: a box is NB nodes x the G heads of a kv head
  const u64 qdims[3] = {Dn, Hq, B * N};
  const u64 qstrides[2] = {Dn * 2, Hq * Dn * 2};
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(ap.G), static_cast<cuuint32_t>(p.NB)};
  // tree K/V viewed as [B][N][Hkv][D]: a box is the node rows of (b, kv head), zeros past N
  const u64 tdims[4] = {Dn, Hkv, N, B};
  const u64 tstrides[3] = {Dn * 2, Hkv * Dn * 2, N * Hkv * Dn * 2};
  const cuuint32_t tbox[4] = {64, 1, static_cast<cuuint32_t>(kHalf), 1};
  if (!encode_bf16(&tk, kp, 4, kdims, kstrides, kbox) || !encode_bf16(&tv, vp, 4, kdims, kstrides, kbox) ||
      !encode_bf16(&tq, q, 3, qdims, qstrides, qbox) || !encode_bf16(&tkt, kt, 4, tdims, tstrides, tbox) ||
      !encode_bf16(&tvt, vt, 4, tdims, tstrides, tbox))
    return EAGLE_ERR_CUDA;
  // either kernel may be launched while the one before it on the stream ends, and waits for it
  // before it touches what that one may
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kNumSMs);
  cfg.blockDim = dim3(kPgThreads);
  cfg.dynamicSmemBytes = PgSmem<D>::kAlloc;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<D>, tq, tk, tv, tkt, tvt, p) != cudaSuccess) {
    cudaGetLastError();
    return EAGLE_ERR_CUDA;
  }
  const eagle_status_t rc = launch_status();
  if (rc != EAGLE_OK) return rc;
  // the merge: eight warps share a row's partials while that does not make more than a few
  // CTAs per SM
  const int64_t rows = static_cast<int64_t>(ap.B) * ap.N * ap.Hq;
  const bool split = (rows + 7) / 8 * (D / 16) <= 4 * kNumSMs;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kPgMergeRows - 1) / kPgMergeRows), split ? D / 16 : 1);
  cfg.blockDim = dim3(split ? 256 : 2 * D);
  cfg.dynamicSmemBytes = 0;
  const cudaError_t e = split ? cudaLaunchKernelEx(&cfg, paged_attn_merge_kernel<D, true>, p)
                              : cudaLaunchKernelEx(&cfg, paged_attn_merge_kernel<D, false>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return EAGLE_ERR_CUDA;
  }
  return launch_status();
}

// ------------------------------------------------------------------ e4m3 LM head

bool encode_bytes(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
  auto enc = get_encode();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {kScBlock, box_rows};
  const cuuint32_t es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <auto kKernel>
eagle_status_t launch_scaled(const CUtensorMap& tw, const CUtensorMap& th, const ScaledParams& prm,
                             unsigned grid, unsigned threads, size_t smem, cudaStream_t st) {
  if (!allow_smem<kKernel>(227 * 1024)) return EAGLE_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  // its set-up may overlap the end of the kernel before it (the quantiser); it waits for
  // that kernel before it touches global memory
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kKernel, tw, th, prm) != cudaSuccess) {
    cudaGetLastError();
    return EAGLE_ERR_CUDA;
  }
  return launch_status();
}

// A quantiser's values, e4m3 values and scales share no byte.
bool quantized_apart(const void* x, const void* x8, const float* scales, size_t n, int32_t dtype, size_t scale_bytes) {
  const size_t in = n * (dtype == EAGLE_DTYPE_F32 ? 4 : 2);
  return !overlap(x, in, x8, n) && !overlap(x, in, scales, scale_bytes) && !overlap(x8, n, scales, scale_bytes);
}

bool dtype_ok(int32_t dtype) { return dtype == EAGLE_DTYPE_F32 || dtype == EAGLE_DTYPE_BF16; }

}  // namespace
}  // namespace eagle

extern "C" {

eagle_status_t eagle_rope_append(const eagle_shape_t* shape, const eagle_pages_t* pages, const eagle_rope_t* rope,
                                 int32_t num_rows, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                 const void* v, int64_t v_stride, const int32_t* positions, const int32_t* seq_ids,
                                 const float* cos_sin, void* k_pages, void* v_pages, const int32_t* page_table,
                                 void* q_out, void* k_out, void* stream) {
  eagle_status_t rc = check_shape(shape);
  if (rc != EAGLE_OK) return rc;
  if (rope == nullptr || num_rows < 0) return EAGLE_ERR_INVALID_ARGUMENT;
  const int D = shape->head_dim, esize = elem_size(shape);
  const int64_t qw = static_cast<int64_t>(shape->num_q_heads) * D, kw = static_cast<int64_t>(shape->num_kv_heads) * D;
  if (qw > INT32_MAX || (rope->interleaved != 0 && rope->interleaved != 1)) return EAGLE_ERR_INVALID_ARGUMENT;
  if (rope->rotary_dim < 0 || rope->rotary_dim > D || rope->rotary_dim % 16 != 0) return EAGLE_ERR_INVALID_ARGUMENT;
  if (rope->rotary_dim > 0 && rope->table_len < 1) return EAGLE_ERR_INVALID_ARGUMENT;
  if (num_rows == 0) return EAGLE_OK;
  if (positions == nullptr || (rope->rotary_dim > 0 && !aligned16(cos_sin))) return EAGLE_ERR_INVALID_ARGUMENT;
  const int64_t n = num_rows;
  if ((q == nullptr) != (q_out == nullptr) || (q == nullptr && k == nullptr)) return EAGLE_ERR_INVALID_ARGUMENT;
  if ((q != nullptr && (!rows_ok(q, q_stride, qw, esize, n) || !aligned16(q_out))) ||
      (k != nullptr && !rows_ok(k, k_stride, kw, esize, n)) ||
      (seq_ids != nullptr && (k == nullptr || v == nullptr || !rows_ok(v, v_stride, kw, esize, n))))
    return EAGLE_ERR_INVALID_ARGUMENT;
  const RowSpan in[3] = {{q, q_stride, qw}, {k, k_stride, kw}, {seq_ids != nullptr ? v : nullptr, v_stride, kw}};
  if (q != nullptr && !rotated_out_ok(q_out, qw, 0, in, n, esize)) return EAGLE_ERR_INVALID_ARGUMENT;
  if (k_out != nullptr &&
      (k == nullptr || !aligned16(k_out) || !rotated_out_ok(k_out, kw, 1, in, n, esize) ||
       (q != nullptr && overlap(q_out, static_cast<size_t>(n * qw * esize), k_out,
                                static_cast<size_t>(n * kw * esize)))))
    return EAGLE_ERR_INVALID_ARGUMENT;
  AppendParams p{};
  if (seq_ids != nullptr) {
    rc = check_pages(pages);
    if (rc != EAGLE_OK) return rc;
    if (!aligned16(k_pages) || !aligned16(v_pages) || page_table == nullptr) return EAGLE_ERR_INVALID_ARGUMENT;
    const size_t pool = pool_bytes(pages, shape, esize);
    for (const void* cache : {k_pages, v_pages}) {
      if ((q != nullptr && overlap(q_out, static_cast<size_t>(n * qw * esize), cache, pool)) ||
          (k_out != nullptr && overlap(k_out, static_cast<size_t>(n * kw * esize), cache, pool)))
        return EAGLE_ERR_INVALID_ARGUMENT;
    }
    p.map = page_map(pages, page_table);
  } else if (k != nullptr && k_out == nullptr) {
    return EAGLE_ERR_INVALID_ARGUMENT;  // keys that go nowhere
  }
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.q_stride = q_stride * esize;
  p.k_stride = k_stride * esize;
  p.v_stride = v_stride * esize;
  p.positions = positions;
  p.seq_ids = seq_ids;
  p.cos_sin = cos_sin;
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.k_out = static_cast<uint8_t*>(k_out);
  p.B = shape->batch;
  p.Hq = shape->num_q_heads;
  p.Hkv = shape->num_kv_heads;
  p.table_len = rope->table_len;
  p.rd = rope->rotary_dim;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool il = rope->interleaved != 0;
  if (shape->dtype == EAGLE_DTYPE_F32) {
    D == 64 ? launch_append<float, 64>(p, il, num_rows, st) : launch_append<float, 128>(p, il, num_rows, st);
  } else {
    D == 64 ? launch_append<__nv_bfloat16, 64>(p, il, num_rows, st)
            : launch_append<__nv_bfloat16, 128>(p, il, num_rows, st);
  }
  return launch_status();
}

size_t eagle_paged_workspace_bytes(const eagle_shape_t* shape, const eagle_pages_t* pages, int32_t shared_len) {
  if (check_paged_shape(shape, pages, shared_len) != EAGLE_OK) return 0;
  return shape->dtype == EAGLE_DTYPE_BF16 ? plan_paged(shape, shared_len).bytes()
                                          : plan_paged_f32(shape, shared_len).bytes();
}

eagle_status_t eagle_tree_attention_paged(const eagle_shape_t* shape, const eagle_pages_t* pages, const void* q,
                                          const void* k_pages, const void* v_pages, const int32_t* page_table,
                                          const int32_t* prefix_lens, int32_t shared_len, const void* k_tree,
                                          const void* v_tree, const int32_t* parents, void* out, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  eagle_status_t rc = check_paged_shape(shape, pages, shared_len);
  if (rc == EAGLE_OK)
    rc = check_attention_args(shape, q, k_pages, v_pages, prefix_lens, k_tree, v_tree, parents, out, workspace,
                              workspace_bytes, eagle_paged_workspace_bytes(shape, pages, shared_len));
  if (rc != EAGLE_OK) return rc;
  if (page_table == nullptr) return EAGLE_ERR_INVALID_ARGUMENT;
  // inputs are read by some CTAs while others write outputs
  const int esize = elem_size(shape);
  const size_t nodes = static_cast<size_t>(shape->batch) * shape->num_nodes, row = nodes * shape->head_dim * esize;
  const size_t qn = row * shape->num_q_heads, tn = row * shape->num_kv_heads, pool = pool_bytes(pages, shape, esize);
  const size_t table = static_cast<size_t>(shape->batch) * pages->max_pages * sizeof(int32_t);
  if (overlap(out, qn, q, qn) || overlap(out, qn, k_tree, tn) || overlap(out, qn, v_tree, tn) ||
      overlap(out, qn, k_pages, pool) || overlap(out, qn, v_pages, pool) || overlap(out, qn, page_table, table) ||
      overlap(out, qn, prefix_lens, shape->batch * sizeof(int32_t)) ||
      overlap(out, qn, parents, nodes * sizeof(int32_t)))
    return EAGLE_ERR_INVALID_ARGUMENT;
  PagedAttnParams p{};
  p.map = page_map(pages, page_table);
  p.prefix_lens = prefix_lens;
  p.parents = parents;
  p.B = shape->batch;
  p.N = shape->num_nodes;
  p.Hq = shape->num_q_heads;
  p.Hkv = shape->num_kv_heads;
  p.G = p.Hq / p.Hkv;
  p.Lmax = shape->max_prefix_len;
  p.shared = shared_len;
  p.scale = softmax_scale(shape);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool d64 = shape->head_dim == 64;
  if (shape->dtype == EAGLE_DTYPE_BF16)
    return d64 ? launch_paged_tc<64>(shape, pages, p, q, k_pages, v_pages, k_tree, v_tree, out, workspace, st)
               : launch_paged_tc<128>(shape, pages, p, q, k_pages, v_pages, k_tree, v_tree, out, workspace, st);
  const PagedF32Plan plan = plan_paged_f32(shape, shared_len);
  if (plan.items > INT32_MAX) return EAGLE_ERR_UNSUPPORTED;
  auto run = [&](auto d, auto rt) {
    return launch_paged_f32<d(), rt()>(plan, q, k_pages, v_pages, k_tree, v_tree, out, workspace, p, st);
  };
  auto with_rows = [&](auto d) {
    switch (plan.rt) {
      case 4: return run(d, std::integral_constant<int, 4>());
      case 16: return run(d, std::integral_constant<int, 16>());
      case 32: return run(d, std::integral_constant<int, 32>());
      default: return run(d, std::integral_constant<int, 64>());
    }
  };
  return d64 ? with_rows(std::integral_constant<int, 64>()) : with_rows(std::integral_constant<int, 128>());
}

eagle_status_t eagle_commit_accepted_paged(const eagle_shape_t* shape, const eagle_pages_t* pages, void* k_pages,
                                           void* v_pages, const int32_t* page_table, const int32_t* prefix_lens,
                                           const void* k_tree, const void* v_tree, const void* hidden,
                                           const int32_t* parents, const int32_t* accepted_nodes,
                                           const int32_t* accept_len, int32_t* new_prefix_lens, void* feat,
                                           void* stream) {
  eagle_status_t rc = check_commit_args(shape, k_pages, v_pages, prefix_lens, k_tree, v_tree, hidden, parents,
                                        accepted_nodes, accept_len, new_prefix_lens, feat);
  if (rc == EAGLE_OK) rc = check_pages(pages);
  if (rc != EAGLE_OK) return rc;
  if (page_table == nullptr) return EAGLE_ERR_INVALID_ARGUMENT;
  const int esize = elem_size(shape);
  const size_t hn = static_cast<size_t>(shape->batch) * shape->num_nodes * shape->hidden * esize;
  if (overlap(feat, hn, hidden, hn)) return EAGLE_ERR_INVALID_ARGUMENT;  // (a gather)
  CommitPagedParams p{};
  p.k_pages = static_cast<uint8_t*>(k_pages);
  p.v_pages = static_cast<uint8_t*>(v_pages);
  p.map = page_map(pages, page_table);
  p.prefix_lens = prefix_lens;
  p.k_tree = static_cast<const uint8_t*>(k_tree);
  p.v_tree = static_cast<const uint8_t*>(v_tree);
  p.hidden = static_cast<const uint8_t*>(hidden);
  p.parents = parents;
  p.accepted_nodes = accepted_nodes;
  p.accept_len = accept_len;
  p.new_lens = new_prefix_lens;
  p.feat = static_cast<uint8_t*>(feat);
  p.N = shape->num_nodes;
  p.Hkv = shape->num_kv_heads;
  p.row_bytes = shape->head_dim * esize;
  p.hrow_bytes = shape->hidden * esize;
  const dim3 grid(shape->batch, shape->num_kv_heads + shape->num_nodes);
  commit_paged_kernel<<<grid, kCommitThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}

eagle_status_t eagle_quantize_rows(int32_t rows, int32_t cols, int32_t dtype, const void* x, void* x_out,
                                   float* scales, void* stream) {
  if (rows < 0 || cols < 16 || cols % 16 != 0 || !dtype_ok(dtype)) return EAGLE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return EAGLE_OK;
  if (!aligned16(x) || !aligned16(x_out) || !aligned16(scales)) return EAGLE_ERR_INVALID_ARGUMENT;
  if (rows > INT32_MAX - 3) return EAGLE_ERR_INVALID_ARGUMENT;
  const int kblocks = (cols + kScBlock - 1) / kScBlock, ldm = (rows + 3) / 4 * 4;
  if (!quantized_apart(x, x_out, scales, static_cast<size_t>(rows) * cols, dtype,
                       static_cast<size_t>(kblocks) * ldm * sizeof(float)))
    return EAGLE_ERR_INVALID_ARGUMENT;
  const int64_t grid = (static_cast<int64_t>(rows) * kblocks + 3) / 4;
  if (grid > INT32_MAX) return EAGLE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == EAGLE_DTYPE_F32)
    quantize_rows_kernel<float><<<static_cast<unsigned>(grid), 128, 0, st>>>(
        static_cast<const float*>(x), static_cast<uint8_t*>(x_out), scales, rows, cols, kblocks, ldm);
  else
    quantize_rows_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), 128, 0, st>>>(
        static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(x_out), scales, rows, cols, kblocks, ldm);
  return launch_status();
}

eagle_status_t eagle_quantize_blocks(int32_t rows, int32_t cols, int32_t dtype, const void* w, void* w_out,
                                     float* scales, void* stream) {
  if (rows < 0 || cols < 16 || cols % 16 != 0 || !dtype_ok(dtype)) return EAGLE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return EAGLE_OK;
  if (!aligned16(w) || !aligned16(w_out) || scales == nullptr || (reinterpret_cast<uintptr_t>(scales) & 3) != 0)
    return EAGLE_ERR_INVALID_ARGUMENT;
  const int kblocks = (cols + kScBlock - 1) / kScBlock;
  const int64_t grid = (static_cast<int64_t>(rows) + kScBlock - 1) / kScBlock * kblocks;
  if (!quantized_apart(w, w_out, scales, static_cast<size_t>(rows) * cols, dtype, grid * sizeof(float)))
    return EAGLE_ERR_INVALID_ARGUMENT;
  if (grid > INT32_MAX) return EAGLE_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == EAGLE_DTYPE_F32)
    quantize_blocks_kernel<float><<<static_cast<unsigned>(grid), 256, 0, st>>>(
        static_cast<const float*>(w), static_cast<uint8_t*>(w_out), scales, rows, cols, kblocks);
  else
    quantize_blocks_kernel<__nv_bfloat16><<<static_cast<unsigned>(grid), 256, 0, st>>>(
        static_cast<const __nv_bfloat16*>(w), static_cast<uint8_t*>(w_out), scales, rows, cols, kblocks);
  return launch_status();
}

eagle_status_t eagle_lm_head_logits_scaled(int32_t rows, int32_t hidden, int32_t vocab, const void* x,
                                           const float* x_scales, const void* w, const float* w_scales,
                                           float* logits, void* stream) {
  if (rows < 0 || hidden < 16 || hidden % 16 != 0 || vocab < 1) return EAGLE_ERR_INVALID_ARGUMENT;
  if (rows == 0) return EAGLE_OK;
  if (!aligned16(x) || !aligned16(x_scales) || !aligned16(w) || w_scales == nullptr ||
      (reinterpret_cast<uintptr_t>(w_scales) & 3) != 0 || logits == nullptr ||
      (reinterpret_cast<uintptr_t>(logits) & 3) != 0)
    return EAGLE_ERR_INVALID_ARGUMENT;
  const int64_t vtiles = (static_cast<int64_t>(vocab) + kScBlock - 1) / kScBlock;
  if (rows > (1 << 24) || vtiles > 65535) return EAGLE_ERR_UNSUPPORTED;
  const int KB = (hidden + kScBlock - 1) / kScBlock;
  const size_t out_bytes = static_cast<size_t>(rows) * vocab * sizeof(float);
  if (overlap(logits, out_bytes, x, static_cast<size_t>(rows) * hidden) ||
      overlap(logits, out_bytes, w, static_cast<size_t>(vocab) * hidden) ||
      overlap(logits, out_bytes, x_scales, static_cast<size_t>(KB) * ((rows + 3) / 4 * 4) * sizeof(float)) ||
      overlap(logits, out_bytes, w_scales, static_cast<size_t>(vtiles) * KB * sizeof(float)))
    return EAGLE_ERR_INVALID_ARGUMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tw, th;
  ScaledParams prm{logits, x_scales, w_scales, rows, vocab, hidden, KB, (rows + 3) / 4 * 4, 0, 0, 0};
  const bool few = rows <= kScFewRows;
  const int bn = few ? (rows + 15) / 16 * 16 : (rows <= 64 ? 64 : kScBlock);  // rows of a box of x
  if (!encode_bytes(&tw, w, static_cast<uint64_t>(hidden), static_cast<uint64_t>(vocab), kScBlock) ||
      !encode_bytes(&th, x, static_cast<uint64_t>(hidden), static_cast<uint64_t>(rows), static_cast<uint32_t>(bn)))
    return EAGLE_ERR_CUDA;
  if (few) {
    // two CTAs per SM, each with as deep a ring as fits
    int stages = 2;
    while (stages < 8 && scaled_smem_bytes(bn, stages + 1) <= 113 * 1024) ++stages;
    prm.bn = bn;
    prm.stages = stages;
    const size_t smem = scaled_smem_bytes(bn, stages);
    const unsigned grid = static_cast<unsigned>(vtiles);
    return launch_scaled<lm_head_scaled_kernel>(tw, th, prm, grid, kScThreads, smem, st);
  }
  // two vocabulary blocks a tile (two thirds of the shared-memory bytes per product) while
  // there are six of them per SM, so that the last round of tiles is a small part
  const int row_tiles = (rows + kScBlock - 1) / kScBlock;
  const int64_t wide = (vtiles + 1) / 2 * row_tiles;
  const int nv = wide >= 6 * kNumSMs && rows > 64 ? 2 : 1;
  prm.bn = row_tiles;
  prm.stages = static_cast<int32_t>((vtiles + nv - 1) / nv);
  prm.vec = vocab % 4 == 0 && aligned16(logits);
  const int64_t tiles = static_cast<int64_t>(prm.stages) * row_tiles;
  const unsigned grid = static_cast<unsigned>(tiles < kNumSMs ? tiles : kNumSMs);
  if (nv == 2) {
    if (!register_shares_fit<lm_head_scaled_rows_kernel<2, 128>>(kScRowsThreads, kScRowsEpiRegs, kScRowsOtherRegs))
      return EAGLE_ERR_CUDA;
    return launch_scaled<lm_head_scaled_rows_kernel<2, 128>>(tw, th, prm, grid, kScRowsThreads,
                                                             ScaledRowsCfg<2, 128>::kAlloc, st);
  }
  if (rows <= 64)
    return launch_scaled<lm_head_scaled_rows_kernel<1, 64>>(tw, th, prm, grid, kScRowsThreads,
                                                            ScaledRowsCfg<1, 64>::kAlloc, st);
  return launch_scaled<lm_head_scaled_rows_kernel<1, 128>>(tw, th, prm, grid, kScRowsThreads,
                                                           ScaledRowsCfg<1, 128>::kAlloc, st);
}

}  // extern "C"
