// paged.cuh -- the paged K/V cache: page look-up, the append of new tokens with the rotary
// position embedding applied on the way, and the post-accept commit into pages.
//
// Layout: k_pages, v_pages [num_pages, Hkv, page_size, D]; position p of sequence b lives on
// page page_table[b, p / page_size], row p % page_size of every kv head.  page_size is a
// power of two, so both are shifts and masks.
#pragma once

#include "commit.cuh"
#include "device_common.cuh"

namespace eagle {

enum PagedError : int32_t {
  kErrPageIndex = 0x206,     // a page index outside [0, num_pages)
  kErrAppendRow = 0x401,     // a position or sequence index outside the cache or the angle table
};

struct PageMap {
  const int32_t* table;  // [B, max_pages]
  int32_t num_pages;
  int32_t page_shift;    // log2(page_size)
  int32_t max_pages;
};

// Page of position p of sequence b (p / page_size < max_pages), or -1 with the error
// recorded when the table holds none.
__device__ __forceinline__ int32_t page_of(const PageMap& m, int b, int p) {
  const int32_t pg = m.table[static_cast<size_t>(b) * m.max_pages + (p >> m.page_shift)];
  if (pg < 0 || pg >= m.num_pages) {
    record_error(kErrPageIndex);
    return -1;
  }
  return pg;
}
// Element offset of (page, head g, position p's row) in the page pool.
__device__ __forceinline__ size_t page_row(const PageMap& m, int32_t page, int g, int Hkv, int p, int D) {
  const int row = p & ((1 << m.page_shift) - 1);
  return ((((static_cast<size_t>(page) * Hkv + g) << m.page_shift) + row) * D);
}

// ------------------------------------------------------------------ append with rotation
// For row r at position p and each head x of its query and key, with (a, b) the pair
// (x[i], x[i + rd/2]) (halves) or (x[2i], x[2i + 1]) (interleaved), i < rd/2:
//     a' = a cos(p, i) - b sin(p, i),   b' = b cos(p, i) + a sin(p, i)
// in fp32 from the table's fp32 cosines and sines, rounded once to the cache's type; columns
// past rd are copied.
//
// Pure streaming: every element is read once and written once.  One CTA per row, so the
// row's cosines come from L1 after the first head; a thread takes two 16-byte chunks at a
// time (for halves the two that hold the pairs), all loads before the stores.  8,191 rows of
// 32/8 heads of 128 in bf16: 35 us, 5.8 TB/s, HBM-bound; 8 rows: 2.8 us, of which an empty
// launch is 2.2.

struct AppendParams {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  int64_t q_stride, k_stride, v_stride;  // bytes between rows
  const int32_t* positions;
  const int32_t* seq_ids;  // NULL: nothing goes to the cache
  const float* cos_sin;    // [table_len, rd]: rd/2 cosines, then rd/2 sines
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* q_out;          // [R, Hq, D]
  uint8_t* k_out;          // [R, Hkv, D] or NULL
  PageMap map;
  int32_t B, Hq, Hkv, table_len, rd;
};

template <typename T>
struct AppendVec;
template <>
struct AppendVec<float> {
  static constexpr int kN = 4;  // elements of a 16-byte chunk
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <>
struct AppendVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};

constexpr int kAppendThreads = 128;

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) rope_append_kernel(const AppendParams p) {
  using V = AppendVec<T>;
  constexpr int N = V::kN;
  constexpr int kItems = D / (2 * N);  // two-chunk items of a head
  const int r = blockIdx.x;
  const int pos = p.positions[r];
  if (pos < 0) return;  // a padding row
  const int seq = p.seq_ids != nullptr ? p.seq_ids[r] : -1;
  // the whole row is checked before any of it is written
  bool ok = (p.rd == 0 || pos < p.table_len) && seq >= -1 && seq < p.B;
  const bool cached = ok && seq >= 0;
  ok = ok && (!cached || (pos >> p.map.page_shift) < p.map.max_pages);
  if (!ok) {
    if (threadIdx.x == 0) record_error(kErrAppendRow);
    return;
  }
  const int32_t page = cached ? page_of(p.map, seq, pos) : 0;
  if (page < 0) return;
  const float* cs = p.cos_sin + static_cast<size_t>(pos) * p.rd;
  const int hq = p.q != nullptr ? p.Hq : 0;
  const int hk = p.k != nullptr ? p.Hkv : 0;
  const int hv = cached ? p.Hkv : 0;
  const int half = p.rd / 2;
  for (int item = threadIdx.x; item < (hq + hk + hv) * kItems; item += kAppendThreads) {
    int h = item / kItems;
    const int c = item % kItems;
    const int kind = h < hq ? 0 : (h < hq + hk ? 1 : 2);  // query, key, value
    h -= kind == 0 ? 0 : (kind == 1 ? hq : hq + hk);
    const uint8_t* src = kind == 0   ? p.q + static_cast<int64_t>(r) * p.q_stride
                         : kind == 1 ? p.k + static_cast<int64_t>(r) * p.k_stride
                                     : p.v + static_cast<int64_t>(r) * p.v_stride;
    src += static_cast<size_t>(h) * D * sizeof(T);
    // columns of the item's two chunks: the two members of its pairs, or neighbours
    const bool turn = kind != 2 && c * 2 * N < p.rd;
    int d0 = c * 2 * N, d1 = d0 + N;
    if (!kInterleaved && turn) {
      d0 = c * N;
      d1 = half + c * N;
    }
    const uint4 w0 = *reinterpret_cast<const uint4*>(src + d0 * sizeof(T));
    const uint4 w1 = *reinterpret_cast<const uint4*>(src + d1 * sizeof(T));
    uint4 o0 = w0, o1 = w1;
    if (turn) {
      float a[N], b[N];
      V::unpack(w0, a);
      V::unpack(w1, b);
      if (kInterleaved) {
        // pairs are neighbours: chunk 0 holds the pairs from d0 / 2, chunk 1 from d1 / 2
        float x[N], y[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          const float c0 = cs[d0 / 2 + i], s0 = cs[half + d0 / 2 + i];
          const float c1 = cs[d1 / 2 + i], s1 = cs[half + d1 / 2 + i];
          x[2 * i] = a[2 * i] * c0 - a[2 * i + 1] * s0;
          x[2 * i + 1] = a[2 * i + 1] * c0 + a[2 * i] * s0;
          y[2 * i] = b[2 * i] * c1 - b[2 * i + 1] * s1;
          y[2 * i + 1] = b[2 * i + 1] * c1 + b[2 * i] * s1;
        }
        o0 = V::pack(x);
        o1 = V::pack(y);
      } else {
        float x[N], y[N];
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 c4 = *reinterpret_cast<const float4*>(cs + d0 + i);
          const float4 s4 = *reinterpret_cast<const float4*>(cs + half + d0 + i);
          const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i + j] = a[i + j] * cc[j] - b[i + j] * ss[j];
            y[i + j] = b[i + j] * cc[j] + a[i + j] * ss[j];
          }
        }
        o0 = V::pack(x);
        o1 = V::pack(y);
      }
    }
    auto store = [&](uint8_t* dst) {
      *reinterpret_cast<uint4*>(dst + d0 * sizeof(T)) = o0;
      *reinterpret_cast<uint4*>(dst + d1 * sizeof(T)) = o1;
    };
    if (kind == 0) {
      store(p.q_out + (static_cast<size_t>(r) * p.Hq + h) * D * sizeof(T));
    } else {
      if (cached)
        store((kind == 1 ? p.k_pages : p.v_pages) + page_row(p.map, page, h, p.Hkv, pos, D) * sizeof(T));
      if (kind == 1 && p.k_out != nullptr)
        store(p.k_out + (static_cast<size_t>(r) * p.Hkv + h) * D * sizeof(T));
    }
  }
}

// ------------------------------------------------------------------ commit into pages
// commit_kernel (commit.cuh) with the cache rows found through the page table: the same
// checks of the path, plus every page the new rows land on, before anything is written.
// Latency-bound: path, page and copy follow one another.  One walk of a 45-node tree, 32 kv
// heads of 128: 2.8 us; 64 walks of 60-node trees, 8 kv heads, hidden 8192: 4.4 us.

struct CommitPagedParams {
  uint8_t* k_pages;
  uint8_t* v_pages;
  PageMap map;
  const int32_t* prefix_lens;
  const uint8_t* k_tree;
  const uint8_t* v_tree;
  const uint8_t* hidden;
  const int32_t* parents;
  const int32_t* accepted_nodes;
  const int32_t* accept_len;
  int32_t* new_lens;
  uint8_t* feat;
  int32_t N, Hkv;
  int32_t row_bytes;   // D * esize
  int32_t hrow_bytes;  // H * esize
};

__global__ void __launch_bounds__(kCommitThreads) commit_paged_kernel(const CommitPagedParams p) {
  __shared__ int32_t path[64];
  __shared__ int32_t page[64];  // page of each new row
  const int b = blockIdx.x;
  const int N = p.N;
  const size_t seq = static_cast<size_t>(b) * N;
  const int32_t L = p.prefix_lens[b];
  const int32_t a = p.accept_len[b];
  // a row of the path: the root, then an accepted node, a child of the row before it (read
  // before it is known whether there is such a row: a load's latency less)
  const int row = threadIdx.x;
  const int32_t c = row == 0 || row >= N ? 0 : p.accepted_nodes[seq + row - 1];
  const int32_t prev = row <= 1 || row >= N ? 0 : p.accepted_nodes[seq + row - 2];
  if (a == -1) {  // the walk found the tree invalid: nothing committed, length unchanged
    if (blockIdx.y == 0 && threadIdx.x == 0) p.new_lens[b] = L;
    return;
  }
  const int64_t cap = static_cast<int64_t>(p.map.max_pages) << p.map.page_shift;
  const bool shape_ok = a >= 0 && a <= N - 1 && L >= 0 && static_cast<int64_t>(L) + a + 1 <= cap;
  int ok = 1;
  if (shape_ok && static_cast<int>(blockIdx.y) - p.Hkv > a) return;  // a hidden row past the path
  if (shape_ok && row <= a) {
    ok = row == 0 || (c >= 1 && c < N && p.parents[seq + c] == prev);
    const int32_t pg = page_of(p.map, b, L + row);
    ok = ok && pg >= 0;
    path[row] = c;
    page[row] = pg;
  }
  ok = __syncthreads_and(ok) && shape_ok;
  if (!ok) {
    if (blockIdx.y == 0 && threadIdx.x == 0) p.new_lens[b] = -1;
    return;
  }
  const int n = a + 1;
  if (blockIdx.y == 0 && threadIdx.x == 0) p.new_lens[b] = L + n;
  const int y = blockIdx.y;
  if (y < p.Hkv) {
    const int g = y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < 2 * n; r += kCommitThreads / 32) {
      const int t = r >> 1;
      const bool is_v = r & 1;
      const size_t src = ((seq + path[t]) * p.Hkv + g) * p.row_bytes;
      const size_t dst = page_row(p.map, page[t], g, p.Hkv, L + t, p.row_bytes);
      commit_copy((is_v ? p.v_pages : p.k_pages) + dst, (is_v ? p.v_tree : p.k_tree) + src, p.row_bytes, lane,
                  32);
    }
  } else {
    const int t = y - p.Hkv;
    commit_copy(p.feat + (seq + t) * p.hrow_bytes, p.hidden + (seq + path[t]) * p.hrow_bytes, p.hrow_bytes,
                threadIdx.x, kCommitThreads);
  }
}

}  // namespace eagle
