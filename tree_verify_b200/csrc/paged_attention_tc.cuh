// paged_attention_tc.cuh -- tree attention over a paged, partly shared K/V cache on the
// 5th-generation tensor cores (bf16).
//
//   out = softmax(scale q K^T) V   over the shared positions, the sequence's own positions
//   and the node's ancestors; with parts p of the keys and m_p, l_p, a_p their maximum,
//   sum and accumulator, out = sum_p 2^(m_p - m) a_p / sum_p 2^(m_p - m) l_p.
//
// Work is cut into items.  A shared item is (kv head, pair of 128-row tiles) over the shared
// positions; its rows are the B * N nodes of the whole batch x the G heads of the kv head,
// so the shared K/V is read for 256 rows at a time whatever sequence they belong to.  An own
// item is (sequence, kv head, pair of row tiles) over the sequence's own positions and its
// tree.  Keys go in tiles of 128.
//
// The lengths live on the device, so the plan is made there: items are laid end to end on
// a line of units (paged_tile_units for a key tile, kPgItemCost more for an item) and the
// line is cut into one equal piece for each of P CTAs, one CTA per SM.  Every CTA finds
// its piece by a scan over the batch's lengths.  A piece that begins or ends inside an item
// leaves a partial result; a second kernel merges each row's partials.
//
// A CTA runs two softmax groups of 128 threads (thread = query row), each with its own
// scores S and accumulator O in TMEM and its own chain S = Q K^T, softmax, O += P V; one
// group's softmax runs under the other's MMAs.  With two row tiles in the item the groups
// take one each and share every K/V tile; with one, they take the even and the odd tiles of
// the CTA's run and add up their sums at the end of an item (an item of one tile is one
// group's alone, and the next item the other's).
//
//   warps 0-3, 4-7   softmax groups 0 and 1
//   warp 8           TMA of the K and V tiles: one box per page and 64 columns, a lane each
//   warps 9, 10      one thread each: MMAs of groups 0 and 1, and TMA of their Q tiles
//   warp 11          walks the CTA's items and hands their descriptions to the others
// P of a tile lies over its S, so a group's next S is issued when its P V has completed.
// P V of a tile's first 64 keys is issued while the softmax of the others runs.
//
// Measured, main kernel and merge: 64 nodes x 8 sequences, 32/8 heads of 128, 8192 shared and
// 131..512 own keys: 82 us, 870 TFLOP/s; there the softmax chain of a tile (some 890
// instructions a thread) bounds it, beside 2,048 of 3,750 clocks of MMAs.  60 nodes x 16
// sequences of 32/32 heads over 500 + 12..3596 keys: 123.5 us, 4.15 TB/s, a tile's chain of
// loads, MMAs and softmax.  One token of each of 32 sequences of 32/8 heads over 2000..6000
// keys: 93 us, 5.6 TB/s, HBM.  One token over 4097 keys: 14.6 us, latency.
#pragma once

#include "attention.cuh"
#include "paged_attention.cuh"

namespace eagle {

constexpr int kPgThreads = 32 * 12;
constexpr int kPgLoadWarp = 8, kPgMmaWarp = 9, kPgItemWarp = 11;
constexpr int kPgReaders = 11;                // readers of an item: 8 softmax warps, the loads, 2 MMA issuers
constexpr int kHalf = kAttnKeys / 2;          // keys of half a tile; rows that a tree has at most
constexpr int kPgItems = 2;                   // items described ahead
constexpr int kPgItemCost = 8;                // units of an item beyond its tiles (see paged_tile_units)
constexpr float kPgRescaleThreshold = 8.0f;   // log2 units
constexpr int kPgPolyPairs = 1;               // of 8 pairs, through the polynomial 2^x (2 % of pair tiles' time)
constexpr int kPgSoftRegs = 208, kPgOtherRegs = 88;  // of the launch's 168 x 384 registers

struct PagedTcParams {
  PagedAttnParams a;
  __nv_bfloat16* out;
  float* part_acc;      // [partial rows, D]: see paged_part_row
  float2* part_ml;      // [partial rows]
  int32_t* run_shared;  // whether the shared part runs
  int2* cuts;           // [items]: the CTAs with an item's first and last tile (see paged_item)
  int32_t NB;           // nodes of a row tile (G * NB <= 128)
  int32_t rb_own, rb_sh;      // row tiles of a sequence, of the batch (0 without a shared part)
  int32_t rows_own, rows_sh;  // rows of a tile that can be real
  int64_t own_row0;           // first partial row of the own part
  int32_t box;          // rows of a TMA box: min(page size, 64)
  float scale_log2;
};

// One sequence's own part.
struct PagedSeq {
  int32_t L;      // its length, clamped
  int32_t begin;  // first own position
  int32_t t0;     // position of tile 0's first key (begin, rounded down to a box)
  int32_t T;      // tiles: of the keys, and of the tree, which takes the upper half of the last
                  // key tile where that one leaves it free, else a tile of its own
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedTcParams& p, int b) {
  PagedSeq s;
  const int L = p.a.prefix_lens[b];
  s.L = L < 0 ? 0 : (L > p.a.Lmax ? p.a.Lmax : L);
  s.begin = s.L >= p.a.shared ? p.a.shared : 0;
  s.t0 = s.begin & ~(p.box - 1);
  const int keys = s.L > s.begin ? s.L - s.t0 : 0;
  s.T = (keys + kAttnKeys / 2 + kAttnKeys - 1) / kAttnKeys;
  return s;
}

// Units of a key tile for `nrow` row tiles: a pair costs about 3,750 clocks, bound by its
// softmax and MMAs; a single row tile half of that, or 2,800 while its K/V come from HBM.
// (All measured with heads of 128; heads of 64 are cut by the same weights, unmeasured.)
__device__ __forceinline__ int paged_tile_units(int nrow) { return nrow == 2 ? 4 : 3; }
// Units of `T` tiles over `rb` row tiles of one kv head.
__device__ __forceinline__ int64_t paged_head_units(int T, int rb) {
  return static_cast<int64_t>(rb >> 1) * (4 * T + kPgItemCost) + (rb & 1) * (3 * T + kPgItemCost);
}
// First unit of row pair pi among its head's.
__device__ __forceinline__ int64_t paged_pair_units(int T, int pi) {
  return static_cast<int64_t>(pi) * (4 * T + kPgItemCost);
}
// Quotient of non-negative numbers, by the short division where it does.
__device__ __forceinline__ int64_t paged_div(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// Pieces of a line of W units: no more than units, so that none is empty.
__device__ __forceinline__ int paged_pieces(int64_t W) { return W < kNumSMs ? static_cast<int>(W) : kNumSMs; }
// Piece c of P is [c W / P, (c + 1) W / P), of one unit each if W < kNumSMs.
__device__ __forceinline__ int64_t paged_cut(int c, int64_t W) {
  return W < kNumSMs ? c : static_cast<int64_t>(static_cast<uint64_t>(c * W) / kNumSMs);
}

// Walks the items of a piece [lo, hi) of the line.
struct PagedCursor {
  int64_t u0;    // first unit of the item
  int32_t b;     // sequence, -1 in the shared part
  int32_t kvh, pi, rb, T;
  PagedSeq s;
  __device__ __forceinline__ int nrow() const { return min(2, rb - 2 * pi); }

  __device__ __forceinline__ void set_seq(const PagedTcParams& p) {
    rb = p.rb_own;
    if (b < p.a.B) {
      s = paged_seq(p, b);
      T = s.T;
    }
  }
  // at unit lo; first_b, first_base: the own sequence that holds lo (or sequence 0) and its start
  __device__ __forceinline__ void init(const PagedTcParams& p, int64_t lo, int64_t shared_units, int first_b,
                                       int64_t first_base) {
    int64_t base = 0;
    if (lo < shared_units) {
      b = -1;
      rb = p.rb_sh;
      T = (p.a.shared + kAttnKeys - 1) / kAttnKeys;
      s.L = p.a.shared;
      s.begin = s.t0 = 0;
      s.T = T;
    } else {
      b = first_b;
      base = first_base;
      set_seq(p);
    }
    const int64_t per = paged_head_units(T, rb);
    kvh = static_cast<int32_t>(paged_div(lo - base, per));
    const int64_t r = lo - base - kvh * per;
    pi = rb <= 2 ? 0
                 : static_cast<int32_t>(min(paged_div(r, 4 * static_cast<int64_t>(T) + kPgItemCost),
                                            static_cast<int64_t>(((rb + 1) >> 1) - 1)));
    u0 = base + kvh * per + paged_pair_units(T, pi);
  }
  __device__ __forceinline__ void next(const PagedTcParams& p) {
    u0 += static_cast<int64_t>(paged_tile_units(nrow())) * T + kPgItemCost;
    if (++pi < ((rb + 1) >> 1)) return;
    pi = 0;
    if (++kvh < p.a.Hkv) return;
    kvh = 0;
    ++b;
    set_seq(p);
  }
  // the item's tiles [a, z) that start in [lo, hi)
  __device__ __forceinline__ void range(int64_t lo, int64_t hi, int& a, int& z) const {
    a = tiles_before(lo);
    z = tiles_before(hi);
  }
  __device__ __forceinline__ int tiles_before(int64_t at) const {
    if (at <= u0) return 0;
    const bool pair = nrow() == 2;
    if (at - u0 >= static_cast<int64_t>(pair ? 4 : 3) * T) return T;
    const uint32_t u = static_cast<uint32_t>(at - u0);  // (T < 2^25)
    return static_cast<int>(pair ? (u + 3) / 4 : (u + 2) / 3);
  }
};

// Index of an item among the shared or the own ones, and among all (shared ones first).
__device__ __forceinline__ int64_t paged_item(const PagedTcParams& p, int b, int kvh, int pi) {
  if (b < 0) return static_cast<int64_t>(kvh) * ((p.rb_sh + 1) >> 1) + pi;
  return (static_cast<int64_t>(b) * p.a.Hkv + kvh) * ((p.rb_own + 1) >> 1) + pi;
}
__device__ __forceinline__ int64_t paged_item_of_all(const PagedTcParams& p, int b, int64_t item) {
  return b < 0 ? item : static_cast<int64_t>(p.a.Hkv) * ((p.rb_sh + 1) >> 1) + item;
}
// Row of the partials where CTA `cta`'s run of an item begins, for group g.  Along the line
// either the item or the CTA grows from run to run, so item + CTA names a run.
__device__ __forceinline__ int64_t paged_part_row(const PagedTcParams& p, int b, int64_t item, int cta, int g) {
  if (b < 0) return (2 * (item + cta) + g) * p.rows_sh;
  return p.own_row0 + (2 * (item + cta) + g) * p.rows_own;
}

// One CTA's run of an item, as the item warp describes it.
struct PagedRun {
  int32_t b;       // sequence, -1 in the shared part, kPgEnd after the last item
  int32_t kvh;
  int32_t a, z;    // tiles [a, z); none when no tile starts in the piece
  int32_t n;       // index of the tile with the tree, the last (none in the shared part)
  int32_t L, begin, t0;
  int32_t nrow;    // row tiles: 2, or 1 whose key tiles the groups take in turn
  int32_t node0;   // first node of row tile 0, in the sequence or (shared) in the batch
  int64_t prow;    // first partial row, of group 0
};
constexpr int32_t kPgEnd = -2;

template <int D>
struct PgSmem {
  static constexpr int kKStages = D == 128 ? 3 : 6;
  static constexpr int kVStages = D == 128 ? 2 : 5;
  static constexpr int kTile = kAttnKeys * D * 2;
  static constexpr int kQOff = 0;                       // two Q tiles
  static constexpr int kKOff = kQOff + 2 * kTile;
  static constexpr int kVOff = kKOff + kKStages * kTile;
  static constexpr int kAncOff = kVOff + kVStages * kTile;       // 64 masks
  static constexpr int kRunOff = kAncOff + 64 * 8;
  // the groups' exchange, [128] float2; before the first item the plan's warp sums and minima
  static constexpr int kXchOff = kRunOff + kPgItems * static_cast<int>(sizeof(PagedRun));
  static constexpr int kFirstOff = kXchOff + 128 * 8;
  static constexpr int kBarOff = kFirstOff + 16;
  // q_full[2], k_full, k_empty, v_full, v_empty, s_full[2], p_half[2], p_full[2], pv_done[2],
  // turn[2], all_done[2],
  // item_full, item_empty, met
  static constexpr int kNumBars = 2 + 2 * kKStages + 2 * kVStages + 12 + 2 * kPgItems + 1;
  static constexpr int kBytes = kBarOff + kNumBars * 8 + 16;
  static constexpr int kAlloc = kBytes + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kOCol = 2 * kAttnKeys;      // O of group g at kOCol + g D
  static_assert(kAlloc <= 227 * 1024, "shared memory");
  static_assert(kXchOff % 8 == 0 && kBarOff % 8 == 0, "alignment");
};

template <int D>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kt,
                         const __grid_constant__ CUtensorMap tm_vt, const __grid_constant__ PagedTcParams prm) {
  using SM = PgSmem<D>;
  constexpr int SK = SM::kKStages, SV = SM::kVStages;
  extern __shared__ uint8_t pg_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pg_smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  uint64_t* anc = reinterpret_cast<uint64_t*>(smem + SM::kAncOff);
  PagedRun* runs = reinterpret_cast<PagedRun*>(smem + SM::kRunOff);
  int64_t* scan_s = reinterpret_cast<int64_t*>(smem + SM::kXchOff);
  int32_t* live_s = reinterpret_cast<int32_t*>(scan_s + 16);
  float2* xch = reinterpret_cast<float2*>(smem + SM::kXchOff);
  int64_t* first_base_s = reinterpret_cast<int64_t*>(smem + SM::kFirstOff);
  int32_t* first_b_s = reinterpret_cast<int32_t*>(first_base_s + 1);
  const uint32_t q_full = sbase + SM::kBarOff;
  const uint32_t k_full = q_full + 16, k_empty = k_full + 8 * SK;
  const uint32_t v_full = k_empty + 8 * SK, v_empty = v_full + 8 * SV;
  const uint32_t s_full = v_empty + 8 * SV, p_half = s_full + 16, p_full = p_half + 16;
  const uint32_t pv_done = p_full + 16, turn = pv_done + 16, all_done = turn + 16;
  const uint32_t item_full = all_done + 16, item_empty = item_full + 8 * kPgItems;
  const uint32_t met = item_empty + 8 * kPgItems;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kBarOff + SM::kNumBars * 8);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = prm.a.B, N = prm.a.N, G = prm.a.G, Hkv = prm.a.Hkv;
  const int cta = blockIdx.x;

  // ------------------------------------------------------------ set-up and plan
  if (tid == 32 * kPgItemWarp) {  // (not a thread that reads lengths in an ordinary batch)
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_full + 8 * g, 1);
      mbar_init(s_full + 8 * g, 1);
      mbar_init(p_half + 8 * g, 4);  // one arrival per warp of the group
      mbar_init(p_full + 8 * g, 4);
      mbar_init(pv_done + 8 * g, 1);
      mbar_init(turn + 8 * g, 1);
      mbar_init(all_done + 8 * g, 1);
    }
    for (int s = 0; s < SK; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(k_empty + 8 * s, 2);  // either group
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(v_full + 8 * s, 1);
      mbar_init(v_empty + 8 * s, 2);
    }
    for (int s = 0; s < kPgItems; ++s) {
      mbar_init(item_full + 8 * s, 1);
      mbar_init(item_empty + 8 * s, kPgReaders);
    }
    mbar_init(met, 8);  // one arrival per warp of both groups
    fence_mbar_init();
  }
  if (warp == kPgMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), SM::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();  // nothing that another kernel writes is read or written before
  // each thread sums the units of a run of sequences; a block scan gives their starts
  const int chunk = (B + kPgThreads - 1) / kPgThreads;
  const int sb0 = min(B, tid * chunk), sb1 = min(B, sb0 + chunk);
  int64_t sum = 0;
  int first_long = INT32_MAX;  // a sequence that holds the whole shared part
  for (int b = sb0; b < sb1; ++b) {
    const PagedSeq s = paged_seq(prm, b);
    sum += Hkv * paged_head_units(s.T, prm.rb_own);
    if (s.L >= prm.a.shared) first_long = min(first_long, b);
    if (cta == 0) {
      const int raw = prm.a.prefix_lens[b];
      if (raw < 0 || raw > prm.a.Lmax) record_error(kErrAttnPrefixLen);
    }
  }
  int64_t incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  first_long = __reduce_min_sync(0xffffffffu, first_long);
  if (lane == 31) {
    scan_s[warp] = incl;
    live_s[warp] = first_long;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t start = incl - sum, own_units = 0;
#pragma unroll
  for (int w = 0; w < kPgThreads / 32; ++w) {
    if (w < warp) start += scan_s[w];
    own_units += scan_s[w];
    first_long = min(first_long, live_s[w]);
  }
  const bool run_shared = prm.a.shared > 0 && first_long < B;
  const int64_t shared_units =
      run_shared ? Hkv * paged_head_units((prm.a.shared + kAttnKeys - 1) / kAttnKeys, prm.rb_sh) : 0;
  const int64_t W = shared_units + own_units;
  const int P = paged_pieces(W);
  const int64_t lo = cta < P ? paged_cut(cta, W) : W, hi = cta < P ? paged_cut(cta + 1, W) : W;
  start += shared_units;
  if (cta == 0 && tid == 0) *prm.run_shared = run_shared ? 1 : 0;
  {
    const int64_t at = max(lo, shared_units);  // the first own unit this CTA may meet
    int64_t u = start;
    if (at >= start && at < start + sum) {
      for (int b = sb0; b < sb1; ++b) {
        const int64_t units = chunk == 1 ? sum : Hkv * paged_head_units(paged_seq(prm, b).T, prm.rb_own);
        if (at >= u && at < u + units) {
          *first_b_s = b;
          *first_base_s = u;
        }
        u += units;
      }
    }
  }
  __syncthreads();
  pdl_launch_dependents();  // the merge waits for this grid
  const uint32_t tmem = *tmem_slot;
  // the i-th description: wait for it, take a copy, release it (a warp's lane 0, once the
  // warp has what it needs)
  auto run_wait = [&](int i, int32_t err) { return mbar_wait(item_full + 8 * (i % kPgItems), (i / kPgItems) & 1, err); };
  auto run_release = [&](int i) { mbar_arrive(item_empty + 8 * (i % kPgItems)); };

  if (warp >= 8) {
    reg_dec<kPgOtherRegs>();
    if (warp == kPgItemWarp) {
      // ---------------------------------------------------------- items
      int i = 0, mask_b = -1;  // the masks are of sequence mask_b
      bool ok = true;
      PagedCursor cur;
      if (lo < hi)
        cur.init(prm, lo, shared_units, *first_b_s, *first_base_s);
      else
        cur.u0 = hi;
      for (;;) {
        const bool end = cur.u0 >= hi;
        int a = 0, z = 0;
        if (!end) {
          // (a piece that ends in what an item costs beyond its tiles has no run of it)
          if (lo >= cur.u0 + static_cast<int64_t>(paged_tile_units(cur.nrow())) * cur.T) {
            cur.next(prm);
            continue;
          }
          cur.range(lo, hi, a, z);
        }
        // the ancestor masks of the tree: a node and every node up its parent chain (a link
        // that does not point to an earlier node ends it); lane j has nodes j and j + 32
        uint64_t m0 = 0, m1 = 0;
        const bool tree = !end && cur.b >= 0 && z == cur.T && cur.b != mask_b;
        if (tree) {
          const int32_t* par = prm.a.parents + static_cast<size_t>(cur.b) * N;
          const int j0 = lane, j1 = lane + 32;
          const int q0 = j0 < N ? par[j0] : -1, q1 = j1 < N ? par[j1] : -1;
          const int p0 = q0 < j0 ? q0 : -1, p1 = q1 < j1 ? q1 : -1;  // negative: no parent
          int a0 = j0, a1 = j1;
          while (__any_sync(0xffffffffu, a0 >= 0 || a1 >= 0)) {
            if (a0 >= 0) m0 |= 1ull << a0;
            if (a1 >= 0) m1 |= 1ull << a1;
            const int u00 = __shfl_sync(0xffffffffu, p0, a0 & 31), u01 = __shfl_sync(0xffffffffu, p1, a0 & 31);
            const int u10 = __shfl_sync(0xffffffffu, p0, a1 & 31), u11 = __shfl_sync(0xffffffffu, p1, a1 & 31);
            a0 = a0 < 0 ? -1 : (a0 < 32 ? u00 : u01);
            a1 = a1 < 0 ? -1 : (a1 < 32 ? u10 : u11);
          }
        }
        const int s = i % kPgItems;
        if (i >= kPgItems) ok = mbar_wait(item_empty + 8 * s, (i / kPgItems - 1) & 1, kErrAttnProducerWait);
        // (new masks only once nobody reads the old ones for the item before)
        if (tree && i > 0) ok = ok && mbar_wait(item_empty + 8 * ((i - 1) % kPgItems), ((i - 1) / kPgItems) & 1, kErrAttnProducerWait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (tree) {
          anc[lane] = m0;
          anc[lane + 32] = m1;
          mask_b = cur.b;
        }
        if (lane == 0) {
          PagedRun& d = runs[s];
          d.b = end ? kPgEnd : cur.b;
          if (!end) {
            d.kvh = cur.kvh;
            d.a = a;
            d.z = z;
            d.n = cur.b < 0 ? INT32_MAX : cur.T - 1;
            d.L = cur.s.L;
            d.begin = cur.s.begin;
            d.t0 = cur.s.t0;
            d.nrow = cur.nrow();
            d.node0 = 2 * cur.pi * prm.NB;
            const int64_t item = paged_item(prm, cur.b, cur.kvh, cur.pi);
            d.prow = paged_part_row(prm, cur.b, item, cta, 0);
            // for the merge: between the two lie the item's runs
            int2* cut = prm.cuts + paged_item_of_all(prm, cur.b, item);
            if (a == 0) cut->x = cta;
            if (a < z && z == cur.T) cut->y = cta;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(item_full + 8 * s);
        ++i;
        if (end) break;
        cur.next(prm);
      }
    } else if (warp == kPgLoadWarp) {
      // ---------------------------------------------------------- K and V tiles
      const int box = prm.box, boxes = kAttnKeys / box;  // boxes of a tile
      const int page_mask = (1 << prm.a.map.page_shift) - 1;
      const int bc = lane / (D / 64), bh = lane % (D / 64);  // this lane's box of a tile
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        prefetch_tmap(&tm_kt);
        prefetch_tmap(&tm_vt);
      }
      int issued_k = 0, issued_v = 0, sk = 0, sv = 0;
      uint32_t pk = 1, pv = 1;  // parity of the slot's last release; the first round waits for none
      bool ok = true;
      for (int i = 0; ok; ++i) {
        ok = __all_sync(0xffffffffu, run_wait(i, kErrAttnProducerWait));
        if (!ok) break;
        const PagedRun& d = runs[i % kPgItems];
        const int b = d.b, kvh = d.kvh, a = d.a, z = d.z, n = d.n, L = d.L, t0 = d.t0;
        __syncwarp();
        if (lane == 0) run_release(i);
        if (b == kPgEnd) break;
        const int32_t* row = prm.a.map.table + static_cast<size_t>(b < 0 ? first_long : b) * prm.a.map.max_pages;
        // lane l holds the page of the l-th box from a tile on: a load per 32 boxes, a
        // group ahead of its use; boxes past the length or on no page read past the pool,
        // which gives zeros
        auto fetch = [&](int t) {
          const int64_t pos = t0 + static_cast<int64_t>(t) * kAttnKeys + static_cast<int64_t>(lane) * box;
          if (pos >= L) return prm.a.map.num_pages;
          const int pg = row[pos >> prm.a.map.page_shift];
          if (pg >= 0 && pg < prm.a.map.num_pages) return pg;
          record_error(kErrPageIndex);
          return prm.a.map.num_pages;
        };
        const int per = 32 / boxes;  // tiles of a group
        int ent = 0, ent_next = fetch(a), k = 0;
        for (int t = a; t < z; ++t) {
          if (k == 0) {
            ent = ent_next;
            ent_next = t + per < z ? fetch(t + per) : 0;
          }
          // boxes of keys in this tile: none of the half that the tree takes
          const int tree_row = t == n ? (L > t0 + t * kAttnKeys ? kHalf : 0) : kAttnKeys;
          const int pg = __shfl_sync(0xffffffffu, ent, (k * boxes + bc) & 31);
          const int at = (t0 + t * kAttnKeys + bc * box) & page_mask;
          if (++k == per) k = 0;
          auto issue = [&](uint32_t fb, uint32_t dst, const CUtensorMap* map, const CUtensorMap* tree) {
            if (lane == 0) mbar_arrive_expect_tx(fb, SM::kTile);
            __syncwarp();
            if (bc * box < tree_row)
              tma_load_4d(dst + bh * kAttnKeys * 128 + bc * box * 128, map, fb, bh * 64, at, kvh, pg);
            else if (t == n && (bc == boxes || (bc == boxes + 1 && tree_row == 0)))  // (nodes past 63: zeros)
              tma_load_4d(dst + bh * kAttnKeys * 128 + (tree_row + (bc - boxes) * kHalf) * 128, tree, fb, bh * 64,
                          kvh, (bc - boxes) * kHalf, b);
          };
          if (issued_k >= SK) ok = mbar_wait(k_empty + 8 * sk, pk, kErrAttnProducerWait);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          issue(k_full + 8 * sk, sbase + SM::kKOff + sk * SM::kTile, &tm_k, &tm_kt);
          ++issued_k;
          if (++sk == SK) {
            sk = 0;
            pk ^= 1;
          }
          if (issued_v >= SV) ok = mbar_wait(v_empty + 8 * sv, pv, kErrAttnProducerWait);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          issue(v_full + 8 * sv, sbase + SM::kVOff + sv * SM::kTile, &tm_v, &tm_vt);
          ++issued_v;
          if (++sv == SV) {
            sv = 0;
            pv ^= 1;
          }
        }
      }
      // every issued copy lands before the CTA can leave
      for (int i = max(0, issued_k - SK); i < issued_k; ++i)
        mbar_wait(k_full + 8 * (i % SK), (i / SK) & 1, kErrAttnProducerWait);
      for (int i = max(0, issued_v - SV); i < issued_v; ++i)
        mbar_wait(v_full + 8 * (i % SV), (i / SV) & 1, kErrAttnProducerWait);
    } else if (elect_one()) {
      // ---------------------------------------------------------- MMAs of a group
      const int g = warp - kPgMmaWarp;
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kAttnKeys);
      constexpr uint32_t idesc_o = idesc_bf16_f32_bmn(128, D);
      const uint32_t s_tmem = tmem + g * kAttnKeys, o_tmem = tmem + SM::kOCol + g * D;
      const uint32_t qb = sbase + SM::kQOff + g * SM::kTile;
      const uint32_t sf = s_full + 8 * g, ph = p_half + 8 * g, pf = p_full + 8 * g, pd = pv_done + 8 * g,
                     qf = q_full + 8 * g;
      bool ok = true;
      int item = 0;               // descriptions read
      int base = 0;               // the next one's first tile in the CTA's run of tiles
      int gi = 0, end = 0, step = 1;  // the tiles this group takes of the item
      int n = 0, q = 0;           // tiles done, Q tiles sent for
      int turns = 0;              // shared tiles done
      prefetch_tmap(&tm_q);
      auto wait = [&](uint32_t bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity, kErrAttnMmaWait); };
      // the next item with a tile for this group, its Q tile on the way
      auto open = [&]() {
        for (;;) {
          ok = ok && run_wait(item, kErrAttnMmaWait);
          if (!ok) return false;
          const PagedRun& d = runs[item % kPgItems];
          const int b = d.b, kvh = d.kvh, tiles = d.z - d.a, nrow = d.nrow, node0 = d.node0;
          run_release(item);
          if (b == kPgEnd) return false;
          ++item;
          step = nrow == 2 ? 1 : 2;
          gi = base + (nrow == 2 ? 0 : (base & 1) ^ g);
          end = base + tiles;
          base = end;
          if (gi >= end) continue;
          mbar_arrive_expect_tx(qf, static_cast<uint32_t>(prm.NB * G * D * 2));
          const int node = (b < 0 ? 0 : b * N) + node0 + (nrow == 2 ? g * prm.NB : 0);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) tma_load_3d(qb + h * 128 * 128, &tm_q, qf, h * 64, kvh * G, node);
          ++q;
          return true;
        }
      };
      // Waits for the K tile of gi.  On the way it sees the other group's tiles land and gives
      // up its claim to their slots: every phase of a slot's barrier is seen by both issuers,
      // and no slot is filled again before, since a wait for a phase is only sound while the
      // barrier is not more than that phase ahead or behind.
      int seen = 0;
      auto reach = [&]() {
        for (; seen < gi && ok; ++seen) {
          wait(k_full + 8 * (seen % SK), (seen / SK) & 1);
          if (ok) mbar_arrive(k_empty + 8 * (seen % SK));
          wait(v_full + 8 * (seen % SV), (seen / SV) & 1);
          if (ok) mbar_arrive(v_empty + 8 * (seen % SV));
        }
        wait(k_full + 8 * (gi % SK), (gi / SK) & 1);
      };
      // (a test of a barrier takes some 300 clocks while the tensor core reads shared memory:
      // those for operands are made under the MMAs issued before)
      bool more = open(), first = true;
      if (more) {
        wait(qf, 0);
        reach();
      }
      while (more && ok) {
        const int sk = gi % SK, sv = gi % SV;
        tc_fence_after();
        const uint64_t ad = smem_desc_k_sw128(qb), bd = smem_desc_k_sw128(sbase + SM::kKOff + sk * SM::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (128 * 128 / 16) + 2 * (kk & 3);
          tc_mma_f16(s_tmem, ad + off, bd + off, idesc_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(sf);
        tc_commit(k_empty + 8 * sk);
        // With shared tiles the groups take turns from P V to the next S: left alone they fall
        // into step, both softmaxes at once and then both pairs of MMAs.
        const bool alternate = step == 1;
        if (!first && alternate) mbar_arrive(turn + 8 * (g ^ 1));
        if (alternate && (g == 1 || turns > 0)) wait(turn + 8 * g, (turns - 1 + g) & 1);
        wait(v_full + 8 * sv, (gi / SV) & 1);
        seen = gi + 1;
        const uint64_t vd = smem_desc_mn_sw128(sbase + SM::kVOff + sv * SM::kTile, kAttnKeys * 128, 1024);
        wait(ph, n & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kAttnKeys / 32; ++kk)
          tc_mma_f16_ts(o_tmem, s_tmem + 8 * kk, vd + kk * (2048 / 16), idesc_o, (!first || kk > 0) ? 1u : 0u);
        wait(pf, n & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = kAttnKeys / 32; kk < kAttnKeys / 16; ++kk)
          tc_mma_f16_ts(o_tmem, s_tmem + 8 * kk, vd + kk * (2048 / 16), idesc_o, 1u);
        tc_commit(pd);
        tc_commit(v_empty + 8 * sv);
        first = false;
        turns += alternate ? 1 : 0;
        gi += step;
        if (gi >= end) {
          if (alternate) mbar_arrive(turn + 8 * (g ^ 1));
          // (P was taken from a complete S: the Q tile of the item that ends here is free)
          first = true;
          more = open();
          if (more) wait(qf, (q - 1) & 1);
        }
        if (more) reach();
        wait(pd, n & 1);
        ++n;
      }
      // every Q tile on its way lands, and every MMA completes, before the CTA can leave
      if (q > 0) mbar_wait(qf, (q - 1) & 1, kErrAttnMmaWait);
      tc_commit(all_done + 8 * g);
      mbar_wait(all_done + 8 * g, 0, kErrAttnMmaWait);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax groups
    reg_inc<kPgSoftRegs>();
    const int g = warp >> 2;
    const int r = tid & 127;                // query row of the tile = TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + g * kAttnKeys, o_col = lane_base + SM::kOCol + g * D;
    const float c = prm.scale_log2;
    const int row_node = r / G;             // node of this row in a row tile
    int n = 0;         // tiles this group has taken
    int base = 0;      // index in the CTA's run of tiles of the item's first tile
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = mbar_wait(bar, parity, kErrAttnConsumerWait);
    };
    // Both groups meet.  A warp whose waits have given up leaves the items on its own, so this
    // is a bounded wait like all others, not a barrier of the hardware's: the rest give up too.
    uint32_t meets = 0;
    auto meet_groups = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(met);
      wait(met, meets++ & 1);
      tc_fence_after();
    };
    for (int i = 0;; ++i) {
      ok = __all_sync(0xffffffffu, ok && run_wait(i, kErrAttnConsumerWait));
      if (!ok) break;
      const PagedRun& d = runs[i % kPgItems];
      const int b = d.b, nrow = d.nrow, a = d.a, z = d.z, tree_t = d.n, L = d.L, begin = d.begin, t0 = d.t0;
      const int node = d.node0 + (nrow == 2 ? g * prm.NB : 0) + row_node;  // in the batch or in the sequence
      const int rows = b < 0 ? prm.rows_sh : prm.rows_own;
      const int64_t prow = d.prow + (nrow == 2 ? g * rows : 0);
      const int kvh = d.kvh;
      const bool in_tile = r < prm.NB * G;
      const uint64_t tree_bits = in_tile && b >= 0 && node < N ? anc[node] : 0ull;
      __syncwarp();
      if (lane == 0) run_release(i);
      if (b == kPgEnd) break;
      bool rvalid;
      if (b < 0)  // rows of a sequence that lacks the shared part take no share of it
        rvalid = in_tile && node < B * N && prm.a.prefix_lens[min(node, B * N - 1) / N] >= prm.a.shared;
      else
        rvalid = in_tile && node < N;
      // a warp without a real row skips the scores and outputs, and keeps every barrier
      const bool live = __any_sync(0xffffffffu, rvalid);
      const int step = nrow == 2 ? 1 : 2, t_first = a + (nrow == 2 ? 0 : (base & 1) ^ g);
      float m_ref = -INFINITY, l = 0.f;
      for (int t = t_first; t < z; t += step, ++n) {
        const bool tree = t == tree_t;
        const int pos = t0 + t * kAttnKeys;
        const int valid = max(0, min(kAttnKeys, L - pos));  // keys of the cache in this tile
        const bool upper = tree ? valid > 0 : valid > kHalf;  // whether its upper half is used
        wait(s_full + 8 * g, n & 1);
        tc_fence_after();
        if (valid > 0 && valid < kAttnKeys) {
          // what the last page holds past the length must not reach P V, whatever it is:
          // zero those rows of the V slot once it has landed (later boxes came in as zeros).
          // The slot's tile before this one has landed -- the issuer saw it before this S --
          // so the wait cannot take its phase for that one's.
          const int gi = base + t - a, s = gi % SV;
          wait(v_full + 8 * s, (gi / SV) & 1);
          const int end = (valid + prm.box - 1) & ~(prm.box - 1);
          const uint32_t vb = sbase + SM::kVOff + s * SM::kTile;
          for (int idx = r; idx < (end - valid) * (D / 8); idx += 128) {
            const int j = valid + idx / (D / 8), dd = (idx % (D / 8)) * 8;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + attn_swz(j, dd)), "r"(0) : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();  // lane 0's arrivals below speak for the whole warp
        }
        if (live) {
          float x[kAttnKeys];
          __syncwarp();  // the TMEM loads below are warp-wide
          {
            uint32_t v0[32], v1[32], v2[32], v3[32];
            tmem_ld_cols<32>(s_col, v0);
            tmem_ld_cols<32>(s_col + 32, v1);
            tmem_ld_cols<32>(s_col + 64, v2);
            tmem_ld_cols<32>(s_col + 96, v3);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              x[j] = __uint_as_float(v0[j]);
              x[32 + j] = __uint_as_float(v1[j]);
              x[64 + j] = __uint_as_float(v2[j]);
              x[96 + j] = __uint_as_float(v3[j]);
            }
          }
          // masked scores become -inf, which also drops what a masked place holds (rows that
          // are not real go on unmasked: nothing reads their P or O but their own lanes)
          const int skip = max(0, begin - pos);
          if (tree || valid < kAttnKeys || skip > 0) {
            uint64_t m0 = valid >= 64 ? ~0ull : (1ull << valid) - 1ull;
            uint64_t m1 = valid >= 128 ? ~0ull : (valid <= 64 ? 0ull : (1ull << (valid - 64)) - 1ull);
            if (skip > 0) m0 = skip >= 64 ? 0ull : m0 & (~0ull << skip);  // (tiles start less than 64 keys before)
            if (tree) {
              if (upper)
                m1 = tree_bits;
              else
                m0 = tree_bits;
            }
#pragma unroll
            for (int j = 0; j < 64; ++j) {
              x[j] = ((m0 >> j) & 1ull) ? x[j] : -INFINITY;
              x[64 + j] = ((m1 >> j) & 1ull) ? x[64 + j] : -INFINITY;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int j = 4; j + 8 <= kAttnKeys; j += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmax3f(mx[k], x[j + 2 * k], x[j + 2 * k + 1]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], x[kAttnKeys - 4 + k]);
          // in scaled log2 units (the scale is positive)
          const float m_new = fmaxf(m_ref, fmax3f(mx[0], mx[1], fmaxf(mx[2], mx[3])) * c);
          // the reference moves only when the maximum grows by more than 2^8 over it; P
          // stays below 2^8 and the rescaling of O is rare
          const bool rebase =
              rvalid && m_new != -INFINITY && (m_ref == -INFINITY || m_new > m_ref + kPgRescaleThreshold);
          const bool scale_o = rebase && m_ref != -INFINITY;
          const float f = scale_o ? fast_exp2(m_ref - m_new) : 1.0f;
          if (rebase) {
            l *= f;
            m_ref = m_new;
          }
          const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
          // O holds the earlier tiles' P V against the old reference (they have completed:
          // S of this tile was issued after them)
          if (__any_sync(0xffffffffu, scale_o)) {
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t ov[16];
              tmem_ld_cols<16>(o_col + c0, ov);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
              tmem_st_cols<16>(o_col + c0, ov);
            }
          }
          float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
            if (h == 1 && !upper) {
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = 0u;
              tmem_st_cols<32>(s_col + 32, w);
              tmem_st_wait();
              break;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 y = ffma2(make_float2(x[64 * h + 2 * e], x[64 * h + 2 * e + 1]), make_float2(c, c),
                                     make_float2(neg_m, neg_m));
              float2 pe;
              if ((e & 7) < kPgPolyPairs) {
                pe = exp2_poly2<true>(y);
              } else {
                pe.x = fast_exp2(y.x);
                pe.y = fast_exp2(y.y);
              }
              // P is rounded to bf16 for the MMA; the denominator sums the fp32 values
              w[e] = pack_bf16x2(pe.x, pe.y);
              if (e & 1)
                ls1 = fadd2(ls1, pe);
              else
                ls0 = fadd2(ls0, pe);
            }
            tmem_st_cols<32>(s_col + 32 * h, w);
            tmem_st_wait();
            if (h == 0) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_half + 8 * g);
            }
          }
          ls0 = fadd2(ls0, ls1);
          l += ls0.x + ls0.y;
        } else if (lane == 0) {
          mbar_arrive(p_half + 8 * g);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * g);
      }
      // ---------------------------------------------------------- the run's result
      // A run of all of an item's tiles, without a shared part beside it, is the output;
      // others leave a partial, [D / 4][rows of the tile][4]: a warp's stores are contiguous.
      const bool direct = b >= 0 && a == 0 && z == tree_t + 1 && !(run_shared && L >= prm.a.shared);
      __nv_bfloat16* orow =
          prm.out + ((static_cast<int64_t>(max(b, 0)) * N + node) * prm.a.Hq + kvh * G + r % G) * D;
      float4* part = reinterpret_cast<float4*>(prm.part_acc + prow * D) + r;
      auto put = [&](int cc, const float (&v)[16]) {
        if (!rvalid) return;
        if (direct) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(orow + cc + k) =
                make_uint4(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]),
                           pack_bf16x2(v[k + 4], v[k + 5]), pack_bf16x2(v[k + 6], v[k + 7]));
        } else {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            part[static_cast<size_t>((cc + k) / 4) * rows] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
      };
      const bool any = nrow == 2 ? z > a : z > t_first;  // this group took a tile
      const bool meet = nrow == 1 && z - a > 1;           // both did, of the same rows
      if (any) {
        wait(pv_done + 8 * g, (n - 1) & 1);
        tc_fence_after();
      }
      // what this row's O, and the other group's where the groups took alternate tiles of the
      // same rows, count for
      float w0 = direct ? 1.0f / l : 1.0f, w1 = 0.f;
      int c0 = 0, c1 = D;
      if (meet) {
        // the sums meet here: both O are in this warp's TMEM lanes, and each group brings half
        // of the columns out
        if (g == 1) xch[r] = make_float2(m_ref, l);
        meet_groups();
        if (g == 0) {
          const float2 x = xch[r];
          const float m = fmaxf(m_ref, x.x);
          w0 = m_ref == -INFINITY ? 0.f : exp2f(m_ref - m);
          w1 = x.x == -INFINITY ? 0.f : exp2f(x.x - m);
          m_ref = m;
          l = l * w0 + x.y * w1;
          if (direct) {
            w0 /= l;
            w1 /= l;
          }
          xch[r] = make_float2(w1, w0);
        }
        meet_groups();
        if (g == 1) {
          w0 = xch[r].x;
          w1 = xch[r].y;
        }
        c0 = g * (D / 2);
        c1 = c0 + D / 2;
      }
      if (live && any) {
        const uint32_t other = lane_base + SM::kOCol + (g ^ 1) * D;
#pragma unroll 1
        for (int cc = c0; cc < c1; cc += 16) {
          uint32_t o[16];
          float v[16];
          __syncwarp();
          tmem_ld_cols<16>(o_col + cc, o);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = w0 != 0.f ? __uint_as_float(o[k]) * w0 : 0.f;
          if (meet) {
            tmem_ld_cols<16>(other + cc, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] += w1 != 0.f ? __uint_as_float(o[k]) * w1 : 0.f;
          }
          put(cc, v);
        }
      }
      // (an empty run's partial says so)
      if (rvalid && !direct && (nrow == 2 || (meet || z == a ? g == 0 : any)))
        prm.part_ml[prow + r] = make_float2(m_ref, l);
      if (meet) meet_groups();  // neither group lets its next P V at its O before the other has read it
      base += z - a;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kPgMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, SM::kTmemCols);
  }
}

// ------------------------------------------------------------------ merge
// Output row = the sum of its partials weighted by 2^(m_p - m), over the sum of their l.
// A CTA takes 8 rows, neighbours in the partials; a thread four columns of one row, kBatch
// partials at a time with all loads issued before any is used.  A warp is 8 rows x 4 column
// groups: it reads 128-byte runs and writes whole sectors.  With kSplit, for few rows, the
// CTA's 8 warps share one such group of columns and take every 8th partial each.  The order of
// the sums does not depend on timing.  Latency-bound: 35 MB of partials of 16384 rows take 9 us
// from L2, a single token's 2.6 (16 rows a CTA: 10.5; 2, 3 or 8 partials at a time: 9 to 30).
constexpr int kPgMergeRows = 8;

template <int D, bool kSplit>
__global__ void __launch_bounds__(kSplit ? 256 : 2 * D, kSplit ? 1 : 640 / D)
    paged_attn_merge_kernel(const __grid_constant__ PagedTcParams prm) {
  constexpr int kBatch = 4, kRows = kPgMergeRows;
  __shared__ int64_t row0_s[2][kRows], out_s[kRows];
  __shared__ int32_t count_s[2][kRows], step_s[2][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();  // (a next call's main kernel sets itself up meanwhile)
  if (threadIdx.x < 2 * kRows) {
    // thread = (own or shared runs, row): the first partial's row, the step to the next,
    // their number
    const uint32_t N = prm.a.N, Hq = prm.a.Hq, G = prm.a.G, Hkv = prm.a.Hkv;
    const int k = threadIdx.x / kRows, j = threadIdx.x % kRows;
    // rows in the order (sequence, kv head, node, head)
    const int64_t x = static_cast<int64_t>(blockIdx.x) * kRows + j;
    int count = 0, step = 0;
    int64_t row0 = 0, orow = -1;
    if (x < static_cast<int64_t>(prm.a.B) * N * Hq) {
      const uint32_t bk = static_cast<uint32_t>(x < (1ll << 32) ? static_cast<uint32_t>(x) / (N * G) : x / (N * G));
      const uint32_t in_head = static_cast<uint32_t>(x - static_cast<int64_t>(bk) * (N * G));
      const int b = bk / Hkv, kvh = bk - b * Hkv;
      const int node = in_head / G, hg = in_head - node * G;
      const uint32_t fnode = b * N + node;
      orow = static_cast<int64_t>(fnode) * Hq + kvh * G + hg;
      const uint32_t nd = k == 0 ? node : fnode;
      const int rb = k == 0 ? prm.rb_own : prm.rb_sh;
      if (rb > 0) {
        const int rt = nd / static_cast<uint32_t>(prm.NB), pi = rt >> 1, nrow = min(2, rb - 2 * pi);
        const int64_t item = paged_item(prm, k == 0 ? b : -1, kvh, pi);
        // (nothing before this is the main kernel's; all of these are on their way before the
        // first is used; without a shared run the shared items' cuts are stale, and not taken)
        pdl_wait();
        int2 cut = prm.cuts[paged_item_of_all(prm, k == 0 ? b : -1, item)];
        const int shared_runs = *prm.run_shared, L = prm.a.prefix_lens[b];
        // (after a wait that gave up an entry may be missing: whatever it holds names CTAs)
        cut.x = max(0, min(cut.x, kNumSMs - 1));
        cut.y = max(0, min(cut.y, kNumSMs - 1));
        // (of a pair, the second row tile has the second slot)
        row0 = paged_part_row(prm, k == 0 ? b : -1, item, cut.x, nrow == 2 ? (rt & 1) : 0);
        step = 2 * (k == 0 ? prm.rows_own : prm.rows_sh);
        count = k == 0 || (shared_runs != 0 && min(L, prm.a.Lmax) >= prm.a.shared) ? cut.y - cut.x + 1 : 0;
        // the row in the tile, below the bits of the partial's first row
        row0 = row0 * 128 + ((nd - rt * prm.NB) * G + hg);
      }
    }
    count_s[k][j] = count;
    step_s[k][j] = step;
    row0_s[k][j] = row0;
    if (k == 0) out_s[j] = orow;
  }
  pdl_wait();
  __syncthreads();
  const int col = (kSplit ? blockIdx.y : warp) * 4 + (lane >> 3);  // group of four columns
  const int first = kSplit ? warp : 0, stride = kSplit ? 8 : 1;
  const int j = lane & 7;
  const int n0 = count_s[0][j], total = n0 + count_s[1][j];
  if (!kSplit && total <= 1) return;  // the run that holds the whole item wrote the output (0: no row)
  const int64_t base0 = row0_s[0][j] >> 7, base1 = row0_s[1][j] >> 7;
  const int r0 = static_cast<int>(row0_s[0][j] & 127), r1 = static_cast<int>(row0_s[1][j] & 127);
  const int st0 = step_s[0][j], st1 = step_s[1][j];
  float m = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = first; i0 < total; i0 += kBatch * stride) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * stride;
      ml[k] = make_float2(-INFINITY, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < total) {
        const bool own = i < n0;
        const int64_t base = own ? base0 + static_cast<int64_t>(i) * st0 : base1 + static_cast<int64_t>(i - n0) * st1;
        const int r = own ? r0 : r1, rows = own ? prm.rows_own : prm.rows_sh;
        ml[k] = prm.part_ml[base + r];
        v[k] = *(reinterpret_cast<const float4*>(prm.part_acc + base * D) + static_cast<size_t>(col) * rows + r);
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
    const float base = mn == -INFINITY ? 0.f : mn;  // (no maximum, but perhaps a NaN sum)
    const float f = exp2f(m - base);
    den *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (ml[k].y == 0.f) continue;  // an empty partial's accumulator was never written
      const float w = exp2f(ml[k].x - base);
      den += w * ml[k].y;
      acc = make_float4(acc.x + w * v[k].x, acc.y + w * v[k].y, acc.z + w * v[k].z, acc.w + w * v[k].w);
    }
    m = mn;
  }
  if constexpr (kSplit) {
    __shared__ float4 acc_s[8][32];
    __shared__ float2 ml_s[8][32];
    acc_s[warp][lane] = acc;
    ml_s[warp][lane] = make_float2(m, den);
    __syncthreads();
    if (warp != 0) return;
    float mn = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = fmaxf(mn, ml_s[k][lane].x);
    if (mn == -INFINITY) mn = 0.f;
    den = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (ml_s[k][lane].y == 0.f) continue;
      const float w = exp2f(ml_s[k][lane].x - mn);
      const float4 t = acc_s[k][lane];
      den += w * ml_s[k][lane].y;
      acc = make_float4(acc.x + w * t.x, acc.y + w * t.y, acc.z + w * t.z, acc.w + w * t.w);
    }
  }
  if (total <= 1) return;
  const float inv = 1.0f / den;  // the node itself is always visible
  *reinterpret_cast<uint2*>(prm.out + out_s[j] * D + col * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

}  // namespace eagle
