// Attention of a few new tokens per sequence over a paged cache: a tree of drafted tokens
// (each sees its ancestors), a run of new tokens, or (n = 1) the decode step; optionally with
// a sliding window and sinks.
//
// Sequence b holds ctx_b committed positions and n new ones (positions ctx_b .. ctx_b + n - 1,
// already written to its pages). Token i sees new token j when bit j of its word is set, and
// committed position p when p > ctx_b + depth_i - window or p < sinks, depth_i being the
// number of its ancestors (its word's bits minus itself).
//
// GB300 mapping. The cache is read once, so HBM bounds the operation: a visible position is
// 4 hd bytes of K and V against 4 hd n group flops. The n x group query rows that share a kv
// head are packed into tiles (row = token * group + head of the group), one TMEM lane each,
// and the cache streams past them in 128-position tiles.
//   * Few rows: a product has 128 rows whether they are used or not, so up to 32 (64) rows are
//     put in the tile kSplit = 4 (2) times. Copy c of a row takes the columns [c, c + 1) 128 /
//     kSplit of every tile, with its own maximum, sum and O (its P is zero elsewhere, written
//     once), and the copies are merged at the end: the softmax of a tile, which is what a CTA
//     waits for, takes a quarter (half) of the time and all four warps.
//   * Work: a unit is (sequence, kv head, row tile) with the position tiles it can see; the
//     units' tiles in order form one line that is cut into equal runs, one per resident CTA,
//     so ragged lengths and windows balance without a plan from the host (the lengths are
//     read on the device: a captured graph follows them).
//   * A run's end cuts a unit: such pieces write (max, sum, unnormalised O) records, and
//     tree_combine_kernel merges each cut unit's records in order.
//   * Short caches (a table of at most kWholeTiles tiles a sequence): runs of whole units, so
//     there is nothing to merge: no records, no scratch and no second kernel, which at that
//     length cost more than the tiles that a CTA takes more. Where a unit a CTA fills the GPU
//     (`tree_choose`) the lengths decide: whole units unless the longest would keep the call waiting
//     for more than the 4 us that cutting costs. A CTA takes about 0.9 us a tile, HBM 0.075 ns
//     a column of one (B64 n16 over 2048 positions 28.8 us cut, 24.1 whole; over 4096 43.6 and
//     42.6; with more units than CTAs cut is better: B64 n1 at hd 128, window 2048 55.0, 57.0).
//   * Roundings: scores, maxima, sums and O are fp32; P is rounded to bf16, V's type, before P V (o
//     0.0023 relative from the exact values, 0.0017 with fp32 products).
//   * Pages: a tile is loaded box by box (one TMA box per page, or per 128 rows of a larger
//     one). A box that no row can see, or whose table entry is no page, is loaded from
//     outside the pool: the TMA unit writes zeros and reads nothing.
// Warps: 0 TMA producer; 1 TMEM owner and MMA issuer; 2-5 softmax, one query row a thread.
// TMEM: S [0,128) fp32 | P [128,192) bf16 pairs | O [192, 192 + hd).
#include <type_traits>

#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kTreeThreads = 192;

// K and V rings of one 128-position tile per slot. At hd 32 and 64 two CTAs fit an SM (256 TMEM
// columns each; the bytes are chosen so that no more do), at hd 128 one.
template <int HD>
struct TreeLayout {
  static constexpr int kCtas = HD == 128 ? 1 : 2;               // resident per SM that fit
  static constexpr int kSlots = HD == 32 ? 4 : 3;               // of K, and of V
  static constexpr uint32_t kRowBytes = HD * 2;
  static constexpr uint32_t kTileBytes = kTileRows * kRowBytes;
  static constexpr uint32_t kAtomBytes = kRowBytes < 128 ? kRowBytes : 128;
  static constexpr int kSubTiles = static_cast<int>(kRowBytes / kAtomBytes);
  static constexpr uint32_t kSubBytes = kTileRows * kAtomBytes;
  static constexpr uint32_t kSwizzle = HD == 32 ? kSwizzle64 : kSwizzle128;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kTileBytes;
  static constexpr uint32_t kV = kK + kSlots * kTileBytes;
  static constexpr uint32_t kBars = kV + kSlots * kTileBytes;
  static constexpr int kNumBars = 4 * kSlots + 6;
  static constexpr uint32_t kPages = kBars + 8 * kNumBars;      // per V slot: boxes that hold a page
  static constexpr uint32_t kMisc = (kPages + 4 * kSlots + 15) / 16 * 16;
  static constexpr uint32_t kUsed = kMisc + 32;
  // The tiles start at the next multiple of 1024; the base is at least 256-byte aligned.
  static constexpr uint32_t kDynBytes = kUsed + 768 > 80 * 1024 ? kUsed + 768 : 80 * 1024;
  static constexpr uint32_t kTmemCols = HD == 128 ? 512 : 256;
  static_assert(kCtas * (kDynBytes + 1024) <= 228 * 1024, "resident CTAs fit the SM");
  static_assert((kCtas + 1) * (kDynBytes + 1024) > 228 * 1024 || kCtas * kTmemCols < 512,
                "no CTA more than the tensor memory holds");
};

__device__ __forceinline__ bool tree_wait(uint32_t bar, uint32_t parity, const WaitCtl &ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}

// The line that holds p into L2. While the rings keep HBM busy a load that misses L2 takes
// about 4 us; what the next piece will read is asked for at the start of the current one.
__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// One arrival for the whole warp, after what every lane has done (128 arrivals of single
// lanes take some 500 cycles).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The position tiles that some new token of one sequence can see, as a list: `heads` sink
// tiles, then the tiles from lo to that of the last new token. Entry e is tile e below heads,
// else e - heads + lo.
struct Sight {
  int ctx, end;      // committed positions; end of the new ones
  int far;           // first committed position inside the first token's window
  int lo, heads, count;
};

__device__ __forceinline__ Sight sight_of(const TreeArgs &a, int b) {
  Sight s;
  s.ctx = min(max(a.ctx_lens[b], 0), a.max_pages * a.page_size - a.n);
  s.end = s.ctx + a.n;
  s.far = max(s.ctx - a.window + 1, 0);
  s.lo = s.far / kTileRows;
  s.heads = min((min(a.sinks, s.end) + kTileRows - 1) / kTileRows, s.lo);
  s.count = s.heads + (s.end - 1) / kTileRows - s.lo + 1;
  return s;
}

// a / b for 0 <= a, 0 < b.
__device__ __forceinline__ int quotient(int a, int b) {
  return static_cast<int>(static_cast<unsigned>(a) / static_cast<unsigned>(b));
}

// The line of `length` tiles (at most 2^30) in `runs` runs: the first length % runs have one more.
struct Runs {
  int each, more;
  __device__ Runs(int length, int runs) : each(quotient(length, runs)), more(length - each * runs) {}
  __device__ int start(int c) const { return c * each + min(c, more); }
  __device__ int of(int pos) const {                           // the run that holds pos
    const int head = more * (each + 1);
    return pos < head ? quotient(pos, each + 1) : more + quotient(pos - head, each);
  }
};

// A run of the line of tiles, walked piece by piece; warp-uniform, every warp of every role
// walks the same pieces. With whole units the line's steps are units.
struct Walk {
  int pos, stop;           // next tile (unit) and end of the run, on the line
  int first;               // where sequence b starts on it
  int b, e0, e1, unit;     // piece: sequence, entries [e0, e1) of its list, unit within it
  int whole;               // the line's steps are units
  Sight s;
};

// Tiles of four sequences (from b on).
__device__ __forceinline__ int four_counts(const TreeArgs &a, int b, int *counts) {
#pragma unroll
  for (int k = 0; k < 4; ++k) counts[k] = b + k < a.B ? sight_of(a, b + k).count : 0;
  return (counts[0] + counts[1]) + (counts[2] + counts[3]);
}

// Tiles of all sequences and units: the line's length. And the sequence that holds tile
// `target` of it, with the line's tiles before that sequence. Four sequences a lane; counts:
// those of the first 128, which the one keeps for the other; longest: tiles of a sequence at most.
template <bool kLongest>
__device__ __forceinline__ int line_length(const TreeArgs &a, int units, int lane, int *counts, int *longest) {
  int total = __reduce_add_sync(0xffffffffu, four_counts(a, 4 * lane, counts));
  int most = max(max(counts[0], counts[1]), max(counts[2], counts[3]));
  for (int b0 = 128; b0 < a.B; b0 += 128) {
    int more[4];
    total += __reduce_add_sync(0xffffffffu, four_counts(a, b0 + 4 * lane, more));
    most = max(most, max(max(more[0], more[1]), max(more[2], more[3])));
  }
  if constexpr (kLongest) *longest = __reduce_max_sync(0xffffffffu, most);
  return total * units;
}

__device__ __forceinline__ void line_find(const TreeArgs &a, int units, int lane, const int *counts, int target,
                                          int *b_out, int *first_out) {
  const int want = quotient(target, units);                    // x units > target as x > want
  int base = 0, c[4] = {counts[0], counts[1], counts[2], counts[3]};
  int mine = (c[0] + c[1]) + (c[2] + c[3]);
#pragma unroll 1
  for (int b0 = 0;;) {
    int incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + incl > want);
    if (past) {
      const int l = __ffs(past) - 1;
      int before = base + incl - mine, k = 0;
#pragma unroll
      for (int x = 0; x < 3; ++x)
        if (k == x && before + c[x] <= want) before += c[x], ++k;
      *b_out = b0 + 4 * l + __shfl_sync(0xffffffffu, k, l);
      *first_out = __shfl_sync(0xffffffffu, before, l) * units;
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
    b0 += 128;
    if (b0 >= a.B) break;                                      // (target is on the line: not reached)
    mine = four_counts(a, b0 + 4 * lane, c);
  }
  *b_out = a.B - 1;
  *first_out = 0;
}

template <bool kChoose>
__device__ __forceinline__ bool walk_piece(Walk &w, const TreeArgs &a, int units) {
  if (w.pos >= w.stop) return false;
  if (kChoose ? w.whole : a.whole) {
    w.b = quotient(w.pos, units);
    w.unit = w.pos - w.b * units;
    w.s = sight_of(a, w.b);
    w.e0 = 0;
    w.e1 = w.s.count;
    ++w.pos;
    return true;
  }
  int at = w.pos - w.first;
  if (at >= w.s.count * units) {                               // the next sequence
    w.first += w.s.count * units;
    if (++w.b >= a.B) return false;                            // (only if the lengths change under the call)
    w.s = sight_of(a, w.b);
    at = 0;
  }
  w.unit = quotient(at, w.s.count);
  w.e0 = at - w.unit * w.s.count;
  w.e1 = min(w.s.count, w.e0 + (w.stop - w.pos));
  w.pos += w.e1 - w.e0;
  return true;
}

// Record of a cut unit's piece: CTA c's piece that starts inside a unit is record 2c, the one
// that starts it record 2c + 1. Layout: [records][rows][hd] O, then [records][rows] (max, sum).
// CTAs an SM: with few rows two (where they fit), so that one streams while the other ends a
// unit (B64 n16 hd 64: 43.2 us, one with twice the slots 47.8; 200 sequences of 1000 positions,
// n 1, 34.2 against 47.0). A tile of 128 rows is bound by its softmax and wants the registers of
// one: a row of 128 scores spills in the 168 registers of two (B8 n64 hd 64 over 8192 positions:
// 42.8 us, one CTA 31.9).
template <int HD, int kSplit>
constexpr int tree_ctas() {
  return kSplit == 1 ? 1 : TreeLayout<HD>::kCtas;
}

// kChoose: a call that tree_choose lets choose (a kernel of its own: the choice in every call
// cost those that have none 1 %).
template <int HD, int kSplit, bool kChoose>
__global__ void __launch_bounds__(kTreeThreads, tree_ctas<HD, kSplit>())
    tree_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const TreeArgs a) {
  using L = TreeLayout<HD>;
  extern __shared__ uint8_t tree_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tree_smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(smem + L::kQ), sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV);
  const uint32_t bar0 = smem_u32(smem + L::kBars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto k_full = [&](int s) { return bar(s); };
  auto k_empty = [&](int s) { return bar(L::kSlots + s); };
  auto v_full = [&](int s) { return bar(2 * L::kSlots + s); };
  auto v_empty = [&](int s) { return bar(3 * L::kSlots + s); };
  const uint32_t s_full = bar(4 * L::kSlots), s_free = bar(4 * L::kSlots + 1), p_full = bar(4 * L::kSlots + 2);
  const uint32_t o_done = bar(4 * L::kSlots + 3), q_full = bar(4 * L::kSlots + 4);
  const uint32_t meet = bar(4 * L::kSlots + 5);              // the softmax warps among themselves
  constexpr int kRows = kTileRows / kSplit, kCols = kTileRows / kSplit;
  volatile uint32_t *pages = reinterpret_cast<volatile uint32_t *>(smem + L::kPages);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 16);
  const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};
  XATTN_DCHECK(smem + L::kUsed <= tree_smem_raw + L::kDynBytes, a.status);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < 4 * L::kSlots; ++s) mbar_init(bar(s), 1);
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(p_full, 4);
    mbar_init(o_done, 1);
    mbar_init(q_full, 4);
    mbar_init(meet, 4);
    fence_mbar_init();
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  grid_dep_wait();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  const uint32_t tS = tmem, tP = tmem + 128, tO = tmem + 192;

  // This CTA's run of the line.
  const int group = a.group, rows_all = a.n * group, row_tiles = a.row_tiles;
  const int units = a.nkv * row_tiles;
  int counts[4];
  Walk walk;
  walk.whole = a.whole;
  int length = a.B * units, longest = 0;
  if (!a.whole) {
    const int tiles = line_length<kChoose>(a, units, lane, counts, &longest);
    if constexpr (kChoose)
      walk.whole = longest * 900.f <= fmaxf(tiles * (HD * 0.075f), tiles * (900.f / gridDim.x)) + 4000.f;
    if (!walk.whole) length = tiles;
  }
  const Runs runs(length, min(static_cast<int>(gridDim.x), length));
  walk.pos = walk.stop = 0;
  if (static_cast<int>(blockIdx.x) < length) {
    walk.pos = runs.start(blockIdx.x);
    walk.stop = runs.start(blockIdx.x + 1);
  }
  if (!walk.whole && walk.pos < walk.stop) {
    line_find(a, units, lane, counts, walk.pos, &walk.b, &walk.first);
    walk.s = sight_of(a, walk.b);
  }

  if (warp == 0) {
    // ---------------- TMA producer: lane l finds box l of each tile ----------------
    const int box_rows = min(a.page_size, kTileRows), boxes = kTileRows / box_rows;
    int R = 0, issued_k = 0, issued_v = 0;
    bool ok = true, have = walk_piece<kChoose>(walk, a, units);
    auto page_of = [&](int p) { return a.page_shift >= 0 ? p >> a.page_shift : quotient(p, a.page_size); };
    // The table entries of a piece, 8 to a 32-byte sector.
    auto prefetch_table = [&](const Walk &w) {
      const int *table = a.page_table + static_cast<size_t>(w.b) * a.max_pages;
      const int t0 = w.e0 < w.s.heads ? w.e0 : w.e0 - w.s.heads + w.s.lo;
      const int t1 = w.e1 - 1 < w.s.heads ? w.e1 - 1 : w.e1 - 1 - w.s.heads + w.s.lo;
      const int last = page_of(min(t1 * kTileRows + kTileRows - 1, w.s.end - 1));
      for (int at = page_of(t0 * kTileRows) + 8 * lane; at <= last + 7; at += 256) prefetch_l2(table + min(at, last));
    };
    // A tile's boxes: their pages come to every lane first, then one elected lane issues the
    // copies back to back from uniform registers (box by box, with a shuffle or a branch per
    // box, took 75 cycles each: at 16-row pages as long as the bytes themselves take). Only
    // pages of more than 128 rows have a row to start at, and those are one box.
    auto load_boxes = [&](uint32_t dst, const CUtensorMap *map, uint32_t full, int kvh, int row, int page) {
      int pg[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) pg[x] = __shfl_sync(0xffffffffu, page, x);
      const int rw = __shfl_sync(0xffffffffu, row, 0);
      const uint32_t box_bytes = box_rows * L::kAtomBytes;
      XATTN_DCHECK(kvh < a.nkv && page >= 0 && page <= a.num_pages && row >= 0 && row + box_rows <= a.page_size &&
                       boxes <= 8 && dst >= sK && dst + L::kTileBytes <= smem_u32(smem + L::kBars),
                   a.status);
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (x < boxes) {
#pragma unroll
            for (int c = 0; c < L::kSubTiles; ++c)
              tma_load_4d(dst + c * L::kSubBytes + x * box_bytes, map, full, 64 * c, kvh, x == 0 ? rw : 0, pg[x]);
          }
      }
      __syncwarp();
    };
    while (ok && have) {
      const Walk here = walk;
      const int kvh = row_tiles == 1 ? here.unit : quotient(here.unit, row_tiles);
      const int *table = a.page_table + static_cast<size_t>(here.b) * a.max_pages;
      // This lane's box of entry e: its table entry (-1 when no row can see the box) and its
      // row in the page. Read one tile ahead, so that no tile waits for the table.
      auto box_of = [&](int e, int *row) -> int {
        const int tile = e < here.s.heads ? e : e - here.s.heads + here.s.lo;
        const int p0 = tile * kTileRows + lane * box_rows, at = page_of(p0);
        *row = p0 - at * a.page_size;
        if (lane >= boxes || e >= here.e1 || p0 >= here.s.end || (p0 + box_rows <= here.s.far && p0 >= a.sinks)) return -1;
        return __ldg(table + at);                               // p0 < end <= max_pages * page_size
      };
      int row_next = 0, id_next = box_of(here.e0, &row_next);
      const bool first = R == 0;
      have = false;
#pragma unroll 1
      for (int e = here.e0; e < here.e1; ++e, ++R) {
        // Looking ahead waits until the run's first copies are on their way.
        if (e == min(here.e0 + (first ? 1 : 0), here.e1 - 1)) {
          if (first) prefetch_table(here);
          have = walk_piece<kChoose>(walk, a, units);
          if (have) prefetch_table(walk);
        }
        // Outside the pool (num_pages) there is nothing to read: the box is zeros.
        const int row = row_next, page = id_next >= 0 && id_next < a.num_pages ? id_next : a.num_pages;
        id_next = box_of(e + 1, &row_next);
        const unsigned held = __ballot_sync(0xffffffffu, page != a.num_pages);
        const int s = R % L::kSlots;
        const uint32_t ph = static_cast<uint32_t>((R / L::kSlots) & 1) ^ 1u;
        if (!tree_wait(k_empty(s), ph, ctl)) { ok = false; break; }
        mbar_expect_tx_elect(k_full(s), L::kTileBytes);
        load_boxes(sK + s * L::kTileBytes, &mk, k_full(s), kvh, row, page);
        issued_k = R + 1;
        if (!tree_wait(v_empty(s), ph, ctl)) { ok = false; break; }
        if (elect_one()) {
          pages[s] = held;                 // read by the softmax warps before P V frees the slot
          mbar_expect_tx(v_full(s), L::kTileBytes);
        }
        __syncwarp();
        load_boxes(sV + s * L::kTileBytes, &mv, v_full(s), kvh, row, page);
        issued_v = R + 1;
      }
    }
    __syncwarp();
    // Every copy in flight has landed before the CTA can exit.
    for (int r = max(issued_k - L::kSlots, 0); r < issued_k; ++r)
      mbar_drain(k_full(r % L::kSlots), (r / L::kSlots) & 1, ctl);
    for (int r = max(issued_v - L::kSlots, 0); r < issued_v; ++r)
      mbar_drain(v_full(r % L::kSlots), (r / L::kSlots) & 1, ctl);
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, HD / L::kSubTiles, false, true);
    constexpr uint32_t kTileDesc = L::kTileBytes >> 4, kSubDesc = L::kSubBytes >> 4;
    constexpr uint32_t kVStep = (16 * L::kAtomBytes) >> 4;       // 16 positions of V
    const uint64_t dQ = smem_desc(sQ, 16, 8 * L::kAtomBytes, L::kSwizzle);
    const uint64_t dK = smem_desc(sK, 16, 8 * L::kAtomBytes, L::kSwizzle);
    const uint64_t dV = smem_desc(sV, 8192, 8 * L::kAtomBytes, L::kSwizzle);
    // S = Q K^T of ring entry r, once K has landed and the last S has been read.
    auto scores = [&](int r) -> bool {
      const int s = r % L::kSlots;
      if (!tree_wait(k_full(s), (r / L::kSlots) & 1, ctl) || !tree_wait(s_free, (r - 1) & 1, ctl)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t off = (kk / 4) * kSubDesc + (kk % 4) * 2;
          mma_ss(tS, dQ + off, dK + s * kTileDesc + off, idesc_qk, kk > 0 ? 1u : 0u);
        }
        mma_commit(s_full);
        mma_commit(k_empty(s));
      }
      __syncwarp();
      return true;
    };
    int R = 0, piece = 0, scored = 0;
    bool ok = true;
    while (ok && walk_piece<kChoose>(walk, a, units)) {
      ok = tree_wait(q_full, piece & 1, ctl) && scores(R);
      if (ok) scored = R + 1;
#pragma unroll 1
      for (int e = walk.e0; ok && e < walk.e1; ++e, ++R) {
        if (e + 1 < walk.e1) {
          if (!scores(R + 1)) { ok = false; break; }
          scored = R + 2;
        }
        const int s = R % L::kSlots;
        if (!tree_wait(v_full(s), (R / L::kSlots) & 1, ctl) || !tree_wait(p_full, R & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kTileRows / 16; ++kk)
#pragma unroll
            for (int c = 0; c < L::kSubTiles; ++c)
              mma_ts(tO + c * (HD / L::kSubTiles), tP + kk * 8, dV + s * kTileDesc + c * kSubDesc + kk * kVStep,
                     idesc_pv, (e > walk.e0 || kk > 0) ? 1u : 0u);
          mma_commit(o_done);
          mma_commit(v_empty(s));
        }
        __syncwarp();
      }
      ++piece;
    }
    __syncwarp();
    // The last products and the copies they released are done before TMEM goes.
    if (scored > 0) mbar_drain(s_full, (scored - 1) & 1, ctl);
    if (R > 0) mbar_drain(o_done, (R - 1) & 1, ctl);
  } else {
    // ---------------- softmax: thread = one copy of a query row ----------------
    const int quarter = warp & 3, lane_row = quarter * 32 + lane;     // TMEM lane
    const int row = lane_row % kRows, copy = lane_row / kRows;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tSx = tS + lane_off + copy * kCols, tPx = tP + lane_off + copy * (kCols / 2), tOx = tO + lane_off;
    const int box_rows = min(a.page_size, kTileRows);
    const unsigned all_boxes = box_rows == kTileRows ? 1u : (1u << (kTileRows / box_rows)) - 1u;
    float2 *stat = reinterpret_cast<float2 *>(smem + L::kQ);        // every lane's (max, sum), at a piece's end
    if constexpr (kSplit > 1) {
      // P of the columns that the other copies take.
      uint32_t zero[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) zero[i] = 0u;
      tmem_st_x32(tP + lane_off, zero);
      tmem_st_x32(tP + lane_off + 32, zero);
      tmem_wait_st();
    }
    int R = 0, meets = 0;
    bool ok = true;
    // All softmax warps have come this far (bounded, like every wait).
    auto meet_all = [&]() -> bool {
      warp_arrive(meet, lane);
      return tree_wait(meet, meets++ & 1, ctl);
    };
    // A piece's query row and word: into L2 while the piece before it runs, into registers
    // before that piece's result is written (after it with kSplit = 1, whose rows of 128 scores
    // leave none: hd 128 48.7 against 45.2 us), and then put in place.
    uint4 xq[HD / 8];
    unsigned long long word = 0, all_words[2] = {0, 0};
    auto load_rows = [&](bool ahead) {
      const int row0 = (walk.unit % row_tiles) * kRows, rho = row0 + row;
      const bool mine = rho < rows_all;
      const int token = mine ? rho / group : 0;
      const size_t at = static_cast<size_t>(walk.b) * a.n + token;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + (at * a.nh + static_cast<size_t>(walk.unit / row_tiles) * group + (mine ? rho - token * group : 0)) * HD);
      if (ahead) {
        if (mine && copy == 0) {
#pragma unroll
          for (int c = 0; c < HD / 8; c += 8) prefetch_l2(src + c);
          if (a.tree) prefetch_l2(a.tree + at);
        }
        return;
      }
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) xq[c] = mine ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
      word = !mine ? 0 : (a.tree ? __ldg(a.tree + at) : (2ull << token) - 1);   // (not used here: no wait)
      // Tokens lane and lane + 32 of the sequence. (Four copies: the warp's own rows are all of them.)
      if (kSplit < 4 && a.tree) {
        const unsigned long long *words = a.tree + static_cast<size_t>(walk.b) * a.n;
        all_words[0] = lane < a.n ? __ldg(words + lane) : 0;
        all_words[1] = lane + 32 < a.n ? __ldg(words + lane + 32) : 0;
      }
    };
    // Nothing for the combine until the run's end says otherwise (a run that gives up says
    // nothing).
    if (!a.whole && warp == 2 && lane == 0) a.plan[blockIdx.x] = make_int4(0, 0, 0, 0);
    bool have = walk_piece<kChoose>(walk, a, units);
    if (kSplit > 1 && have) load_rows(false);
    while (ok && have) {
      const Sight s = walk.s;
      const int b = walk.b, e0 = walk.e0, e1 = walk.e1;
      const int kvh = walk.unit / row_tiles, row0 = (walk.unit % row_tiles) * kRows;
      const int unit = walk.unit;
      if (kSplit == 1) load_rows(false);
      // From here on `walk` is the next piece.
      have = walk_piece<kChoose>(walk, a, units);
      if (have) load_rows(true);
      // A run that ends inside the unit it started last says so to the combine.
      if (!have && !a.whole && warp == 2 && lane == 0) {
        const int start = walk.stop - (e1 - e0);
        if (e0 == 0 && e1 < s.count)
          a.plan[blockIdx.x] = make_int4(b, unit, runs.of(start + s.count - 1), 1);
      }
      const int rows = min(rows_all - row0, kRows);
      const bool live = kSplit > 1 || quarter * 32 < rows;    // the warp has a row
      const bool mine = row < rows;
      // The rows into the Q tile, swizzled as TMA would (0 past the last).
      if (live) {
        constexpr int kChunks = static_cast<int>(L::kAtomBytes / 16);
#pragma unroll
        for (int c = 0; c < HD / 8; ++c) {
          const int ch = c % kChunks, sw = L::kAtomBytes == 128 ? (ch ^ (lane_row & 7)) : (ch ^ ((lane_row >> 1) & 3));
          *reinterpret_cast<uint4 *>(smem + L::kQ + (c / kChunks) * L::kSubBytes + lane_row * L::kAtomBytes +
                                     (sw << 4)) = xq[c];
        }
      }
      fence_proxy_async_smem();
      warp_arrive(q_full, lane);
      // The row's ancestors and how far its window reaches.
      // Bits past the last new token mean nothing.
      const unsigned long long in_tree = a.n == 64 ? ~0ull : (1ull << a.n) - 1, seen = word & in_tree;
      auto depth_of = [&](unsigned long long w) { return max(__popcll(w & in_tree) - 1, 0); };
      const int far = s.ctx + depth_of(word) - a.window + 1;
      // What some token of the sequence sees: new tokens, and committed positions from far_any on.
      unsigned long long seen_any = in_tree;
      int far_any = s.far;
      if (a.tree) {
        const unsigned long long x = kSplit == 4 ? seen : (all_words[0] | all_words[1]) & in_tree;
        seen_any = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(x)) |
                   static_cast<unsigned long long>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(x >> 32))) << 32;
        int depth = 64;
        if (kSplit == 4 ? mine : lane < a.n) depth = depth_of(kSplit == 4 ? word : all_words[0]);
        if (kSplit < 4 && lane + 32 < a.n) depth = min(depth, depth_of(all_words[1]));
        far_any = s.ctx + __reduce_min_sync(0xffffffffu, depth) - a.window + 1;
      }
      float mrow = -INFINITY, lrow = 0.f;
      // One tile: this copy's kCols columns. vis: a word per 32 columns. With few columns a
      // thread always masks; 128 have a copy without masks for the tiles that every row sees
      // whole. One copy of the code instead of two: batch of trees at
      // hd 64 45.6 -> 44.6 us (its first pass runs from L2).
      auto step = [&](auto masked, const uint32_t *vis, bool first) -> bool {
        float x[kCols];
        uint32_t *xr = reinterpret_cast<uint32_t *>(x);
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld_x32(tSx + c, xr + c);
        tmem_wait_ld();
        reg_fence<kCols>(xr);
        tc_fence_before();
        warp_arrive(s_free, lane);
        // Scaled scores (log2 domain) and their maximum.
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          fmul2(x[c], x[c + 1], x[c], x[c + 1], a.scale_log2, a.scale_log2);
          if constexpr (decltype(masked)::value) {
            if (((vis[c >> 5] >> (c & 31)) & 1u) == 0u) x[c] = -INFINITY;
            if (((vis[c >> 5] >> ((c + 1) & 31)) & 1u) == 0u) x[c + 1] = -INFINITY;
          }
          float &m = mx[(c >> 1) & 3];
          m = fmax3(m, x[c], x[c + 1]);
        }
        const float mnew = fmax3(fmaxf(mrow, mx[0]), mx[1], fmaxf(mx[2], mx[3]));
        // O is rescaled only when some row's maximum grew by more than 2^8.
        const bool rescale = __any_sync(0xffffffffu, mnew > mrow + 8.0f);
        const float m_use = rescale ? mnew : mrow;
        float alpha = 1.f;
        if (rescale && mnew > mrow) alpha = ex2_approx(mrow - mnew);
        const float base = m_use == -INFINITY ? 0.f : -m_use;         // a row that has seen nothing yet
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[kCols / 2];
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          float p0, p1;
          fadd2(p0, p1, x[c], x[c + 1], base, base);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          const int e = (c >> 1) & 1;
          fadd2(ps[2 * e], ps[2 * e + 1], ps[2 * e], ps[2 * e + 1], p0, p1);
          pk[c / 2] = pack_bf16x2(p0, p1);
        }
        // P over the last tile's, which its P V has read then.
        if (!tree_wait(o_done, (R - 1) & 1, ctl)) return false;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kCols / 2; c += 16) tmem_st_x16(tPx + c, pk + c);
        if (rescale && !first) {
#pragma unroll
          for (int c = 0; c < HD; c += 32) {
            uint32_t ov[32];
            tmem_ld_x32(tOx + c, ov);
            tmem_wait_ld();
            reg_fence<32>(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st_x32(tOx + c, ov);
          }
        }
        lrow = lrow * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
        mrow = m_use;
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(p_full, lane);
        return true;
      };
#pragma unroll 1
      for (int e = e0; e < e1; ++e, ++R) {
        const int tile = e < s.heads ? e : e - s.heads + s.lo, t0 = tile * kTileRows;
        const int slot = R % L::kSlots;
        // V has landed (so pages[slot] is there to read; its slot is not loaded again before
        // this tile's P V), and the scores.
        if (!tree_wait(v_full(slot), (R / L::kSlots) & 1, ctl) || !tree_wait(s_full, R & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        const unsigned held = pages[slot];
        XATTN_DCHECK(t0 >= 0 && t0 < s.end && s.end <= a.max_pages * a.page_size, a.status);
        // Positions that some row does not see: new ones, those behind a window, missing pages.
        const bool edge = t0 + kTileRows > s.ctx || held != all_boxes ||
                          (t0 <= s.end - 1 - a.window && t0 + kTileRows > a.sinks);
        uint32_t vis[kCols / 32];
        if (edge) {
#pragma unroll
          for (int w = 0; w < kCols / 32; ++w) {
            const int col = copy * kCols + 32 * w, base = t0 + col, off = base - s.ctx;
            uint32_t m = bit_range(0, s.ctx - 1 - base) & (bit_range(far - base, 31) | bit_range(0, a.sinks - 1 - base));
            if (off >= 0) {
              if (off < 64) m |= static_cast<uint32_t>(seen >> off);
            } else if (off > -32) {
              m |= static_cast<uint32_t>(seen << -off);
            }
            uint32_t there = 0;
            if (box_rows >= 32)
              there = (held >> (col / box_rows)) & 1u ? 0xffffffffu : 0u;
            else
              there = ((held >> (col / 16)) & 1u ? 0x0000ffffu : 0u) | ((held >> (col / 16 + 1)) & 1u ? 0xffff0000u : 0u);
            vis[w] = m & there;
          }
          // V rows that no token sees may hold anything -- behind the cache, behind every token's
          // window, drafted rows that no word names (the spare ones of a smaller tree) -- and are
          // zeroed before P V, in which their P is 0 (0 x NaN would not be). Missing pages were
          // loaded as zeros.
          const int p = t0 + lane_row, off = p - s.ctx;
          if (off < 0 ? p < far_any && p >= a.sinks : off >= a.n || ((seen_any >> off) & 1u) == 0u) {
#pragma unroll
            for (int c = 0; c < L::kSubTiles; ++c)
#pragma unroll
              for (uint32_t x = 0; x < L::kAtomBytes; x += 16)
                *reinterpret_cast<uint4 *>(smem + L::kV + slot * L::kTileBytes + c * L::kSubBytes +
                                           lane_row * L::kAtomBytes + x) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (!live) {
          warp_arrive(s_free, lane);
          // P of the previous tile has been read before anyone moves on.
          if (!tree_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
          warp_arrive(p_full, lane);
          continue;
        }
        if constexpr (kSplit > 1) {
          if (!edge)
#pragma unroll
            for (int w = 0; w < kCols / 32; ++w) vis[w] = 0xffffffffu;
          ok = step(std::true_type{}, vis, e == e0);
        } else {
          ok = edge ? step(std::true_type{}, vis, e == e0) : step(std::false_type{}, vis, e == e0);
        }
        if (!ok) break;
      }
      if (!ok) break;
      // The piece's result: O and the LSE of a whole unit, else a record (its O not divided by
      // its sum).
      const bool whole = e0 == 0 && e1 == s.count;
      const size_t rec0 = (2 * static_cast<size_t>(blockIdx.x) + (e0 == 0 ? 1 : 0)) * a.rec_rows;
      XATTN_DCHECK(rec0 + rows <= 2 * static_cast<size_t>(gridDim.x) * a.rec_rows || a.whole, a.status);
      auto out_of = [&](int r) {                              // row r of the tile, in o and lse
        const int rho = row0 + r;
        const size_t at = (static_cast<size_t>(b) * a.n + rho / group) * a.nh + static_cast<size_t>(kvh) * group + rho % group;
        XATTN_DCHECK(r >= rows || at < static_cast<size_t>(a.B) * a.n * a.nh, a.status);
        return at;
      };
      // (Here and in the combine a sum of 0 is a row that saw nothing; NaN, of a query or of scores
      // that are no numbers, is not 0 and stays.)
      auto put_stats = [&](float M, float sum) {
        if (whole)
          a.lse[out_of(row)] = sum != 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
        else
          *reinterpret_cast<float2 *>(a.ws_ml + 2 * (rec0 + row)) = make_float2(M, sum);
      };
      if constexpr (kSplit > 1) {
        // The copies' (max, sum) meet in the Q tile, which the last scores have read, while the
        // last P V runs; each copy then weighs its own O, and the copies meet there again. Of
        // two copies each adds half of the columns. Of four, few rows and many columns, all
        // warps add, some lanes a row, so that a piece's end goes with its rows: a token's 4 at
        // hd 128 2600 cycles, 5100 with copy 0's warp adding its lanes' rows (B64 n1 window
        // 2048: 59.0 -> 55.1 us; B64 n8 hd 64 44.6 -> 41.1; with two copies this way loses, B64
        // n16 45.2 against 44.0).
        stat[lane_row] = make_float2(mrow, lrow);
        warp_arrive(meet, lane);
        if (have) load_rows(false);
        if (!tree_wait(meet, meets++ & 1, ctl)) { ok = false; break; }
        float M = -INFINITY, sum = 0.f, weight = 0.f;
#pragma unroll
        for (int k = 0; k < kSplit; ++k) M = fmaxf(M, stat[k * kRows + row].x);
#pragma unroll
        for (int k = 0; k < kSplit; ++k) {
          const float2 ml = stat[k * kRows + row];
          const float w = ml.y != 0.f ? ex2_approx(ml.x - M) : 0.f;
          sum = fmaf(ml.y, w, sum);
          if (k == copy) weight = w;
        }
        if (whole && sum != 0.f) weight /= sum;
        warp_arrive(meet, lane);
        if (mine && copy == 0) put_stats(M, sum);
        if (!tree_wait(o_done, (R - 1) & 1, ctl) || !tree_wait(meet, meets++ & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        float4 *part = reinterpret_cast<float4 *>(smem + L::kQ);
        if constexpr (kSplit == 2) {
          // Each copy hands one half of its columns over and adds the other: the Q tile holds a
          // half of every lane.
          constexpr int kCols2 = HD / 2, kOnce = kCols2 < 32 ? kCols2 : 32, kPieces = kCols2 / 4;
          static_assert(kTileRows * kPieces * 16 <= L::kTileBytes, "half of every lane's O fits the Q tile");
          auto piece = [](int l, int i) { return l * kPieces + (i ^ (l & (kPieces < 8 ? kPieces - 1 : 7))); };
          auto o_columns = [&](float *x, int c) {            // kOnce weighed columns of this copy's O
            uint32_t ov[kOnce];
            if constexpr (kOnce == 32) tmem_ld_x32(tOx + c, ov);
            else tmem_ld_x16(tOx + c, ov);
            tmem_wait_ld();
            reg_fence<kOnce>(ov);
            // A copy that saw nothing counts 0, whatever its O holds.
#pragma unroll
            for (int e = 0; e < kOnce; ++e) x[e] = weight != 0.f ? __uint_as_float(ov[e]) * weight : 0.f;
          };
          float x[kOnce];
#pragma unroll 1
          for (int c = 0; c < kCols2; c += kOnce) {
            o_columns(x, (1 - copy) * kCols2 + c);
            if (mine)
#pragma unroll
              for (int e = 0; e < kOnce; e += 4)
                part[piece(lane_row, (c + e) / 4)] = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            __syncwarp();                                    // (the reads of TMEM are the warp's)
          }
          if (!meet_all()) { ok = false; break; }
          const size_t out = mine ? out_of(row) : 0;
#pragma unroll 1
          for (int c = 0; c < kCols2; c += kOnce) {
            const int col = copy * kCols2 + c;
            o_columns(x, col);
            if (mine)
#pragma unroll
              for (int e = 0; e < kOnce; e += 4) {
                const float4 z = part[piece(lane_row ^ kRows, (c + e) / 4)];
                x[e] += z.x, x[e + 1] += z.y, x[e + 2] += z.z, x[e + 3] += z.w;
              }
            if (mine && whole) {
              uint4 *dst = reinterpret_cast<uint4 *>(a.o + out * HD + col);
#pragma unroll
              for (int e = 0; e < kOnce; e += 8)
                dst[e / 8] = make_uint4(pack_bf16x2(x[e], x[e + 1]), pack_bf16x2(x[e + 2], x[e + 3]),
                                        pack_bf16x2(x[e + 4], x[e + 5]), pack_bf16x2(x[e + 6], x[e + 7]));
            } else if (mine) {
              float4 *dst = reinterpret_cast<float4 *>(a.ws_o + (rec0 + row) * HD + col);
#pragma unroll
              for (int e = 0; e < kOnce; e += 4) dst[e / 4] = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
            __syncwarp();                                    // (the reads of TMEM are the warp's)
          }
          if (have && !meet_all()) { ok = false; break; }    // read before the next queries go there
        } else {
          // The tile takes every column of up to half of its rows, or half the columns of all.
          constexpr int kHalf = kRows / 2;
          static_assert(kSplit * kHalf * HD * 4 <= L::kTileBytes, "half of the copies' O fits the Q tile");
          const bool few = rows <= kHalf;
          const int pieces = few ? HD / 4 : HD / 8, at = few ? copy * kHalf + row : lane_row;   // 16 bytes each
          const bool here = mine && (!few || row < kHalf);
          auto piece = [&](int l, int i) { return l * pieces + (i ^ (l & min(7, pieces - 1))); };   // against bank conflicts
          XATTN_DCHECK(!here || (at + 1) * pieces * 16 <= static_cast<int>(L::kTileBytes), a.status);
#pragma unroll 1
          for (int p0 = 0; p0 < HD / 4; p0 += pieces) {
#pragma unroll 1
            for (int c = p0 / 8 * 8; c < p0 + pieces; c += 8) {
              uint32_t ov[32];
              tmem_ld_x32(tOx + 4 * c, ov);
              tmem_wait_ld();
              reg_fence<32>(ov);
              // A copy that saw nothing counts 0, whatever its O holds.
              auto val = [&](int x) { return weight != 0.f ? __uint_as_float(ov[x]) * weight : 0.f; };
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (here && (HD > 32 || (c + x >= p0 && c + x < p0 + pieces)))
                  part[piece(at, c + x - p0)] = make_float4(val(4 * x), val(4 * x + 1), val(4 * x + 2), val(4 * x + 3));
              __syncwarp();                                  // (the reads of TMEM are the warp's)
            }
            if (!meet_all()) { ok = false; break; }
            const int i = lane & (pieces - 1), each = 32 / pieces;
            for (int r = quarter * each + lane / pieces; r < rows; r += 4 * each) {
              const int step = few ? kHalf : kRows;
              float4 x = part[piece(r, i)];
#pragma unroll
              for (int k = 1; k < kSplit; ++k) {
                const float4 z = part[piece(r + k * step, i)];
                x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
              }
              if (whole)
                *reinterpret_cast<uint2 *>(a.o + out_of(r) * HD + 4 * (p0 + i)) =
                    make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
              else
                *reinterpret_cast<float4 *>(a.ws_o + (rec0 + r) * HD + 4 * (p0 + i)) = x;
            }
            // The Q tile is read before the next columns, or queries, go there.
            if ((have || p0 + pieces < HD / 4) && !meet_all()) { ok = false; break; }
          }
        }
        if (!ok) break;
      } else {
        if (!tree_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        const size_t out = mine ? out_of(row) : 0;
        const float inv = lrow != 0.f ? 1.f / lrow : 0.f;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t ov[32];
          if (live) tmem_ld_x32(tOx + c, ov);
          tmem_wait_ld();
          reg_fence<32>(ov);
          if (mine && whole) {
            auto val = [&](int i) { return lrow != 0.f ? __uint_as_float(ov[i]) * inv : 0.f; };
            uint4 *dst = reinterpret_cast<uint4 *>(a.o + out * HD + c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(val(8 * i), val(8 * i + 1)), pack_bf16x2(val(8 * i + 2), val(8 * i + 3)),
                                  pack_bf16x2(val(8 * i + 4), val(8 * i + 5)), pack_bf16x2(val(8 * i + 6), val(8 * i + 7)));
          } else if (mine) {
            uint4 *dst = reinterpret_cast<uint4 *>(a.ws_o + (rec0 + row) * HD + c);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
          }
          __syncwarp();
        }
        if (mine) put_stats(mrow, lrow);
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Merges the records of the cut units: block (c, y) takes rows of the unit that run c starts
// and does not finish, if there is one (plan[c]: sequence, unit, last run, yes); with kSearch
// of the c-th such unit, so that a few units of many rows over many runs are not 30 idle blocks
// to each that has work. The search takes 1.2 us, so it is for calls that would otherwise launch
// more blocks than the GPU holds twice (B8 n16 over 8192 positions: 22.5 us, 26.9 without; with
// one token each 17.0 and 15.8). HD / 4 lanes
// hold a row, four columns each. Up to 8 records are added by one warp; more (a long cache
// over many runs) by the block's warps, every eighth record each, and then in order.
template <int HD, bool kSearch>
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeArgs a, int runs) {
  constexpr int kLanes = HD / 4, kSub = 32 / kLanes, kWarps = 8;
  __shared__ float4 part[kWarps][32];
  __shared__ float2 part_ml[kWarps][32];
  grid_dep_launch();
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = lane % kLanes, sub = lane / kLanes;
  int c0 = blockIdx.x;
  if constexpr (kSearch) {
    __shared__ int found, counts[kWarps];
    if (threadIdx.x == 0) found = -1;
    int want = c0;
#pragma unroll 1
    for (int r0 = 0; r0 < runs; r0 += 256) {
      const int c = r0 + static_cast<int>(threadIdx.x);
      const unsigned cut = __ballot_sync(0xffffffffu, c < runs && a.plan[c].w != 0);
      if (lane == 0) counts[warp] = __popc(cut);
      __syncthreads();
      int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = all;
        all += counts[w];
      }
      if (((cut >> lane) & 1u) && before + __popc(cut & ((1u << lane) - 1u)) == want) found = c;
      want -= all;
      __syncthreads();
    }
    c0 = found;
    if (c0 < 0) return;
  }
  const int4 plan = a.plan[c0];
  if (!plan.w) return;
  const int group = a.group, rows_all = a.n * group, row_tiles = a.row_tiles;
  const int kvh = plan.y / row_tiles, row0 = (plan.y % row_tiles) * a.tile_rows;
  const int rows = min(rows_all - row0, a.tile_rows);
  const int records = plan.z - c0 + 1;
  const bool wide = records > kWarps;
  const int first = wide ? warp : 0, step = wide ? kWarps : 1;
  const int stride = kSub * static_cast<int>(gridDim.y) * (wide ? 1 : kWarps);
  for (int rb = (wide ? blockIdx.y : blockIdx.y * kWarps + warp) * kSub; rb < rows; rb += stride) {
    const int row = min(rb + sub, rows - 1);                // (a spare lane repeats the last row)
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // One pass, the next record on its way while one is added. A record that saw nothing holds
    // anything but a sum of 0. (Small code on purpose: this kernel's instructions come from L2
    // every time, the other kernel's having taken their place; unrolled by four, in two passes,
    // it took 9.4 us.)
    auto rec_of = [&](int k) { return static_cast<size_t>(2 * (c0 + k) + (k == 0 ? 1 : 0)) * a.rec_rows + row; };
    size_t rec = rec_of(first);
    float2 ml = first < records ? *reinterpret_cast<const float2 *>(a.ws_ml + 2 * rec) : make_float2(0.f, 0.f);
    float4 x = first < records ? *reinterpret_cast<const float4 *>(a.ws_o + rec * HD + 4 * i) : acc;
#pragma unroll 1
    for (int k = first; k < records; k += step) {
      const float2 ml_here = ml;
      const float4 x_here = x;
      if (k + step < records) {
        rec = rec_of(k + step);
        ml = *reinterpret_cast<const float2 *>(a.ws_ml + 2 * rec);
        x = *reinterpret_cast<const float4 *>(a.ws_o + rec * HD + 4 * i);
      }
      if (ml_here.y != 0.f) {
        const float m2 = fmaxf(M, ml_here.x), f0 = ex2_approx(M - m2), f1 = ex2_approx(ml_here.x - m2);
        M = m2;
        sum = sum * f0 + ml_here.y * f1;
        acc.x = acc.x * f0 + x_here.x * f1, acc.y = acc.y * f0 + x_here.y * f1;
        acc.z = acc.z * f0 + x_here.z * f1, acc.w = acc.w * f0 + x_here.w * f1;
      }
    }
    if (wide) {
      part[warp][lane] = acc;
      part_ml[warp][lane] = make_float2(M, sum);
      __syncthreads();
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      M = -INFINITY, sum = 0.f;
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_ml[w][lane].x);
#pragma unroll 1
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = part_ml[w][lane];
        const float4 x = part[w][lane];
        const float f = ml.y != 0.f ? ex2_approx(ml.x - M) : 0.f;
        sum = fmaf(ml.y, f, sum);
        acc.x = fmaf(x.x, f, acc.x), acc.y = fmaf(x.y, f, acc.y);
        acc.z = fmaf(x.z, f, acc.z), acc.w = fmaf(x.w, f, acc.w);
      }
      __syncthreads();                                      // before the next rows overwrite part
    }
    if (rb + sub < rows && (!wide || warp == 0)) {
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      const int rho = row0 + row;
      const size_t out =
          (static_cast<size_t>(plan.x) * a.n + rho / group) * a.nh + static_cast<size_t>(kvh) * group + rho % group;
      *reinterpret_cast<uint2 *>(a.o + out * HD + 4 * i) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (i == 0) a.lse[out] = sum != 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
    }
  }
}

// A unit a CTA, or nearly: whole units may be faster than cut ones.
bool tree_choose(const TreeArgs &a, int grid) {
  const double units = static_cast<double>(a.B) * a.nkv * a.row_tiles;
  return !a.whole && units <= grid && 2 * units >= grid;
}

template <int HD, int kSplit, bool kChoose>
cudaError_t launch_tree_kernel(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int grid,
                               cudaStream_t stream) {
  using L = TreeLayout<HD>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t err = allow_smem(tree_kernel<HD, kSplit, kChoose>, L::kDynBytes, allowed);
  if (err != cudaSuccess) return err;
  return launch_pdl(tree_kernel<HD, kSplit, kChoose>, static_cast<unsigned>(grid), kTreeThreads, L::kDynBytes, stream,
                    mk, mv, a);
}

template <int HD, int kSplit>
cudaError_t launch_tree_split(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, bool choose, int grid,
                              cudaStream_t stream) {
  const cudaError_t err = choose ? launch_tree_kernel<HD, kSplit, true>(mk, mv, a, grid, stream)
                                 : launch_tree_kernel<HD, kSplit, false>(mk, mv, a, grid, stream);
  if (err != cudaSuccess || grid == 1 || a.whole) return err;
  // A block for the rows that 8 warps hold at once; where a unit spans many runs (few units),
  // one for each warp's rows.
  const int rows_once = 128 / HD * (static_cast<long long>(a.B) * a.nkv * 8 > grid ? 8 : 1);
  const long long units = static_cast<long long>(a.B) * a.nkv * a.row_tiles;
  const unsigned by_rows = static_cast<unsigned>((a.rec_rows + rows_once - 1) / rows_once);
  constexpr long long kTwice = 2 * 8 * 152;                    // blocks, 8 an SM
  if (units < (grid - 1) / 2 && (grid - 1ll) * by_rows > kTwice)
    return launch_pdl(tree_combine_kernel<HD, true>, dim3(static_cast<unsigned>(units), by_rows), 256, 0, stream, a, grid);
  return launch_pdl(tree_combine_kernel<HD, false>, dim3(static_cast<unsigned>(grid - 1), by_rows), 256, 0, stream, a, grid);
}

template <int HD>
cudaError_t launch_tree_hd(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int grid,
                           cudaStream_t stream) {
  const bool choose = tree_choose(a, grid);
  if (a.tile_rows == 32) return launch_tree_split<HD, 4>(mk, mv, a, choose, grid, stream);
  if (a.tile_rows == 64) return launch_tree_split<HD, 2>(mk, mv, a, choose, grid, stream);
  return launch_tree_split<HD, 1>(mk, mv, a, choose, grid, stream);
}

}  // namespace

// Rows of a row tile: the smallest of 32, 64 and 128 that holds every row of a kv head, else
// 128 (and several tiles).
int tree_tile_rows(int n, int nh, int nkv) {
  const long long rows = static_cast<long long>(n) * (nh / nkv);
  return rows <= 32 ? 32 : (rows <= 64 ? 64 : kTileRows);
}

// Runs are whole units when no sequence can have more tiles than this. At 1000 positions (8
// tiles; n 8, hd 64, 4 kv heads) whole against cut units: 64 sequences 12.9 and 21.6 us; one
// sequence 9.6 and 10.8 us on the GPU, 10.4 and 12.0 us with the host's part of a call.
constexpr int kWholeTiles = 8;
bool tree_whole(int page_size, int max_pages) {
  return static_cast<long long>(max_pages) * page_size <= kWholeTiles * kTileRows;
}

// The longest line that the table allows, in tiles (whole units).
double tree_line(const TreeArgs &a) {
  const long long tiles = a.whole ? 1 : (static_cast<long long>(a.max_pages) * a.page_size + kTileRows - 1) / kTileRows;
  return static_cast<double>(tiles) * a.B * a.nkv * a.row_tiles;
}

// CTAs of a call on a GPU with `sms` SMs: one resident wave, or one per tile (whole unit) of
// the longest line that the table allows when that is shorter.
int tree_grid(const TreeArgs &a, int hd, int sms) {
  const double most = tree_line(a);
  const int resident = sms * (a.tile_rows == kTileRows || hd == 128 ? 1 : tree_ctas<64, 2>());
  return most < resident ? static_cast<int>(most) : resident;
}

size_t tree_workspace_bytes(int grid, int rec_rows, int hd) {
  return static_cast<size_t>(grid) * (sizeof(int4) + 2 * rec_rows * (static_cast<size_t>(hd) + 2) * sizeof(float));
}

cudaError_t launch_tree_bf16(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int hd, int grid,
                             cudaStream_t stream) {
  if (hd == 32) return launch_tree_hd<32>(mk, mv, a, grid, stream);
  if (hd == 64) return launch_tree_hd<64>(mk, mv, a, grid, stream);
  if (hd == 128) return launch_tree_hd<128>(mk, mv, a, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace xattn
