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
// head are packed into tiles of 128 rows (row = token * group + head of the group), one TMEM
// lane each, and the cache streams past them in 128-position tiles.
//   * Work: a unit is (sequence, kv head, row tile) with the position tiles it can see; the
//     units' tiles in order form one line that is cut into equal runs, one per resident CTA,
//     so ragged lengths and windows balance without a plan from the host (the lengths are
//     read on the device: a captured graph follows them).
//   * A run's end cuts a unit: such pieces write (max, sum, unnormalised O) records, and
//     tree_combine_kernel merges each cut unit's records in order.
//   * Pages: a tile is loaded box by box (one TMA box per page, or per 128 rows of a larger
//     one). A box that no row can see, or whose table entry is no page, is loaded from
//     outside the pool: the TMA unit writes zeros and reads nothing.
// Warps: 0 TMA producer; 1 TMEM owner and MMA issuer; 2-5 softmax, one query row a thread.
// TMEM: S [0,128) fp32 | P [128,192) bf16 pairs | O [192, 192 + hd).
#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kTreeThreads = 192;

// K and V rings of one 128-position tile per slot. hd 32 and 64 take two CTAs an SM (256 TMEM
// columns each), hd 128 one; the bytes are chosen so that no more fit.
template <int HD>
struct TreeLayout {
  static constexpr int kCtas = HD == 128 ? 1 : 2;               // resident per SM
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
  static constexpr int kNumBars = 4 * kSlots + 5;
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

// Bits lo..hi of a 32-bit word (clipped to it; none when hi < lo).
__device__ __forceinline__ uint32_t word_range(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 31);
  return hi < lo ? 0u : (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
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

// A run of the line of tiles, walked piece by piece; warp-uniform, every warp of every role
// walks the same pieces. All counts in 64 bits.
struct Walk {
  long long pos, stop;     // next tile and end of the run, on the line
  long long first;         // where sequence b starts on it
  int b, e0, e1, unit;     // piece: sequence, entries [e0, e1) of its list, unit within it
  Sight s;
};

// Tiles of all sequences, and (for the warp's target tile) the sequence that holds it.
__device__ __forceinline__ long long line_length(const TreeArgs &a, int units, int lane) {
  long long t = 0;
  for (int b = lane; b < a.B; b += 32) t += sight_of(a, b).count;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  return t * units;
}

__device__ __forceinline__ void line_find(const TreeArgs &a, int units, int lane, long long target, int *b_out,
                                          long long *first_out) {
  long long base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const long long mine = b < a.B ? static_cast<long long>(sight_of(a, b).count) * units : 0;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, b < a.B && base + incl > target);
    if (past) {
      const int l = __ffs(past) - 1;
      *b_out = b0 + l;
      *first_out = base + __shfl_sync(0xffffffffu, incl - mine, l);
      return;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  *b_out = a.B;
  *first_out = base;
}

__device__ __forceinline__ bool walk_piece(Walk &w, const TreeArgs &a, int units) {
  if (w.pos >= w.stop) return false;
  long long at = w.pos - w.first;
  if (at >= static_cast<long long>(w.s.count) * units) {       // the next sequence
    w.first += static_cast<long long>(w.s.count) * units;
    w.s = sight_of(a, ++w.b);
    at = 0;
  }
  w.unit = static_cast<int>(at / w.s.count);
  w.e0 = static_cast<int>(at % w.s.count);
  w.e1 = static_cast<int>(min(static_cast<long long>(w.s.count), w.e0 + (w.stop - w.pos)));
  w.pos += w.e1 - w.e0;
  return true;
}

// Record of a cut unit's piece: CTA c's piece that starts inside a unit is record 2c, the one
// that starts it record 2c + 1. Layout: [records][rows][hd] O, then [records][rows] (max, sum).
template <int HD>
__global__ void __launch_bounds__(kTreeThreads, TreeLayout<HD>::kCtas)
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
  volatile uint32_t *pages = reinterpret_cast<volatile uint32_t *>(smem + L::kPages);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 16);
  const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};
  XATTN_DCHECK(smem + L::kUsed <= tree_smem_raw + L::kDynBytes, a.status);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < 4 * L::kSlots; ++s) mbar_init(bar(s), 1);
    mbar_init(s_full, 1);
    mbar_init(s_free, 128);
    mbar_init(p_full, 128);
    mbar_init(o_done, 1);
    mbar_init(q_full, 128);
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
  const int group = a.nh / a.nkv, rows_all = a.n * group;
  const int row_tiles = (rows_all + kTileRows - 1) / kTileRows;
  const int units = a.nkv * row_tiles;
  const long long length = line_length(a, units, lane);
  const long long runs = min(static_cast<long long>(gridDim.x), length);
  Walk walk;
  walk.pos = walk.stop = 0;
  if (blockIdx.x < runs) {
    walk.pos = blockIdx.x * length / runs;
    walk.stop = (blockIdx.x + 1) * length / runs;
    line_find(a, units, lane, walk.pos, &walk.b, &walk.first);
    walk.s = sight_of(a, walk.b);
  }

  if (warp == 0) {
    // ---------------- TMA producer: lane l loads box l of each tile ----------------
    const int box_rows = min(a.page_size, kTileRows), boxes = kTileRows / box_rows;
    int R = 0, issued_k = 0, issued_v = 0;
    bool ok = true;
    while (ok && walk_piece(walk, a, units)) {
      const int kvh = walk.unit / row_tiles;
      const int *table = a.page_table + static_cast<size_t>(walk.b) * a.max_pages;
#pragma unroll 1
      for (int e = walk.e0; e < walk.e1; ++e, ++R) {
        const int tile = e < walk.s.heads ? e : e - walk.s.heads + walk.s.lo;
        // The box's page, or num_pages (outside the pool) when it holds nothing to see.
        const int p0 = tile * kTileRows + lane * box_rows;
        int page = a.num_pages, row = 0;
        if (lane < boxes && p0 < walk.s.end && (p0 + box_rows > walk.s.far || p0 < a.sinks)) {
          const int id = table[p0 / a.page_size];               // p0 < end <= max_pages * page_size
          if (id >= 0 && id < a.num_pages) page = id, row = p0 % a.page_size;
        }
        const unsigned held = __ballot_sync(0xffffffffu, page != a.num_pages);
        const int s = R % L::kSlots;
        const uint32_t ph = static_cast<uint32_t>((R / L::kSlots) & 1) ^ 1u;
        if (!tree_wait(k_empty(s), ph, ctl)) { ok = false; break; }
        if (lane == 0) mbar_expect_tx(k_full(s), L::kTileBytes);
        __syncwarp();
        if (lane < boxes)
#pragma unroll
          for (int c = 0; c < L::kSubTiles; ++c)
            tma_load_4d(sK + s * L::kTileBytes + c * L::kSubBytes + lane * box_rows * L::kAtomBytes, &mk, k_full(s),
                        64 * c, kvh, row, page);
        issued_k = R + 1;
        if (!tree_wait(v_empty(s), ph, ctl)) { ok = false; break; }
        if (lane == 0) {
          pages[s] = held;                 // read by the softmax warps before P V frees the slot
          mbar_expect_tx(v_full(s), L::kTileBytes);
        }
        __syncwarp();
        if (lane < boxes)
#pragma unroll
          for (int c = 0; c < L::kSubTiles; ++c)
            tma_load_4d(sV + s * L::kTileBytes + c * L::kSubBytes + lane * box_rows * L::kAtomBytes, &mv, v_full(s),
                        64 * c, kvh, row, page);
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
    while (ok && walk_piece(walk, a, units)) {
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
    // ---------------- softmax: thread = query row of the tile ----------------
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tSx = tS + lane_off, tPx = tP + lane_off, tOx = tO + lane_off;
    const int box_rows = min(a.page_size, kTileRows);
    const unsigned all_boxes = box_rows == kTileRows ? 1u : (1u << (kTileRows / box_rows)) - 1u;
    int R = 0;
    bool ok = true;
    while (ok && walk_piece(walk, a, units)) {
      const Sight s = walk.s;
      const int kvh = walk.unit / row_tiles, row0 = (walk.unit % row_tiles) * kTileRows;
      const int rows = min(rows_all - row0, kTileRows);
      const bool live = quarter * 32 < rows;                 // the warp has a row
      const int rho = row0 + row, token = rho / group;
      const bool mine = row < rows;
      const size_t out = (static_cast<size_t>(walk.b) * a.n + token) * a.nh + static_cast<size_t>(kvh) * group +
                         rho % group;                         // row of q, o and lse
      // The row's query into the Q tile, swizzled as TMA would (dead rows of a live warp: 0).
      if (live) {
        constexpr int kChunks = static_cast<int>(L::kAtomBytes / 16);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (mine ? out : 0) * HD);
#pragma unroll
        for (int c = 0; c < HD / 8; ++c) {
          const uint4 x = mine ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          const int ch = c % kChunks, sw = L::kAtomBytes == 128 ? (ch ^ (row & 7)) : (ch ^ ((row >> 1) & 3));
          *reinterpret_cast<uint4 *>(smem + L::kQ + (c / kChunks) * L::kSubBytes + row * L::kAtomBytes + (sw << 4)) = x;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
      // The row's ancestors, its position, and how far its window reaches.
      unsigned long long word = 0;
      if (mine) {
        const unsigned long long all = a.n == 64 ? ~0ull : (1ull << a.n) - 1;
        word = a.tree ? a.tree[static_cast<size_t>(walk.b) * a.n + token] & all : (2ull << token) - 1;
      }
      const int pos = s.ctx + max(__popcll(word) - 1, 0);
      const int far = pos - a.window + 1;
      float mrow = -INFINITY, lrow = 0.f;
#pragma unroll 1
      for (int e = walk.e0; e < walk.e1; ++e, ++R) {
        const int tile = e < s.heads ? e : e - s.heads + s.lo, t0 = tile * kTileRows;
        const int slot = R % L::kSlots;
        // V has landed (so pages[slot] is there to read; its slot is not loaded again before
        // this tile's P V), and the scores.
        if (!tree_wait(v_full(slot), (R / L::kSlots) & 1, ctl) || !tree_wait(s_full, R & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        const unsigned held = pages[slot];
        // Positions that some row does not see: new ones, those behind a window, missing pages.
        const bool edge = t0 + kTileRows > s.ctx || held != all_boxes ||
                          (t0 <= s.end - 1 - a.window && t0 + kTileRows > a.sinks);
        uint32_t vis[4];
        if (edge) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int base = t0 + 32 * w, off = base - s.ctx;
            uint32_t m = word_range(0, s.ctx - 1 - base) & (word_range(far - base, 31) | word_range(0, a.sinks - 1 - base));
            if (off >= 0) {
              if (off < 64) m |= static_cast<uint32_t>(word >> off);
            } else if (off > -32) {
              m |= static_cast<uint32_t>(word << -off);
            }
            uint32_t there = 0;
            if (box_rows >= 32)
              there = (held >> (32 * w / box_rows)) & 1u ? 0xffffffffu : 0u;
            else
              there = ((held >> (2 * w)) & 1u ? 0x0000ffffu : 0u) | ((held >> (2 * w + 1)) & 1u ? 0xffff0000u : 0u);
            vis[w] = m & there;
          }
          // V rows that no row sees may hold anything: they are zeroed before P V, in which
          // their P is 0 (0 x NaN would not be). Missing pages were loaded as zeros.
          const int p = t0 + row;
          if (p >= s.end || (p < s.far && p >= a.sinks)) {
#pragma unroll
            for (int c = 0; c < L::kSubTiles; ++c)
#pragma unroll
              for (uint32_t x = 0; x < L::kAtomBytes; x += 16)
                *reinterpret_cast<uint4 *>(smem + L::kV + slot * L::kTileBytes + c * L::kSubBytes +
                                           row * L::kAtomBytes + x) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (!live) {
          mbar_arrive(s_free);
          // P of the previous tile has been read before anyone moves on.
          if (!tree_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
          mbar_arrive(p_full);
          continue;
        }
        uint32_t r[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld_x32(tSx + c, r + c);
        tmem_wait_ld();
        reg_fence<128>(r);
        tc_fence_before();
        mbar_arrive(s_free);
        // Scaled, masked scores in place (the log2 domain), their maximum, P and its sum.
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; ++c) {
          float x = __uint_as_float(r[c]) * a.scale_log2;
          if (edge && ((vis[c >> 5] >> (c & 31)) & 1u) == 0u) x = -INFINITY;
          r[c] = __float_as_uint(x);
          mx[c & 3] = fmaxf(mx[c & 3], x);
        }
        const float mnew = fmaxf(mrow, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        // O is rescaled only when some row's maximum grew by more than 2^8.
        const bool rescale = __any_sync(0xffffffffu, mnew > mrow + 8.0f);
        const float m_use = rescale ? mnew : mrow;
        const float alpha = (rescale && mnew > mrow) ? ex2_approx(mrow - mnew) : 1.f;
        const float base = m_use == -INFINITY ? 0.f : m_use;       // a row that has seen nothing yet
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          const float p0 = ex2_approx(__uint_as_float(r[2 * c]) - base);
          const float p1 = ex2_approx(__uint_as_float(r[2 * c + 1]) - base);
          ps[(c & 1) * 2] += p0;
          ps[(c & 1) * 2 + 1] += p1;
          r[c] = pack_bf16x2(p0, p1);
        }
        if (!tree_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        tmem_st_x32(tPx, r);
        tmem_st_x32(tPx + 32, r + 32);
        if (rescale && e > walk.e0) {
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
        mbar_arrive(p_full);
      }
      if (!ok) break;
      // The piece's result: O and the LSE of a whole unit, else a record.
      if (!tree_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
      if (!live) continue;
      tc_fence_after();
      const bool whole = walk.e0 == 0 && walk.e1 == s.count;
      const size_t rec = 2 * static_cast<size_t>(blockIdx.x) + (walk.e0 == 0 ? 1 : 0);
      const float inv = lrow > 0.f ? 1.f / lrow : 0.f;
      float *ws_o = a.ws_o + (rec * a.rec_rows + row) * HD;
#pragma unroll
      for (int c = 0; c < HD; c += 32) {
        uint32_t ov[32];
        tmem_ld_x32(tOx + c, ov);
        tmem_wait_ld();
        reg_fence<32>(ov);
        if (mine && whole) {
          // A row that sees nothing gives 0, whatever its O columns hold.
          uint4 *dst = reinterpret_cast<uint4 *>(a.o + out * HD + c);
          auto val = [&](int i) { return lrow > 0.f ? __uint_as_float(ov[i]) * inv : 0.f; };
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16x2(val(8 * i), val(8 * i + 1)), pack_bf16x2(val(8 * i + 2), val(8 * i + 3)),
                                pack_bf16x2(val(8 * i + 4), val(8 * i + 5)), pack_bf16x2(val(8 * i + 6), val(8 * i + 7)));
        } else if (mine) {
          XATTN_DCHECK(rec < 2 * static_cast<size_t>(gridDim.x) && row < a.rec_rows, a.status);
          uint4 *dst = reinterpret_cast<uint4 *>(ws_o + c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
        }
        __syncwarp();
      }
      if (mine && whole) a.lse[out] = lrow > 0.f ? (mrow + __log2f(lrow)) * kLn2 : -INFINITY;
      if (mine && !whole) *reinterpret_cast<float2 *>(a.ws_ml + 2 * (rec * a.rec_rows + row)) = make_float2(mrow, lrow);
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

// One warp per (sequence, token, head): merges the records of its unit if a run's end cut it.
template <int HD>
__global__ void __launch_bounds__(128) tree_combine_kernel(const TreeArgs a, int runs_max) {
  constexpr int kPerLane = HD / 32;
  grid_dep_launch();
  grid_dep_wait();
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<long long>(a.B) * a.n * a.nh) return;
  const int h = static_cast<int>(w % a.nh), token = static_cast<int>(w / a.nh % a.n);
  const int b = static_cast<int>(w / a.nh / a.n);
  const int group = a.nh / a.nkv, kvh = h / group, rho = token * group + h % group;
  const int row_tiles = (a.n * group + kTileRows - 1) / kTileRows, units = a.nkv * row_tiles;
  // The unit's place on the line.
  long long before = 0, length = 0;
  for (int i = lane; i < a.B; i += 32) {
    const long long c = static_cast<long long>(sight_of(a, i).count) * units;
    length += c;
    if (i < b) before += c;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    length += __shfl_xor_sync(0xffffffffu, length, off);
    before += __shfl_xor_sync(0xffffffffu, before, off);
  }
  const int count = sight_of(a, b).count;
  const long long u0 = before + static_cast<long long>(kvh * row_tiles + rho / kTileRows) * count, u1 = u0 + count;
  const long long runs = min(static_cast<long long>(runs_max), length);
  const long long c0 = ((u0 + 1) * runs - 1) / length, c1 = (u1 * runs - 1) / length;   // first and last run
  if (c0 == c1) return;                                   // in one piece: already written
  const int row = rho % kTileRows;
  auto record = [&](long long c) { return (static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * a.rec_rows + row); };
  float M = -INFINITY;
  for (long long c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, a.ws_ml[2 * record(c)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float sum = 0.f, acc[kPerLane];
#pragma unroll
  for (int e = 0; e < kPerLane; ++e) acc[e] = 0.f;
  for (long long c = c0; c <= c1; ++c) {
    const size_t rec = record(c);
    const float2 ml = *reinterpret_cast<const float2 *>(a.ws_ml + 2 * rec);
    if (!(ml.y > 0.f)) continue;                          // saw nothing
    const float wgt = ex2_approx(ml.x - base);
    sum = fmaf(ml.y, wgt, sum);
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) acc[e] = fmaf(a.ws_o[rec * HD + lane * kPerLane + e], wgt, acc[e]);
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int e = 0; e < kPerLane; ++e)
    a.o[static_cast<size_t>(w) * HD + lane * kPerLane + e] = __float2bfloat16_rn(acc[e] * inv);
  if (lane == 0) a.lse[w] = sum > 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
}

template <int HD>
cudaError_t launch_tree_hd(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int grid,
                           cudaStream_t stream) {
  using L = TreeLayout<HD>;
  cudaError_t err = cudaFuncSetAttribute(tree_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(L::kDynBytes));
  if (err != cudaSuccess) return err;
  err = launch_pdl(tree_kernel<HD>, static_cast<unsigned>(grid), kTreeThreads, L::kDynBytes, stream, mk, mv, a);
  if (err != cudaSuccess || grid == 1) return err;
  const long long warps = static_cast<long long>(a.B) * a.n * a.nh;
  return launch_pdl(tree_combine_kernel<HD>, static_cast<unsigned>((warps + 3) / 4), 128, 0, stream, a, grid);
}

}  // namespace

// CTAs of a call on a GPU with `sms` SMs: one resident wave, or one per tile of the longest
// line that the table allows when that is shorter.
int tree_grid(int B, int n, int nh, int nkv, int hd, int page_size, int max_pages, int sms) {
  const long long tiles = (static_cast<long long>(max_pages) * page_size + kTileRows - 1) / kTileRows;
  const long long row_tiles = (static_cast<long long>(n) * (nh / nkv) + kTileRows - 1) / kTileRows;
  const long long most = tiles * B * nkv * row_tiles;
  const int resident = sms * (hd == 128 ? TreeLayout<128>::kCtas : TreeLayout<64>::kCtas);
  return static_cast<int>(most < resident ? most : resident);
}

int tree_record_rows(int n, int nh, int nkv) {
  const long long rows = static_cast<long long>(n) * (nh / nkv);
  return rows < kTileRows ? static_cast<int>(rows) : kTileRows;
}

size_t tree_workspace_bytes(int grid, int rec_rows, int hd) {
  return static_cast<size_t>(grid) * 2 * rec_rows * (static_cast<size_t>(hd) + 2) * sizeof(float);
}

cudaError_t launch_tree_bf16(const CUtensorMap &mk, const CUtensorMap &mv, const TreeArgs &a, int hd, int grid,
                             cudaStream_t stream) {
  if (hd == 32) return launch_tree_hd<32>(mk, mv, a, grid, stream);
  if (hd == 64) return launch_tree_hd<64>(mk, mv, a, grid, stream);
  if (hd == 128) return launch_tree_hd<128>(mk, mv, a, grid, stream);
  return cudaErrorInvalidValue;
}

}  // namespace xattn
