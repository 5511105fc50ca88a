// Latent attention in its absorbed form: a few new tokens per sequence over a paged cache whose rows
// (c, k_rope) are the keys of every head, and whose c are the values.
//
// GB300 mapping. A cached position is 2 (dc + dr) bytes for all heads, and 2 (2 dc + dr) flops a query row:
// with 16 rows HBM bounds the operation, with 128 the tensor cores come near to it. The cache is read once per
// row tile, in tiles of 64 positions:
//   * S^T = C Q^T : positions are the M = 64 rows, the query rows (token, head) the N columns, so that a few
//     heads do not cost the 128 rows that a query tile has; and O^T += C^T P^T with the 128 numbers of a latent
//     block as M. One copy of the tile in shared memory is K-major for the first product and MN-major for the
//     second. O^T [dc, N] fp32 takes dc / 128 x N of the 512 TMEM columns, so N is at most 64: 16, 32 or 64
//     query rows a row tile, and several row tiles where there are more.
//   * Rings: a tile is dc / 128 pairs of 64-column sub-tiles (16 KB) and the shared part (8 KB); a pair is free
//     again as soon as its block of O^T has been added, so loads go on while a tile is worked on.
//   * Softmax: a thread has one position and half of the columns; a column's maximum over the positions would be a
//     reduction over lanes. It is needed only where some score exceeds the column's running maximum by more than
//     2^8 (the stale one is exact because the final division uses the same): each tile asks just that, in one vote,
//     and only where the answer is yes are the maxima taken and O^T rescaled. Sums stay with the threads
//     until the end.
//   * Work: the sequences' tiles form one line that is cut into equal runs, one per group of CTAs, a CTA of the
//     group per row tile (they read the same tiles at the same time, the second from L2); lengths are read on the
//     device, so a captured graph follows them. A run's end cuts a sequence: such pieces write (max, sum, O)
//     records, and latent_combine_kernel merges them in order.
//   * Measured: 64 sequences of 8192 positions, one token of 16 heads, 512 + 64: 106 us, 5.7 TB/s; of 4096 62 us, and 79 with 64
//     heads, 115 with 128 (two row tiles: 2560 cycles of shared-memory reads a tile of 64 rows, 3200 taken). A batch of
//     64 takes 15 us and 10.7 us for every 1000 positions beyond 2048 (7 TB/s; 9.5 us with 16 positions): the 15 are the start, the last
//     tiles' chain, records and the combine. One sequence of 16 positions takes 9.5 us, of 1000 11.
//   * Roundings: scores, maxima, sums and O are fp32; P is rounded to bf16, C's type.
//   * Pages as in attn_tree.cu: a box whose table entry is no page is loaded from outside the pool (zeros).
// Warps: 0 TMA producer; 1 TMEM owner and issuer of S^T; 10 issuer of O^T (apart, so that a tile's P is not kept waiting
// behind scores whose tile has not landed); 2-9 softmax (warp & 3: lane quarter; two halves of the columns).
// TMEM: S^T buffers [0, N), [N, 2N); O^T block j [2N + j N, 2N + (j + 1) N).
#include <cfloat>
#include <type_traits>

#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kTilePos = 64;                       // positions of a tile
constexpr int kLatThreads = 352;
constexpr int kSoftWarps = 8;

// N: query rows (columns) of a row tile.
template <int N>
struct LatLayout {
  static constexpr uint32_t kSub = kTilePos * 128;               // a sub-tile of 64 columns
  static constexpr uint32_t kPair = 2 * kSub;
  static constexpr int kPairs = N == 64 ? 8 : 10;
  static constexpr int kQBufs = N == 16 ? 2 : 1;                 // query rows of this piece, and of the next
  static constexpr int kRopes = N == 64 ? 2 : 3;
  static constexpr uint32_t kQSub = N * 128;                     // 64 columns of the query rows
  static constexpr uint32_t kPRow = N * 2;
  static constexpr uint32_t kSwizzleP = N == 64 ? kSwizzle128 : (N == 32 ? kSwizzle64 : kSwizzle32);
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kP = kQ + kQBufs * 9 * kQSub;
  static constexpr uint32_t kC = kP + kTilePos * kPRow;
  static constexpr uint32_t kR = kC + kPairs * kPair;
  static constexpr uint32_t kBars = kR + kRopes * kSub;
  static constexpr int kNumBars = 2 * kPairs + 2 * kRopes + 7 + 2 * kQBufs;
  static constexpr uint32_t kBase = (kBars + 8 * kNumBars + 15) / 16 * 16;   // float [N] maxima, [N] factors, [4][N] parts
  static constexpr uint32_t kFlags = kBase + 6 * N * 4;
  static constexpr uint32_t kHeld = kFlags + 2 * kSoftWarps * 4;             // per rope slot: boxes that hold a page
  static constexpr uint32_t kMisc = (kHeld + 4 * kRopes + 15) / 16 * 16;
  static constexpr uint32_t kUsed = kMisc + 32;
  static constexpr uint32_t kDynBytes = kUsed + 1024;
  static_assert(kP % 1024 == 0 && kC % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  static_assert(kDynBytes <= 227 * 1024, "exceeds the opt-in shared memory of one CTA");
  static_assert(kDynBytes > 114 * 1024, "one CTA an SM: each holds all TMEM columns");
};

__device__ __forceinline__ bool lat_wait(uint32_t bar, uint32_t parity, const WaitCtl &ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void lat_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

__device__ __forceinline__ int lat_ctx(const LatentDecodeArgs &a, int b) {
  return min(max(a.ctx_lens[b], 0), a.max_pages * a.page_size - a.n);
}
__device__ __forceinline__ int lat_tiles(const LatentDecodeArgs &a, int b) {
  return (lat_ctx(a, b) + a.n + kTilePos - 1) / kTilePos;
}

// The line of `length` tiles in `runs` runs: the first length % runs have one more.
struct LatRuns {
  int each, more;
  __device__ LatRuns(int length, int runs) : each(length / runs), more(length - length / runs * runs) {}
  __device__ int start(int c) const { return c * each + min(c, more); }
  __device__ int of(int pos) const {
    const int head = more * (each + 1);
    return pos < head ? pos / (each + 1) : more + (pos - head) / each;
  }
};

// A run of the line, walked piece by piece; warp-uniform, every role walks the same pieces.
struct LatWalk {
  int pos, stop;           // next tile and end of the run, on the line
  int first;               // where sequence b starts on it
  int b, ctx, count;       // sequence, its committed positions and tiles
  int e0, e1;              // the piece: tiles [e0, e1) of the sequence
};

// What a walk holds is the same in every lane; the broadcasts let the compiler see it, so that loops over it keep the counters, and the
// descriptors made of them, in uniform registers. With those issued from a converged warp, a product of 64 x 64 x 16 takes its
// 33 cycles; with loop bounds as loaded 47, and issued by one lane in a branch of its own 53.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ bool lat_piece(LatWalk &w, const LatentDecodeArgs &a) {
  if (w.pos >= w.stop) return false;
  if (w.pos - w.first >= w.count) {
    w.first += w.count;
    if (++w.b >= a.B) return false;                              // (only if the lengths change under the call)
    w.ctx = uniform(lat_ctx(a, w.b));
    w.count = (w.ctx + a.n + kTilePos - 1) / kTilePos;
  }
  w.e0 = w.pos - w.first;
  w.e1 = min(w.count, w.e0 + (w.stop - w.pos));
  w.pos += w.e1 - w.e0;
  return true;
}

// The line's length, and this group's run of it. Lane l takes B / 32 sequences in a row.
__device__ __forceinline__ LatRuns lat_start(const LatentDecodeArgs &a, int group, int groups, int lane, LatWalk &w) {
  const int each = (a.B + 31) / 32, b0 = lane * each, b1 = min(a.B, b0 + each);
  int mine = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) mine += lat_tiles(a, b);
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  const int total = uniform(__shfl_sync(0xffffffffu, incl, 31));
  const LatRuns runs(total, min(groups, total));
  w.pos = w.stop = 0;
  if (group >= total) return runs;
  w.pos = runs.start(group);
  w.stop = runs.start(group + 1);
  const unsigned past = __ballot_sync(0xffffffffu, incl > w.pos);
  const int l = __ffs(past) - 1;
  int b = b0, at = incl - mine;
  if (lane == l) {
    for (int c = lat_tiles(a, b); at + c <= w.pos; c = lat_tiles(a, b)) at += c, ++b;
  }
  w.b = uniform(__shfl_sync(0xffffffffu, b, l));
  w.first = uniform(__shfl_sync(0xffffffffu, at, l));
  w.ctx = uniform(lat_ctx(a, w.b));
  w.count = (w.ctx + a.n + kTilePos - 1) / kTilePos;
  return runs;
}

// Sixteen TMEM lanes (S^T with M = 64 has 16 of its rows in the first lanes of each quarter) by 8 K columns: thread t
// gets rows t / 4 (x[4 i], x[4 i + 1]) and t / 4 + 8 (x[4 i + 2], x[4 i + 3]) of columns 8 i + 2 (t % 4), + 1.
template <int K>
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t addr, uint32_t *r) {
  if constexpr (K == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  } else if constexpr (K == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  }
}

// Eight-by-eight matrices of 16-bit numbers in that layout into rows of 16 bytes: lane l gives row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix_x2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t *r) {
  if constexpr (C == 32) tmem_ld_x32(addr, r);
  else if constexpr (C == 16) tmem_ld_x16(addr, r);
  else tmem_ld_x8(addr, r);
}
__device__ __forceinline__ void tmem_st_x8_words(uint32_t addr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <int C>
__device__ __forceinline__ void tmem_st_cols(uint32_t addr, const uint32_t *r) {
  if constexpr (C == 32) tmem_st_x32(addr, r);
  else if constexpr (C == 16) tmem_st_x16(addr, r);
  else tmem_st_x8_words(addr, r);
}

template <int N>
__global__ void __launch_bounds__(kLatThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mc,
                         const __grid_constant__ CUtensorMap mqc, const __grid_constant__ CUtensorMap mpair,
                         const LatentDecodeArgs a) {
  using L = LatLayout<N>;
  constexpr int kPairs = L::kPairs, kRopes = L::kRopes;
  extern __shared__ uint8_t latent_smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(latent_smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t sQ = smem_u32(smem + L::kQ), sP = smem_u32(smem + L::kP), sC = smem_u32(smem + L::kC),
                 sR = smem_u32(smem + L::kR), bar0 = smem_u32(smem + L::kBars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto c_full = [&](int s) { return bar(s); };
  auto c_empty = [&](int s) { return bar(kPairs + s); };
  auto r_full = [&](int s) { return bar(2 * kPairs + s); };
  auto r_empty = [&](int s) { return bar(2 * kPairs + kRopes + s); };
  constexpr int kB = 2 * kPairs + 2 * kRopes;
  auto s_full = [&](int x) { return bar(kB + x); };
  auto s_free = [&](int x) { return bar(kB + 2 + x); };
  const uint32_t p_full = bar(kB + 4), o_done = bar(kB + 5), meet = bar(kB + 6);
  constexpr int kQBufs = L::kQBufs;
  auto q_full = [&](int x) { return bar(kB + 7 + x); };
  auto q_empty = [&](int x) { return bar(kB + 7 + kQBufs + x); };
  float *base = reinterpret_cast<float *>(smem + L::kBase), *factor = base + N, *parts = base + 2 * N;
  volatile int *flags = reinterpret_cast<volatile int *>(smem + L::kFlags);
  volatile uint32_t *held_boxes = reinterpret_cast<volatile uint32_t *>(smem + L::kHeld);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 16);
  const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};
  XATTN_DCHECK(smem + L::kUsed <= latent_smem_raw + L::kDynBytes, a.status);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kB; ++s) mbar_init(bar(s), 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(s_free(x), kSoftWarps);
    }
    mbar_init(p_full, kSoftWarps);
    mbar_init(o_done, 1);
    for (int x = 0; x < kQBufs; ++x) {
      mbar_init(q_full(x), 1);
      mbar_init(q_empty(x), 1);
    }
    mbar_init(meet, kSoftWarps);
    fence_mbar_init();
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mc);
    tma_prefetch_desc(&mqc);
    tma_prefetch_desc(&mpair);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  grid_dep_wait();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  const uint32_t tS = tmem, tO = tmem + 2 * N;

  const int group = static_cast<int>(blockIdx.x) / a.row_tiles, rt = static_cast<int>(blockIdx.x) - group * a.row_tiles;
  const int groups = static_cast<int>(gridDim.x) / a.row_tiles, blocks = a.dc / 128;
  LatWalk walk;
  const LatRuns runs = lat_start(a, group, groups, lane, walk);


  if (warp == 0) {
    // ---------------- TMA producer: lane l finds box l of each tile ----------------
    const int box_rows = min(a.page_size, kTilePos), boxes = kTilePos / box_rows;
    const uint32_t box_bytes = box_rows * 128u;
    int R = 0, Rj = 0, issued_c = 0, issued_r = 0, pieces = 0;
    bool ok = true;
    while (ok && lat_piece(walk, a)) {
      const int qb = pieces % kQBufs;
      if (!lat_wait(q_empty(qb), ((pieces / kQBufs) & 1) ^ 1, ctl)) break;
      mbar_expect_tx_elect(q_full(qb), (2 * blocks + 1) * L::kQSub);
      tma_load_4d_elect(sQ + qb * 9 * L::kQSub, &mqc, q_full(qb), 0, rt * N, 0, walk.b);
      tma_load_4d_elect(sQ + (9 * qb + 2 * blocks) * L::kQSub, &mq, q_full(qb), a.dc, rt * N, walk.b, 0);
      ++pieces;
      const int *table = a.page_table + static_cast<size_t>(walk.b) * a.max_pages;
      const int end = walk.ctx + a.n;
      // This lane's box of tile e: its table entry (-1 past the end), read one tile ahead.
      auto box_of = [&](int e, int *row) -> int {
        const int p0 = e * kTilePos + lane * box_rows, at = p0 / a.page_size;
        *row = p0 - at * a.page_size;
        if (lane >= boxes || e >= walk.e1 || p0 >= end) return -1;
        return __ldg(table + at);
      };
      int row_next = 0, id_next = box_of(walk.e0, &row_next);
#pragma unroll 1
      for (int e = walk.e0; ok && e < walk.e1; ++e, ++R) {
        const int page = id_next >= 0 && id_next < a.num_pages ? id_next : a.num_pages, row = row_next;
        id_next = box_of(e + 1, &row_next);
        const unsigned held = __ballot_sync(0xffffffffu, page != a.num_pages);
        int pg[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) pg[x] = __shfl_sync(0xffffffffu, page, x);
        const int rw = __shfl_sync(0xffffffffu, row, 0);
        XATTN_DCHECK(page >= 0 && page <= a.num_pages && row >= 0 && row + box_rows <= a.page_size && boxes <= 4, a.status);
        auto load_sub = [&](uint32_t dst, uint32_t full, int col) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (x < boxes) tma_load_4d(dst + x * box_bytes, &mc, full, col, x == 0 ? rw : 0, pg[x], 0);
        };
#pragma unroll 1
        for (int j = 0; j < blocks; ++j, ++Rj) {
          const int s = Rj % kPairs;
          if (!lat_wait(c_empty(s), ((Rj / kPairs) & 1) ^ 1, ctl)) { ok = false; break; }
          if (boxes == 1) {                                     // both sub-tiles in one box
            mbar_expect_tx_elect(c_full(s), L::kPair);
            tma_load_4d_elect(sC + s * L::kPair, &mpair, c_full(s), 0, rw, 2 * j, pg[0]);
          } else if (elect_one()) {
            mbar_expect_tx(c_full(s), L::kPair);
            load_sub(sC + s * L::kPair, c_full(s), 128 * j);
            load_sub(sC + s * L::kPair + L::kSub, c_full(s), 128 * j + 64);
          }
          __syncwarp();
          issued_c = Rj + 1;
        }
        if (!ok) break;
        const int s = R % kRopes;
        if (!lat_wait(r_empty(s), ((R / kRopes) & 1) ^ 1, ctl)) { ok = false; break; }
        if (elect_one()) {
          held_boxes[s] = held;                                  // read by the softmax warps before the slot's next use
          mbar_expect_tx(r_full(s), L::kSub);
          load_sub(sR + s * L::kSub, r_full(s), a.dc);
        }
        __syncwarp();
        issued_r = R + 1;
      }
    }
    __syncwarp();
    // Every copy in flight has landed before the CTA can exit.
    for (int r = max(pieces - kQBufs, 0); r < pieces; ++r) mbar_drain(q_full(r % kQBufs), (r / kQBufs) & 1, ctl);
    for (int r = max(issued_c - kPairs, 0); r < issued_c; ++r) mbar_drain(c_full(r % kPairs), (r / kPairs) & 1, ctl);
    for (int r = max(issued_r - kRopes, 0); r < issued_r; ++r) mbar_drain(r_full(r % kRopes), (r / kRopes) & 1, ctl);
  } else if (warp == 1) {
    // ---------------- issuer of S^T = C Q^T ----------------
    constexpr uint32_t idesc_s = idesc_bf16_f32(64, N, false, false);
    const uint64_t dQ0 = smem_desc(sQ, 16, 1024, kSwizzle128);
    const uint64_t dC = smem_desc(sC, 16, 1024, kSwizzle128), dR = smem_desc(sR, 16, 1024, kSwizzle128);
    const int rope_steps = a.dr / 16;
    int R = 0, Rj = 0, piece = 0;
    bool ok = true;
    while (ok && lat_piece(walk, a)) {
      const int qb = piece % kQBufs;
      if (!lat_wait(q_full(qb), (piece / kQBufs) & 1, ctl)) break;
      const uint64_t dQ = dQ0 + qb * 9 * (L::kQSub >> 4);
#pragma unroll 1
      for (int e = walk.e0; e < walk.e1; ++e) {
        if (!lat_wait(s_free(R & 1), ((R >> 1) & 1) ^ 1, ctl)) { ok = false; break; }
        const uint32_t d = tS + (R & 1) * N;
#pragma unroll 1
        for (int j = 0; j < blocks; ++j, ++Rj) {
          const int s = Rj % kPairs;
          if (!lat_wait(c_full(s), (Rj / kPairs) & 1, ctl)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss_elect(d, dC + s * (L::kPair >> 4) + (kk / 4) * (L::kSub >> 4) + (kk % 4) * 2,
                         dQ + (2 * j + kk / 4) * (L::kQSub >> 4) + (kk % 4) * 2, idesc_s, (j > 0 || kk > 0) ? 1u : 0u);
        }
        const int s = R % kRopes;
        if (!ok || !lat_wait(r_full(s), (R / kRopes) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        for (int kk = 0; kk < rope_steps; ++kk)
          mma_ss_elect(d, dR + s * (L::kSub >> 4) + kk * 2, dQ + 2 * blocks * (L::kQSub >> 4) + kk * 2, idesc_s, 1u);
        mma_commit_elect(s_full(R & 1));
        if (e + 1 == walk.e1) mma_commit_elect(q_empty(qb));
        ++R;
      }
      ++piece;
    }
    __syncwarp();
    if (R > 0) mbar_drain(s_full((R - 1) & 1), ((R - 1) >> 1) & 1, ctl);   // the products are done before TMEM goes
  } else if (warp == 10) {
    // ---------------- issuer of O^T += C^T P^T ----------------
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, N, true, true);
    const uint64_t dCt = smem_desc(sC, L::kSub, 1024, kSwizzle128);      // MN-major: 64 columns a sub-tile
    const uint64_t dP = smem_desc(sP, 16, 8 * L::kPRow, L::kSwizzleP);   // MN-major
    int R = 0, Rj = 0;
    bool ok = true;
    while (ok && lat_piece(walk, a)) {
#pragma unroll 1
      for (int e = walk.e0; e < walk.e1; ++e, ++R) {
        if (!lat_wait(p_full, R & 1, ctl)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < blocks; ++j, ++Rj) {
          const int s = Rj % kPairs;
#pragma unroll
          for (int kk = 0; kk < kTilePos / 16; ++kk)
            mma_ss_elect(tO + j * N, dCt + s * (L::kPair >> 4) + kk * 128, dP + kk * L::kPRow, idesc_o,
                         (e > walk.e0 || kk > 0) ? 1u : 0u);
          mma_commit_elect(c_empty(s));
        }
        mma_commit_elect(o_done);
      }
    }
    __syncwarp();
    if (R > 0) mbar_drain(o_done, (R - 1) & 1, ctl);
  } else {
    // ---------------- softmax: thread = two positions, a quarter of its warp's columns ----------------
    constexpr int C = N / 2, K = C / 8;
    const int quarter = warp & 3, half = (warp - 2) >> 2, tid = static_cast<int>(threadIdx.x) - 64;
    const int pos = quarter * 16 + (lane >> 2);                    // and pos + 8 (M = 64: a quarter's first 16 lanes)
    const int col = half * C + 2 * (lane & 3);                     // and + 1, + 8, + 9, ..
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int box_rows = min(a.page_size, kTilePos);
    const unsigned all_boxes = (1u << (kTilePos / box_rows)) - 1u;
    const int rows_all = a.n * a.nh, row0 = rt * N, rows = min(rows_all - row0, N);
    // Where this lane's row of the P matrices goes: rows pos, chunks of 8 columns, swizzled.
    auto p_chunk = [&](int k) -> uint32_t {
      const int at = quarter * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), chunk = half * K + k;
      const int sw = N == 64 ? (chunk ^ (at & 7)) : (N == 32 ? (chunk ^ ((at >> 1) & 3)) : (chunk ^ ((at >> 2) & 1)));
      return sP + at * L::kPRow + (sw << 4);
    };
    int R = 0, meets = 0;
    bool ok = true;
    auto meet_all = [&]() -> bool {
      lat_arrive(meet, lane);
      return lat_wait(meet, meets++ & 1, ctl);
    };
    // (One group has no plan and no records: its one run cuts no sequence.)
    if (warp == 2 && lane == 0 && rt == 0 && groups > 1) a.plan[group] = make_int2(0, 0);
    while (ok && lat_piece(walk, a)) {
      const int e0 = walk.e0, e1 = walk.e1, b = walk.b, ctx = walk.ctx, end = ctx + a.n;
      const bool whole = groups == 1 || (e0 == 0 && e1 == walk.count);
      // A run that ends inside the sequence it started last says so to the combine.
      if (warp == 2 && lane == 0 && rt == 0 && !whole && e0 == 0)
        a.plan[group] = make_int2(b, runs.of(walk.first + walk.count - 1) + 1);
      float l[2 * K];
#pragma unroll
      for (int k = 0; k < 2 * K; ++k) l[k] = 0.f;
#pragma unroll 1
      for (int e = e0; e < e1; ++e, ++R) {
        const bool first = e == e0;
        if (!lat_wait(s_full(R & 1), (R >> 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        const unsigned held = held_boxes[R % kRopes];
        float x[4 * K];
        uint32_t *xr = reinterpret_cast<uint32_t *>(x);
        tmem_ld_16x256b<K>(tS + (R & 1) * N + half * C + lane_off, xr);
        tmem_wait_ld();
        reg_fence<4 * K>(xr);
        tc_fence_before();
        lat_arrive(s_free(R & 1), lane);
#pragma unroll
        for (int k = 0; k < 2 * K; ++k) fmul2(x[2 * k], x[2 * k + 1], x[2 * k], x[2 * k + 1], a.scale_log2, a.scale_log2);
        if (e * kTilePos + kTilePos > ctx + 1 || held != all_boxes) {
          // Positions that some row does not see: new ones, those behind the last, missing pages.
          const int p = e * kTilePos + pos;
          const bool there0 = (held >> (pos / box_rows)) & 1u, there1 = (held >> ((pos + 8) / box_rows)) & 1u;
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int last = min(ctx + (row0 + col + 8 * k + h) / a.nh, end - 1);
              if (!there0 || p > last) x[4 * k + h] = -INFINITY;
              if (!there1 || p + 8 > last) x[4 * k + 2 + h] = -INFINITY;
            }
          // Rows behind the last position may hold anything and are zeroed before P meets them (0 x NaN would not
          // be 0).
          const int r = tid >> 2;
          if (e * kTilePos + r >= end) {
            for (int j = tid & 3; j < 2 * blocks; j += 4) {
              uint8_t *row = smem + L::kC + ((R * blocks + j / 2) % kPairs) * L::kPair + (j & 1) * L::kSub + r * 128;
#pragma unroll
              for (int v = 0; v < 8; ++v) reinterpret_cast<uint4 *>(row)[(v + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);   // (banks)
            }
          }
        }
        // Does some score pass its column's base by more than 2^8? A piece's first tile always asks.
        bool grow = first;
        if (!first) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            const float2 m = *reinterpret_cast<const float2 *>(base + col + 8 * k);
            float d0, d1, d2, d3;
            fadd2(d0, d1, x[4 * k], x[4 * k + 1], m.x, m.y);
            fadd2(d2, d3, x[4 * k + 2], x[4 * k + 3], m.x, m.y);
            top = fmax3(fmax3(top, d0, d1), d2, d3);
          }
          grow = top > 8.f;
        }
        const bool warp_grows = __any_sync(0xffffffffu, grow);
        if (lane == 0) flags[(R & 1) * kSoftWarps + warp - 2] = warp_grows;
        if (!meet_all()) { ok = false; break; }
        int any = 0;
#pragma unroll
        for (int w = 0; w < kSoftWarps; ++w) any |= flags[(R & 1) * kSoftWarps + w];
        if (any) {
          // The columns' maxima: over a warp's positions, then over the four quarters.
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float m = fmaxf(x[4 * k + h], x[4 * k + 2 + h]);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
              if (lane < 4) parts[quarter * N + col + 8 * k + h] = m;
            }
          if (!meet_all()) { ok = false; break; }
          if (tid < N) {
            // (-FLT_MAX stands for nothing seen: any score is far above it, and differences stay numbers.)
            const float old = first ? -FLT_MAX : -base[tid];
            const float m = fmaxf(fmax3(old, parts[tid], parts[N + tid]), fmaxf(parts[2 * N + tid], parts[3 * N + tid]));
            factor[tid] = ex2_approx(old - m);
            base[tid] = -m;
          }
          if (!meet_all()) { ok = false; break; }
        }
        uint32_t pk[2 * K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float2 m = *reinterpret_cast<const float2 *>(base + col + 8 * k);
          if (any) {
            const float2 f = *reinterpret_cast<const float2 *>(factor + col + 8 * k);
            if (!first) l[2 * k] *= f.x, l[2 * k + 1] *= f.y;
          }
          float d0, d1, d2, d3;
          fadd2(d0, d1, x[4 * k], x[4 * k + 1], m.x, m.y);
          fadd2(d2, d3, x[4 * k + 2], x[4 * k + 3], m.x, m.y);
          d0 = ex2_approx(d0), d1 = ex2_approx(d1), d2 = ex2_approx(d2), d3 = ex2_approx(d3);
          fadd2(l[2 * k], l[2 * k + 1], l[2 * k], l[2 * k + 1], d0, d1);
          fadd2(l[2 * k], l[2 * k + 1], l[2 * k], l[2 * k + 1], d2, d3);
          pk[2 * k] = pack_bf16x2(d0, d1);
          pk[2 * k + 1] = pack_bf16x2(d2, d3);
        }
        // P over the last tile's, which its product has read then; O^T is at rest too.
        if (!lat_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        if (any && !first) {
          const float *f = factor + half * C;
#pragma unroll 1
          for (int j = 0; j < blocks; ++j) {
            uint32_t ov[C];
            const uint32_t at = tO + j * N + half * C + lane_off;
            tmem_ld_cols<C>(at, ov);
            tmem_wait_ld();
            reg_fence<C>(ov);
#pragma unroll
            for (int c = 0; c < C; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * f[c]);
            tmem_st_cols<C>(at, ov);
          }
          tmem_wait_st();
        }
        if constexpr (K == 1) {
          stmatrix_x2(p_chunk(0), pk[0], pk[1]);
        } else {
#pragma unroll
          for (int k = 0; k < K; k += 2) stmatrix_x4(p_chunk(k + (lane >> 4)), pk[2 * k], pk[2 * k + 1], pk[2 * k + 2], pk[2 * k + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        if (warp == 2 && lane == 0) mbar_arrive(r_empty(R % kRopes));
        lat_arrive(p_full, lane);
      }
      if (!ok) break;
      // The piece's sums meet in `parts`; its O^T and LSE, or its record (O not divided by the sum).
#pragma unroll
      for (int k = 0; k < 2 * K; ++k) {
        float s = l[k];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (lane < 4) parts[quarter * N + col + 8 * (k / 2) + (k & 1)] = s;
      }
      if (!meet_all()) { ok = false; break; }
      const size_t rec = (2 * static_cast<size_t>(blockIdx.x) + (e0 == 0 ? 1 : 0)) * N;
      const size_t out = static_cast<size_t>(b) * rows_all + row0;
      if (tid < N) {
        const float sum = (parts[tid] + parts[N + tid]) + (parts[2 * N + tid] + parts[3 * N + tid]), m = -base[tid];
        factor[tid] = !whole ? 1.f : (sum != 0.f ? 1.f / sum : 0.f);
        if (tid < rows) {
          if (whole)
            a.lse[out + tid] = sum != 0.f ? (m + __log2f(sum)) * kLn2 : -INFINITY;
          else
            a.ws_ml[rec + tid] = make_float2(m, sum);
        }
      }
      if (!meet_all() || !lat_wait(o_done, (R - 1) & 1, ctl)) { ok = false; break; }
      tc_fence_after();
      // Eight rows of a block a load, a lane a number of the latent; with few rows four loads together.
      constexpr int kOnce = N == 64 ? 1 : 4;
      const int d = quarter * 32 + lane;
#pragma unroll 1
      for (int x0 = 0; x0 < blocks * K; x0 += kOnce) {
        uint32_t ov[kOnce][8];
        auto row_of = [&](int x) { return half * C + (x - x / K * K) * 8; };
#pragma unroll
        for (int y = 0; y < kOnce; ++y)
          if (x0 + y < blocks * K) tmem_ld_x8(tO + (x0 + y) / K * N + row_of(x0 + y) + lane_off, ov[y]);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < kOnce; ++y) {
          reg_fence<8>(ov[y]);
          const int x = x0 + y, j = x / K, r0 = row_of(x);
          if (x >= blocks * K || r0 >= rows) continue;
          if (whole) {
            __nv_bfloat16 *to = a.o + (out + r0) * a.dc + j * 128 + d;
#pragma unroll
            for (int c = 0; c < 8; ++c, to += a.dc) {
              const float f = factor[r0 + c];
              if (r0 + c < rows) *to = __float2bfloat16_rn(f != 0.f ? __uint_as_float(ov[y][c]) * f : 0.f);
            }
          } else {
            float *to = a.ws_o + (rec + r0) * a.dc + j * 128 + d;
#pragma unroll
            for (int c = 0; c < 8; ++c, to += a.dc)
              if (r0 + c < rows) *to = __uint_as_float(ov[y][c]);
          }
        }
        __syncwarp();                                            // (the reads of TMEM are the warp's)
      }
      tc_fence_before();
      if (!meet_all()) { ok = false; break; }                    // factor and parts are read
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merges the records of the cut sequences: block (c, y) takes rows of the sequence that run c starts and does not finish, if
// there is one (plan[c]: sequence, past the last run). dc / 4 threads hold a row, four columns each, and add the records in
// order, the next one's numbers on their way while one is added; `passes` rows a thread. kWide, for calls whose sequences spread
// over many runs: with more than kFewRecords records the block's warps take every eighth each, and add up in the order of the
// warps. (The other form has no shared memory, so that its blocks are there before the decode kernel's leave the SM.)
constexpr int kCombineThreads = 256, kFewRecords = 8;
__device__ __forceinline__ void merge_record(float &M, float &sum, float4 &acc, float2 ml, float4 x) {
  if (ml.y == 0.f) return;                                      // a record that saw nothing holds anything but this
  const float m = fmaxf(M, ml.x), f0 = ex2_approx(M - m), f1 = ex2_approx(ml.x - m);
  M = m;
  sum = sum * f0 + ml.y * f1;
  acc.x = acc.x * f0 + x.x * f1, acc.y = acc.y * f0 + x.y * f1, acc.z = acc.z * f0 + x.z * f1, acc.w = acc.w * f0 + x.w * f1;
}
template <bool kWide>
__global__ void __launch_bounds__(kCombineThreads) latent_combine_kernel(const LatentDecodeArgs a, int tile_rows, int passes) {
  grid_dep_launch();
  grid_dep_wait();
  const int c0 = blockIdx.x;
  const int2 plan = a.plan[c0];
  if (plan.y == 0) return;
  const int records = plan.y - c0, quads = a.dc / 4, rows = a.n * a.nh;
  auto rec_of = [&](int k, int row) {
    const int rt = row / tile_rows;
    return (2 * (static_cast<size_t>(c0 + k) * a.row_tiles + rt) + (k == 0 ? 1 : 0)) * tile_rows + (row - rt * tile_rows);
  };
  auto put = [&](int row, int i, float M, float sum, float4 acc) {
    const size_t out = static_cast<size_t>(plan.x) * rows + row;
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<uint2 *>(a.o + out * a.dc + 4 * i) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (i == 0) a.lse[out] = sum != 0.f ? (M + __log2f(sum)) * kLn2 : -INFINITY;
  };
  const int each = kCombineThreads / quads, row0 = static_cast<int>(blockIdx.y) * each * passes;
  if (!kWide || records <= kFewRecords) {
    const int sub = threadIdx.x / quads, i = threadIdx.x - sub * quads;
    if (sub >= each) return;                                    // (dc = 384: some threads are over)
#pragma unroll 2
    for (int p = 0; p < passes; ++p) {
      const int row = row0 + p * each + sub;
      if (row >= rows) break;
      float M = -FLT_MAX, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      size_t rec = rec_of(0, row);
      float2 ml = a.ws_ml[rec];
      float4 x = *reinterpret_cast<const float4 *>(a.ws_o + rec * a.dc + 4 * i);
#pragma unroll 1
      for (int k = 0; k < records; ++k) {
        const float2 ml_here = ml;
        const float4 x_here = x;
        if (k + 1 < records) {
          rec = rec_of(k + 1, row);
          ml = a.ws_ml[rec];
          x = *reinterpret_cast<const float4 *>(a.ws_o + rec * a.dc + 4 * i);
        }
        merge_record(M, sum, acc, ml_here, x_here);
      }
      put(row, i, M, sum, acc);
    }
    return;
  }
  if constexpr (kWide) {
    __shared__ float4 part[8][128];
    __shared__ float2 part_ml[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int row = row0; row < min(row0 + each * passes, rows); ++row) {
      float M = -FLT_MAX, sum = 0.f;
      float4 acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int k = warp; k < records; k += 8) {
        const size_t rec = rec_of(k, row);
        const float2 ml = a.ws_ml[rec];
        float4 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          x[q] = lane + 32 * q < quads ? *reinterpret_cast<const float4 *>(a.ws_o + rec * a.dc + 4 * (lane + 32 * q))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
        float m1 = M, s1 = sum;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          m1 = M, s1 = sum;
          merge_record(m1, s1, acc[q], ml, x[q]);
        }
        M = m1, sum = s1;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) part[warp][lane + 32 * q] = acc[q];
      if (lane == 0) part_ml[warp] = make_float2(M, sum);
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < quads) {
        M = -FLT_MAX, sum = 0.f;
        float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 8; ++w) merge_record(M, sum, all, part_ml[w], part[w][threadIdx.x]);
        put(row, threadIdx.x, M, sum, all);
      }
      __syncthreads();                                            // before the next row's parts
    }
  }
}

template <int N>
cudaError_t launch_latent_n(const LatentDecodeMaps &maps, const LatentDecodeArgs &a, int groups, int sms, cudaStream_t stream) {
  using L = LatLayout<N>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t err = allow_smem(latent_decode_kernel<N>, L::kDynBytes, allowed);
  if (err != cudaSuccess) return err;
  err = launch_pdl(latent_decode_kernel<N>, static_cast<unsigned>(groups) * a.row_tiles, kLatThreads, L::kDynBytes, stream,
                   maps.q, maps.pages, maps.q_latents, maps.latents, a);
  if (err != cudaSuccess || groups == 1) return err;
  // Rows a thread: as many as make one wave of blocks; one where sequences spread over many runs.
  const int rows = a.n * a.nh, each = kCombineThreads / (a.dc / 4);
  const long long blocks = static_cast<long long>(groups - 1) * ((rows + each - 1) / each);
  const bool wide = groups >= 4 * a.B;
  const int passes = wide ? 1 : static_cast<int>(min(max(blocks / (sms * 8), 1ll), 8ll));
  return launch_pdl(wide ? latent_combine_kernel<true> : latent_combine_kernel<false>,
                    dim3(static_cast<unsigned>(groups - 1), static_cast<unsigned>((rows + each * passes - 1) / (each * passes))),
                    kCombineThreads, 0, stream, a, N, passes);
}

}  // namespace

// The fewest columns that hold the rows: 64 sequences of 4096, 16 rows 62 us (by 32 columns 63, by 64 66 to 68), 32 rows 66 (by 64
// 70).
int latent_tile_rows(int n, int nh) {
  const long long rows = static_cast<long long>(n) * nh;
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
}

// Groups of CTAs (runs of the line), a CTA of each per row tile: as many as the GPU holds at once, and no more than
// the tables allow tiles. With more row tiles than SMs one group, whose CTAs come in waves.
int latent_groups(const LatentDecodeArgs &a, int sms) {
  const long long most = static_cast<long long>(a.B) * ((static_cast<long long>(a.max_pages) * a.page_size + kTilePos - 1) / kTilePos);
  long long groups = sms / a.row_tiles;
  if (groups > kMaxLatentRuns) groups = kMaxLatentRuns;
  if (groups > most) groups = most;
  return groups < 1 ? 1 : static_cast<int>(groups);
}

size_t latent_decode_workspace_bytes(const LatentDecodeArgs &a, int groups, int tile_rows) {
  if (groups == 1) return 0;
  return static_cast<size_t>(groups) * a.row_tiles * 2 * tile_rows * (a.dc * sizeof(float) + sizeof(float2)) +
         static_cast<size_t>(groups) * sizeof(int2);
}

cudaError_t launch_latent_decode(const LatentDecodeMaps &maps, const LatentDecodeArgs &a, int groups, int tile_rows, int sms,
                                 cudaStream_t stream) {
  if (tile_rows == 16) return launch_latent_n<16>(maps, a, groups, sms, stream);
  if (tile_rows == 32) return launch_latent_n<32>(maps, a, groups, sms, stream);
  return launch_latent_n<64>(maps, a, groups, sms, stream);
}

}  // namespace xattn
