// Rows of a paged K/V cache: appending new tokens' rows, and compacting drafted rows to the
// accepted path. Position p of sequence b is row p % page_size of page
// page_table[b][p / page_size]; a position past the table, or whose entry is no page of the
// pool, has no row: nothing is read or written for it.
//
// Both move 16-byte vectors, K and V in one launch, and are bound by HBM (large appends) or
// by the launch itself (a decode step's rows).
#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kPageThreads = 256;

// Row of the pool (all pages' rows in order) that holds position p of sequence b, or -1.
__device__ __forceinline__ long long pool_row(const PageArgs &a, int b, long long p) {
  if (p < 0 || p >= a.max_pages * a.page_size) return -1;   // (at most 2^30)
  const unsigned at = static_cast<unsigned>(p) / a.page_size, row = static_cast<unsigned>(p) - at * a.page_size;
  const int id = a.page_table[static_cast<size_t>(b) * a.max_pages + at];
  return id >= 0 && id < a.num_pages ? static_cast<long long>(id) * a.page_size + row : -1;
}

// One thread per (sequence, new row, 16-byte vector of the row): its K and its V. 16 sequences of
// 4096 rows, 4 heads of 128: 41.1 us, 6.5 TB/s (96 % of the measured copy).
__global__ void __launch_bounds__(kPageThreads) cache_append_kernel(const PageArgs a, const uint4 *__restrict__ k_new,
                                                                   const uint4 *__restrict__ v_new) {
  grid_dep_launch();
  grid_dep_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kPageThreads + threadIdx.x;
  if (t >= static_cast<long long>(a.B) * a.n * a.row_vecs) return;
  int vec, b, i;
  if (t >> 32) {
    const long long row = t / a.row_vecs;
    vec = static_cast<int>(t - row * a.row_vecs);
    b = static_cast<int>(row / a.n);
    i = static_cast<int>(row - static_cast<long long>(b) * a.n);
  } else {                                                   // divisions in 32 bits
    const unsigned row = static_cast<unsigned>(t) / a.row_vecs;
    vec = static_cast<int>(static_cast<unsigned>(t) - row * a.row_vecs);
    b = static_cast<int>(row / a.n);
    i = static_cast<int>(row - static_cast<unsigned>(b) * a.n);
  }
  const uint4 k = k_new[t], v = v_new[t];
  const long long dst = pool_row(a, b, static_cast<long long>(a.ctx_lens[b]) + i);
  if (dst < 0) return;
  a.k_pages[dst * a.row_vecs + vec] = k;
  a.v_pages[dst * a.row_vecs + vec] = v;
}

// One block per (`lanes` vectors of a row, sequence, K or V): it holds every accepted row's share
// of them, a group of 256 / lanes x kRowsEach rows at a time. A group's rows are all read before
// any is written (the barrier), and a later group reads none that an earlier one wrote: a path
// that ascends has path[i] >= i. lanes is 32, 64 or 128, as many as a row has vectors for: few
// rows are accepted, and blocks are what the launch costs. One thread a vector that moved its
// rows in order, a chain of reads, took 6.8 us for 64 sequences with trees of 16 (32 vectors);
// this way 2.7. With always 32 lanes and 8 rows a thread, 256 sequences of 128 vectors took 8.0
// us; this way 4.7.
constexpr int kRowsEach = 4;
__global__ void __launch_bounds__(kPageThreads) cache_compact_kernel(const PageArgs a, const int *__restrict__ path,
                                                                    const int *__restrict__ accepted, int lanes,
                                                                    int vec_blocks) {
  grid_dep_launch();
  grid_dep_wait();
  const unsigned chunk = blockIdx.x % vec_blocks, rest = blockIdx.x / vec_blocks;
  const int b = static_cast<int>(rest >> 1), row = threadIdx.x / lanes, row_lanes = kPageThreads / lanes;
  const int vec = static_cast<int>(chunk) * lanes + threadIdx.x - row * lanes;
  uint4 *pool = (rest & 1) ? a.v_pages : a.k_pages;
  const long long ctx = a.ctx_lens[b];
  const int count = min(accepted[b], a.n);
  for (int i0 = 0; i0 < count; i0 += row_lanes * kRowsEach) {
    uint4 x[kRowsEach];
    long long dst[kRowsEach];
#pragma unroll
    for (int e = 0; e < kRowsEach; ++e) {
      const int i = i0 + row + e * row_lanes;
      dst[e] = -1;
      if (i >= count || vec >= a.row_vecs) continue;
      const int from = path[static_cast<size_t>(b) * a.n + i];
      if (from <= i || from >= a.n) continue;                // already in place, or no drafted row
      const long long src = pool_row(a, b, ctx + from);
      dst[e] = src < 0 ? -1 : pool_row(a, b, ctx + i);
      if (dst[e] >= 0) x[e] = pool[src * a.row_vecs + vec];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kRowsEach; ++e)
      if (dst[e] >= 0) pool[dst[e] * a.row_vecs + vec] = x[e];
    __syncthreads();
  }
}

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + kPageThreads - 1) / kPageThreads); }

}  // namespace

cudaError_t launch_cache_append(const PageArgs &a, const void *k_new, const void *v_new, cudaStream_t stream) {
  return launch_pdl(cache_append_kernel, blocks_for(static_cast<long long>(a.B) * a.n * a.row_vecs), kPageThreads, 0,
                    stream, a, static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new));
}

cudaError_t launch_cache_compact(const PageArgs &a, const int *path, const int *accepted, cudaStream_t stream) {
  const int lanes = a.row_vecs <= 32 ? 32 : (a.row_vecs <= 64 ? 64 : 128);
  const int vec_blocks = (a.row_vecs + lanes - 1) / lanes;
  return launch_pdl(cache_compact_kernel, dim3(static_cast<unsigned>(2ll * a.B * vec_blocks)), kPageThreads, 0, stream,
                    a, path, accepted, lanes, vec_blocks);
}

}  // namespace xattn
