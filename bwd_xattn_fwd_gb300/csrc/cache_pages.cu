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
  if (p < 0 || p >= static_cast<long long>(a.max_pages) * a.page_size) return -1;
  const int id = a.page_table[static_cast<size_t>(b) * a.max_pages + p / a.page_size];
  if (id < 0 || id >= a.num_pages) return -1;
  return static_cast<long long>(id) * a.page_size + p % a.page_size;
}

// One thread per (sequence, new row, 16-byte vector of the row): its K and its V.
__global__ void __launch_bounds__(kPageThreads) cache_append_kernel(const PageArgs a, const uint4 *__restrict__ k_new,
                                                                   const uint4 *__restrict__ v_new) {
  grid_dep_launch();
  grid_dep_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kPageThreads + threadIdx.x;
  if (t >= static_cast<long long>(a.B) * a.n * a.row_vecs) return;
  const long long row = t / a.row_vecs;
  const int vec = static_cast<int>(t % a.row_vecs), b = static_cast<int>(row / a.n), i = static_cast<int>(row % a.n);
  const uint4 k = k_new[t], v = v_new[t];
  const long long dst = pool_row(a, b, static_cast<long long>(a.ctx_lens[b]) + i);
  if (dst < 0) return;
  a.k_pages[dst * a.row_vecs + vec] = k;
  a.v_pages[dst * a.row_vecs + vec] = v;
}

// One thread per (sequence, K or V, 16-byte vector): moves the accepted rows down in order.
// Ascending paths have path[i] >= i, so a row is read before the row that lands on it is
// written, also with kRun loads ahead of their stores.
__global__ void __launch_bounds__(kPageThreads) cache_compact_kernel(const PageArgs a, const int *__restrict__ path,
                                                                    const int *__restrict__ accepted) {
  grid_dep_launch();
  grid_dep_wait();
  constexpr int kRun = 8;
  const long long t = static_cast<long long>(blockIdx.x) * kPageThreads + threadIdx.x;
  if (t >= 2ll * a.B * a.row_vecs) return;
  const int vec = static_cast<int>(t % a.row_vecs), which = static_cast<int>(t / a.row_vecs % 2);
  const int b = static_cast<int>(t / a.row_vecs / 2);
  uint4 *pool = which ? a.v_pages : a.k_pages;
  const int count = min(accepted[b], a.n);
  const long long ctx = a.ctx_lens[b];
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += kRun) {
    uint4 x[kRun];
    long long dst[kRun];
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      dst[e] = -1;
      if (i0 + e >= count) continue;
      const int from = path[static_cast<size_t>(b) * a.n + i0 + e];
      if (from <= i0 + e || from >= a.n) continue;             // already in place, or no drafted row
      const long long src = pool_row(a, b, ctx + from);
      dst[e] = src < 0 ? -1 : pool_row(a, b, ctx + i0 + e);
      if (dst[e] >= 0) x[e] = pool[src * a.row_vecs + vec];
    }
#pragma unroll
    for (int e = 0; e < kRun; ++e)
      if (dst[e] >= 0) pool[dst[e] * a.row_vecs + vec] = x[e];
  }
}

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + kPageThreads - 1) / kPageThreads); }

}  // namespace

cudaError_t launch_cache_append(const PageArgs &a, const void *k_new, const void *v_new, cudaStream_t stream) {
  return launch_pdl(cache_append_kernel, blocks_for(static_cast<long long>(a.B) * a.n * a.row_vecs), kPageThreads, 0,
                    stream, a, static_cast<const uint4 *>(k_new), static_cast<const uint4 *>(v_new));
}

cudaError_t launch_cache_compact(const PageArgs &a, const int *path, const int *accepted, cudaStream_t stream) {
  return launch_pdl(cache_compact_kernel, blocks_for(2ll * a.B * a.row_vecs), kPageThreads, 0, stream, a, path,
                    accepted);
}

}  // namespace xattn
