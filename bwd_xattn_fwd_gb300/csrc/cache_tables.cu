// The paged cache's bookkeeping on the GPU: pages taken from a stack of free ones for the new
// positions of a batch, with the slot map of its tokens (reserve); pages given back (release); and rows
// written to the places that a slot map names (write).
//
// A slot is a row of the pool: page * page_size + row in the page. With held_b = ceil(ctx_b / page_size)
// pages in the table already, sequence b needs ceil((ctx_b + new_b) / page_size) - held_b more; prefix
// sums of these and of new_b give each sequence its stretch of the stack and of the slot map.
#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kPlanThreads = 1024, kFillThreads = 256;

struct Pair {
  long long x, y;
};

// Inclusive sums of a pair over the block's threads; part: one pair a warp, shared. total: the block's.
template <int kThreads>
__device__ __forceinline__ Pair block_scan(Pair v, Pair *part, Pair *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, off), y = __shfl_up_sync(0xffffffffu, v.y, off);
    if (lane >= off) v.x += x, v.y += y;
  }
  __syncthreads();                                           // part is read from the last time
  if (lane == 31) part[warp] = v;
  __syncthreads();
  Pair before{0, 0}, all{0, 0};
#pragma unroll 8
  for (int w = 0; w < kThreads / 32; ++w) {
    const Pair p = part[w];
    if (w == warp) before = all;
    all.x += p.x, all.y += p.y;
  }
  *total = all;
  return {v.x + before.x, v.y + before.y};
}

__device__ __forceinline__ int pages_of(int positions, int page_size) { return (positions + page_size - 1) / page_size; }

__device__ __forceinline__ int clamp_len(int len, int most) { return min(max(len, 0), most); }

// Sequences in order, 1024 at a time: what each needs, whether it gets it, and where its tokens start.
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const ReserveArgs a) {
  __shared__ Pair part[kPlanThreads / 32];
  __shared__ long long taken_part[kPlanThreads / 32];
  grid_dep_launch();
  grid_dep_wait();
  const int most = a.max_pages * a.page_size;                // (at most 2^30)
  const int count = clamp_len(a.free_count[0], a.num_pages);
  Pair base{0, 0};
  long long taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int need = 0, room = 0, fresh = 0;
    if (b < a.B) {
      const int ctx = clamp_len(a.ctx_lens[b], most);
      fresh = max(a.new_lens[b], 0);
      room = min(fresh, most - ctx);
      need = pages_of(ctx + room, a.page_size) - pages_of(ctx, a.page_size);
    }
    Pair total;
    Pair upto = block_scan<kPlanThreads>({need, fresh}, part, &total);
    upto.x += base.x, upto.y += base.y;
    base.x += total.x, base.y += total.y;
    if (b < a.B) {
      const bool ok = (need == 0 || upto.x <= count) && upto.y <= a.tokens;
      if (ok && need > 0) taken = upto.x;
      a.first[b] = ok ? static_cast<int>(min(upto.x - need, static_cast<long long>(a.num_pages))) : 0;
      a.granted[b] = ok ? room : 0;
      a.offsets[b + 1] = static_cast<int>(min(upto.y, 0x7fffffffll));
    }
  }
  // The pages taken: the largest running need that was met (each thread's last is its largest).
#pragma unroll
  for (int off = 16; off; off >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, off));
  if ((threadIdx.x & 31) == 0) taken_part[threadIdx.x >> 5] = taken;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kPlanThreads / 32; ++w) taken = max(taken, taken_part[w]);
    a.offsets[0] = 0;
    a.first[a.B] = count;
    a.free_count[0] = count - static_cast<int>(taken);
  }
}

// One thread a token: its slot, and the table entry of a page that begins with it.
__global__ void __launch_bounds__(kFillThreads) reserve_fill_kernel(const ReserveArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kFillThreads + threadIdx.x;
  if (t >= a.tokens) return;
  long long slot = -1;
  if (t < a.offsets[a.B]) {
    int lo = 0, hi = a.B;                                    // offsets[lo] <= t < offsets[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.offsets[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int at = static_cast<int>(t - a.offsets[lo]);
    if (at < a.granted[lo]) {
      const int ctx = clamp_len(a.ctx_lens[lo], a.max_pages * a.page_size), pos = ctx + at, page = pos / a.page_size;
      const int row = pos - page * a.page_size, held = pages_of(ctx, a.page_size);
      int *entry = a.page_table + static_cast<size_t>(lo) * a.max_pages + page;
      int id;
      if (page >= held) {
        const int place = a.first[a.B] - 1 - (a.first[lo] + page - held);
        id = place >= 0 && place < a.num_pages ? a.free_pages[place] : -1;   // (outside only if the lengths change)
        if (row == 0) *entry = id;
      } else {
        id = *entry;
      }
      if (id >= 0 && id < a.num_pages) slot = static_cast<long long>(id) * a.page_size + row;
    }
  }
  a.slots[t] = slot;
}

// One warp a sequence: how many pages it gives back.
__global__ void __launch_bounds__(kFillThreads) release_count_kernel(const ReleaseArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, b = static_cast<int>(blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.counts[a.B] = clamp_len(a.free_count[0], a.num_pages);
  if (b >= a.B) return;
  const int most = a.max_pages * a.page_size;
  const int from = pages_of(clamp_len(a.keep_lens[b], most), a.page_size), to = pages_of(clamp_len(a.held_lens[b], most), a.page_size);
  const int *row = a.page_table + static_cast<size_t>(b) * a.max_pages;
  int n = 0;
  for (int j = from + lane; j < to; j += 32) n += row[j] >= 0 && row[j] < a.num_pages;
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) a.counts[b] = n;
}

// One warp a sequence, `each` sequences a block: its pages onto the stack, the first sequence's first page
// topmost, so that a release undoes the reserve before it.
__global__ void __launch_bounds__(kFillThreads) release_push_kernel(const ReleaseArgs a, int each) {
  __shared__ Pair part[kFillThreads / 32];
  __shared__ int before[kFillThreads / 32];
  grid_dep_launch();
  grid_dep_wait();
  constexpr int kWarps = kFillThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = static_cast<int>(blockIdx.x) * each;
  Pair mine{0, 0}, total;
  for (int b = threadIdx.x; b < a.B; b += kFillThreads) {
    const int n = a.counts[b];
    mine.x += n;
    if (b < b0) mine.y += n;
  }
  block_scan<kFillThreads>(mine, part, &total);
  const int count = a.counts[a.B];
  const long long top = count + total.x;                     // one past the stack's new top
  if (blockIdx.x == 0 && threadIdx.x == 0) a.free_count[0] = static_cast<int>(min(top, static_cast<long long>(a.num_pages)));
  const int most = a.max_pages * a.page_size;
  long long rank = total.y;
  for (int g = 0; g < each; g += kWarps) {
    const int b = b0 + g + warp;
    const bool live = g + warp < each && b < a.B;
    __syncthreads();
    if (lane == 0) before[warp] = live ? a.counts[b] : 0;
    __syncthreads();
    long long r = rank;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) r += before[w];
      rank += before[w];
    }
    if (!live) continue;
    const int from = pages_of(clamp_len(a.keep_lens[b], most), a.page_size), to = pages_of(clamp_len(a.held_lens[b], most), a.page_size);
    int *row = a.page_table + static_cast<size_t>(b) * a.max_pages;
    for (int j0 = from; j0 < to; j0 += 32) {
      const int j = j0 + lane, id = j < to ? row[j] : -1;
      const bool real = id >= 0 && id < a.num_pages;
      const unsigned all = __ballot_sync(0xffffffffu, real);
      const long long place = top - 1 - (r + __popc(all & ((1u << lane) - 1u)));
      if (real && place >= 0 && place < a.num_pages) a.free_pages[place] = id;
      if (j < to) row[j] = -1;
      r += __popc(all);
    }
  }
}

// One thread a 16-byte vector of a row of either source.
__global__ void __launch_bounds__(kFillThreads) cache_write_kernel(const WriteArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kFillThreads + threadIdx.x;
  const int each = a.vecs[0] + a.vecs[1];
  long long r;
  int v;
  if (t >> 32) {
    r = t / each;
    v = static_cast<int>(t - r * each);
  } else {                                                   // division in 32 bits
    r = static_cast<unsigned>(t) / static_cast<unsigned>(each);
    v = static_cast<int>(static_cast<unsigned>(t) - static_cast<unsigned>(r) * each);
  }
  if (r >= a.rows) return;
  const long long slot = a.slots[r];
  if (slot < 0 || slot >= a.num_slots) return;
  const int x = v < a.vecs[0] ? 0 : 1;
  if (x) v -= a.vecs[0];
  a.dst[x][slot * a.stride[x] + v] = a.src[x][r * a.vecs[x] + v];
}

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + kFillThreads - 1) / kFillThreads); }

}  // namespace

cudaError_t launch_cache_reserve(const ReserveArgs &a, cudaStream_t stream) {
  const cudaError_t err = launch_pdl(reserve_plan_kernel, 1, kPlanThreads, 0, stream, a);
  if (err != cudaSuccess || a.tokens == 0) return err;
  return launch_pdl(reserve_fill_kernel, blocks_for(a.tokens), kFillThreads, 0, stream, a);
}

cudaError_t launch_cache_release(const ReleaseArgs &a, cudaStream_t stream) {
  constexpr int kWarps = kFillThreads / 32;
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.B) + kWarps - 1) / kWarps);
  const cudaError_t err = launch_pdl(release_count_kernel, blocks, kFillThreads, 0, stream, a);
  if (err != cudaSuccess) return err;
  const int each = (static_cast<int>((blocks + 511) / 512)) * kWarps;
  return launch_pdl(release_push_kernel, static_cast<unsigned>((static_cast<long long>(a.B) + each - 1) / each), kFillThreads, 0, stream, a,
                    each);
}

cudaError_t launch_cache_write(const WriteArgs &a, cudaStream_t stream) {
  return launch_pdl(cache_write_kernel, blocks_for(a.rows * (a.vecs[0] + a.vecs[1])), kFillThreads, 0, stream, a);
}

}  // namespace xattn
