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

constexpr int kPlanThreads = 1024, kFewThreads = 256, kFillThreads = 256;

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

// One thread a sequence: what sequence b needs (y: its tokens), and what it may get at most.
__device__ __forceinline__ Pair reserve_need(const ReserveArgs &a, int b, int *room) {
  *room = 0;
  if (b >= a.B) return {0, 0};
  const int most = a.max_pages * a.page_size;                // (at most 2^30)
  const int ctx = clamp_len(a.ctx_lens[b], most), fresh = max(a.new_lens[b], 0);
  *room = min(fresh, most - ctx);
  return {pages_of(ctx + *room, a.page_size) - pages_of(ctx, a.page_size), fresh};
}

// The slot of token t, the at-th of sequence b, whose new pages begin `first` below the stack's top `count`; the page that
// begins with it goes into the table.
__device__ __forceinline__ long long reserve_slot(const ReserveArgs &a, int b, int at, int first, int count) {
  const int ctx = clamp_len(a.ctx_lens[b], a.max_pages * a.page_size), pos = ctx + at, page = pos / a.page_size;
  const int row = pos - page * a.page_size, held = pages_of(ctx, a.page_size);
  XATTN_DCHECK(b >= 0 && b < a.B && at >= 0 && pos >= ctx && page < a.max_pages && first >= 0 && first <= a.num_pages, a.status);
  int *entry = a.page_table + static_cast<size_t>(b) * a.max_pages + page;
  int id;
  if (page >= held) {
    const int place = count - 1 - (first + page - held);
    id = place >= 0 && place < a.num_pages ? a.free_pages[place] : -1;   // (outside only if the lengths change)
    if (row == 0) *entry = id;
  } else {
    id = *entry;
  }
  return id >= 0 && id < a.num_pages ? static_cast<long long>(id) * a.page_size + row : -1;
}

// What each sequence needs, whether it gets it, and where its tokens start. A thread takes ceil(B / kThreads) sequences in a row:
// their sums, then, behind one scan of the block, each in its place. With kFill the block also does what reserve_fill_kernel
// does (B <= kThreads; what it needs for that stays in shared memory).
template <bool kFill, int kThreads>
__global__ void __launch_bounds__(kThreads) reserve_plan_kernel(const ReserveArgs a) {
  __shared__ Pair part[kThreads / 32];
  __shared__ int taken_part[kThreads / 32];
  __shared__ int starts[kFill ? kThreads + 1 : 1], got[kFill ? kThreads : 1], firsts[kFill ? kThreads : 1];
  grid_dep_launch();
  grid_dep_wait();
  const int count = clamp_len(a.free_count[0], a.num_pages);
  const int each = kFill ? 1 : (a.B + kThreads - 1) / kThreads, b0 = static_cast<int>(threadIdx.x) * each;
  const int b1 = min(b0 + each, a.B);
  int room;
  Pair mine{0, 0}, total;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) {
    const Pair need = reserve_need(a, b, &room);
    mine.x += need.x, mine.y += need.y;
  }
  Pair upto = block_scan<kThreads>(mine, part, &total);
  upto.x -= mine.x, upto.y -= mine.y;
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const Pair need = reserve_need(a, b, &room);
    upto.x += need.x, upto.y += need.y;
    const bool ok = (need.x == 0 || upto.x <= count) && upto.y <= a.tokens;
    if (ok && need.x > 0) taken = static_cast<int>(upto.x);
    const int first = ok ? static_cast<int>(min(upto.x - need.x, static_cast<long long>(a.num_pages))) : 0;
    const int end = static_cast<int>(min(upto.y, 0x7fffffffll));
    XATTN_DCHECK(b >= 0 && room >= 0 && upto.x >= need.x && end >= 0 && (!kFill || a.B <= kThreads), a.status);
    a.granted[b] = ok ? room : 0;
    a.offsets[b + 1] = end;
    if constexpr (kFill)
      starts[b + 1] = end, got[b] = ok ? room : 0, firsts[b] = first;
    else
      a.first[b] = first;
  }
  // The pages taken: the largest running need that was met (each thread's last is its largest).
  taken = __reduce_max_sync(0xffffffffu, taken);
  if ((threadIdx.x & 31) == 0) taken_part[threadIdx.x >> 5] = taken;
  if (kFill && threadIdx.x == 0) starts[0] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    taken = __reduce_max_sync(0xffffffffu, threadIdx.x < kThreads / 32 ? taken_part[threadIdx.x] : 0);
    if (threadIdx.x == 0) {
      a.offsets[0] = 0;
      if (!kFill) a.first[a.B] = count;
      a.free_count[0] = count - taken;
    }
  }
  if constexpr (kFill) {
    for (int t = threadIdx.x; t < a.tokens; t += kThreads) {
      long long slot = -1;
      if (t < starts[a.B]) {
        int lo = 0, hi = a.B;                                // starts[lo] <= t < starts[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (starts[mid] <= t) lo = mid;
          else hi = mid;
        }
        XATTN_DCHECK(lo < a.B && starts[lo] <= t && t < starts[lo + 1], a.status);
        if (t - starts[lo] < got[lo]) slot = reserve_slot(a, lo, t - starts[lo], firsts[lo], count);
      }
      a.slots[t] = slot;
    }
  }
}

// A warp has kTokensEach x 32 tokens in a row: their slots, and the table entries of pages that begin with them. It looks for
// its first token's sequence 32 places at a time (two steps for 1024 sequences), and each thread goes on from there. (32 registers;
// 8 bytes are spilled.)
constexpr int kTokensEach = 4;
__global__ void __launch_bounds__(kFillThreads) reserve_fill_kernel(const ReserveArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const long long t0 = (static_cast<long long>(blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5)) * (32 * kTokensEach);
  const int end = a.offsets[a.B], count = a.first[a.B];
  int lo = 0;
  if (t0 < end) {                                            // (warp-uniform)
    int hi = a.B;                                            // offsets[lo] <= t0 < offsets[hi]
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = min(lo + lane * step, hi);
      XATTN_DCHECK(at >= 0 && at <= a.B, a.status);
      const unsigned below = __ballot_sync(0xffffffffu, at < hi && a.offsets[at] <= t0);   // lanes 0 .. k
      const int k = 31 - __clz(below);
      lo += k * step;
      hi = min(lo + step, hi);
    }
  }
  int next = t0 < end ? a.offsets[lo + 1] : 0;
  long long slot[kTokensEach];
#pragma unroll
  for (int e = 0; e < kTokensEach; ++e) {
    const long long t = t0 + 32 * e + lane;
    slot[e] = -1;
    if (t < end) {
      while (next <= t) next = a.offsets[++lo + 1];
      const int at = static_cast<int>(t) - a.offsets[lo];
      XATTN_DCHECK(lo < a.B && at >= 0, a.status);
      if (at < a.granted[lo]) slot[e] = reserve_slot(a, lo, at, a.first[lo], count);
    }
  }
#pragma unroll
  for (int e = 0; e < kTokensEach; ++e) {
    const long long t = t0 + 32 * e + lane;
    if (t < a.tokens) a.slots[t] = slot[e];
  }
}

// Pages that sequence b gives back: entries [from, to) of its row.
__device__ __forceinline__ int *release_row(const ReleaseArgs &a, int b, int *from, int *to) {
  const int most = a.max_pages * a.page_size;
  *from = pages_of(clamp_len(a.keep_lens[b], most), a.page_size);
  *to = pages_of(clamp_len(a.held_lens[b], most), a.page_size);
  XATTN_DCHECK(b >= 0 && b < a.B && *from >= 0 && *to <= a.max_pages, a.status);
  return a.page_table + static_cast<size_t>(b) * a.max_pages;
}

// (warp) How many pages sequence b gives back.
__device__ __forceinline__ int release_count(const ReleaseArgs &a, int b, int lane) {
  int from, to, n = 0;
  const int *row = release_row(a, b, &from, &to);
#pragma unroll 4
  for (int j = from + lane; j < to; j += 32) n += row[j] >= 0 && row[j] < a.num_pages;
  return __reduce_add_sync(0xffffffffu, n);
}

// (warp) Sequence b's pages onto the stack, downwards from place top - 1 - rank.
__device__ __forceinline__ void release_push(const ReleaseArgs &a, int b, long long top, long long rank, int lane) {
  int from, to;
  int *row = release_row(a, b, &from, &to);
  for (int j0 = from; j0 < to; j0 += 32) {
    const int j = j0 + lane, id = j < to ? row[j] : -1;
    const bool real = id >= 0 && id < a.num_pages;
    const unsigned all = __ballot_sync(0xffffffffu, real);
    const long long place = top - 1 - (rank + __popc(all & ((1u << lane) - 1u)));
    if (real && place >= 0 && place < a.num_pages) a.free_pages[place] = id;
    if (j < to) row[j] = -1;
    rank += __popc(all);
  }
}

// Few sequences with short rows: all in one block. The first sequence's first page ends topmost, so that a release undoes
// the reserve before it.
template <int kThreads>
__global__ void __launch_bounds__(kThreads) release_small_kernel(const ReleaseArgs a) {
  __shared__ Pair part[kThreads / 32];
  __shared__ int ranks[kThreads];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int count = clamp_len(a.free_count[0], a.num_pages);
  XATTN_DCHECK(a.B <= kThreads, a.status);
  for (int b = warp; b < a.B; b += kThreads / 32) {
    const int n = release_count(a, b, lane);
    if (lane == 0) ranks[b] = n;
  }
  __syncthreads();
  const int mine = tid < a.B ? ranks[tid] : 0;
  Pair total;
  const Pair upto = block_scan<kThreads>({mine, 0}, part, &total);
  if (tid < a.B) ranks[tid] = static_cast<int>(upto.x) - mine;
  const long long top = count + total.x;                     // one past the stack's new top
  __syncthreads();
  if (tid == 0) a.free_count[0] = static_cast<int>(min(top, static_cast<long long>(a.num_pages)));
  for (int b = warp; b < a.B; b += kThreads / 32) release_push(a, b, top, ranks[b], lane);
}

// One warp a sequence: how many pages it gives back.
__global__ void __launch_bounds__(kFillThreads) release_count_kernel(const ReleaseArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, b = static_cast<int>(blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.counts[a.B] = clamp_len(a.free_count[0], a.num_pages);
  if (b >= a.B) return;
  const int n = release_count(a, b, lane);
  if (lane == 0) a.counts[b] = n;
}

// One warp a sequence, `each` sequences a block, which adds up for itself what the sequences before it give back.
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
  const long long top = a.counts[a.B] + total.x;             // one past the stack's new top
  if (blockIdx.x == 0 && threadIdx.x == 0) a.free_count[0] = static_cast<int>(min(top, static_cast<long long>(a.num_pages)));
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
    if (live) release_push(a, b, top, r, lane);
  }
}

// A thread has kVecsEach 16-byte vectors of the rows of both sources, a block's width apart; what it reads of the source does
// not wait for the slot. (The slot first, then the row: 41 us for 65536 rows of 576, 3.7 TB/s.)
template <int kVecsEach>
__global__ void __launch_bounds__(kFillThreads) cache_write_kernel(const WriteArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const long long t0 = static_cast<long long>(blockIdx.x) * (kFillThreads * kVecsEach) + threadIdx.x;
  const unsigned each = a.vecs0 + a.vecs1;
  uint4 x[kVecsEach];
  uint4 *to[kVecsEach];
#pragma unroll
  for (int e = 0; e < kVecsEach; ++e) {
    const long long t = t0 + e * kFillThreads;
    long long r;
    unsigned v;
    if (t >> 32) {
      r = t / each;
      v = static_cast<unsigned>(t - r * each);
    } else {                                                 // division in 32 bits
      r = static_cast<unsigned>(t) / each;
      v = static_cast<unsigned>(t) - static_cast<unsigned>(r) * each;
    }
    to[e] = nullptr;
    if (r >= a.rows) continue;
    const long long slot = a.slots[r];
    const bool second = v >= a.vecs0;
    if (second) v -= a.vecs0;
    x[e] = second ? a.src1[r * a.vecs1 + v] : a.src0[r * a.vecs0 + v];
    XATTN_DCHECK(r >= 0 && v < (second ? a.vecs1 : a.vecs0) && static_cast<int>(a.vecs0) <= a.stride0 &&
                     static_cast<int>(a.vecs1) <= a.stride1,
                 a.status);
    if (slot >= 0 && slot < a.num_slots) to[e] = second ? a.dst1 + slot * a.stride1 + v : a.dst0 + slot * a.stride0 + v;
  }
#pragma unroll
  for (int e = 0; e < kVecsEach; ++e)
    if (to[e]) *to[e] = x[e];
}

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + kFillThreads - 1) / kFillThreads); }

// One block does all of a small call: no scratch and no second kernel. A reserve of 1000 tokens of 1000 sequences takes 6 us
// so (two kernels 14), of 2048 of 128 7.4 (9.3), of 4000 of 4 8.1 (7.4), of 8192 of 512 12.4 (7.9). A release of 64
// sequences takes 3.7 us on the GPU (3.3) and less of the host's time (2.2 for 4.9), of 8 1.8 (3.3), of 256 7.8 (3.4).
constexpr int kSmallTokens = 2048, kSmallSeqs = 64, kSmallEntries = 16384;

}  // namespace

bool reserve_small(int B, long long tokens) { return B <= kPlanThreads && tokens <= kSmallTokens; }
bool release_small(int B, int max_pages) {
  return B <= kSmallSeqs && static_cast<long long>(B) * max_pages <= kSmallEntries;
}

cudaError_t launch_cache_reserve(const ReserveArgs &a, cudaStream_t stream) {
  if (reserve_small(a.B, a.tokens)) {
    // A block of 256 threads starts and scans sooner: one token of 64 sequences 3.8 us, with 1024 threads 6.1.
    if (a.B <= kFewThreads && a.tokens <= 2 * kFewThreads)
      return launch_pdl(reserve_plan_kernel<true, kFewThreads>, 1, kFewThreads, 0, stream, a);
    return launch_pdl(reserve_plan_kernel<true, kPlanThreads>, 1, kPlanThreads, 0, stream, a);
  }
  const cudaError_t err = launch_pdl(reserve_plan_kernel<false, kPlanThreads>, 1, kPlanThreads, 0, stream, a);
  if (err != cudaSuccess || a.tokens == 0) return err;
  return launch_pdl(reserve_fill_kernel, blocks_for((a.tokens + kTokensEach - 1) / kTokensEach), kFillThreads, 0, stream, a);
}

cudaError_t launch_cache_release(const ReleaseArgs &a, cudaStream_t stream) {
  if (release_small(a.B, a.max_pages)) {
    if (a.B <= kFewThreads / 32)                               // (8 sequences: 1.8 us, with 1024 threads 2.8)
      return launch_pdl(release_small_kernel<kFewThreads>, 1, kFewThreads, 0, stream, a);
    return launch_pdl(release_small_kernel<kPlanThreads>, 1, kPlanThreads, 0, stream, a);
  }
  constexpr int kWarps = kFillThreads / 32;
  const unsigned blocks = static_cast<unsigned>((static_cast<long long>(a.B) + kWarps - 1) / kWarps);
  const cudaError_t err = launch_pdl(release_count_kernel, blocks, kFillThreads, 0, stream, a);
  if (err != cudaSuccess) return err;
  const int each = (static_cast<int>((blocks + 511) / 512)) * kWarps;
  return launch_pdl(release_push_kernel, static_cast<unsigned>((static_cast<long long>(a.B) + each - 1) / each), kFillThreads, 0,
                    stream, a, each);
}

cudaError_t launch_cache_write(const WriteArgs &a, int sms, cudaStream_t stream) {
  // One vector a thread where that is less than the GPU holds at once (64 rows of 576: 1.3 us, 2.5 with four), else two (65536
  // rows: 24.6 us, 6.2 TB/s; one 25.6, four 26.8, eight 32.2).
  const long long vecs = a.rows * (a.vecs0 + a.vecs1);
  constexpr int kMany = 2;
  if (vecs <= static_cast<long long>(sms) * 2048) return launch_pdl(cache_write_kernel<1>, blocks_for(vecs), kFillThreads, 0, stream, a);
  return launch_pdl(cache_write_kernel<kMany>, blocks_for((vecs + kMany - 1) / kMany), kFillThreads, 0, stream, a);
}

}  // namespace xattn
