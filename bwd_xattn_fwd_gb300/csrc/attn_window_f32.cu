// Window attention with sinks in IEEE fp32 on the CUDA cores: query i sees key j <= i only if
// i - j < window or j < sinks.
//
// The method is the bf16 path's: an online softmax over the key tiles that hold a visible
// pair, and a backward that recomputes the scores from the saved LSE and uses D_i = dO_i . o_i.
// Products are FMA chains over tiles of 32 x 32 pairs, the operands in shared memory (rows of
// hd rounded up to 32, 64 or 128, zero-filled), loaded one tile ahead by asynchronous copies.
// A tile belongs to a group of 64 threads with 4 x 4 pairs each: shared-memory reads, not the
// FMA pipe, bound a product (8 16-byte reads for 64 FMAs). The two groups of a block take its
// tiles in turn, and dK/dV a cluster of blocks as well, because the problems this mode serves
// (gradient checks, small models) are chains of a few tiles on a GPU that they do not fill.
// Forward and backward of B2 S499 4 heads on 2, hd 64, window 100: 64.5 us (13.4 + 17.8 + 34.4 alone);
// one group of 128 threads with 2 x 4 pairs (6 reads for 32 FMAs) took 98 us, a warp per row
// and one key at a time 643 us.
// Three kernels: the forward, dQ (query tile, walking keys), dK/dV (key tile, walking queries
// of every head of the group). Every output is a sum in a fixed order, without atomics.
#include <cooperative_groups.h>

#include <cmath>

#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kT = 32;                 // rows of a tile, queries and keys
constexpr int kGroup = 64;             // threads of a tile: rows 4 ty .. + 3, columns tx + 8 j
constexpr int kF32Threads = 128;       // two groups
constexpr int kPairStride = kT + 4;    // of a 32 x 32 tile of P or dS
constexpr int kPairs = kT * kPairStride;

struct F32Args {
  const float *q, *k, *v, *o, *dO, *lse;
  float *out, *out2, *stat;            // o, or dq, or dk and dv; lse, or D (written by dQ)
  int B, S, nh, nkv, hd, window, sinks;
  float scale;
  bool vec;                            // 16-byte accesses: hd a multiple of 4, pointers aligned
};

template <int HDP>
__host__ __device__ constexpr int tile_floats() {
  return kT * (HDP + 4);
}

// Starts the copy of 32 rows (from row0 on, of one head) of a [B, S, heads, hd] tensor by
// `threads` threads; rows past S and columns past hd become zeros.
template <int HDP>
__device__ __forceinline__ void load_rows(float *dst, const float *src, const F32Args &a, int heads, int b, int head,
                                          int row0, int t, int threads) {
  for (int x = t; x < kT * HDP / 4; x += threads) {
    const int r = x / (HDP / 4), c = x % (HDP / 4) * 4;
    const bool in = row0 + r < a.S;
    const float *from = src + ((static_cast<size_t>(b) * a.S + (in ? row0 + r : 0)) * heads + head) * a.hd;
    const uint32_t to = smem_u32(dst + r * (HDP + 4) + c);
    if (a.vec) {
      const int bytes = in && c < a.hd ? 16 : 0;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from + (bytes ? c : 0)), "r"(bytes)
                   : "memory");
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int bytes = in && c + e < a.hd ? 4 : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * e), "l"(from + (bytes ? c + e : 0)),
                     "r"(bytes)
                     : "memory");
      }
    }
  }
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last `kLeft` committed groups of copies of this thread have landed.
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// The 64 threads of group g.
__device__ __forceinline__ void group_sync(int g) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "n"(kGroup) : "memory");
}

// acc[r][j] = x_(4 ty + r) . y_(tx + 8 j).
template <int HDP>
__device__ __forceinline__ void products(float (&acc)[4][4], const float *x, const float *y, int ty, int tx) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[r][j] = 0.f;
  const float *x0 = x + 4 * ty * (HDP + 4), *y0 = y + tx * (HDP + 4);
#pragma unroll 4
  for (int d = 0; d < HDP; d += 4) {
    float4 xv[4], yv[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) xv[r] = *reinterpret_cast<const float4 *>(x0 + r * (HDP + 4) + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) yv[j] = *reinterpret_cast<const float4 *>(y0 + 8 * j * (HDP + 4) + d);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[r][j] = fmaf(xv[r].x, yv[j].x, acc[r][j]);
        acc[r][j] = fmaf(xv[r].y, yv[j].y, acc[r][j]);
        acc[r][j] = fmaf(xv[r].z, yv[j].z, acc[r][j]);
        acc[r][j] = fmaf(xv[r].w, yv[j].w, acc[r][j]);
      }
  }
}

// A thread's accumulators: rows 4 ty + r, columns 4 tx + 32 c .. + 3.
template <int HDP>
struct Acc {
  float4 x[4][HDP / 32];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < HDP / 32; ++c) x[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // += sum_j w_(row, j) y_j
  __device__ __forceinline__ void add(const float *w, const float *y, int ty, int tx) {
#pragma unroll 2
    for (int j0 = 0; j0 < kT; j0 += 4) {
      float wv[4][4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4 *>(wv[r]) = *reinterpret_cast<const float4 *>(w + (4 * ty + r) * kPairStride + j0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < HDP / 32; ++c) {
          const float4 yv = *reinterpret_cast<const float4 *>(y + (j0 + j) * (HDP + 4) + 4 * tx + 32 * c);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r][c].x = fmaf(wv[r][j], yv.x, x[r][c].x);
            x[r][c].y = fmaf(wv[r][j], yv.y, x[r][c].y);
            x[r][c].z = fmaf(wv[r][j], yv.z, x[r][c].z);
            x[r][c].w = fmaf(wv[r][j], yv.w, x[r][c].w);
          }
        }
    }
  }
  __device__ __forceinline__ void put(float *tile, int ty, int tx) const {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < HDP / 32; ++c)
        *reinterpret_cast<float4 *>(tile + (4 * ty + r) * (HDP + 4) + 4 * tx + 32 * c) = x[r][c];
  }
  // row r: own * mine + tile * other
  __device__ __forceinline__ void merge(int r, const float *tile, int ty, int tx, float mine, float other) {
#pragma unroll
    for (int c = 0; c < HDP / 32; ++c) {
      const float4 y = *reinterpret_cast<const float4 *>(tile + (4 * ty + r) * (HDP + 4) + 4 * tx + 32 * c);
      x[r][c].x = x[r][c].x * mine + y.x * other;
      x[r][c].y = x[r][c].y * mine + y.y * other;
      x[r][c].z = x[r][c].z * mine + y.z * other;
      x[r][c].w = x[r][c].w * mine + y.w * other;
    }
  }
  // Row r to a row of a [.., hd] tensor, times mult.
  __device__ __forceinline__ void store(int r, float *dst, const F32Args &a, int tx, float mult) const {
#pragma unroll
    for (int c = 0; c < HDP / 32; ++c) {
      const int d = 4 * tx + 32 * c;
      const float y[4] = {x[r][c].x * mult, x[r][c].y * mult, x[r][c].z * mult, x[r][c].w * mult};
      if (a.vec) {
        if (d < a.hd) *reinterpret_cast<float4 *>(dst + d) = make_float4(y[0], y[1], y[2], y[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (d + e < a.hd) dst[d + e] = y[e];
      }
    }
  }
};

__device__ __forceinline__ bool sees(const F32Args &a, int i, int j) {
  return j <= i && (i - j < a.window || j < a.sinks);
}

// Sum and maximum over the 8 lanes tx of one ty (a group of 8 neighbouring lanes).
__device__ __forceinline__ float sum8(float x) {
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ float max8(float x) {
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// The key tiles that query tile m sees, as a list: `heads` sink tiles, then lo .. m.
struct KeyTiles {
  int lo, heads, count;
  __device__ KeyTiles(const F32Args &a, int m) {
    lo = max(m * kT - a.window + 1, 0) / kT;
    heads = min((a.sinks + kT - 1) / kT, lo);
    count = heads + m - lo + 1;
  }
  __device__ int at(int e) const { return e < heads ? e : e - heads + lo; }
};

// What a query-tile kernel's block and thread work on.
struct Place {
  int m, h, b, kvh, g, t, tx, ty;
  __device__ Place(const F32Args &a) {
    const int tiles = (a.S + kT - 1) / kT, bh = blockIdx.x / tiles;
    m = blockIdx.x % tiles;
    h = bh % a.nh;
    b = bh / a.nh;
    kvh = h / (a.nh / a.nkv);
    g = threadIdx.x / kGroup;
    t = threadIdx.x % kGroup;
    tx = t % 8;
    ty = t / 8;
  }
};

// Shared memory of the query-tile kernels: `kQueryTiles` tiles, then per group K, V twice, then
// per group a 32 x 32 tile of pairs.
template <int HDP, int kQueryTiles>
__host__ __device__ constexpr int query_floats() {
  return (kQueryTiles + 8) * tile_floats<HDP>() + 2 * kPairs;
}

// Forward: block = (batch, head, query tile).
template <int HDP>
__global__ void __launch_bounds__(kF32Threads) window_fwd_f32_kernel(const F32Args a) {
  grid_dep_wait();
  extern __shared__ __align__(16) float f32_smem[];
  constexpr int kTile = tile_floats<HDP>();
  const Place w(a);
  float *sq = f32_smem, *skv = sq + kTile + w.g * 4 * kTile, *sp = sq + 9 * kTile + w.g * kPairs;
  const KeyTiles keys(a, w.m);
  auto load = [&](int e, int slot) {
    float *dst = skv + slot * 2 * kTile;
    load_rows<HDP>(dst, a.k, a, a.nkv, w.b, w.kvh, keys.at(e) * kT, w.t, kGroup);
    load_rows<HDP>(dst + kTile, a.v, a, a.nkv, w.b, w.kvh, keys.at(e) * kT, w.t, kGroup);
    copies_commit();
  };
  load_rows<HDP>(sq, a.q, a, a.nh, w.b, w.h, w.m * kT, threadIdx.x, kF32Threads);
  copies_commit();
  if (w.g < keys.count) load(w.g, 0);
  copies_wait<1>();
  if (w.g >= keys.count) copies_wait<0>();
  __syncthreads();                          // q is everyone's
  Acc<HDP> acc;
  acc.zero();
  float mrow[4], lrow[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) mrow[r] = -INFINITY, lrow[r] = 0.f;
  for (int e = w.g, slot = 0; e < keys.count; e += 2, slot ^= 1) {
    if (e + 2 < keys.count) {
      load(e + 2, slot ^ 1);
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    group_sync(w.g);
    const float *sk = skv + slot * 2 * kTile, *sv = sk + kTile;
    float s[4][4];
    products<HDP>(s, sq, sk, w.ty, w.tx);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = w.m * kT + 4 * w.ty + r;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[r][j] = sees(a, i, keys.at(e) * kT + w.tx + 8 * j) ? s[r][j] * a.scale : -INFINITY;
        mx = fmaxf(mx, s[r][j]);
      }
      const float mnew = fmaxf(mrow[r], max8(mx));
      const float base = mnew == -INFINITY ? 0.f : mnew;      // no key of these tiles seen yet
      const float alpha = expf(mrow[r] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(s[r][j] - base);
        sum += p;
        sp[(4 * w.ty + r) * kPairStride + w.tx + 8 * j] = p;
      }
      lrow[r] = lrow[r] * alpha + sum8(sum);
      mrow[r] = mnew;
#pragma unroll
      for (int c = 0; c < HDP / 32; ++c)
        acc.x[r][c].x *= alpha, acc.x[r][c].y *= alpha, acc.x[r][c].z *= alpha, acc.x[r][c].w *= alpha;
    }
    __syncwarp();                          // a row of P is written and read by one warp
    acc.add(sp, sv, w.ty, w.tx);
    group_sync(w.g);                       // before the tiles are overwritten
  }
  // Group 1 hands its rows to group 0 (its K, V and P are done with).
  float *other = sq + 5 * kTile, *stats = sq + 9 * kTile + kPairs;
  if (w.g == 1) {
    acc.put(other, w.ty, w.tx);
    if (w.tx == 0)
#pragma unroll
      for (int r = 0; r < 4; ++r) stats[2 * (4 * w.ty + r)] = mrow[r], stats[2 * (4 * w.ty + r) + 1] = lrow[r];
  }
  __syncthreads();
  if (w.g == 1) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = w.m * kT + 4 * w.ty + r;
    const float m1 = stats[2 * (4 * w.ty + r)], l1 = stats[2 * (4 * w.ty + r) + 1];
    const float M = fmaxf(mrow[r], m1);      // finite for i < S: a row sees itself
    const float w0 = expf(mrow[r] - M), w1 = expf(m1 - M), sum = lrow[r] * w0 + l1 * w1;
    if (i >= a.S) continue;
    acc.merge(r, other, w.ty, w.tx, w0 / sum, w1 / sum);
    const size_t row = (static_cast<size_t>(w.b) * a.S + i) * a.nh + w.h;
    acc.store(r, a.out + row * a.hd, a, w.tx, 1.f);
    if (w.tx == 0) a.stat[row] = M + logf(sum);
  }
}

// dQ: block = (batch, head, query tile); dQ_i = scale sum_j P_ij (dO_i . v_j - D_i) k_j. Also
// writes D_i = dO_i . o_i for the dK/dV kernel.
template <int HDP>
__global__ void __launch_bounds__(kF32Threads) window_dq_f32_kernel(const F32Args a) {
  grid_dep_wait();
  extern __shared__ __align__(16) float f32_smem[];
  constexpr int kTile = tile_floats<HDP>();
  const Place w(a);
  float *sq = f32_smem, *sdo = sq + kTile, *so = sdo + kTile;
  float *skv = sq + 3 * kTile + w.g * 4 * kTile, *sds = sq + 11 * kTile + w.g * kPairs;
  const KeyTiles keys(a, w.m);
  auto load = [&](int e, int slot) {
    float *dst = skv + slot * 2 * kTile;
    load_rows<HDP>(dst, a.k, a, a.nkv, w.b, w.kvh, keys.at(e) * kT, w.t, kGroup);
    load_rows<HDP>(dst + kTile, a.v, a, a.nkv, w.b, w.kvh, keys.at(e) * kT, w.t, kGroup);
    copies_commit();
  };
  load_rows<HDP>(sq, a.q, a, a.nh, w.b, w.h, w.m * kT, threadIdx.x, kF32Threads);
  load_rows<HDP>(sdo, a.dO, a, a.nh, w.b, w.h, w.m * kT, threadIdx.x, kF32Threads);
  load_rows<HDP>(so, a.o, a, a.nh, w.b, w.h, w.m * kT, threadIdx.x, kF32Threads);
  copies_commit();
  if (w.g < keys.count) load(w.g, 0);
  copies_wait<1>();
  if (w.g >= keys.count) copies_wait<0>();
  __syncthreads();
  float D[4], L[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int at = (4 * w.ty + r) * (HDP + 4) + 4 * w.tx, i = w.m * kT + 4 * w.ty + r;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < HDP; c += 32) {
      const float4 x = *reinterpret_cast<const float4 *>(sdo + at + c), y = *reinterpret_cast<const float4 *>(so + at + c);
      s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
    }
    D[r] = sum8(s);
    const size_t row = (static_cast<size_t>(w.b) * a.S + i) * a.nh + w.h;
    L[r] = i < a.S ? a.lse[row] : 0.f;
    if (w.g == 0 && w.tx == 0 && i < a.S) a.stat[row] = D[r];
  }
  Acc<HDP> acc;
  acc.zero();
  for (int e = w.g, slot = 0; e < keys.count; e += 2, slot ^= 1) {
    if (e + 2 < keys.count) {
      load(e + 2, slot ^ 1);
      copies_wait<1>();
    } else {
      copies_wait<0>();
    }
    group_sync(w.g);
    const float *sk = skv + slot * 2 * kTile, *sv = sk + kTile;
    float s[4][4], dp[4][4];
    products<HDP>(s, sq, sk, w.ty, w.tx);
    products<HDP>(dp, sdo, sv, w.ty, w.tx);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = sees(a, w.m * kT + 4 * w.ty + r, keys.at(e) * kT + w.tx + 8 * j);
        sds[(4 * w.ty + r) * kPairStride + w.tx + 8 * j] = in ? expf(s[r][j] * a.scale - L[r]) * (dp[r][j] - D[r]) : 0.f;
      }
    __syncwarp();
    acc.add(sds, sk, w.ty, w.tx);
    group_sync(w.g);
  }
  float *other = sq + 7 * kTile;
  if (w.g == 1) acc.put(other, w.ty, w.tx);
  __syncthreads();
  if (w.g == 1) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = w.m * kT + 4 * w.ty + r;
    if (i >= a.S) continue;
    acc.merge(r, other, w.ty, w.tx, 1.f, 1.f);
    acc.store(r, a.out + ((static_cast<size_t>(w.b) * a.S + i) * a.nh + w.h) * a.hd, a, w.tx, a.scale);
  }
}

// dK, dV: a cluster of kParts blocks = (batch, kv head, key tile); its (head of the group,
// query tile) pairs go round the 2 kParts groups, so that a sink tile, which every query sees,
// is not one block's chain; the parts are added in order through distributed shared memory.
// kParts is 4, or 8 where that leaves a block an SM (B1 S200, 14 key tiles: 11.5 us, 16.5 with 4;
// B4 S300, 80 key tiles: 39.3 and 27.2).
constexpr int kSms = 152;

// Shared memory: K, V; per group q, dO twice; per group P and dS; per group lse and D of 32 rows.
template <int HDP>
__host__ __device__ constexpr int key_floats() {
  return 10 * tile_floats<HDP>() + 4 * kPairs + 4 * kT;
}

template <int HDP, int kParts>
__global__ void __cluster_dims__(kParts, 1, 1) __launch_bounds__(kF32Threads) window_dkdv_f32_kernel(const F32Args a) {
  namespace cg = cooperative_groups;
  grid_dep_wait();
  extern __shared__ __align__(16) float f32_smem[];
  constexpr int kTile = tile_floats<HDP>();
  const int g = threadIdx.x / kGroup, t = threadIdx.x % kGroup, tx = t % 8, ty = t / 8;
  float *sk = f32_smem, *sv = sk + kTile, *sx = sv + kTile + g * 4 * kTile;
  float *sp = sk + 10 * kTile + g * 2 * kPairs, *sds = sp + kPairs, *sl = sk + 10 * kTile + 4 * kPairs + g * 2 * kT;
  float *sd = sl + kT;
  cg::cluster_group cluster = cg::this_cluster();
  const int part = static_cast<int>(cluster.block_rank());
  const int tiles = (a.S + kT - 1) / kT, group = a.nh / a.nkv;
  const int unit = blockIdx.x / kParts, n = unit % tiles, bk = unit / tiles, kvh = bk % a.nkv, b = bk / a.nkv;
  // Query tiles n .. last see some key of the tile.
  const int last_key = min(n * kT + kT, a.S) - 1;
  const int last = n * kT < a.sinks ? tiles - 1 : min((last_key + a.window - 1) / kT, tiles - 1);
  const int per_head = last - n + 1, count = per_head * group;
  auto load = [&](int it, int slot) {
    const int h = kvh * group + it / per_head, row0 = (n + it % per_head) * kT;
    float *dst = sx + slot * 2 * kTile;
    load_rows<HDP>(dst, a.q, a, a.nh, b, h, row0, t, kGroup);
    load_rows<HDP>(dst + kTile, a.dO, a, a.nh, b, h, row0, t, kGroup);
    copies_commit();
  };
  load_rows<HDP>(sk, a.k, a, a.nkv, b, kvh, n * kT, threadIdx.x, kF32Threads);
  load_rows<HDP>(sv, a.v, a, a.nkv, b, kvh, n * kT, threadIdx.x, kF32Threads);
  copies_commit();
  const int first = 2 * part + g;
  if (first < count) load(first, 0);
  copies_wait<1>();
  if (first >= count) copies_wait<0>();
  __syncthreads();                          // k and v are everyone's
  Acc<HDP> dk, dv;
  dk.zero();
  dv.zero();
  for (int it = first, slot = 0; it < count; it += 2 * kParts, slot ^= 1) {
    const int h = kvh * group + it / per_head, i0 = (n + it % per_head) * kT;
    if (it + 2 * kParts < count) load(it + 2 * kParts, slot ^ 1);
    {
      const size_t row = (static_cast<size_t>(b) * a.S + min(i0 + t % kT, a.S - 1)) * a.nh + h;
      (t < kT ? sl : sd)[t % kT] = t < kT ? a.lse[row] : a.stat[row];
    }
    if (it + 2 * kParts < count) copies_wait<1>();
    else copies_wait<0>();
    group_sync(g);
    const float *q = sx + slot * 2 * kTile, *dO = q + kTile;
    float s[4][4], dp[4][4];                                          // rows: keys; columns: queries
    products<HDP>(s, sk, q, ty, tx);
    products<HDP>(dp, sv, dO, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = tx + 8 * j, at = (4 * ty + r) * kPairStride + i;
        const bool in = i0 + i < a.S && sees(a, i0 + i, n * kT + 4 * ty + r);
        const float p = in ? expf(s[r][j] * a.scale - sl[i]) : 0.f;
        sp[at] = p;
        sds[at] = in ? p * (dp[r][j] - sd[i]) : 0.f;
      }
    __syncwarp();
    dv.add(sp, dO, ty, tx);
    dk.add(sds, q, ty, tx);
    group_sync(g);
  }
  // The parts, in order: each group's dK and dV into its own q, dO tiles (done with); block
  // `part` adds and writes rows part, part + kParts, ..
  dk.put(sx, ty, tx);
  dv.put(sx + kTile, ty, tx);
  cluster.sync();
  float *parts = sv + kTile;
  for (int x = threadIdx.x; x < 2 * (kT / kParts) * (HDP / 4); x += kF32Threads) {
    const int c = x % (HDP / 4) * 4, r = x / (HDP / 4) % (kT / kParts) * kParts + part, which = x / (HDP / 4) / (kT / kParts);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < 2 * kParts; ++p) {
      const float4 y = *reinterpret_cast<const float4 *>(cluster.map_shared_rank(parts, p / 2) + (p % 2) * 4 * kTile +
                                                         which * kTile + r * (HDP + 4) + c);
      sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
    }
    const int j = n * kT + r;
    if (j >= a.S) continue;
    const float mult = which ? 1.f : a.scale;
    const float val[4] = {sum.x * mult, sum.y * mult, sum.z * mult, sum.w * mult};
    float *dst = (which ? a.out2 : a.out) + ((static_cast<size_t>(b) * a.S + j) * a.nkv + kvh) * a.hd;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < a.hd) dst[c + e] = val[e];
  }
  cluster.sync();                          // nobody leaves while its parts are being read
}

bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Programmatic launches that no kernel triggers early: a kernel is set up while the one before it
// ends, but its blocks do not start on the SMs that one leaves free, where they would pile up
// (the three kernels 140 us instead of 98 with 2 x 4 pairs).
template <typename Kernel>
cudaError_t launch(Kernel *kernel, std::atomic<unsigned long long> &allowed, long long blocks, int floats,
                   const F32Args &a, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(floats) * sizeof(float);
  const cudaError_t err = allow_smem(kernel, smem, allowed);
  if (err != cudaSuccess) return err;
  return launch_pdl(kernel, static_cast<unsigned>(blocks), kF32Threads, smem, stream, a);
}

template <int HDP>
cudaError_t launch_fwd(const F32Args &a, cudaStream_t stream) {
  static std::atomic<unsigned long long> allowed{0};
  const long long tiles = (a.S + kT - 1) / kT;
  return launch(window_fwd_f32_kernel<HDP>, allowed, tiles * a.B * a.nh, query_floats<HDP, 1>(), a, stream);
}

template <int HDP>
cudaError_t launch_bwd(const F32Args &a, float *dk, float *dv, cudaStream_t stream) {
  static std::atomic<unsigned long long> allowed_q{0}, allowed_kv{0}, allowed_kv8{0};
  const long long tiles = (a.S + kT - 1) / kT;
  const cudaError_t err =
      launch(window_dq_f32_kernel<HDP>, allowed_q, tiles * a.B * a.nh, query_floats<HDP, 3>(), a, stream);
  if (err != cudaSuccess) return err;
  F32Args kv = a;
  kv.out = dk;
  kv.out2 = dv;
  const long long units = tiles * a.B * a.nkv;
  if (units * 8 <= kSms)
    return launch(window_dkdv_f32_kernel<HDP, 8>, allowed_kv8, units * 8, key_floats<HDP>(), kv, stream);
  return launch(window_dkdv_f32_kernel<HDP, 4>, allowed_kv, units * 4, key_floats<HDP>(), kv, stream);
}

}  // namespace

cudaError_t launch_window_fwd_f32(const float *q, const float *k, const float *v, float *o, float *lse, int B, int S,
                                  int nh, int nkv, int hd, float scale, int window, int sinks, cudaStream_t stream) {
  const bool vec = hd % 4 == 0 && aligned(q) && aligned(k) && aligned(v) && aligned(o);
  const F32Args a = {q, k, v, nullptr, nullptr, nullptr, o, nullptr, lse, B, S, nh, nkv, hd, window, sinks, scale, vec};
  return hd <= 32 ? launch_fwd<32>(a, stream) : (hd <= 64 ? launch_fwd<64>(a, stream) : launch_fwd<128>(a, stream));
}

cudaError_t launch_window_bwd_f32(const float *q, const float *k, const float *v, const float *o, const float *dO,
                                  const float *lse, float *dq, float *dk, float *dv, float *D, int B, int S, int nh,
                                  int nkv, int hd, float scale, int window, int sinks, cudaStream_t stream) {
  const bool vec = hd % 4 == 0 && aligned(q) && aligned(k) && aligned(v) && aligned(o) && aligned(dO) && aligned(dq);
  const F32Args a = {q, k, v, o, dO, lse, dq, nullptr, D, B, S, nh, nkv, hd, window, sinks, scale, vec};
  return hd <= 32 ? launch_bwd<32>(a, dk, dv, stream)
                  : (hd <= 64 ? launch_bwd<64>(a, dk, dv, stream) : launch_bwd<128>(a, dk, dv, stream));
}

}  // namespace xattn
