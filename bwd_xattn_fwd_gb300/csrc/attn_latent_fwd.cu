// Latent attention in its expanded form, forward, on sm_103a tensor cores.
//
// Head h's key of token j is (kv[j, h, :dn], k_rope[j]) and its value kv[j, h, dn:]; the shared part k_rope is read from
// its one copy, so no key is put together in memory. Causal, online softmax over key tiles, each row's log-sum-exp kept.
//
// GB300 mapping: that of attn_fwd_sm103.cu (a unit is two 128-row query tiles A, B of one head that share every K and V
// tile; two MMA issuers, two softmax warpgroups; P in bf16 over S in TMEM), with heads of unlike widths:
//   * A tile is 64-column sub-tiles of 128 rows (16 KB, 128-byte swizzle): dn's, one of dr, and dv's. Columns behind dn, dr
//     or dv are other columns or zeros that no product touches: the scores take (dn + dr) / 16 steps, P V has N = dv.
//   * At dn, dv > 64 the two query tiles take 96 KB, and 8 sub-tiles are left for K (3) and V (2). They form one ring of
//     sub-tiles in the order K(0) V(0) K(1) V(1) ..: V(n) takes the place of K(n - 1)'s first two as soon as both scores
//     have read them, K(n) that of V(n - 2). (Two stages of K and one of V are as much memory, but V(n) could only be
//     fetched when P V(n - 1) has ended, right before it is needed.) Where dn, dv <= 64: three whole stages.
//   * P V is a product a sub-tile (P from TMEM: 32 cycles a K step and 64 columns, as much as half of one over 128), so V's
//     two may lie anywhere in the ring.
// Roundings: P to bf16, V's type, before P V; o to bf16. All exponentials on the special-function unit: one pair in eight on the FMA
// pipe, as in attn_fwd_sm103.cu, was 1 % slower here, one in four 5 %.
// Bound by the tensor cores, and between units by the softmax's turn: B4 S4093, 16 heads of 128 + 64 / 128 243 us, 1411 TFLOP/s of
// visible pairs (71 % of the measured peak); 64 + 32 / 64 at S4096 133 us, 1293, at B8 S1024, 12 heads 24 us, 665.
// Registers: a softmax thread holds a row of S (128). At the cap of 168 that 384 threads leave, NS = 2 spills 16 bytes and NS = 1 none.
// TMEM: S_A [0,128) S_B [128,256) fp32 | O_A, O_B from 256, 64 NS columns each | NS = 1: P_A [384,448) P_B [448,512), so that the
// next scores are issued as soon as these are read; NS = 2: P_X over the first half of S_X, the next scores behind P V.
#include <type_traits>

#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kFwdThreads = 384;   // 12 warps
constexpr uint32_t kSubTile = kTileRows * 128;

// NS: sub-tiles of dn, and of dv, that there is room for (dn, dv <= 64 NS).
template <int NS>
struct LatentFwdLayout {
  static constexpr int kBlocks = NS == 2 ? 8 : 9;                  // ring of sub-tiles
  static constexpr int kEach = 2 * NS + 1;                         // of one K and V tile
  static constexpr int kDepth = NS == 2 ? 2 : 3;                   // barriers of K, and of V
  static constexpr bool kAliasP = NS == 2;
  static constexpr uint32_t kQ = 0;                                // Q_A, Q_B
  static constexpr uint32_t kRing = 2 * (NS + 1) * kSubTile;
  static constexpr uint32_t kBars = kRing + kBlocks * kSubTile;
  static constexpr int kNumBars = 4 * kDepth + 12;
  static constexpr uint32_t kMisc = kBars + 8 * kNumBars;
  static constexpr uint32_t kUsed = kMisc + 32;
  static constexpr uint32_t kDynBytes = kUsed + 1024;
  static_assert(kDynBytes <= 227 * 1024, "exceeds the opt-in shared memory of one CTA");
  static_assert(kDynBytes > 114 * 1024, "one CTA an SM: each holds all TMEM columns");
};

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl &ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}

// kNegScale: scale < 0, so the row maximum of the scaled scores is the scaled minimum of the raw ones.
template <int NS, bool kFull, bool kNegScale>
__global__ void __maxnreg__(168)
    latent_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkv,
                      const __grid_constant__ CUtensorMap mrope, const LatentArgs a) {
  using L = LatentFwdLayout<NS>;
  constexpr int kDepth = L::kDepth, kBlocks = L::kBlocks;
  extern __shared__ uint8_t latent_fwd_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(latent_fwd_smem) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int S = a.S, nh = a.nh, dn = kFull ? 64 * NS : a.dn, dv = kFull ? 64 * NS : a.dv;
  const int dn_steps = dn / 16, dr_steps = a.dr / 16;
  const int k_subs = (dn + 63) / 64, v_subs = (dv + 63) / 64;

  // Units (tile pair jp of one (batch, head)), longest first; CTA c of G takes unit k G + c in even rounds and
  // k G + G - 1 - c in odd ones. Every role walks the same units; barriers' phases count over all of them.
  const int num_m = (S + kTileRows - 1) / kTileRows, num_pairs = (num_m + 1) / 2, BH = a.B * nh;
  const int num_units = num_pairs * BH;
  const int G = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  auto unit_at = [G, cta](int k) { return k * G + ((k & 1) ? G - 1 - cta : cta); };
#define XATTN_LATENT_UNIT(u)                                       \
  const int jp = num_pairs - 1 - (u) / BH;                         \
  const int b = ((u) % BH) / nh, h = (u) % nh;                     \
  const int mA = 2 * jp, mB = 2 * jp + 1;                          \
  const bool hasB = mB < num_m;                                    \
  const int count = (hasB ? mB : mA) + 1; /* key tiles */          \
  (void)b;                                                         \
  (void)h;                                                         \
  (void)count

  const uint32_t sQ = smem_u32(smem + L::kQ), sRing = smem_u32(smem + L::kRing), bar0 = smem_u32(smem + L::kBars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto k_full = [&](int s) { return bar(s); };
  auto k_empty = [&](int s) { return bar(kDepth + s); };
  auto v_full = [&](int s) { return bar(2 * kDepth + s); };
  auto v_empty = [&](int s) { return bar(3 * kDepth + s); };
  constexpr int kB = 4 * kDepth;
  auto s_full = [&](int x) { return bar(kB + x); };
  auto p_full = [&](int x) { return bar(kB + 2 + x); };
  auto o_done = [&](int x) { return bar(kB + 4 + x); };
  auto s_free = [&](int x) { return bar(kB + 6 + x); };
  auto o_free = [&](int x) { return bar(kB + 8 + x); };
  const uint32_t q_full = bar(kB + 10), q_empty = bar(kB + 11);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 16);
  const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kDepth; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(k_empty(s), 2);          // both issuers release each tile, used or passed
      mbar_init(v_empty(s), 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 128);
      mbar_init(o_done(x), 1);
      mbar_init(s_free(x), 128);
      mbar_init(o_free(x), 128);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);                   // both issuers' last scores of a unit
    fence_mbar_init();
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mkv);
    tma_prefetch_desc(&mrope);
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
  auto tS = [&](int x) { return tmem + 128u * x; };
  auto tO = [&](int x) { return tmem + 256u + 64u * NS * x; };
  auto tP = [&](int x) { return L::kAliasP ? tS(x) : tmem + 384u + 64u * x; };
  // Ring position of K(R) and V(R), R counting tiles over all units.
  auto k_block = [](int R, int c) { return (R * L::kEach + c) % kBlocks; };
  auto v_block = [](int R, int c) { return (R * L::kEach + NS + 1 + c) % kBlocks; };

  if (warp == 0) {
    // ---------------- TMA producer (converged warp, one elected lane issues) ----------------
    int units = 0, R = 0, issued_v = 0;
    bool ok = true;
    auto load = [&](uint32_t dst, const CUtensorMap *map, uint32_t full, int col, int head, int row0, int bb) {
      XATTN_DCHECK(col % 8 == 0 && head >= 0 && head < nh && row0 >= 0 && row0 < S && bb >= 0 && bb < a.B && dst >= sQ &&
                       dst + kSubTile <= bar0,
                   a.status);
      tma_load_4d_elect(dst, map, full, col, head, row0, bb);
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_LATENT_UNIT(u);
      if (!warp_wait(q_empty, (units & 1) ^ 1, ctl)) break;        // the unit before has taken its last scores
      mbar_expect_tx_elect(q_full, (hasB ? 2 : 1) * (k_subs + 1) * kSubTile);
      for (int x = 0; x < (hasB ? 2 : 1); ++x) {
        for (int c = 0; c < k_subs; ++c)
          load(sQ + (x * (NS + 1) + c) * kSubTile, &mq, q_full, 64 * c, h, (mA + x) * kTileRows, b);
        load(sQ + (x * (NS + 1) + NS) * kSubTile, &mq, q_full, dn, h, (mA + x) * kTileRows, b);
      }
      ++units;
#pragma unroll 1
      for (int n = 0; n < count; ++n, ++R) {
        const int s = R % kDepth, r0 = n * kTileRows;
        const uint32_t ph = static_cast<uint32_t>((R / kDepth) & 1) ^ 1u;
        // K(R)'s place was V(R - 2)'s (and K's third), or K(R - 3)'s; V(R)'s was K(R - 1)'s, or V(R - 3)'s.
        if (!warp_wait(NS == 2 ? v_empty(s) : k_empty(s), ph, ctl)) { ok = false; break; }
        mbar_expect_tx_elect(k_full(s), (k_subs + 1) * kSubTile);
        for (int c = 0; c < k_subs; ++c) load(sRing + k_block(R, c) * kSubTile, &mkv, k_full(s), 64 * c, h, r0, b);
        load(sRing + k_block(R, NS) * kSubTile, &mrope, k_full(s), 0, 0, r0, b);
        if (NS == 2) {
          if (R > 0) ok = warp_wait(k_empty((R - 1) % kDepth), ((R - 1) / kDepth) & 1, ctl);
        } else {
          ok = warp_wait(v_empty(s), ph, ctl);
        }
        if (!ok) { ++R; break; }                                   // (K(R) is on its way)
        mbar_expect_tx_elect(v_full(s), v_subs * kSubTile);
        for (int c = 0; c < v_subs; ++c) load(sRing + v_block(R, c) * kSubTile, &mkv, v_full(s), dn + 64 * c, h, r0, b);
        issued_v = R + 1;
      }
    }
    // Every copy in flight has landed before the CTA can exit.
    if (units > 0) mbar_drain(q_full, (units - 1) & 1, ctl);
    for (int r = max(R - kDepth, 0); r < R; ++r) mbar_drain(k_full(r % kDepth), (r / kDepth) & 1, ctl);
    for (int r = max(issued_v - kDepth, 0); r < issued_v; ++r) mbar_drain(v_full(r % kDepth), (r / kDepth) & 1, ctl);
  } else if (warp == 1 || warp == 3) {
    // ---------------- MMA issuers: warp 1 for query tile A, warp 3 for tile B ----------------
    // Each waits for and releases every key tile, those its query tile does not use too, so that no wait falls two
    // phases behind (a barrier tells only its last two apart).
    const int x = warp == 1 ? 0 : 1;
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
    const uint32_t idesc_pv0 = idesc_bf16_f32(128, min(dv, 64), false, true),
                   idesc_pv1 = idesc_bf16_f32(128, max(dv - 64, 16), false, true);
    constexpr uint32_t kSubDesc = kSubTile >> 4, kRowStep = (16 * 128) >> 4;
    const uint64_t dQ = smem_desc(sQ, 16, 1024, kSwizzle128) + x * (NS + 1) * kSubDesc;
    const uint64_t dK = smem_desc(sRing, 16, 1024, kSwizzle128);
    const uint64_t dV = smem_desc(sRing, 8192, 1024, kSwizzle128);       // MN-major
    const uint32_t tSx = tS(x), tOx = tO(x), tPx = tP(x);
    auto issue_qk = [&](int R, bool last) {
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < NS; ++c) {
          const uint64_t q = dQ + c * kSubDesc, kd = dK + k_block(R, c) * kSubDesc;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (4 * c + kk < dn_steps) mma_ss(tSx, q + kk * 2, kd + kk * 2, idesc_qk, c + kk > 0 ? 1u : 0u);
        }
        const uint64_t q = dQ + NS * kSubDesc, kd = dK + k_block(R, NS) * kSubDesc;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < dr_steps) mma_ss(tSx, q + kk * 2, kd + kk * 2, idesc_qk, 1u);
        mma_commit(s_full(x));
        mma_commit(k_empty(R % kDepth));
        if (last) mma_commit(q_empty);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int R, bool first) {
      const uint64_t v0 = dV + v_block(R, 0) * kSubDesc, v1 = dV + v_block(R, NS - 1) * kSubDesc;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTileRows / 16; ++kk) {
          mma_ts(tOx, tPx + kk * 8, v0 + kk * kRowStep, idesc_pv0, (!first || kk > 0) ? 1u : 0u);
          if (NS == 2 && dv > 64) mma_ts(tOx + 64, tPx + kk * 8, v1 + kk * kRowStep, idesc_pv1, (!first || kk > 0) ? 1u : 0u);
        }
        mma_commit(o_done(x));
        mma_commit(v_empty(R % kDepth));
      }
      __syncwarp();
    };
    auto landed_k = [&](int R) { return warp_wait(k_full(R % kDepth), (R / kDepth) & 1, ctl); };
    auto landed_v = [&](int R) { return warp_wait(v_full(R % kDepth), (R / kDepth) & 1, ctl); };
    auto pass_tile = [&](int R) -> bool {
      if (!landed_k(R)) return false;
      if (elect_one()) mbar_arrive(k_empty(R % kDepth));
      __syncwarp();
      if (!landed_v(R)) return false;
      if (elect_one()) mbar_arrive(v_empty(R % kDepth));
      __syncwarp();
      return true;
    };
    bool ok = true;
    int units = 0, unitsx = 0, steps = 0;
#pragma unroll 1
    for (int k = 0, R = 0, gx = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_LATENT_UNIT(u);
      const int used = x == 0 ? mA + 1 : (hasB ? mB + 1 : 0);
      if (!warp_wait(q_full, units & 1, ctl)) break;
      if (used > 0) {
        // The unit's first scores: S_X of the unit before has been read; its first P V overwrites O_X, which that unit's
        // epilogue has read.
        ok = landed_k(R) && warp_wait(s_free(x), (gx - 1) & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        issue_qk(R, used == 1);
        if (!warp_wait(o_free(x), (unitsx - 1) & 1, ctl)) break;
#pragma unroll 1
        for (int n = 0; n < used; ++n, ++gx) {
          const bool more = n + 1 < used;
          if constexpr (!L::kAliasP) {
            if (more) {
              if (!warp_wait(s_free(x), gx & 1, ctl) || !landed_k(R + n + 1)) { ok = false; break; }
              tc_fence_after();
              issue_qk(R + n + 1, n + 2 == used);
            }
          }
          if (!landed_v(R + n) || !warp_wait(p_full(x), gx & 1, ctl)) { ok = false; break; }
          tc_fence_after();
          issue_pv(R + n, n == 0);
          if constexpr (L::kAliasP) {
            // P_X(n) lies in S_X's columns: the next scores over them behind its product.
            if (more) {
              if (!landed_k(R + n + 1)) { ok = false; break; }
              tc_fence_after();
              issue_qk(R + n + 1, n + 2 == used);
            }
          }
        }
        if (!ok) break;
        ++unitsx;
      } else {
        if (elect_one()) mbar_arrive(q_empty);
        __syncwarp();
      }
      for (int n = used; ok && n < count; ++n) ok = pass_tile(R + n);
      if (!ok) break;
      R += count;
      ++units;
      steps = gx;
    }
    if (steps > 0) mbar_drain(o_done(x), (steps - 1) & 1, ctl);      // covers every MMA of this issuer
  } else if (warp >= 4) {
    // ---------------- softmax + epilogue: one thread per query row of tile X ----------------
    const int x = (warp - 4) >> 2;          // 0 = tile A, 1 = tile B
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tSx = tS(x) + lane_off, tOx = tO(x) + lane_off, tPx = tP(x) + lane_off;
    const float scale_log2 = a.scale * kLog2e;
    bool ok = true;
#pragma unroll 1
    for (int k = 0, gx = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_LATENT_UNIT(u);
      const int mX = x == 0 ? mA : mB;
      if (x == 1 && !hasB) continue;
      float mrow = -INFINITY, lrow = 0.f;
      // One key step; `masked` selects the diagonal tile's copy, compiled apart from the
      // loop over the other tiles so that their code carries no mask. On the diagonal
      // tile the warp's rows are 32 q .. 32 q + 31 (q = quarter): 32-column chunks below q
      // are wholly visible, chunk q is masked per lane (key column > row), chunks above q
      // are wholly masked (P = 0 without exponentials); q is warp-uniform, so each chunk
      // takes one branch-free path.
      auto step = [&](auto masked, bool first) -> bool {
        constexpr bool kDiag = decltype(masked)::value;
        if (!warp_wait(s_full(x), gx & 1, ctl)) return false;
        tc_fence_after();
        // The whole row of S_X(n) comes into registers with one TMEM read, and the buffer
        // is released at once: S_X(n+1) is computed while this softmax runs.
        uint32_t r[128];
#pragma unroll
        for (int c = 0; c < 128; c += 32) tmem_ld_x32(tSx + c, r + c);
        tmem_wait_ld();
        reg_fence<128>(r);
        tc_fence_before();
        mbar_arrive(s_free(x));
        // The row maximum of the scaled scores: the scaled maximum of the raw scores
        // (scale >= 0) or their scaled minimum (scale < 0); masked columns do not count.
        constexpr float kFill = kNegScale ? INFINITY : -INFINITY;
        float mx4[4] = {kFill, kFill, kFill, kFill};
        auto max_chunk = [&](auto mask_chunk, int c32) {
#pragma unroll
          for (int c = c32; c < c32 + 32; c += 2) {
            float v0 = __uint_as_float(r[c]), v1 = __uint_as_float(r[c + 1]);
            if (decltype(mask_chunk)::value) {
              if (c > row) v0 = kFill;
              if (c + 1 > row) v1 = kFill;
            }
            float &a = mx4[(c >> 1) & 3];
            a = kNegScale ? fmin3(a, v0, v1) : fmax3(a, v0, v1);
          }
        };
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          if (!kDiag || cc < quarter) max_chunk(std::false_type{}, 32 * cc);
          else if (cc == quarter) max_chunk(std::true_type{}, 32 * cc);
        }
        const float mx = (kNegScale ? fmin3(mx4[0], mx4[1], fminf(mx4[2], mx4[3]))
                                    : fmax3(mx4[0], mx4[1], fmaxf(mx4[2], mx4[3]))) * scale_log2;
        // Conditional rescaling: keep the stale max unless some row of the warp grew by
        // more than 2^8; the decision is per warp because TMEM loads/stores are collective.
        const float mnew = fmaxf(mrow, mx);
        const bool rescale = __any_sync(0xffffffffu, mnew > mrow + 8.0f);
        const float m_use = rescale ? mnew : mrow;
        // rescale is warp-uniform, so this is a uniform branch: the common path issues no
        // special-function op here (one would queue behind the other warpgroup's
        // exponentials on the shared unit).
        float alpha = 1.f;
        if (rescale) alpha = ex2_approx(mrow - mnew);
        const float neg_m = -m_use;
        // Exponents, the causal mask on them (-inf -> exact zeros for any scale, 0
        // included), the exponentials, row sums and bf16 P, packed in place into r[0, 64).
        // The first three quarters of P are computed before waiting for the previous PV_X
        // (which still reads P_X), so that product's latency overlaps the exponentials;
        // storing them before the last quarter keeps the register peak at one S row.
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
        auto exp_chunk = [&](auto mask_chunk, int c32) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = c32 + 2 * e;
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(r[c]), __uint_as_float(r[c + 1]), scale_log2, scale_log2,
                  neg_m, neg_m);
            if (decltype(mask_chunk)::value) {
              if (c > row) x0 = -INFINITY;
              if (c + 1 > row) x1 = -INFINITY;
            }
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            const int a = (e & 1) * 2;
            fadd2(ps[a], ps[a + 1], ps[a], ps[a + 1], p0, p1);
            r[c32 / 2 + e] = pack_bf16x2(p0, p1);
          }
        };
        auto chunk = [&](int cc) {
          if (!kDiag || cc < quarter) {
            exp_chunk(std::false_type{}, 32 * cc);
          } else if (cc == quarter) {
            exp_chunk(std::true_type{}, 32 * cc);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) r[16 * cc + e] = 0u;
          }
        };
        chunk(0);
        chunk(1);
        chunk(2);
        if (!warp_wait(o_done(x), (gx - 1) & 1, ctl)) return false;
        tc_fence_after();
        tmem_st_x32(tPx, r);
        tmem_st_x16(tPx + 32, r + 32);
        chunk(3);
        tmem_st_x16(tPx + 48, r + 48);
        if (rescale && !first) {
#pragma unroll 1
          for (int c = 0; c < dv; c += 16) {
            uint32_t ov[16];
            tmem_ld_x16(tOx + c, ov);
            tmem_wait_ld();
            reg_fence<16>(ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st_x16(tOx + c, ov);
          }
        }
        lrow = lrow * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
        mrow = m_use;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(x));
        return true;
      };
#pragma unroll 1
      for (int n = 0; n < mX; ++n, ++gx) {
        if (!step(std::false_type{}, n == 0)) { ok = false; break; }
      }
      if (ok) {
        if (!step(std::true_type{}, mX == 0)) ok = false;
        ++gx;
      }
      if (!ok) break;
      // Epilogue: O / l in bf16 and the LSE; then O_X is free for the next unit.
      if (!warp_wait(o_done(x), (gx - 1) & 1, ctl)) break;
      tc_fence_after();
      const int i = mX * kTileRows + row;
      const float inv = 1.f / lrow;
      const size_t at = (static_cast<size_t>(b) * S + i) * nh + h;
      XATTN_DCHECK(i >= S || at < static_cast<size_t>(a.B) * S * nh, a.status);
#pragma unroll 1
      for (int c = 0; c < dv; c += 16) {
        uint32_t ov[16];
        tmem_ld_x16(tOx + c, ov);
        tmem_wait_ld();
        reg_fence<16>(ov);
        if (i < S) {
          auto pair = [&](int e) { return pack_bf16x2(__uint_as_float(ov[e]) * inv, __uint_as_float(ov[e + 1]) * inv); };
          store_32(a.o + at * dv + c, pair(0), pair(2), pair(4), pair(6), pair(8), pair(10), pair(12), pair(14));
        }
        __syncwarp();
      }
      if (i < S) a.lse[at] = (mrow + __log2f(lrow)) * kLn2;
      tc_fence_before();
      mbar_arrive(o_free(x));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
#undef XATTN_LATENT_UNIT

template <int NS, bool kFull, bool kNegScale>
cudaError_t launch_latent_fwd_ns(const LatentMaps &maps, const LatentArgs &a, int sms, cudaStream_t stream) {
  using L = LatentFwdLayout<NS>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t err = allow_smem(latent_fwd_kernel<NS, kFull, kNegScale>, L::kDynBytes, allowed);
  if (err != cudaSuccess) return err;
  const int num_m = (a.S + kTileRows - 1) / kTileRows;
  const long long units = static_cast<long long>(a.B) * a.nh * ((num_m + 1) / 2);
  return launch_pdl(latent_fwd_kernel<NS, kFull, kNegScale>, static_cast<unsigned>(units < sms ? units : sms), kFwdThreads,
                    L::kDynBytes, stream, maps.q, maps.kv, maps.rope, a);
}

}  // namespace

cudaError_t launch_latent_fwd(const LatentMaps &maps, const LatentArgs &a, int sms, cudaStream_t stream) {
  // One sub-tile that is full: products without conditions (B8 S1024, 12 heads of 64 + 32 / 64: 27.5 -> 24.5 us, B4 S4096, 16
  // heads 144 -> 133). With two the
  // same is slower: S and P V of one query tile then go out in a row and keep the other's waiting (B4 S4093, 16 heads of 128 + 64 /
  // 128: 250 -> 278 us).
  if (a.dn == 64 && a.dv == 64 && a.scale >= 0.f) return launch_latent_fwd_ns<1, true, false>(maps, a, sms, stream);
  if (a.dn <= 64 && a.dv <= 64)
    return a.scale < 0.f ? launch_latent_fwd_ns<1, false, true>(maps, a, sms, stream)
                         : launch_latent_fwd_ns<1, false, false>(maps, a, sms, stream);
  return a.scale < 0.f ? launch_latent_fwd_ns<2, false, true>(maps, a, sms, stream)
                       : launch_latent_fwd_ns<2, false, false>(maps, a, sms, stream);
}

}  // namespace xattn
