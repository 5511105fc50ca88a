// Latent attention in its expanded form, backward, on sm_103a tensor cores: the scores are recomputed, D = rowsum(dO * O)
// stands for the softmax Jacobian, and the gradient of the shared part k_rope is the sum over the heads.
//   P = exp(scale S - LSE), dS = P (dO V^T - D);
//   dV = P^T dO, dK = scale dS^T Q (its first dn numbers to dkv, the others summed over the heads to dk_rope), dQ = scale dS K.
//
// Three kernels:
//   1. latent_dq_kernel (query-stationary): S and dP, dQ += dS K in TMEM over the key tiles. It also makes -LSE log2 e and -D of
//      its rows and leaves them, transposed to [B, nh, S_pad] (a tile's 64 of a head are one contiguous copy), for the next.
//   2. latent_dkv_kernel (key-stationary): a unit is (batch, head, 128 keys); dV [128, dv] and dK [128, dn + dr] stay in TMEM,
//      320 of its 512 columns, so queries come in tiles of 64 and three 64-column places hold the scores: S^T(t) in place
//      t % 2 (P^T over it), dP^T(t) in the third (dS^T over it). S^T is issued two tiles ahead, so it runs while the warps
//      work on P and dS. A score product of 64 columns takes 48 cycles a K step where its arithmetic is 32 (shared memory
//      feeds 128 + 64 rows); with 128 columns the places would not fit. Per 64 queries 576 (S) + 384 (dP) + 256 (dV) + 384 (dK).
//      S and dP are made twice: dQ [., dn + dr] does not fit beside dV and dK, and summed with atomics it would not be
//      reproducible.
//   3. latent_rope_kernel: k_rope's gradient from the heads' fp32 parts, in order.
// Every output is bit-for-bit reproducible. Roundings: P and dS to bf16, Q's, K's and dO's type, before their products; dS is
// made of the unrounded P. B2 S4001, 16 heads of 128 + 64 / 128: dQ 181 us, 1445 TFLOP/s of its products (73 % of the measured
// peak; tensor cores), dK/dV 273 us, 1203 (61 %; the shared-memory reads of its products and their
// chain), k_rope 8. B8 S1024, 12 heads of 64 + 32 / 64: 41, 56 and 5 us (units' starts and ends, the P / dS chain).
#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kBwdThreads = 384;                       // 12 warps
constexpr int kQRows = 64;                             // queries of a tile (dkv)
constexpr uint32_t kKeySub = kTileRows * 128;          // 64 columns of 128 rows
constexpr uint32_t kQuerySub = kQRows * 128;           // 64 columns of 64 rows

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl &ctl) {
  const bool ok = mbar_wait(bar, parity, ctl);
  return __all_sync(0xffffffffu, ok);
}

// NS: sub-tiles of dn, and of dv, that there is room for (dn, dv <= 64 NS). kFull: they are full (dn = dv = 64 NS), so that the
// products' steps have no conditions (backward of B8 S1024, 12 heads of 64 + 32 / 64: 101 -> 99 us, B4 S4096,
// 16 heads 646 -> 632; of 128 + 64 / 128 at B4 S4093 940 -> 936).

// dQ: a unit is (batch, head, 128 queries). Q stays in shared memory and dO in TMEM (the A operand of dP), which leaves room
// for three stages of K: K(n) is needed from S(n) to dQ(n), and with two the next scores waited for it. V has one stage: only
// dP(n) reads it.
template <int NS>
struct LatentDqLayout {
  static constexpr int kStages = 3;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + (NS + 1) * kKeySub;
  static constexpr uint32_t kV = kK + kStages * (NS + 1) * kKeySub;
  static constexpr uint32_t kBars = kV + NS * kKeySub;
  static constexpr int kNumBars = 2 * kStages + 13;
  static constexpr uint32_t kRows = (kBars + 8 * kNumBars + 15) / 16 * 16;   // -LSE log2 e and -D
  static constexpr uint32_t kMisc = kRows + kTileRows * 8;
  static constexpr uint32_t kUsed = kMisc + 32;
  static constexpr uint32_t kDynBytes = kUsed + 1024 > 116 * 1024 ? kUsed + 1024 : 116 * 1024;   // one CTA an SM (TMEM)
  static_assert(kDynBytes <= 227 * 1024, "exceeds the opt-in shared memory of one CTA");
};

// Warps: 0 TMA; 1 MMA issuer and TMEM owner; 2-3 the rows' numbers; 4-7 and 8-11 P and dS, a query row a thread, 64 key columns
// a group.
// TMEM: S [0, 128) | dP [128, 256), dS bf16 over [128, 160) and [192, 224) | dO bf16 [256, 320) | dQ [320, 512), its part for
// k_rope from 448.
template <int NS, bool kFull>
__global__ void __maxnreg__(168)
    latent_dq_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkv,
                     const __grid_constant__ CUtensorMap mrope, const LatentArgs a) {
  using L = LatentDqLayout<NS>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t latent_dq_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(latent_dq_smem) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int S = a.S, nh = a.nh, dn = kFull ? 64 * NS : a.dn, dr = a.dr, dv = kFull ? 64 * NS : a.dv;
  const int dn_steps = dn / 16, dr_steps = dr / 16, dv_steps = dv / 16;
  const int k_subs = (dn + 63) / 64, v_subs = (dv + 63) / 64;
  const int num_m = (S + kTileRows - 1) / kTileRows, BH = a.B * nh, num_units = num_m * BH;
  // Units, most key tiles first; CTA c of G takes unit k G + c in even rounds and k G + G - 1 - c in odd ones.
  auto unit_at = [&](int k) {
    const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
    return k * G + ((k & 1) ? G - 1 - c : c);
  };
#define XATTN_DQ_UNIT(u)                                             \
  const int m = num_m - 1 - (u) / BH, bh = (u) % BH;                 \
  const int b = bh / nh, h = bh - b * nh, T = m + 1; /* key tiles */ \
  (void)b;                                                           \
  (void)h
  const uint32_t sQ = smem_u32(smem + L::kQ), sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV),
                 bar0 = smem_u32(smem + L::kBars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto k_full = [&](int s) { return bar(s); };
  auto k_empty = [&](int s) { return bar(kStages + s); };
  constexpr int kB = 2 * kStages;
  const uint32_t v_full = bar(kB), v_empty = bar(kB + 1), q_full = bar(kB + 2), s_full = bar(kB + 3), dp_full = bar(kB + 4),
                 dq_done = bar(kB + 5), q_empty = bar(kB + 6), s_free = bar(kB + 7), ds_full = bar(kB + 8), do_full = bar(kB + 9),
                 rows_empty = bar(kB + 10), rows_first = bar(kB + 11), rows_full = bar(kB + 12);
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 16);
  const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar(i), i == kB + 12 ? 64 : (i >= kB + 7 ? 256 : 1));
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
  const uint32_t tS = tmem, tdP = tmem + 128, tdO = tmem + 256, tdQ = tmem + 320, tdQr = tmem + 448;

  // -LSE log2 e and -D of a unit's rows r0 .. r0 + count - 1, by a warp, 8 NS lanes a row of o and dO. (A kernel of its own
  // for them took 10 us of B8 S1024, 12 heads of 64 + 32 / 64; by the threads whose rows they are a unit began 2 us later.)
  auto row_numbers = [&](int u, int r0, int count) {
    XATTN_DQ_UNIT(u);
    (void)T;
    constexpr int kLanes = 8 * NS, kAtOnce = 32 / kLanes;
    const int part = lane % kLanes;
    float2 *rows = reinterpret_cast<float2 *>(smem + L::kRows) + r0;
    constexpr int kOnce = 8;                                          // rows that kLanes lanes have in flight
#pragma unroll 1
    for (int from = lane / kLanes; from < count; from += kAtOnce * kOnce) {
      uint4 x[kOnce], y[kOnce];
      float lse[kOnce];
#pragma unroll
      for (int e = 0; e < kOnce; ++e) {
        const int at = from + kAtOnce * e, ig = m * kTileRows + r0 + at;
        const size_t row = (static_cast<size_t>(b) * S + ig) * nh + h;
        x[e] = y[e] = make_uint4(0u, 0u, 0u, 0u);
        lse[e] = INFINITY;                                            // rows behind the last get a weight of 0
        if (ig >= S || at >= count) continue;
        lse[e] = a.lse[row];
        if (8 * part < dv) {
          x[e] = __ldg(reinterpret_cast<const uint4 *>(a.o + row * dv + 8 * part));
          y[e] = __ldg(reinterpret_cast<const uint4 *>(a.dO + row * dv + 8 * part));
        }
      }
#pragma unroll
      for (int e = 0; e < kOnce; ++e) {
        float dot = 0.f;
        auto add = [&](uint32_t v, uint32_t w) {
          dot = fmaf(bf16lo_to_f32(v), bf16lo_to_f32(w), dot);
          dot = fmaf(bf16hi_to_f32(v), bf16hi_to_f32(w), dot);
        };
        add(x[e].x, y[e].x), add(x[e].y, y[e].y), add(x[e].z, y[e].z), add(x[e].w, y[e].w);
#pragma unroll
        for (int off = kLanes / 2; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (part == 0 && from + kAtOnce * e < count) rows[from + kAtOnce * e] = make_float2(-lse[e] * kLog2e, -dot);
      }
    }
    __syncwarp();
    for (int r = lane; r < count; r += 32) {
      const size_t at = static_cast<size_t>(bh) * padded_rows(S) + m * kTileRows + r0 + r;
      const float2 v = rows[r];
      a.nlse[at] = v.x;
      a.nD[at] = v.y;
    }
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    bool ok = true;
    int units = 0, issued_k = 0, issued_v = 0;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_DQ_UNIT(u);
      auto load = [&](uint32_t dst, const CUtensorMap *map, uint32_t full, int col, int head, int row0) {
        XATTN_DCHECK(col % 8 == 0 && head >= 0 && head < nh && row0 >= 0 && row0 < S && dst >= sQ && dst + kKeySub <= bar0, a.status);
        tma_load_4d_elect(dst, map, full, col, head, row0, b);
      };
      // The unit's first K before its Q: a stage is free sooner.
      for (int n = 0; n < T; ++n) {
        const int s = issued_k % kStages;
        if (!warp_wait(k_empty(s), ((issued_k / kStages) & 1) ^ 1, ctl)) { ok = false; break; }
        mbar_expect_tx_elect(k_full(s), (k_subs + 1) * kKeySub);
        const uint32_t dk = sK + s * (NS + 1) * kKeySub;
        for (int c = 0; c < k_subs; ++c) load(dk + c * kKeySub, &mkv, k_full(s), 64 * c, h, n * kTileRows);
        load(dk + NS * kKeySub, &mrope, k_full(s), 0, 0, n * kTileRows);
        ++issued_k;
        if (n == 0) {
          if (!warp_wait(q_empty, (units & 1) ^ 1, ctl)) { ok = false; break; }
          mbar_expect_tx_elect(q_full, (k_subs + 1) * kKeySub);
          for (int c = 0; c < k_subs; ++c) load(sQ + c * kKeySub, &mq, q_full, 64 * c, h, m * kTileRows);
          load(sQ + NS * kKeySub, &mq, q_full, dn, h, m * kTileRows);
          ++units;
        }
        if (!warp_wait(v_empty, (issued_v & 1) ^ 1, ctl)) { ok = false; break; }
        mbar_expect_tx_elect(v_full, v_subs * kKeySub);
        for (int c = 0; c < v_subs; ++c) load(sV + c * kKeySub, &mkv, v_full, dn + 64 * c, h, n * kTileRows);
        ++issued_v;
      }
    }
    // Every copy in flight has landed before the CTA can exit.
    if (units > 0) mbar_drain(q_full, (units - 1) & 1, ctl);
    for (int n = max(issued_k - kStages, 0); n < issued_k; ++n) mbar_drain(k_full(n % kStages), (n / kStages) & 1, ctl);
    if (issued_v > 0) mbar_drain(v_full, (issued_v - 1) & 1, ctl);
  } else if (warp == 1) {
    // ---------------- MMA issuer: S(n + 1) before dQ(n), dP(n + 1) behind it (dS(n) lies in dP's place) ----------------
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
    const uint32_t idesc_dq = idesc_bf16_f32(128, dn, false, true), idesc_dr = idesc_bf16_f32(128, dr, false, true);
    constexpr uint32_t kSubDesc = kKeySub >> 4;
    const uint64_t dQ = smem_desc(sQ, 16, 1024, kSwizzle128);
    const uint64_t dK = smem_desc(sK, 16, 1024, kSwizzle128), dV = smem_desc(sV, 16, 1024, kSwizzle128);
    const uint64_t dKt = smem_desc(sK, kKeySub, 1024, kSwizzle128);       // MN-major: 64 columns a sub-tile
    // (t counts the tiles of all units.)
    auto scores = [&](int t, bool last) -> bool {
      const int s = t % kStages;
      if (!warp_wait(k_full(s), (t / kStages) & 1, ctl) || !warp_wait(s_free, (t & 1) ^ 1, ctl)) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t kd = dK + s * (NS + 1) * kSubDesc;
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (4 * c + kk < dn_steps) mma_ss(tS, dQ + c * kSubDesc + kk * 2, kd + c * kSubDesc + kk * 2, idesc_s, c + kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < dr_steps) mma_ss(tS, dQ + NS * kSubDesc + kk * 2, kd + NS * kSubDesc + kk * 2, idesc_s, 1u);
        mma_commit(s_full);
        if (last) mma_commit(q_empty);
      }
      __syncwarp();
      return true;
    };
    auto issue_dp = [&](int t) -> bool {
      if (!warp_wait(v_full, t & 1, ctl)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (4 * c + kk < dv_steps) mma_ts(tdP, tdO + 32 * c + 8 * kk, dV + c * kSubDesc + kk * 2, idesc_s, c + kk > 0 ? 1u : 0u);
        mma_commit(dp_full);
        mma_commit(v_empty);
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    int units = 0, t = 0;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_DQ_UNIT(u);
      (void)bh;
      ok = warp_wait(q_full, units & 1, ctl) && scores(t, T == 1) && warp_wait(do_full, units & 1, ctl) && issue_dp(t);
#pragma unroll 1
      for (int n = 0; ok && n < T; ++n, ++t) {
        const int s = t % kStages;
        const bool more = n + 1 < T;
        // (dS of the unit's first tile comes from threads that have read the dQ before: it may be overwritten.)
        ok = (!more || scores(t + 1, n + 2 == T)) && warp_wait(ds_full, t & 1, ctl);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {                                          // dQ += dS K_n
          const uint64_t kd = dKt + s * (NS + 1) * kSubDesc;
#pragma unroll
          for (int kk = 0; kk < kTileRows / 16; ++kk) {
            const uint32_t ds = tdP + (kk / 4) * 64 + (kk % 4) * 8;
            mma_ts(tdQ, ds, kd + kk * 128, idesc_dq, (n > 0 || kk > 0) ? 1u : 0u);
            mma_ts(tdQr, ds, kd + NS * kSubDesc + kk * 128, idesc_dr, (n > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(k_empty(s));
          if (!more) mma_commit(dq_done);
        }
        __syncwarp();
        ok = !more || issue_dp(t + 1);
      }
      if (ok) ++units;
    }
    __syncwarp();
    if (units > 0) mbar_drain(dq_done, (units - 1) & 1, ctl);
  } else if (warp < 4) {
    // ---------------- The rows' numbers, a unit ahead ----------------
#pragma unroll 1
    for (int k = 1;; ++k) {
      const int u = unit_at(k);
      if (u >= num_units || !warp_wait(rows_empty, (k & 1) ^ 1, ctl)) break;
      row_numbers(u, 64 * (warp - 2), 64);
      mbar_arrive(rows_full);
    }
  } else {
    // ---------------- P and dS: one query row per thread, 64 key columns per group ----------------
    const int g = (warp - 4) >> 2, quarter = warp & 3;
    const int i = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int c0 = 64 * g;                              // first key column of this group
    const float scale_log2 = a.scale * kLog2e;
    float nlse2 = 0.f, nD = 0.f;
    // A unit's dO of this thread's row, 64 columns a group, into TMEM (rows behind the last, and columns behind dv: zeros), and
    // the row's numbers.
    auto begin = [&](int u, int k) -> bool {
      XATTN_DQ_UNIT(u);
      (void)T;
      const int ig = m * kTileRows + i;
      const size_t row = (static_cast<size_t>(b) * S + ig) * nh + h;
      XATTN_DCHECK(ig >= S || row < static_cast<size_t>(a.B) * S * nh, a.status);
      if (NS == 2 || g == 0) {
        uint32_t x[32];
        uint4 *v = reinterpret_cast<uint4 *>(x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = ig < S && c0 + 8 * e < dv ? __ldg(reinterpret_cast<const uint4 *>(a.dO + row * dv + c0 + 8 * e))
                                           : make_uint4(0u, 0u, 0u, 0u);
        tmem_st_x32(tdO + lane_off + 32 * g, x);
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(do_full);
      if (!(k == 0 ? warp_wait(rows_first, 0, ctl) : warp_wait(rows_full, (k & 1) ^ 1, ctl))) return false;
      const float2 r = reinterpret_cast<const float2 *>(smem + L::kRows)[i];
      nlse2 = r.x, nD = r.y;
      mbar_arrive(rows_empty);
      return true;
    };
    int units = 0, t = 0;
    // (The first unit's numbers by these warps: by the two that make them later a short call took 1.5 us more.)
    bool ok = unit_at(0) < num_units;
    if (ok) {
      row_numbers(unit_at(0), 16 * (warp - 4), 16);
      mbar_arrive(rows_first);
      ok = begin(unit_at(0), 0);
    }
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_DQ_UNIT(u);
#pragma unroll 1
      for (int n = 0; n < T; ++n, ++t) {
        if (!warp_wait(s_full, t & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        uint32_t p[64];
        tmem_ld_x32(tS + lane_off + c0, p);
        tmem_ld_x32(tS + lane_off + c0 + 32, p + 32);
        tmem_wait_ld();
        reg_fence<64>(p);
        tc_fence_before();
        mbar_arrive(s_free);
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(p[e]), __uint_as_float(p[e + 1]), scale_log2, scale_log2, nlse2, nlse2);
          p[e] = __float_as_uint(ex2_approx(x0));
          p[e + 1] = __float_as_uint(ex2_approx(x1));
        }
        if (n == m) {                                     // keys behind the query
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (c0 + e > i) p[e] = 0u;
        }
        // dS = P (dP - D), bf16 over the first half of this group's dP.
        if (!warp_wait(dp_full, t & 1, ctl)) { ok = false; break; }
        tc_fence_after();
        uint32_t ds[32];
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint32_t d[32];
          tmem_ld_x32(tdP + lane_off + c0 + 32 * part, d);
          tmem_wait_ld();
          reg_fence<32>(d);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float t0, t1;
            fadd2(t0, t1, __uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]), nD, nD);
            fmul2(t0, t1, t0, t1, __uint_as_float(p[32 * part + 2 * e]), __uint_as_float(p[32 * part + 2 * e + 1]));
            ds[16 * part + e] = pack_bf16x2(t0, t1);
          }
        }
        tmem_st_x32(tdP + lane_off + c0, ds);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(ds_full);
      }

      if (!ok) break;
      // The next unit's dO (its place was read by dP of the last tile), then dq = bf16(scale * sum) while its S and dP are
      // made; group g writes every second 16 columns of the thread's row.
      ok = (unit_at(k + 1) >= num_units || begin(unit_at(k + 1), k + 1)) && warp_wait(dq_done, units & 1, ctl);
      if (!ok) break;
      ++units;
      tc_fence_after();
      const int ig = m * kTileRows + i;
      __nv_bfloat16 *to = a.dq + ((static_cast<size_t>(b) * S + ig) * nh + h) * (dn + dr);
#pragma unroll 1
      for (int c = 16 * g; c < dn + dr; c += 32) {
        uint32_t v[16];
        tmem_ld_x16((c < dn ? tdQ + c : tdQr + (c - dn)) + lane_off, v);
        tmem_wait_ld();
        reg_fence<16>(v);
        if (ig < S) {
          auto pair = [&](int e) { return pack_bf16x2(__uint_as_float(v[e]) * a.scale, __uint_as_float(v[e + 1]) * a.scale); };
          store_32(to + c, pair(0), pair(2), pair(4), pair(6), pair(8), pair(10), pair(12), pair(14));
        }
        __syncwarp();
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
#undef XATTN_DQ_UNIT

template <int NS>
struct DkvLayout {
  static constexpr int kStages = NS == 1 ? 6 : 3;                    // (NS = 1 with three: B4 S4096, 16 heads 661 us for 632)
  static constexpr uint32_t kK = 0;                                  // NS sub-tiles and the shared part
  static constexpr uint32_t kV = kK + (NS + 1) * kKeySub;
  static constexpr uint32_t kQ = kV + NS * kKeySub;                  // stages of Q (NS + 1 sub-tiles)
  static constexpr uint32_t kdO = kQ + kStages * (NS + 1) * kQuerySub;
  static constexpr uint32_t kRows = kdO + kStages * NS * kQuerySub;  // stages of -LSE log2 e and -D
  static constexpr uint32_t kBars = kRows + kStages * 2 * kQRows * 4;
  static constexpr int kPlaces = NS == 1 ? 2 : 1;                    // of dP^T and dS^T
  static constexpr int kIssuers = NS == 1 ? 2 : 1;
  static constexpr int kNumBars = 2 * kStages + 16;
  static constexpr uint32_t kMisc = (kBars + 8 * kNumBars + 15) / 16 * 16;
  static constexpr uint32_t kUsed = kMisc + 32;
  static constexpr uint32_t kDynBytes = kUsed + 1024 > 116 * 1024 ? kUsed + 1024 : 116 * 1024;   // one CTA an SM (TMEM)
  static_assert(kDynBytes <= 227 * 1024, "exceeds the opt-in shared memory of one CTA");
};

// Warps: 0 TMA; 1 MMA issuer and TMEM owner (NS = 1: 3 another issuer); 4-7 P^T; 8-11 dS^T; a thread is a key row.
// TMEM (columns): dV 64 NS | dK 64 NS, its shared part 64 | two places of S^T, 64 each | one (NS = 1: two) of dP^T |
// NS = 1: two of P^T, 32 each.
template <int NS, bool kFull>
__global__ void __maxnreg__(168)
    latent_dkv_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mkv,
                      const __grid_constant__ CUtensorMap mrope, const __grid_constant__ CUtensorMap mdo, const LatentArgs a) {
  using L = DkvLayout<NS>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t latent_dkv_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(latent_dkv_smem) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int S = a.S, nh = a.nh, dn = kFull ? 64 * NS : a.dn, dr = a.dr, dv = kFull ? 64 * NS : a.dv;
  const int dn_steps = dn / 16, dr_steps = dr / 16, dv_steps = dv / 16;
  const int k_subs = (dn + 63) / 64, v_subs = (dv + 63) / 64;
  const int num_n = (S + kTileRows - 1) / kTileRows, num_q = (S + kQRows - 1) / kQRows, BH = a.B * nh;
  const int S_pad = padded_rows(S);
  // Units, most query tiles first; CTA c of G takes unit k G + c in even rounds and k G + G - 1 - c in odd ones.
  const int num_units = num_n * BH, G = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  auto unit_at = [G, cta](int k) { return k * G + ((k & 1) ? G - 1 - cta : cta); };
#define XATTN_DKV_UNIT(u)                                          \
  const int n = (u) / BH, bh = (u) - n * BH;                       \
  const int b = bh / nh, h = bh - b * nh;                          \
  const int m0 = 2 * n, T = num_q - m0; /* query tiles */          \
  (void)b;                                                         \
  (void)h

  const uint32_t sK = smem_u32(smem + L::kK), sV = smem_u32(smem + L::kV), sQ = smem_u32(smem + L::kQ),
                 sdO = smem_u32(smem + L::kdO), sRows = smem_u32(smem + L::kRows), bar0 = smem_u32(smem + L::kBars);
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto q_full = [&](int s) { return bar(s); };                       // Q, dO and the rows' numbers of a tile
  auto q_empty = [&](int s) { return bar(kStages + s); };
  constexpr int kB = 2 * kStages;
  const uint32_t k_full = bar(kB), v_full = bar(kB + 1), k_empty = bar(kB + 2), v_empty = bar(kB + 3), acc_done = bar(kB + 4),
                 acc_free = bar(kB + 5);
  auto s_full = [&](int x) { return bar(kB + 6 + x); };
  auto p_full = [&](int x) { return bar(kB + 8 + x); };
  auto s_read = [&](int x) { return bar(kB + 14 + x); };             // by the dS warps: its place may be overwritten
  // dP^T's (and dS^T's) place and its phase, of tile g.
  constexpr int kPlaces = L::kPlaces;
  auto dp_full = [&](int g) { return bar(kB + 10 + g % kPlaces); };
  auto ds_full = [&](int g) { return bar(kB + 12 + g % kPlaces); };
  auto dp_phase = [](int g) { return static_cast<uint32_t>((g / kPlaces) & 1); };
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + L::kMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 16);
  const WaitCtl ctl{abort_flag, a.status, a.timeout_ns};

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), L::kIssuers);
    }
    mbar_init(k_full, 1);
    mbar_init(v_full, 1);
    mbar_init(k_empty, 1);
    mbar_init(v_empty, 1);
    mbar_init(acc_done, L::kIssuers);
    mbar_init(acc_free, 256);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kB + 10 + x), 1);
      mbar_init(bar(kB + 12 + x), 128);
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 128);
      mbar_init(s_read(x), 128);
    }
    fence_mbar_init();
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mkv);
    tma_prefetch_desc(&mrope);
    tma_prefetch_desc(&mdo);
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
  constexpr uint32_t kAcc = 64 * NS;                                  // columns of dV, and of dK
  const uint32_t tdV = tmem, tdK = tmem + kAcc, tdKr = tmem + 2 * kAcc;
  auto tS = [&](int x) { return tmem + 2 * kAcc + 64u + 64u * x; };
  auto tP = [&](int x) { return NS == 1 ? tmem + 448u + 32u * x : tS(x); };      // bf16; NS = 2: over S^T
  auto tdP = [&](int g) { return tmem + 2 * kAcc + 192u + 64u * (g % kPlaces); };

  if (warp == 0) {
    // ---------------- TMA producer (converged warp, one elected lane issues) ----------------
    auto load = [&](uint32_t dst, const CUtensorMap *map, uint32_t full, int col, int head, int row0, int bb) {
      XATTN_DCHECK(col % 8 == 0 && head >= 0 && head < nh && row0 >= 0 && row0 < S && bb >= 0 && bb < a.B && dst >= sK &&
                       dst < sRows,
                   a.status);
      tma_load_4d_elect(dst, map, full, col, head, row0, bb);
    };
    int g = 0, units = 0, units_k = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_DKV_UNIT(u);
      const size_t rows = static_cast<size_t>(bh) * S_pad;
      auto load_tile = [&](int t) -> bool {
        const int s = g % kStages, q0 = (m0 + t) * kQRows;
        if (!warp_wait(q_empty(s), ((g / kStages) & 1) ^ 1, ctl)) return false;
        mbar_expect_tx_elect(q_full(s), (k_subs + 1 + v_subs) * kQuerySub + 2 * kQRows * 4);
        const uint32_t dq = sQ + s * (NS + 1) * kQuerySub, ddo = sdO + s * NS * kQuerySub, dr0 = sRows + s * 2 * kQRows * 4;
        for (int c = 0; c < k_subs; ++c) load(dq + c * kQuerySub, &mq, q_full(s), 64 * c, h, q0, b);
        load(dq + NS * kQuerySub, &mq, q_full(s), dn, h, q0, b);
        for (int c = 0; c < v_subs; ++c) load(ddo + c * kQuerySub, &mdo, q_full(s), 64 * c, h, q0, b);
        XATTN_DCHECK(q0 + kQRows <= S_pad, a.status);
        bulk_load_elect(dr0, a.nlse + rows + q0, kQRows * 4, q_full(s));
        bulk_load_elect(dr0 + kQRows * 4, a.nD + rows + q0, kQRows * 4, q_full(s));
        ++g;
        return true;
      };
      // In the order in which the unit before frees the places: K's with its last S^T, V's with its last dP^T (before its sums
      // are written), a stage with each tile.
      ok = load_tile(0) && warp_wait(k_empty, (units & 1) ^ 1, ctl);
      if (!ok) break;
      mbar_expect_tx_elect(k_full, (k_subs + 1) * kKeySub);
      for (int c = 0; c < k_subs; ++c) load(sK + c * kKeySub, &mkv, k_full, 64 * c, h, n * kTileRows, b);
      load(sK + NS * kKeySub, &mrope, k_full, 0, 0, n * kTileRows, b);
      ++units_k;
      ok = (T < 2 || load_tile(1)) && warp_wait(v_empty, (units & 1) ^ 1, ctl);
      if (!ok) break;
      mbar_expect_tx_elect(v_full, v_subs * kKeySub);
      for (int c = 0; c < v_subs; ++c) load(sV + c * kKeySub, &mkv, v_full, dn + 64 * c, h, n * kTileRows, b);
      ++units;
      for (int t = 2; ok && t < T; ++t) ok = load_tile(t);
      // The next unit's K and V into L2: they are fetched when this one's products have ended, with nothing to do meanwhile.
      const int u1 = unit_at(k + 1);
      if (ok && u1 < num_units) {
        const int n1 = u1 / BH, bh1 = u1 - n1 * BH, b1 = bh1 / nh, h1 = bh1 - b1 * nh;
        for (int c = 0; c < k_subs; ++c) tma_prefetch_4d_elect(&mkv, 64 * c, h1, n1 * kTileRows, b1);
        for (int c = 0; c < v_subs; ++c) tma_prefetch_4d_elect(&mkv, dn + 64 * c, h1, n1 * kTileRows, b1);
      }
    }
    // Every copy in flight has landed before the CTA can exit.
    if (units_k > 0) mbar_drain(k_full, (units_k - 1) & 1, ctl);
    if (units > 0) mbar_drain(v_full, (units - 1) & 1, ctl);
    for (int r = max(g - kStages, 0); r < g; ++r) mbar_drain(q_full(r % kStages), (r / kStages) & 1, ctl);
  } else if (warp == 1 || (L::kIssuers == 2 && warp == 3)) {
    // ---------------- MMA issuers: of S^T and dV (p_side), and of dP^T and dK (s_side) ----------------
    // NS = 2: one thread, so one order: dV(t), dK(t), dP^T(t + 1), S^T(t + 2). dK -> dP^T -> dS^T -> dK is the longest chain (dP^T and
    // dS^T have one place), and S^T, dV fill the time that the dS warps take. (With two issuers the pipe took S^T between dK
    // and dP^T: 2430 cycles a tile, 2200 so.)
    // NS = 1: the products are short and their issue is what takes time (1750 cycles a tile by one thread), so two threads (B4 S4096,
    // 16 heads of 64 + 32 / 64: 695 -> 632 us);
    // dP^T has two places and need not wait for dK.
    const bool p_side = warp == 1, s_side = L::kIssuers == 1 || warp == 3;
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kQRows, false, false);
    const uint32_t idesc_dv = idesc_bf16_f32(128, dv, false, true), idesc_dk = idesc_bf16_f32(128, dn, false, true),
                   idesc_dr = idesc_bf16_f32(128, dr, false, true);
    const uint64_t dK = smem_desc(sK, 16, 1024, kSwizzle128), dQ = smem_desc(sQ, 16, 1024, kSwizzle128);
    const uint64_t dV = smem_desc(sV, 16, 1024, kSwizzle128), ddO = smem_desc(sdO, 16, 1024, kSwizzle128);
    const uint64_t dQt = smem_desc(sQ, kQuerySub, 1024, kSwizzle128);    // MN-major: 64 columns a sub-tile
    const uint64_t ddOt = smem_desc(sdO, kQuerySub, 1024, kSwizzle128);
    auto landed = [&](int g) { return warp_wait(q_full(g % kStages), (g / kStages) & 1, ctl); };
    // S^T of tile g (over all units); its place's P^T and the dS warps' reading of it lie two tiles back.
    // NS = 2: P^T was written after that reading; NS = 1 waits for it here.
    auto issue_s = [&](int g, bool last) {
      if (NS == 1 && g >= 2 && !warp_wait(s_read(g & 1), ((g - 2) >> 1) & 1, ctl)) return false;
      if (NS == 1) tc_fence_after();
      if (elect_one()) {
        const uint64_t q = dQ + (g % kStages) * (NS + 1) * (kQuerySub >> 4);
        const uint32_t d = tS(g & 1);
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (4 * c + kk < dn_steps)
              mma_ss(d, dK + c * (kKeySub >> 4) + kk * 2, q + c * (kQuerySub >> 4) + kk * 2, idesc_s, c + kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < dr_steps) mma_ss(d, dK + NS * (kKeySub >> 4) + kk * 2, q + NS * (kQuerySub >> 4) + kk * 2, idesc_s, 1u);
        mma_commit(s_full(g & 1));
        if (last) mma_commit(k_empty);
      }
      __syncwarp();
      return true;
    };
    auto issue_dp = [&](int g, bool last) {

      if (elect_one()) {
        const uint64_t o = ddO + (g % kStages) * NS * (kQuerySub >> 4);
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            if (4 * c + kk < dv_steps)
              mma_ss(tdP(g), dV + c * (kKeySub >> 4) + kk * 2, o + c * (kQuerySub >> 4) + kk * 2, idesc_s, c + kk > 0 ? 1u : 0u);
        mma_commit(dp_full(g));
        if (last) mma_commit(v_empty);
      }
      __syncwarp();
    };
    bool ok = true;
    int units = 0, g = 0;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_DKV_UNIT(u);
      if (!landed(g)) break;
      if (p_side) {
        if (!warp_wait(k_full, units & 1, ctl)) break;
        tc_fence_after();
        if (!issue_s(g, T == 1)) break;
      }
      if (s_side) {
        if (!warp_wait(v_full, units & 1, ctl)) break;
        tc_fence_after();
        issue_dp(g, T == 1);
      }
      if (T > 1) {
        if (!landed(g + 1)) break;
        tc_fence_after();
        if (p_side && !issue_s(g + 1, T == 2)) break;
      }
      // The first dV and dK overwrite the accumulators, which the unit before has read.
      if (!warp_wait(acc_free, (units & 1) ^ 1, ctl)) break;
#pragma unroll 1
      for (int t = 0; t < T; ++t, ++g) {
        const int s = g % kStages;
        const bool last = t + 1 == T;
        if (kPlaces == 2 && s_side && !last) issue_dp(g + 1, t + 2 == T);   // (its place's dK went before; the tile has landed)
        if (p_side) {
          if (!warp_wait(p_full(g & 1), (g >> 1) & 1, ctl)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t o = ddOt + s * NS * (kQuerySub >> 4);
#pragma unroll
            for (int kk = 0; kk < kQRows / 16; ++kk)
              mma_ts(tdV, tP(g & 1) + kk * 8, o + kk * 128, idesc_dv, (t > 0 || kk > 0) ? 1u : 0u);
            if (L::kIssuers == 2) {
              mma_commit(q_empty(s));
              if (last) mma_commit(acc_done);
            }
          }
          __syncwarp();
        }
        if (s_side) {
          if (!warp_wait(ds_full(g), dp_phase(g), ctl)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t q = dQt + s * (NS + 1) * (kQuerySub >> 4);
#pragma unroll
            for (int kk = 0; kk < kQRows / 16; ++kk) {
              mma_ts(tdK, tdP(g) + kk * 8, q + kk * 128, idesc_dk, (t > 0 || kk > 0) ? 1u : 0u);
              mma_ts(tdKr, tdP(g) + kk * 8, q + NS * (kQuerySub >> 4) + kk * 128, idesc_dr, (t > 0 || kk > 0) ? 1u : 0u);
            }
            mma_commit(q_empty(s));
            if (last) mma_commit(acc_done);
          }
          __syncwarp();
          if (kPlaces == 1 && !last) issue_dp(g + 1, t + 2 == T);    // (the tile has landed: its S^T went before)
        }
        if (t + 2 < T) {
          if (!landed(g + 2)) { ok = false; break; }
          tc_fence_after();
          if (p_side && !issue_s(g + 2, t + 3 == T)) { ok = false; break; }
        }
      }
      ++units;
    }
    if (ok && units > 0) mbar_drain(acc_done, (units - 1) & 1, ctl);
  } else if (warp >= 4) {
    const bool p_side = warp < 8;
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float scale_log2 = a.scale * kLog2e;
    auto probabilities = [&](uint32_t *s, float4 m) {              // of four queries; m: -LSE log2 e
      float x0, x1, x2, x3;
      ffma2(x0, x1, __uint_as_float(s[0]), __uint_as_float(s[1]), scale_log2, scale_log2, m.x, m.y);
      ffma2(x2, x3, __uint_as_float(s[2]), __uint_as_float(s[3]), scale_log2, scale_log2, m.z, m.w);
      s[0] = __float_as_uint(ex2_approx(x0));
      s[1] = __float_as_uint(ex2_approx(x1));
      s[2] = __float_as_uint(ex2_approx(x2));
      s[3] = __float_as_uint(ex2_approx(x3));
    };
    bool ok = true;
    int units = 0, g = 0;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int u = unit_at(k);
      if (u >= num_units) break;
      XATTN_DKV_UNIT(u);
      if (p_side) {
        // ---------------- P^T = exp2(S^T scale log2 e - LSE log2 e) ----------------
#pragma unroll 1
        for (int t = 0; t < T; ++t, ++g) {
          if (!warp_wait(s_full(g & 1), (g >> 1) & 1, ctl)) { ok = false; break; }
          tc_fence_after();
          const uint32_t at = tS(g & 1) + lane_off;
          uint32_t r[64];
          tmem_ld_x32(at, r);
          tmem_ld_x32(at + 32, r + 32);
          tmem_wait_ld();
          reg_fence<64>(r);
          const float4 *nl = reinterpret_cast<const float4 *>(smem + L::kRows + (g % kStages) * 2 * kQRows * 4);
          // Queries before the key (of the first two tiles) do not see it.
          const int hidden = row - t * kQRows;                     // columns below it
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            probabilities(r + c, nl[c / 4]);
            pk[c / 2] = pack_bf16x2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]));
            pk[c / 2 + 1] = pack_bf16x2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
          }
          if (t < 2) {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              if (2 * c < hidden) pk[c] &= 0xffff0000u;
              if (2 * c + 1 < hidden) pk[c] &= 0x0000ffffu;
            }
            if (NS == 1) {
#pragma unroll
              for (int c = 0; c < 64; ++c) r[c] = c < hidden ? 0u : r[c];
            }
          }
          if (NS == 1) {
            tmem_st_x32(at, r);
            tmem_st_x32(at + 32, r + 32);
          } else {
            if (!warp_wait(s_read(g & 1), (g >> 1) & 1, ctl)) { ok = false; break; }
            tc_fence_after();
          }
          tmem_st_x32(tP(g & 1) + lane_off, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full(g & 1));
        }
      } else {
        // ---------------- dS^T = P^T (dP^T - D) ----------------
#pragma unroll 1
        for (int t = 0; t < T; ++t, ++g) {
          // P in fp32 (from the bf16 numbers dK had one rounding more, 2.9e-3 of its norm for 2.4e-3). NS = 1: the P warps leave
          // it over S^T. NS = 2 has no room for both and takes the exponentials here again, while dP^T is on its way. (NS = 1
          // so: B4 S4096, 16 heads of 64 + 32 / 64 668 us, from the P warps 651.)
          if (!warp_wait(NS == 1 ? p_full(g & 1) : s_full(g & 1), (g >> 1) & 1, ctl)) { ok = false; break; }
          tc_fence_after();
          uint32_t p[64], r[32];
          tmem_ld_x32(tS(g & 1) + lane_off, p);
          tmem_ld_x32(tS(g & 1) + lane_off + 32, p + 32);
          tmem_wait_ld();
          reg_fence<64>(p);
          tc_fence_before();
          mbar_arrive(s_read(g & 1));
          const float4 *nl = reinterpret_cast<const float4 *>(smem + L::kRows + (g % kStages) * 2 * kQRows * 4),
                       *nd = nl + kQRows / 4;
          if (NS == 2) {
#pragma unroll
            for (int c = 0; c < 64; c += 4) probabilities(p + c, nl[c / 4]);
            if (t < 2) {
              const int hidden = row - t * kQRows;
#pragma unroll
              for (int c = 0; c < 64; ++c) p[c] = c < hidden ? 0u : p[c];
            }
          }
          if (!warp_wait(dp_full(g), dp_phase(g), ctl)) { ok = false; break; }
          tc_fence_after();
          const uint32_t at = tdP(g) + lane_off;
#pragma unroll
          for (int half = 0; half < 64; half += 32) {
            tmem_ld_x32(at + half, r);
            tmem_wait_ld();
            reg_fence<32>(r);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const int c = half + e;
              const float4 d = nd[c / 4];
              float x0, x1, x2, x3;
              fadd2(x0, x1, __uint_as_float(r[e]), __uint_as_float(r[e + 1]), d.x, d.y);
              fadd2(x2, x3, __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]), d.z, d.w);
              fmul2(x0, x1, x0, x1, __uint_as_float(p[c]), __uint_as_float(p[c + 1]));
              fmul2(x2, x3, x2, x3, __uint_as_float(p[c + 2]), __uint_as_float(p[c + 3]));
              p[c / 2] = pack_bf16x2(x0, x1);
              p[c / 2 + 1] = pack_bf16x2(x2, x3);
            }
          }
          tmem_st_x32(at, p);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(ds_full(g));
        }
      }
      // The unit's sums: the P warps write dV, the dS warps dK.
      if (!ok || !warp_wait(acc_done, units & 1, ctl)) break;
      tc_fence_after();
      const int j = n * kTileRows + row;
      const size_t tok = (static_cast<size_t>(b) * S + j) * nh + h;
      XATTN_DCHECK(j >= S || tok < static_cast<size_t>(a.B) * S * nh, a.status);
      // 32 columns at once (they may end after 16: the rest is read and dropped).
      auto put = [&](uint32_t from, int cols, float mult, __nv_bfloat16 *to) {
#pragma unroll 1
        for (int c = 0; c < cols; c += 32) {
          uint32_t r[32];
          tmem_ld_x32(from + lane_off + c, r);
          tmem_wait_ld();
          reg_fence<32>(r);
          auto pair = [&](int e) { return pack_bf16x2(__uint_as_float(r[e]) * mult, __uint_as_float(r[e + 1]) * mult); };
          if (j < S) {
            store_32(to + c, pair(0), pair(2), pair(4), pair(6), pair(8), pair(10), pair(12), pair(14));
            if (c + 32 <= cols) store_32(to + c + 16, pair(16), pair(18), pair(20), pair(22), pair(24), pair(26), pair(28), pair(30));
          }
          __syncwarp();
        }
      };
      if (p_side) put(tdV, dv, 1.f, a.dkv + tok * (dn + dv) + dn);
      else put(tdK, dn, a.scale, a.dkv + tok * (dn + dv));
      // This head's part of k_rope's gradient, every second 16 columns a group.
#pragma unroll 1
      for (int c = p_side ? 0 : 16; c < dr; c += 32) {
        uint32_t v[16];
        tmem_ld_x16(tdKr + lane_off + c, v);
        tmem_wait_ld();
        reg_fence<16>(v);
        if (j < S) {
          float *dst = a.rope_parts + tok * dr + c;
          store_32(dst, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
          store_32(dst + 8, v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]);
        }
        __syncwarp();
      }
      tc_fence_before();
      mbar_arrive(acc_free);
      ++units;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}
#undef XATTN_DKV_UNIT

// k_rope's gradient: the heads' parts added in order, four columns a thread.
__global__ void __launch_bounds__(256) latent_rope_kernel(const LatentArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const size_t t = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  const int quads = a.dr / 4;
  const size_t tok = t / quads;
  if (tok >= static_cast<size_t>(a.B) * a.S) return;
  const int c = static_cast<int>(t - tok * quads) * 4;
  const float *from = a.rope_parts + tok * a.nh * a.dr + c;
  float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int h = 0; h < a.nh; ++h) {
    const float4 x = *reinterpret_cast<const float4 *>(from + static_cast<size_t>(h) * a.dr);
    g.x += x.x, g.y += x.y, g.z += x.z, g.w += x.w;
  }
  *reinterpret_cast<uint2 *>(a.dk_rope + tok * a.dr + c) =
      make_uint2(pack_bf16x2(g.x * a.scale, g.y * a.scale), pack_bf16x2(g.z * a.scale, g.w * a.scale));
}

template <int NS, bool kFull>
cudaError_t launch_latent_bwd_ns(const LatentMaps &q64, const LatentMaps &q128, const LatentArgs &a, int sms,
                                 cudaStream_t stream) {
  using LK = DkvLayout<NS>;
  using LQ = LatentDqLayout<NS>;
  static std::atomic<unsigned long long> allowed_k{0}, allowed_q{0};
  cudaError_t err = allow_smem(latent_dkv_kernel<NS, kFull>, LK::kDynBytes, allowed_k);
  if (err == cudaSuccess) err = allow_smem(latent_dq_kernel<NS, kFull>, LQ::kDynBytes, allowed_q);
  if (err != cudaSuccess) return err;
  const long long num_n = (a.S + kTileRows - 1) / kTileRows, units = num_n * a.B * a.nh;
  const unsigned grid = static_cast<unsigned>(units < sms ? units : sms);
  err = launch_pdl(latent_dq_kernel<NS, kFull>, grid, kBwdThreads, LQ::kDynBytes, stream, q128.q, q128.kv, q128.rope, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(latent_dkv_kernel<NS, kFull>, grid, kBwdThreads, LK::kDynBytes, stream, q64.q, q128.kv, q128.rope, q64.dO, a);
}

}  // namespace

size_t latent_bwd_workspace_bytes(const LatentArgs &a) {
  return (2 * static_cast<size_t>(a.B) * a.nh * padded_rows(a.S) + static_cast<size_t>(a.B) * a.S * a.nh * a.dr) * sizeof(float);
}
void latent_bwd_workspace_carve(LatentArgs &a, void *base) {
  const size_t rows = static_cast<size_t>(a.B) * a.nh * padded_rows(a.S);
  a.nlse = static_cast<float *>(base);
  a.nD = a.nlse + rows;
  a.rope_parts = a.nD + rows;
}

cudaError_t launch_latent_bwd(const LatentMaps &q64, const LatentMaps &q128, const LatentArgs &a, int sms,
                              cudaStream_t stream) {
  cudaError_t err;
  const bool one = a.dn <= 64 && a.dv <= 64;
  if (a.dn == (one ? 64 : 128) && a.dv == a.dn)
    err = one ? launch_latent_bwd_ns<1, true>(q64, q128, a, sms, stream) : launch_latent_bwd_ns<2, true>(q64, q128, a, sms, stream);
  else
    err = one ? launch_latent_bwd_ns<1, false>(q64, q128, a, sms, stream) : launch_latent_bwd_ns<2, false>(q64, q128, a, sms, stream);
  if (err != cudaSuccess) return err;
  const size_t threads = static_cast<size_t>(a.B) * a.S * (a.dr / 4);
  return launch_pdl(latent_rope_kernel, static_cast<unsigned>((threads + 255) / 256), 256, 0, stream, a);
}

}  // namespace xattn
