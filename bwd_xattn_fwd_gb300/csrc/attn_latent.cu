// Latent attention, plainly: one block a query row (dQ) or a key row (dK, dV), products on
// the CUDA cores in fp32.
#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

constexpr int kPlain = 256;

__device__ __forceinline__ float block_reduce(float x, bool max, float *part) {
  for (int off = 16; off; off >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, off);
    x = max ? fmaxf(x, y) : x + y;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  x = part[0];
  for (int w = 1; w < kPlain / 32; ++w) x = max ? fmaxf(x, part[w]) : x + part[w];
  return x;
}

// Row j's key of head h against the fp32 row x: its own part and the shared one.
__device__ __forceinline__ float key_dot(const LatentArgs &a, const float *x, size_t tok, int h) {
  const __nv_bfloat16 *k = a.kv + (tok * a.nh + h) * (a.dn + a.dv), *r = a.k_rope + tok * a.dr;
  float s = 0.f;
  for (int d = 0; d < a.dn; ++d) s = fmaf(x[d], __bfloat162float(k[d]), s);
  for (int d = 0; d < a.dr; ++d) s = fmaf(x[a.dn + d], __bfloat162float(r[d]), s);
  return s;
}
__device__ __forceinline__ float value_dot(const LatentArgs &a, const float *x, size_t tok, int h) {
  const __nv_bfloat16 *v = a.kv + (tok * a.nh + h) * (a.dn + a.dv) + a.dn;
  float s = 0.f;
  for (int d = 0; d < a.dv; ++d) s = fmaf(x[d], __bfloat162float(v[d]), s);
  return s;
}

__global__ void __launch_bounds__(kPlain) latent_dq_plain(const LatentArgs a) {
  __shared__ float qs[192], os[128], ps[kPlain], part[kPlain / 32];
  const int h = blockIdx.x % a.nh, i = static_cast<int>(blockIdx.x / a.nh % a.S);
  const size_t b = blockIdx.x / a.nh / a.S, tok = b * a.S + i, row = tok * a.nh + h;
  const int dq = a.dn + a.dr, tid = threadIdx.x;
  float dot = 0.f;
  for (int d = tid; d < dq; d += kPlain) qs[d] = __bfloat162float(a.q[row * dq + d]);
  for (int d = tid; d < a.dv; d += kPlain) {
    os[d] = __bfloat162float(a.dO[row * a.dv + d]);
    dot = os[d] * __bfloat162float(a.o[row * a.dv + d]);
  }
  const float D = block_reduce(dot, false, part), lse = a.lse[row];
  if (tid == 0) a.D[row] = D;
  float g = 0.f;
  for (int j0 = 0; j0 <= i; j0 += kPlain) {
    const int j = j0 + tid;
    const size_t tj = b * a.S + j;
    ps[tid] = j <= i ? expf(key_dot(a, qs, tj, h) * a.scale - lse) * (value_dot(a, os, tj, h) - D) : 0.f;
    __syncthreads();
    if (tid < dq)
      for (int x = 0; x < kPlain && j0 + x <= i; ++x) {
        const size_t tx = b * a.S + j0 + x;
        const __nv_bfloat16 k = tid < a.dn ? a.kv[(tx * a.nh + h) * (a.dn + a.dv) + tid] : a.k_rope[tx * a.dr + tid - a.dn];
        g = fmaf(ps[x], __bfloat162float(k), g);
      }
    __syncthreads();
  }
  if (tid < dq) a.dq[row * dq + tid] = __float2bfloat16(g * a.scale);
}

__global__ void __launch_bounds__(kPlain) latent_dkv_plain(const LatentArgs a) {
  __shared__ float ks[192], vs[128], ps[kPlain], ds[kPlain];
  const int h = blockIdx.x % a.nh, j = static_cast<int>(blockIdx.x / a.nh % a.S);
  const size_t b = blockIdx.x / a.nh / a.S, tok = b * a.S + j, row = tok * a.nh + h;
  const int dq = a.dn + a.dr, tid = threadIdx.x;
  for (int d = tid; d < dq; d += kPlain)
    ks[d] = __bfloat162float(d < a.dn ? a.kv[row * (a.dn + a.dv) + d] : a.k_rope[tok * a.dr + d - a.dn]);
  for (int d = tid; d < a.dv; d += kPlain) vs[d] = __bfloat162float(a.kv[row * (a.dn + a.dv) + a.dn + d]);
  __syncthreads();
  float gk = 0.f, gv = 0.f;
  for (int i0 = j; i0 < a.S; i0 += kPlain) {
    const int i = i0 + tid;
    float p = 0.f, d_s = 0.f;
    if (i < a.S) {
      const size_t ri = (b * a.S + i) * a.nh + h;
      float s = 0.f, dp = 0.f;
      for (int d = 0; d < dq; ++d) s = fmaf(ks[d], __bfloat162float(a.q[ri * dq + d]), s);
      for (int d = 0; d < a.dv; ++d) dp = fmaf(vs[d], __bfloat162float(a.dO[ri * a.dv + d]), dp);
      p = expf(s * a.scale - a.lse[ri]);
      d_s = p * (dp - a.D[ri]);
    }
    ps[tid] = p;
    ds[tid] = d_s;
    __syncthreads();
    for (int x = 0; x < kPlain && i0 + x < a.S; ++x) {
      const size_t ri = (b * a.S + i0 + x) * a.nh + h;
      if (tid < dq) gk = fmaf(ds[x], __bfloat162float(a.q[ri * dq + tid]), gk);
      if (tid < a.dv) gv = fmaf(ps[x], __bfloat162float(a.dO[ri * a.dv + tid]), gv);
    }
    __syncthreads();
  }
  if (tid < a.dn) a.dkv[row * (a.dn + a.dv) + tid] = __float2bfloat16(gk * a.scale);
  if (tid < a.dv) a.dkv[row * (a.dn + a.dv) + a.dn + tid] = __float2bfloat16(gv);
  if (tid >= a.dn && tid < dq) a.rope_parts[row * a.dr + tid - a.dn] = gk * a.scale;
}

__global__ void __launch_bounds__(kPlain) latent_rope_plain(const LatentArgs a) {
  const size_t t = static_cast<size_t>(blockIdx.x) * kPlain + threadIdx.x, tok = t / a.dr;
  if (tok >= static_cast<size_t>(a.B) * a.S) return;
  float g = 0.f;
  for (int h = 0; h < a.nh; ++h) g += a.rope_parts[(tok * a.nh + h) * a.dr + t % a.dr];
  a.dk_rope[t] = __float2bfloat16(g);
}

}  // namespace

size_t latent_bwd_workspace_bytes(const LatentArgs &a) {
  return static_cast<size_t>(a.B) * a.S * a.nh * (1 + a.dr) * sizeof(float);
}
void latent_bwd_workspace_carve(LatentArgs &a, void *base) {
  a.D = static_cast<float *>(base);
  a.rope_parts = a.D + static_cast<size_t>(a.B) * a.S * a.nh;
}

cudaError_t launch_latent_bwd(const LatentArgs &a, cudaStream_t stream) {
  latent_dq_plain<<<static_cast<unsigned>(a.B) * a.S * a.nh, kPlain, 0, stream>>>(a);
  latent_dkv_plain<<<static_cast<unsigned>(a.B) * a.S * a.nh, kPlain, 0, stream>>>(a);
  latent_rope_plain<<<static_cast<unsigned>((static_cast<size_t>(a.B) * a.S * a.dr + kPlain - 1) / kPlain), kPlain, 0, stream>>>(a);
  return cudaGetLastError();
}
}  // namespace xattn
