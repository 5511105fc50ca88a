// C ABI of libxattn (declared in include/xattn.h): argument checks, TMA tensor maps,
// scratch handling and kernel launches. No call synchronises the device except
// xattn_check_device_status.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "xattn.h"
#include "sm103_ptx.cuh"
#include "xattn_internal.h"

namespace xattn {
namespace {

// Device status word, written by kernels whose bounded waits expire.
__device__ int g_device_status;

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  bool sm103 = false;
  int sms = 0;
  int *status = nullptr;
  std::once_flag pool_once;       // scratch_alloc's
  cudaError_t pool_err = cudaSuccess;
  cudaMemPool_t pool = nullptr;
};
DeviceInfo g_dev[kMaxDevices];

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

uint64_t wait_limit_ns() {
  static const uint64_t v = [] {
    const char *s = std::getenv("XATTN_WAIT_LIMIT_NS");
    const unsigned long long x = s ? std::strtoull(s, nullptr, 10) : 0ull;
    return x > 0 ? static_cast<uint64_t>(x) : static_cast<uint64_t>(2000000000ull);
  }();
  return v;
}

}  // namespace

bool pdl_enabled() {
  static const bool v = std::getenv("XATTN_NO_PDL") == nullptr;
  return v;
}

namespace {

// Self-test of the bounded waits: one CTA waits on an mbarrier that nothing ever arrives
// on (phase 0 of a barrier expecting one arrival), with the same wait the kernels use.
// The wait runs out after limit_ns and records XATTN_ERR_DEVICE_TIMEOUT in the status
// word; nothing else happens on the device.
__global__ void wait_selftest_kernel(int *status, unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitCtl ctl{&abort_flag, status, limit_ns};
  (void)mbar_wait(smem_u32(&bar), 0, ctl);
}

// A bounds check that fails by construction (index n of a range of n elements, never
// used for an access): in a debug build it records XATTN_ERR_DEVICE_BOUNDS.
__global__ void bounds_selftest_kernel(int *status, int n) {
  const int i = n;
  XATTN_DCHECK(i < n, status);
  (void)i;
  (void)status;
}

#define XATTN_TRY(expr)                          \
  do {                                           \
    const xattn_status st_ = (expr);             \
    if (st_ != XATTN_OK) return st_;             \
  } while (0)

xattn_status device_info(DeviceInfo **out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return XATTN_ERR_CUDA;
  DeviceInfo &d = g_dev[dev];
  std::call_once(d.once, [&d, dev] {
    const OutsideCapture outside;
    int major = 0, minor = 0;
    d.err = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (d.err == cudaSuccess) d.err = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    d.sm103 = (major == 10 && minor == 3);
    if (d.err == cudaSuccess) d.err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (d.err == cudaSuccess) d.err = cudaGetSymbolAddress(reinterpret_cast<void **>(&d.status), g_device_status);
  });
  if (d.err != cudaSuccess) return XATTN_ERR_CUDA;
  *out = &d;
  return XATTN_OK;
}

// Scratch of one call on `stream`, released with cudaFreeAsync on it. It comes from a pool of
// the library's own that keeps what it has grown to: the default pool gives its memory back
// at every synchronisation, and the next call would map it again (step of B8 S2048, each
// call waited for: 471 us with the default pool against 134 us back to back). xattn_trim_scratch
// gives it back.
cudaError_t scratch_pool(DeviceInfo &d) {
  std::call_once(d.pool_once, [&d] {
    const OutsideCapture outside;
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = static_cast<int>(&d - g_dev);
    unsigned long long keep = ~0ull;
    d.pool_err = cudaMemPoolCreate(&d.pool, &props);
    if (d.pool_err == cudaSuccess)
      d.pool_err = cudaMemPoolSetAttribute(d.pool, cudaMemPoolAttrReleaseThreshold, &keep);
  });
  return d.pool_err;
}

xattn_status scratch_alloc(DeviceInfo &d, size_t bytes, cudaStream_t stream, void **out) {
  if (scratch_pool(d) == cudaSuccess && cudaMallocFromPoolAsync(out, bytes, d.pool, stream) == cudaSuccess) return XATTN_OK;
  cudaGetLastError();   // do not leave the failure for the caller's next error check
  return XATTN_ERR_CUDA;
}

xattn_status get_encode() {
  std::call_once(g_encode_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode ? XATTN_OK : XATTN_ERR_CUDA;
}

// 4-D map over a contiguous [B, S, H, hd] bf16 tensor; box = one head's 128-row tile, or
// at hd = 128 one 64-column half of it (a swizzled box row is at most 128 bytes; the
// kernels load the two halves as two sub-tiles). The 128-byte (hd = 64, 128) or 64-byte
// (hd = 32) swizzle matches the UMMA operand layout. Rows past S read as zeros.
xattn_status make_map(CUtensorMap *map, const void *ptr, int B, int S, int H, int hd) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(B)};
  const cuuint64_t row = static_cast<cuuint64_t>(hd) * 2;
  const cuuint64_t strides[3] = {row, row * H, row * H * S};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(hd > 64 ? 64 : hd), 1, static_cast<cuuint32_t>(kTileRows), 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims,
                              strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              hd == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? XATTN_OK : XATTN_ERR_CUDA;
}

// 4-D fp32 map over the [B, S, nh, hd] dQ accumulator. The box is half a head row
// (hd/2 floats: 128 bytes at hd = 64, 64 bytes at hd = 32, with the matching swizzle)
// by 128 rows; the backward adds shared-memory tiles into it with TMA reduce-adds.
// Rows past S are skipped by the TMA unit.
xattn_status make_map_dq(CUtensorMap *map, float *ptr, int B, int S, int nh, int hd) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(nh),
                              static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(B)};
  const cuuint64_t row = static_cast<cuuint64_t>(hd) * 4;
  const cuuint64_t strides[3] = {row, row * nh, row * nh * S};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(hd / 2), 1, static_cast<cuuint32_t>(kTileRows), 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, ptr, dims, strides, box, elem,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              hd == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? XATTN_OK : XATTN_ERR_CUDA;
}

// 4-D map over the backward's [B, nh, S_pad, 16] bf16 auxiliary rows; box = 16 columns
// (32 bytes, 32-byte swizzle) by 128 rows.
xattn_status make_map_aux(CUtensorMap *map, void *ptr, int B, int S, int nh) {
  const cuuint64_t S_pad = static_cast<cuuint64_t>(padded_rows(S));
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kAuxCols), S_pad, static_cast<cuuint64_t>(nh),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t row = kAuxCols * 2;
  const cuuint64_t strides[3] = {row, row * S_pad, row * S_pad * nh};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(kAuxCols), static_cast<cuuint32_t>(kTileRows), 1, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, ptr, dims, strides, box, elem,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? XATTN_OK : XATTN_ERR_CUDA;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
template <typename... T>
bool aligned4(const T *...p) {
  return (((reinterpret_cast<uintptr_t>(p) & 3u) == 0) && ...);
}

xattn_status check_shape(int B, int S, int nh, int nkv, int hd, float scale) {
  if (B <= 0 || S <= 0 || nh <= 0 || nkv <= 0 || hd <= 0) return XATTN_ERR_BAD_SHAPE;
  // Keep every element index and grid size well inside their integer types (in doubles: the
  // products of four ints pass 64 bits).
  const double heads = static_cast<double>(B) * nh;
  if (heads * S * hd > 0x1p40 || heads * ((static_cast<long long>(S) + 127) / 128) > 0x1p31 - 1)
    return XATTN_ERR_BAD_SHAPE;
  if (nh % nkv != 0) return XATTN_ERR_GROUP;
  if (!std::isfinite(scale)) return XATTN_ERR_BAD_SCALE;
  return XATTN_OK;
}

// The bf16 kernels take exponentials to base 2 of scores times scale log2 e, which has to be a number.
xattn_status check_bf16_scale(float scale) {
  return std::isfinite(scale * kLog2e) ? XATTN_OK : XATTN_ERR_BAD_SCALE;
}

// The bf16 backward folds -LSE/scale into a tensor-core operand; it takes scale == 0
// exactly, and any |scale| >= 2^-64 (so that LSE/scale stays far from overflow).
xattn_status check_bwd_scale(float scale) {
  XATTN_TRY(check_bf16_scale(scale));
  if (scale != 0.f && std::fabs(scale) < 0x1p-64f) return XATTN_ERR_BAD_SCALE;
  return XATTN_OK;
}

xattn_status check_bf16(int hd) { return (hd == 32 || hd == 64) ? XATTN_OK : XATTN_ERR_UNSUPPORTED_HD; }
xattn_status check_bf16_fwd(int hd) {
  return (hd == 32 || hd == 64 || hd == 128) ? XATTN_OK : XATTN_ERR_UNSUPPORTED_HD;
}

// With XATTN_VERBOSE set in the environment, CUDA failures are also reported on stderr.
xattn_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return XATTN_OK;
  static const bool verbose = std::getenv("XATTN_VERBOSE") != nullptr;
  if (verbose) std::fprintf(stderr, "libxattn: CUDA error %d: %s\n", static_cast<int>(e), cudaGetErrorString(e));
  return XATTN_ERR_CUDA;
}

// Window and sinks of a window call; on success *w and *s are clipped to S (a window of S
// or more keeps every key, sinks beyond S mean all of them).
xattn_status check_window(int S, int window, int sinks, int *w, int *s) {
  if (window < 1 || sinks < 0) return XATTN_ERR_WINDOW;
  if (S > (1 << 30)) return XATTN_ERR_BAD_SHAPE;   // tile sums stay inside int32
  *w = window < S ? window : S;
  *s = sinks < S ? sinks : S;
  return XATTN_OK;
}

// Sizes of a paged cache [num_pages, page_size, nkv, hd] and a table of max_pages entries a
// sequence, for n new tokens a sequence.
xattn_status check_pages(int B, int n, int nkv, int hd, int num_pages, int page_size, int max_pages) {
  if (B <= 0 || n <= 0 || nkv <= 0 || hd <= 0 || num_pages <= 0 || max_pages <= 0) return XATTN_ERR_BAD_SHAPE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && (page_size <= 0 || page_size % 128 != 0))
    return XATTN_ERR_PAGES;
  const long long most = 1ll << 30;   // positions and rows of one sequence's table stay far inside int32
  if (page_size > most || static_cast<long long>(max_pages) * page_size > most ||
      n > static_cast<long long>(max_pages) * page_size)
    return XATTN_ERR_PAGES;
  // Element offsets stay inside int64, grids inside int32.
  if (static_cast<double>(nkv) * hd > 0x1p30 || static_cast<double>(num_pages) * page_size * nkv * hd > 0x1p60 ||
      static_cast<double>(B) * n * nkv * hd > 0x1p38 || static_cast<double>(B) * max_pages > 0x1p40)
    return XATTN_ERR_BAD_SHAPE;
  return XATTN_OK;
}

// 4-D map over a pool [num_pages, page_size, nkv, hd]: box = up to 128 rows of one kv head in
// one page (64 columns at hd = 128). Pages outside the pool read as zeros. L2 fetches as much
// as a head's row has: at hd = 64 fetches of 256 bytes, half of them the next head's row, made
// a batch of trees 4 % slower (that row's reader comes after it has left L2).
xattn_status make_map_pages(CUtensorMap *map, const void *ptr, int num_pages, int page_size, int nkv, int hd) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(nkv),
                              static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(hd) * 2;
  const cuuint64_t strides[3] = {row, row * nkv, row * nkv * page_size};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(hd > 64 ? 64 : hd), 1,
                             static_cast<cuuint32_t>(page_size < kTileRows ? page_size : kTileRows), 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dims,
                              strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              hd == 32 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              hd == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                        : (hd == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B), CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? XATTN_OK : XATTN_ERR_CUDA;
}

// The fp32 window kernels' largest grid: four blocks per 32 rows of a head.
bool window_f32_grid_ok(int B, int S, int nh) {
  return static_cast<double>(B) * nh * ((S + 31) / 32) * 4 < 0x1p31;
}

xattn_status bf16_device(DeviceInfo **dev) {
  XATTN_TRY(device_info(dev));
  if (!(*dev)->sm103) return XATTN_ERR_NO_DEVICE_SUPPORT;
  return get_encode();
}

xattn_status check_workspace(void *ws, size_t bytes, int B, int S, int nh, int hd) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return XATTN_ERR_WORKSPACE;
  if (bytes < bwd_workspace_bytes(B, S, nh, hd, true)) return XATTN_ERR_WORKSPACE;
  return XATTN_OK;
}

}  // namespace
}  // namespace xattn

using namespace xattn;

extern "C" {

xattn_status xattn_fwd(const void *q, const void *k, const void *v, int B, int S, int nh, int nkv,
                       int hd, float scale, void *o, float *lse, void *stream) {
  if (!q || !k || !v || !o || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  XATTN_TRY(check_bf16_fwd(hd));
  XATTN_TRY(check_bf16_scale(scale));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned4(lse)) return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  CUtensorMap mq, mk, mv;
  XATTN_TRY(make_map(&mq, q, B, S, nh, hd));
  XATTN_TRY(make_map(&mk, k, B, S, nkv, hd));
  XATTN_TRY(make_map(&mv, v, B, S, nkv, hd));
  return cuda_status(launch_fwd_bf16(mq, mk, mv, static_cast<__nv_bfloat16 *>(o), lse, B, S, nh, nkv,
                                     hd, scale, dev->status, wait_limit_ns(),
                                     static_cast<cudaStream_t>(stream)));
}

int xattn_bwd_dq_mode(int S, int nh, int nkv, int hd, int deterministic) {
  if (S <= 0 || nh <= 0 || nkv <= 0 || nh % nkv != 0) return -1;
  if (hd != 32 && hd != 64 && hd != 128) return -1;
  if (!deterministic && hd != 128) return XATTN_BWD_FUSED_DQ;
  return bwd_resident_dq_ok(S, nh, nkv, hd) ? XATTN_BWD_RESIDENT_DQ : XATTN_BWD_QUERY_DQ;
}

int xattn_decode_runs(int B, int T, int nh, int nkv, int hd, int num_sms) {
  if (B <= 0 || T <= 0 || nh <= 0 || nkv <= 0 || nh % nkv != 0 || num_sms <= 0) return -1;
  if (nh / nkv > kMaxDecodeGroup || (hd != 32 && hd != 64 && hd != 128)) return -1;
  const long long chunks = (static_cast<long long>(T) + decode_chunk_keys(hd) - 1) / decode_chunk_keys(hd);
  if (static_cast<long long>(B) * nkv * chunks > 0x7fffffffLL) return -1;
  return decode_runs(B, T, nh, nkv, hd, num_sms);
}

size_t xattn_bwd_workspace_bytes(int B, int S, int nh, int hd) {
  if (B <= 0 || S <= 0 || nh <= 0 || hd <= 0) return 0;
  return bwd_workspace_bytes(B, S, nh, hd, true);
}

xattn_status xattn_bwd_preprocess(const void *o, const void *dO, const float *lse, int B, int S,
                                  int nh, int hd, float scale, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  if (!o || !dO || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nh, hd, scale));
  XATTN_TRY(check_bwd_scale(scale));
  XATTN_TRY(check_bf16(hd));
  if (!aligned16(o) || !aligned16(dO) || !aligned4(lse)) return XATTN_ERR_MISALIGNED;
  XATTN_TRY(check_workspace(workspace, workspace_bytes, B, S, nh, hd));
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  const BwdWorkspace ws = bwd_workspace_carve(workspace, B, S, nh, hd);
  return cuda_status(launch_bwd_preprocess(static_cast<const __nv_bfloat16 *>(o),
                                           static_cast<const __nv_bfloat16 *>(dO), lse, B, S, nh, hd,
                                           scale, ws, true, static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_bwd_main(const void *q, const void *k, const void *v, const void *dO, int B,
                            int S, int nh, int nkv, int hd, float scale, void *dk, void *dv,
                            void *workspace, size_t workspace_bytes, void *stream) {
  if (!q || !k || !v || !dO || !dk || !dv) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  XATTN_TRY(check_bwd_scale(scale));
  XATTN_TRY(check_bf16(hd));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(dk) ||
      !aligned16(dv))
    return XATTN_ERR_MISALIGNED;
  XATTN_TRY(check_workspace(workspace, workspace_bytes, B, S, nh, hd));
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  CUtensorMap mq, mk, mv, mdo;
  XATTN_TRY(make_map(&mq, q, B, S, nh, hd));
  XATTN_TRY(make_map(&mk, k, B, S, nkv, hd));
  XATTN_TRY(make_map(&mv, v, B, S, nkv, hd));
  XATTN_TRY(make_map(&mdo, dO, B, S, nh, hd));
  const BwdWorkspace ws = bwd_workspace_carve(workspace, B, S, nh, hd);
  CUtensorMap maux, mdq;
  XATTN_TRY(make_map_aux(&maux, ws.aux, B, S, nh));
  XATTN_TRY(make_map_dq(&mdq, ws.dqacc, B, S, nh, hd));
  return cuda_status(launch_bwd_main_bf16(mq, mk, mv, mdo, maux, &mdq, static_cast<__nv_bfloat16 *>(dk),
                                          static_cast<__nv_bfloat16 *>(dv), B, S, nh, nkv, hd, scale,
                                          dev->status, wait_limit_ns(),
                                          static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_bwd_dq_convert(int B, int S, int nh, int hd, float scale, void *dq,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  if (!dq) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nh, hd, scale));
  XATTN_TRY(check_bf16(hd));
  if (!aligned16(dq)) return XATTN_ERR_MISALIGNED;
  XATTN_TRY(check_workspace(workspace, workspace_bytes, B, S, nh, hd));
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  const BwdWorkspace ws = bwd_workspace_carve(workspace, B, S, nh, hd);
  return cuda_status(launch_dq_convert(ws.dqacc, static_cast<__nv_bfloat16 *>(dq),
                                       static_cast<size_t>(B) * S * nh * hd, scale,
                                       static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_bwd(const void *q, const void *k, const void *v, const void *o, const void *dO,
                       const float *lse, int B, int S, int nh, int nkv, int hd, float scale, void *dq,
                       void *dk, void *dv, void *stream) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  XATTN_TRY(check_bwd_scale(scale));
  XATTN_TRY(check_bf16_fwd(hd));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned4(lse))
    return XATTN_ERR_MISALIGNED;
  // hd = 128: dV, dK and a dQ accumulator do not fit in TMEM together, so dQ comes from
  // the query-stationary kernel (the deterministic backward).
  if (hd == 128) return xattn_bwd_deterministic(q, k, v, o, dO, lse, B, S, nh, nkv, hd, scale, dq, dk, dv, stream);
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t bytes = bwd_workspace_bytes(B, S, nh, hd, true);
  void *ws = nullptr;
  if (cudaMallocAsync(&ws, bytes, st) != cudaSuccess) return XATTN_ERR_CUDA;
  xattn_status r = xattn_bwd_preprocess(o, dO, lse, B, S, nh, hd, scale, ws, bytes, stream);
  if (r == XATTN_OK) r = xattn_bwd_main(q, k, v, dO, B, S, nh, nkv, hd, scale, dk, dv, ws, bytes, stream);
  if (r == XATTN_OK) r = xattn_bwd_dq_convert(B, S, nh, hd, scale, dq, ws, bytes, stream);
  const cudaError_t fe = cudaFreeAsync(ws, st);
  if (r == XATTN_OK && fe != cudaSuccess) r = XATTN_ERR_CUDA;
  return r;
}

xattn_status xattn_decode(const void *q, const void *k_cache, const void *v_cache, int B, int T,
                          int nh, int nkv, int hd, float scale, void *o, float *lse, void *stream) {
  if (!q || !k_cache || !v_cache || !o || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, T, nh, nkv, hd, scale));
  XATTN_TRY(check_bf16_scale(scale));
  if (nh / nkv > kMaxDecodeGroup) return XATTN_ERR_GROUP;
  if (hd != 32 && hd != 64 && hd != 128) return XATTN_ERR_UNSUPPORTED_HD;
  // One CTA per (batch, kv head, chunk): the grid is one-dimensional.
  const long long chunks = (static_cast<long long>(T) + decode_chunk_keys(hd) - 1) / decode_chunk_keys(hd);
  if (static_cast<long long>(B) * nkv * chunks > 0x7fffffffLL) return XATTN_ERR_BAD_SHAPE;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned4(lse))
    return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  CUtensorMap mk, mv;
  XATTN_TRY(make_map(&mk, k_cache, B, T, nkv, hd));
  XATTN_TRY(make_map(&mv, v_cache, B, T, nkv, hd));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *ws = nullptr;
  if (cudaMallocAsync(&ws, decode_workspace_bytes(B, T, nh, hd), st) != cudaSuccess) return XATTN_ERR_CUDA;
  xattn_status r = cuda_status(launch_decode_bf16(mk, mv, static_cast<const __nv_bfloat16 *>(q),
                                                  static_cast<__nv_bfloat16 *>(o), lse, B, T, nh, nkv, hd, scale, ws,
                                                  dev->status, wait_limit_ns(), st));
  const cudaError_t fe = cudaFreeAsync(ws, st);
  if (r == XATTN_OK && fe != cudaSuccess) r = XATTN_ERR_CUDA;
  return r;
}

xattn_status xattn_tree_decode(const void *q, const void *k_pages, const void *v_pages, const int *page_table,
                               const int *ctx_lens, const unsigned long long *tree, int B, int n, int nh, int nkv,
                               int hd, int num_pages, int page_size, int max_pages, int window, int sinks,
                               float scale, void *o, float *lse, void *stream) {
  if (!q || !k_pages || !v_pages || !page_table || !ctx_lens || !o || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, n, nh, nkv, hd, scale));
  XATTN_TRY(check_bf16_scale(scale));
  XATTN_TRY(check_pages(B, n, nkv, hd, num_pages, page_size, max_pages));
  if (n > XATTN_TREE_MAX) return XATTN_ERR_BAD_SHAPE;
  if (window < n || sinks < 0) return XATTN_ERR_WINDOW;
  if (hd != 32 && hd != 64 && hd != 128) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(o) || !aligned4(lse) ||
      !aligned4(page_table) || !aligned4(ctx_lens) || (reinterpret_cast<uintptr_t>(tree) & 7u) != 0)
    return XATTN_ERR_MISALIGNED;
  TreeArgs a = {};
  a.B = B, a.n = n, a.nh = nh, a.nkv = nkv;
  a.num_pages = num_pages, a.page_size = page_size, a.max_pages = max_pages;
  a.group = nh / nkv;
  a.tile_rows = tree_tile_rows(n, nh, nkv);
  const long long rows = static_cast<long long>(n) * a.group;
  if (rows > (1 << 30)) return XATTN_ERR_BAD_SHAPE;
  a.row_tiles = static_cast<int>((rows + a.tile_rows - 1) / a.tile_rows);
  a.rec_rows = rows < a.tile_rows ? static_cast<int>(rows) : a.tile_rows;
  a.whole = tree_whole(page_size, max_pages) ? 1 : 0;
  a.page_shift = (page_size & (page_size - 1)) ? -1 : __builtin_ctz(page_size);
  if (tree_line(a) > 0x1p30) return XATTN_ERR_BAD_SHAPE;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  CUtensorMap mk, mv;
  XATTN_TRY(make_map_pages(&mk, k_pages, num_pages, page_size, nkv, hd));
  XATTN_TRY(make_map_pages(&mv, v_pages, num_pages, page_size, nkv, hd));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = tree_grid(a, hd, dev->sms);
  void *ws = nullptr;
  if (!a.whole) XATTN_TRY(scratch_alloc(*dev, tree_workspace_bytes(grid, a.rec_rows, hd), st, &ws));
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.page_table = page_table;
  a.ctx_lens = ctx_lens;
  a.tree = tree;
  a.o = static_cast<__nv_bfloat16 *>(o);
  a.lse = lse;
  if (!a.whole) {
    a.plan = static_cast<int4 *>(ws);
    a.ws_o = reinterpret_cast<float *>(a.plan + grid);
    a.ws_ml = a.ws_o + static_cast<size_t>(grid) * 2 * a.rec_rows * hd;
  }
  a.window = window < (1 << 30) ? window : (1 << 30);   // a table holds at most 2^30 positions
  a.sinks = sinks < (1 << 30) ? sinks : (1 << 30);
  a.scale_log2 = scale * kLog2e;
  a.status = dev->status;
  a.timeout_ns = wait_limit_ns();
  xattn_status r = cuda_status(launch_tree_bf16(mk, mv, a, hd, grid, st));
  if (a.whole) return r;
  const cudaError_t fe = cudaFreeAsync(ws, st);
  if (r == XATTN_OK && fe != cudaSuccess) r = XATTN_ERR_CUDA;
  return r;
}

xattn_status xattn_cache_append(const void *k_new, const void *v_new, void *k_pages, void *v_pages,
                                const int *page_table, const int *ctx_lens, int B, int n, int nkv, int hd,
                                int num_pages, int page_size, int max_pages, void *stream) {
  if (!k_new || !v_new || !k_pages || !v_pages || !page_table || !ctx_lens) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_pages(B, n, nkv, hd, num_pages, page_size, max_pages));
  if (hd % 8 != 0) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned4(page_table) ||
      !aligned4(ctx_lens))
    return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  const PageArgs a = {static_cast<uint4 *>(k_pages), static_cast<uint4 *>(v_pages), page_table, ctx_lens, B, n,
                      nkv * hd / 8, num_pages, page_size, max_pages};
  return cuda_status(launch_cache_append(a, k_new, v_new, static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_cache_compact(void *k_pages, void *v_pages, const int *page_table, const int *ctx_lens,
                                 const int *path, const int *accepted, int B, int n, int nkv, int hd, int num_pages,
                                 int page_size, int max_pages, void *stream) {
  if (!k_pages || !v_pages || !page_table || !ctx_lens || !path || !accepted) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_pages(B, n, nkv, hd, num_pages, page_size, max_pages));
  if (hd % 8 != 0) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned4(page_table) || !aligned4(ctx_lens) || !aligned4(path) ||
      !aligned4(accepted))
    return XATTN_ERR_MISALIGNED;
  if (2.0 * B * ((nkv * hd / 8 + 31) / 32) > 0x7fffffff) return XATTN_ERR_BAD_SHAPE;   // its grid
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  const PageArgs a = {static_cast<uint4 *>(k_pages), static_cast<uint4 *>(v_pages), page_table, ctx_lens, B, n,
                      nkv * hd / 8, num_pages, page_size, max_pages};
  return cuda_status(launch_cache_compact(a, path, accepted, static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_bwd_deterministic(const void *q, const void *k, const void *v, const void *o,
                                     const void *dO, const float *lse, int B, int S, int nh,
                                     int nkv, int hd, float scale, void *dq, void *dk, void *dv,
                                     void *stream) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  XATTN_TRY(check_bwd_scale(scale));
  XATTN_TRY(check_bf16_fwd(hd));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned4(lse))
    return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  CUtensorMap mq, mk, mv, mdo;
  XATTN_TRY(make_map(&mq, q, B, S, nh, hd));
  XATTN_TRY(make_map(&mk, k, B, S, nkv, hd));
  XATTN_TRY(make_map(&mv, v, B, S, nkv, hd));
  XATTN_TRY(make_map(&mdo, dO, B, S, nh, hd));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t bytes = bwd_workspace_bytes(B, S, nh, hd, false);
  void *base = nullptr;
  if (cudaMallocAsync(&base, bytes, st) != cudaSuccess) return XATTN_ERR_CUDA;
  const BwdWorkspace ws = bwd_workspace_carve(base, B, S, nh, hd);
  CUtensorMap maux;
  xattn_status r = make_map_aux(&maux, ws.aux, B, S, nh);
  if (r == XATTN_OK)
    r = cuda_status(launch_bwd_preprocess(static_cast<const __nv_bfloat16 *>(o),
                                          static_cast<const __nv_bfloat16 *>(dO), lse, B, S, nh, hd,
                                          scale, ws, false, st));
  if (r == XATTN_OK && bwd_resident_dq_ok(S, nh, nkv, hd)) {
    // Small problems: one kernel, dQ resident in TMEM over each head's key tiles.
    r = cuda_status(launch_bwd_main_resident_bf16(mq, mk, mv, mdo, maux, static_cast<__nv_bfloat16 *>(dk),
                                                  static_cast<__nv_bfloat16 *>(dv), static_cast<__nv_bfloat16 *>(dq),
                                                  B, S, nh, nkv, hd, scale, dev->status, wait_limit_ns(), st));
  } else {
    if (r == XATTN_OK)
      r = cuda_status(launch_bwd_main_bf16(mq, mk, mv, mdo, maux, nullptr, static_cast<__nv_bfloat16 *>(dk),
                                           static_cast<__nv_bfloat16 *>(dv), B, S, nh, nkv, hd, scale,
                                           dev->status, wait_limit_ns(), st));
    if (r == XATTN_OK)
      r = cuda_status(launch_bwd_dq_bf16(mq, mk, mv, mdo, lse, ws, static_cast<__nv_bfloat16 *>(dq), B, S,
                                         nh, nkv, hd, scale, dev->status, wait_limit_ns(), st));
  }
  const cudaError_t fe = cudaFreeAsync(base, st);
  if (r == XATTN_OK && fe != cudaSuccess) r = XATTN_ERR_CUDA;
  return r;
}

xattn_status xattn_window_fwd(const void *q, const void *k, const void *v, int B, int S, int nh, int nkv, int hd,
                              int window, int sinks, float scale, void *o, float *lse, void *stream) {
  if (!q || !k || !v || !o || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  int w = 0, s = 0;
  XATTN_TRY(check_window(S, window, sinks, &w, &s));
  XATTN_TRY(check_bf16_fwd(hd));
  XATTN_TRY(check_bf16_scale(scale));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      !aligned4(lse))
    return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  CUtensorMap mq, mk, mv;
  XATTN_TRY(make_map(&mq, q, B, S, nh, hd));
  XATTN_TRY(make_map(&mk, k, B, S, nkv, hd));
  XATTN_TRY(make_map(&mv, v, B, S, nkv, hd));
  return cuda_status(launch_window_fwd_bf16(mq, mk, mv, static_cast<__nv_bfloat16 *>(o), lse, B, S, nh, nkv, hd,
                                            scale, w, s, dev->status, wait_limit_ns(),
                                            static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_window_bwd(const void *q, const void *k, const void *v, const void *o, const void *dO,
                              const float *lse, int B, int S, int nh, int nkv, int hd, int window, int sinks,
                              float scale, int deterministic, void *dq, void *dk, void *dv, void *stream) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  int w = 0, s = 0;
  XATTN_TRY(check_window(S, window, sinks, &w, &s));
  XATTN_TRY(check_bwd_scale(scale));
  XATTN_TRY(check_bf16_fwd(hd));
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned4(lse))
    return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(bf16_device(&dev));
  // dQ: added across key tiles by the main kernel, or (deterministic, and at hd = 128, where
  // its accumulator does not fit the tensor memory) from the query-stationary kernel.
  const bool fused = !deterministic && hd != 128;
  CUtensorMap mq, mk, mv, mdo, maux, mdq;
  XATTN_TRY(make_map(&mq, q, B, S, nh, hd));
  XATTN_TRY(make_map(&mk, k, B, S, nkv, hd));
  XATTN_TRY(make_map(&mv, v, B, S, nkv, hd));
  XATTN_TRY(make_map(&mdo, dO, B, S, nh, hd));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t base_bytes = (bwd_workspace_bytes(B, S, nh, hd, fused) + 255) / 256 * 256;
  void *base = nullptr;
  XATTN_TRY(scratch_alloc(*dev, base_bytes + window_parts_bytes(B, S, nkv, hd, w, s), st, &base));
  float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(base) + base_bytes);
  const BwdWorkspace ws = bwd_workspace_carve(base, B, S, nh, hd);
  xattn_status r = make_map_aux(&maux, ws.aux, B, S, nh);
  if (r == XATTN_OK && fused) r = make_map_dq(&mdq, ws.dqacc, B, S, nh, hd);
  if (r == XATTN_OK)
    r = cuda_status(launch_bwd_preprocess(static_cast<const __nv_bfloat16 *>(o), static_cast<const __nv_bfloat16 *>(dO),
                                          lse, B, S, nh, hd, scale, ws, fused, st));
  if (r == XATTN_OK)
    r = cuda_status(launch_window_bwd_main_bf16(mq, mk, mv, mdo, maux, fused ? &mdq : nullptr,
                                                static_cast<__nv_bfloat16 *>(dk), static_cast<__nv_bfloat16 *>(dv), B,
                                                S, nh, nkv, hd, scale, w, s, parts, dev->status, wait_limit_ns(), st));
  if (r == XATTN_OK && fused)
    r = cuda_status(launch_dq_convert(ws.dqacc, static_cast<__nv_bfloat16 *>(dq), static_cast<size_t>(B) * S * nh * hd,
                                      scale, st));
  else if (r == XATTN_OK)
    r = cuda_status(launch_window_bwd_dq_bf16(mq, mk, mv, mdo, lse, ws, static_cast<__nv_bfloat16 *>(dq), B, S, nh,
                                              nkv, hd, scale, w, s, dev->status, wait_limit_ns(), st));
  const cudaError_t fe = cudaFreeAsync(base, st);
  if (r == XATTN_OK && fe != cudaSuccess) r = XATTN_ERR_CUDA;
  return r;
}

xattn_status xattn_window_fwd_f32(const float *q, const float *k, const float *v, int B, int S, int nh, int nkv,
                                  int hd, int window, int sinks, float scale, float *o, float *lse, void *stream) {
  if (!q || !k || !v || !o || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  int w = 0, s = 0;
  XATTN_TRY(check_window(S, window, sinks, &w, &s));
  if (hd > 128) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned4(q, k, v, o, lse)) return XATTN_ERR_MISALIGNED;
  if (!window_f32_grid_ok(B, S, nh)) return XATTN_ERR_BAD_SHAPE;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  return cuda_status(launch_window_fwd_f32(q, k, v, o, lse, B, S, nh, nkv, hd, scale, w, s,
                                           static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_window_bwd_f32(const float *q, const float *k, const float *v, const float *o, const float *dO,
                                  const float *lse, int B, int S, int nh, int nkv, int hd, int window, int sinks,
                                  float scale, float *dq, float *dk, float *dv, void *stream) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  int w = 0, s = 0;
  XATTN_TRY(check_window(S, window, sinks, &w, &s));
  if (hd > 128) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned4(q, k, v, o, dO, lse, dq, dk, dv)) return XATTN_ERR_MISALIGNED;
  if (!window_f32_grid_ok(B, S, nh)) return XATTN_ERR_BAD_SHAPE;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *D = nullptr;
  XATTN_TRY(scratch_alloc(*dev, static_cast<size_t>(B) * S * nh * sizeof(float), st, &D));
  xattn_status r = cuda_status(launch_window_bwd_f32(q, k, v, o, dO, lse, dq, dk, dv, static_cast<float *>(D), B, S, nh,
                                                     nkv, hd, scale, w, s, st));
  const cudaError_t fe = cudaFreeAsync(D, st);
  if (r == XATTN_OK && fe != cudaSuccess) r = XATTN_ERR_CUDA;
  return r;
}

xattn_status xattn_fwd_f32(const float *q, const float *k, const float *v, int B, int S, int nh,
                           int nkv, int hd, float scale, float *o, float *lse, void *stream) {
  if (!q || !k || !v || !o || !lse) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  if (hd > 128) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned4(q, k, v, o, lse)) return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  return cuda_status(launch_fwd_f32(q, k, v, o, lse, B, S, nh, nkv, hd, scale,
                                    static_cast<cudaStream_t>(stream)));
}

xattn_status xattn_bwd_f32(const float *q, const float *k, const float *v, const float *o,
                           const float *dO, const float *lse, int B, int S, int nh, int nkv, int hd,
                           float scale, float *dq, float *dk, float *dv, void *stream) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return XATTN_ERR_NULL_PTR;
  XATTN_TRY(check_shape(B, S, nh, nkv, hd, scale));
  if (hd > 128) return XATTN_ERR_UNSUPPORTED_HD;
  if (!aligned4(q, k, v, o, dO, lse, dq, dk, dv)) return XATTN_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  return cuda_status(launch_bwd_f32(q, k, v, o, dO, lse, dq, dk, dv, B, S, nh, nkv, hd, scale,
                                    static_cast<cudaStream_t>(stream)));
}

const char *xattn_status_string(xattn_status s) {
  switch (s) {
    case XATTN_OK: return "ok";
    case XATTN_ERR_NULL_PTR: return "a required pointer is NULL";
    case XATTN_ERR_BAD_SHAPE: return "B, S, nh, nkv and hd must be positive and within size limits";
    case XATTN_ERR_GROUP: return "nh must be a multiple of nkv";
    case XATTN_ERR_UNSUPPORTED_HD: return "unsupported head dimension (bf16: 32, 64 or 128; the backward's stage calls and xattn_bwd_noalloc: 32 or 64; fp32: <= 128)";
    case XATTN_ERR_MISALIGNED: return "a bf16 tensor pointer is not 16-byte aligned, or a float or int array not 4-byte";
    case XATTN_ERR_CUDA: return "a CUDA runtime or driver call failed";
    case XATTN_ERR_NO_DEVICE_SUPPORT: return "the current device is not compute capability 10.3 (sm_103)";
    case XATTN_ERR_DEVICE_TIMEOUT: return "a bounded on-device wait expired";
    case XATTN_ERR_BAD_SCALE: return "scale (bf16: scale log2 e) must be finite";
    case XATTN_ERR_WORKSPACE: return "workspace is NULL, not 256-byte aligned, or too small";
    case XATTN_ERR_SCRATCH_LIMIT:
      return "these sizes need more scratch than xattn_bwd_noalloc's fixed array holds";
    case XATTN_ERR_WINDOW: return "window must be positive (xattn_tree_decode: at least n) and sinks not negative";
    case XATTN_ERR_PAGES:
      return "page_size must be 16, 32, 64 or a multiple of 128, and the table hold n to 2^30 positions a sequence";
    case XATTN_ERR_DEVICE_BOUNDS:
      return "an on-device bounds check failed (debug build)";
  }
  return "unknown xattn status";
}

xattn_status xattn_selftest_wait_timeout(unsigned long long limit_ns, void *stream) {
  if (limit_ns < 1000ull || limit_ns > 10000000000ull) return XATTN_ERR_BAD_SHAPE;
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  wait_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(dev->status, limit_ns);
  return cuda_status(cudaGetLastError());
}

int xattn_build_flags(void) {
#ifdef XATTN_DEBUG
  return XATTN_BUILD_DEVICE_CHECKS;
#else
  return 0;
#endif
}

xattn_status xattn_selftest_bounds_check(void *stream) {
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  bounds_selftest_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(dev->status, 1);
  return cuda_status(cudaGetLastError());
}

xattn_status xattn_trim_scratch(size_t keep_bytes) {
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  const OutsideCapture outside;
  cudaError_t err = scratch_pool(*dev);
  if (err == cudaSuccess) err = cudaMemPoolTrimTo(dev->pool, keep_bytes);
  if (err != cudaSuccess) cudaGetLastError();   // do not leave the failure for the caller's next error check
  return cuda_status(err);
}

xattn_status xattn_check_device_status(void *stream) {
  DeviceInfo *dev = nullptr;
  XATTN_TRY(device_info(&dev));
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return XATTN_ERR_CUDA;
  int word = 0;
  if (cudaMemcpy(&word, dev->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess)
    return XATTN_ERR_CUDA;
  if (word != 0) {
    const int zero = 0;
    if (cudaMemcpy(dev->status, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
      return XATTN_ERR_CUDA;
    return static_cast<xattn_status>(word);
  }
  return XATTN_OK;
}

}  // extern "C"
