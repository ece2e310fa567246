// Host side shared by tg_prefill_attn and tg_prefix_attn: plan checks, tensor maps, launches.
#pragma once

#include "tile_attn.cuh"

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

namespace tgk {

inline PFN_cuTensorMapEncodeTiled_v12000 tile_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// TMA map of a bf16 array seen as [n2][n1][d], boxes of 64 columns x b1 x b2, 128-byte swizzle
inline int tile_map(CUtensorMap *map, const char *fn, const char *what, const uint16_t *p, int64_t d, int64_t n1,
                    int64_t n2, int b1, int b2) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tile_encode_fn();
  if (!enc) return tgi::fail(TG_ERR_CUDA, "%s: cuTensorMapEncodeTiled is unavailable", fn);
  const cuuint64_t gdim[3] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2};
  const cuuint64_t gstride[2] = {(cuuint64_t)d * 2, (cuuint64_t)(d * n1 * 2)};
  const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
  const cuuint32_t estride[3] = {1, 1, 1};
  const CUresult cr = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p), gdim, gstride, box,
                          estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS)
    return tgi::fail(TG_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed for %s (%d)", fn, what, (int)cr);
  return TG_OK;
}

inline bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// what both calls check of their plan, scale and buffers; *hd points into plan_host
inline int check_tile_call(const char *fn, int kind, const void *plan_host, const void *plan_dev, const void *q,
                           const void *out, const float *lse, float scale, const void *workspace,
                           int64_t workspace_bytes, const tg_tile_header **hd) {
  if (!plan_host || !plan_dev) return tgi::fail(TG_ERR_INVALID_ARG, "%s: NULL plan", fn);
  const tg_tile_header *h = static_cast<const tg_tile_header *>(plan_host);
  if (h->magic != TG_TILE_MAGIC || h->version != TG_TILE_VERSION || h->kind != kind)
    return tgi::fail(TG_ERR_INVALID_ARG, "%s: plan_host is not a plan of this call", fn);
  if (h->rows > 0 && (!q || !out)) return tgi::fail(TG_ERR_INVALID_ARG, "%s: NULL q or out", fn);
  if (!std::isfinite(scale)) return tgi::fail(TG_ERR_NONFINITE, "%s: scale is not finite", fn);
  if (scale <= 0.f) return tgi::fail(TG_ERR_INVALID_ARG, "%s: scale=%g must be positive", fn, (double)scale);
  if (misaligned(plan_dev, 16) || misaligned(q, 16) || misaligned(out, 32) || misaligned(lse, 4))
    return tgi::fail(TG_ERR_INVALID_ARG, "%s: plan_dev and q must be 16-byte, out 32-byte aligned", fn);
  if (h->workspace_bytes > 0) {
    if (!workspace) return tgi::fail(TG_ERR_INVALID_ARG, "%s: the plan needs a workspace", fn);
    if (workspace_bytes < h->workspace_bytes)
      return tgi::fail(TG_ERR_CAPACITY, "%s: workspace %lld < %lld bytes", fn, (long long)workspace_bytes,
                       (long long)h->workspace_bytes);
    if (misaligned(workspace, 256)) return tgi::fail(TG_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  }
  *hd = h;
  return TG_OK;
}

inline TileArgs tile_args(const tg_tile_header *hd, const void *plan_dev, float scale, void *workspace, uint16_t *out,
                          float *lse, int32_t *status) {
  TileArgs a = {};
  const uint8_t *pd = static_cast<const uint8_t *>(plan_dev);
  a.lead = reinterpret_cast<const tg_tile_item *>(pd + hd->lead);
  a.items = reinterpret_cast<const tg_tile_item *>(pd + hd->items);
  a.out = out;
  a.lse = lse;
  if (hd->n_slots) {
    float *ws = static_cast<float *>(workspace);
    a.ws_ml = ws;
    a.ws_own = ws + (int64_t)hd->n_slots * 512;
    a.ws_o = ws + (int64_t)hd->n_slots * 768;
  }
  a.status = status;
  a.H = hd->H;
  a.H_q = hd->H_q;
  a.g = hd->H_q / hd->H;
  a.tq = tgi::tile_tokens(a.g);
  a.window = hd->window;
  a.signal = hd->n_merge > 0;
  a.scale_log2 = scale * kTileLog2e;
  return a;
}

// The tile kernel, ready to launch.  It comes ahead of the tensor maps: a host thread's first call into the runtime makes the
// context current that the driver's encoder needs.
template <bool PAGED>
int ready_tiles(const char *fn, int d) {
  void *kernel = d == 128 ? reinterpret_cast<void *>(&tile_attn_kernel<128, PAGED>) : reinterpret_cast<void *>(&tile_attn_kernel<256, PAGED>);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTileSmem);
  if (e != cudaSuccess) return tgi::fail(TG_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", fn, cudaGetErrorString(e));
  return TG_OK;
}

// the tile kernel and, where the plan cut runs, the merge as its programmatic dependent
template <int D, bool PAGED>
int launch_tiles(const char *fn, tg_stream_t stream, const tg_tile_header *hd, const void *plan_dev,
                 const CUtensorMap &qm, const CUtensorMap &km, const CUtensorMap &vm, const TileArgs &a) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)hd->N_CTA);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, tile_attn_kernel<D, PAGED>, qm, km, vm, a);
  if (e != cudaSuccess) return tgi::fail(TG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  if (!hd->n_merge) return tgi::ok();
  MergeArgs m;
  m.merges = reinterpret_cast<const tg_tile_merge *>(static_cast<const uint8_t *>(plan_dev) + hd->merges);
  m.ws_ml = a.ws_ml, m.ws_own = a.ws_own, m.ws_o = a.ws_o, m.out = a.out, m.lse = a.lse;
  m.own_out = a.own_out;
  m.H_q = a.H_q, m.g = a.g, m.tq = a.tq;
  cfg.gridDim = dim3((unsigned)(hd->n_merge * merge_blocks(D)));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, tile_merge_kernel<D>, m);
  if (e != cudaSuccess) return tgi::fail(TG_ERR_CUDA, "%s: merge launch failed: %s", fn, cudaGetErrorString(e));
  return tgi::ok();
}

}  // namespace tgk
