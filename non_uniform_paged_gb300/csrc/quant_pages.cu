// bf16 pages into 4-bit pages and back (tg_quant_pages, tg_dequant_pages).
//
// Mathematics: tg.h, page formats.  A value is 2 bytes on one side and 9/16 on the other, read once and written once:
// bound by memory.
//
// The work is tiles of 16 tokens of every (request, place in the groups); their number is known on the device
// alone.  Each block of threads adds up the tiles of all heads, takes an even share of them, and its warps walk over that
// share.  A tile's 4-bit side passes through shared memory, because its 16-byte pieces (V by blocks of
// values, scales) are not the pieces of 8 values that a lane has of a bf16 row.
#include "page4.cuh"
#include "ptx.cuh"
#include "tg_internal.h"

#include <cuda_runtime.h>

namespace {

using namespace tgk;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kBlocksPerSm = 3;

struct PagesArgs {
  const int32_t *head_order, *ntok, *added, *src_ids, *dst_ids;
  const int64_t *src_off, *dst_off;
  const uint8_t *src;
  uint8_t *dst;
  int64_t src_pages, dst_pages;
  int32_t *status;
  int batch, H, H_p, P, plus, reserve;
  float k_unit, v_unit;  // into 4 bits: their reciprocals
};

// tokens of the head at place p of request b
__device__ __forceinline__ int64_t tokens_of(const PagesArgs &a, int b, int p) {
  const int h = __ldg(a.head_order + p);
  if (h < 0 || h >= a.H) {
    report(a.status, TG_STATUS_BAD_INPUT);
    return 0;
  }
  const int64_t asked = (int64_t)(a.added ? __ldg(a.added + b) : 0) + a.plus;
  const int64_t extra = min(max(asked, (int64_t)0), (int64_t)a.reserve);
  if (extra != asked) report(a.status, TG_STATUS_BAD_INPUT);
  return max(__ldg(a.ntok + (int64_t)b * a.H + h), 0) + extra;
}

// page of token 16 k of list l, -1 if the list or the pool has none
__device__ __forceinline__ int64_t page_of(const PagesArgs &a, const int64_t *off, const int32_t *ids, int64_t pages, int64_t l,
                                           int64_t token) {
  const int64_t at = __ldg(off + l) + token / a.P;
  if (at >= __ldg(off + l + 1)) return -1;
  const int32_t page = __ldg(ids + at);
  return page >= 0 && page < pages ? page : -1;
}

// TO4: bf16 -> 4 bits, else 4 bits -> bf16
template <int D, bool TO4>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) convert_pages_kernel(const PagesArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES, C = D / 128, TILE = C * kTile4;
  constexpr int CHUNKS = TILE / 16;  // 16-byte pieces of a tile
  __shared__ __align__(16) uint8_t tiles[kWarps][TILE];
  __shared__ int64_t sums[kWarps], s_at[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % LANES, side = lane / LANES;
  const int entries = a.batch * a.H;
  griddep_wait();
  // tiles of an entry (request, place): of 16 tokens that are there, or of all pages that hold one
  auto tiles_of = [&](int e) -> int64_t {
    const int64_t n = tokens_of(a, e / a.H, e % a.H);
    return TO4 ? (n + 15) / 16 : (n + a.P - 1) / a.P * (a.P / 16);
  };
  // all tiles, then the entry and the tile in it at which this block's share begins
  auto block_scan = [&](int64_t v, int64_t &before) -> int64_t {  // exclusive prefix of v, and the block's sum
    int64_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int64_t total = 0;
    before = incl - v;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    return total;
  };
  int64_t all = 0, before;
  for (int e = 0; e < entries; e += kThreads) all += block_scan(e + tid < entries ? tiles_of(e + tid) : 0, before);
  const int64_t lo = all / gridDim.x * blockIdx.x + min((int64_t)blockIdx.x, all % gridDim.x);
  const int64_t hi = lo + all / gridDim.x + (blockIdx.x < all % gridDim.x);
  if (lo >= hi) return;
  int64_t sum = 0;
  for (int e = 0; e < entries; e += kThreads) {
    const int64_t n = e + tid < entries ? tiles_of(e + tid) : 0;
    const int64_t total = block_scan(n, before);
    if (sum + before <= lo && lo < sum + before + n) s_at[0] = e + tid, s_at[1] = sum + before;
    sum += total;
  }
  __syncthreads();
  int e = (int)s_at[0];
  int64_t begin = s_at[1], count = tiles_of(e);
  uint8_t *mine = tiles[warp];

  for (int64_t n = lo + warp; n < hi; n += kWarps) {
    while (n >= begin + count) {
      begin += count;
      count = tiles_of(++e);
    }
    const int b = e / a.H, p = e % a.H;
    const int64_t list = (int64_t)b * (a.H / a.H_p) + p / a.H_p, token = (n - begin) * 16;
    const int64_t from = page_of(a, a.src_off, a.src_ids, a.src_pages, list, token);
    const int64_t to = page_of(a, a.dst_off, a.dst_ids, a.dst_pages, list, token);
    if (from < 0 || to < 0) {
      if (lane == 0) report(a.status, TG_STATUS_BAD_PAGE);
      continue;
    }
    const int r0 = (int)(token % a.P), hp = p % a.H_p;
    const int64_t left = tokens_of(a, b, p) - token;  // rows [0, left) are tokens
    const int64_t bf16_at = (((TO4 ? from : to) * a.H_p + hp) * 2 * a.P + r0) * D;
    const int64_t e2m1_at = (((TO4 ? to : from) * a.H_p + hp) * (a.P / 16) + r0 / 16) * TILE;
    __syncwarp();
    if (TO4) {
      const uint16_t *src = reinterpret_cast<const uint16_t *>(a.src) + bf16_at + sub * 8;
      bool odd = false;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        constexpr int STEPS = 16 / PER, GO = STEPS < 8 ? STEPS : 8;
#pragma unroll
        for (int s0 = 0; s0 < STEPS; s0 += GO) {
          uint4 v[GO];
#pragma unroll
          for (int s = 0; s < GO; ++s) {
            const int r = (s0 + s) * PER + side;
            v[s] = r < left ? __ldcs(reinterpret_cast<const uint4 *>(src + ((int64_t)kv * a.P + r) * D)) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int s = 0; s < GO; ++s) {
            const int r = (s0 + s) * PER + side;
            const uint32_t w[4] = {v[s].x, v[s].y, v[s].z, v[s].w};
            float2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            const Code8 o = encode_exact(x, kv ? a.v_unit : a.k_unit, odd);  // (the units' reciprocals)
            uint8_t *tile = mine + sub / 16 * kTile4;
            const int c = sub % 16;
            *reinterpret_cast<uint32_t *>(tile + (kv ? v_codes4(r, c) : k_codes4(r, c))) = o.codes;
            if (!(c & 1)) tile[kv ? v_scale4(r, c / 2) : k_scale4(r, c / 2)] = (uint8_t)o.scale;
          }
        }
      }
      if (odd) report(a.status, TG_STATUS_NONFINITE);
      __syncwarp();
      for (int i = lane; i < CHUNKS; i += 32)
        *reinterpret_cast<uint4 *>(a.dst + e2m1_at + 16 * i) = *reinterpret_cast<const uint4 *>(mine + 16 * i);
    } else {
      for (int i = lane; i < CHUNKS; i += 32)
        *reinterpret_cast<uint4 *>(mine + 16 * i) = __ldcs(reinterpret_cast<const uint4 *>(a.src + e2m1_at + 16 * i));
      __syncwarp();
      uint16_t *dst = reinterpret_cast<uint16_t *>(a.dst) + bf16_at + sub * 8;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll 4
        for (int s = 0; s < 16 / PER; ++s) {
          const int r = s * PER + side, c = sub % 16;
          const uint8_t *tile = mine + sub / 16 * kTile4;
          Code8 o;
          o.codes = *reinterpret_cast<const uint32_t *>(tile + (kv ? v_codes4(r, c) : k_codes4(r, c)));
          o.scale = tile[kv ? v_scale4(r, c / 2) : k_scale4(r, c / 2)];
          uint4 v = held8(o, kv ? a.v_unit : a.k_unit);
          if (r >= left) v = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(dst + ((int64_t)kv * a.P + r) * D) = v;
        }
    }
  }
}

int convert(const char *fn, bool to4, tg_stream_t stream, int d, const PagesArgs &a) {
  using tgi::fail;
  if (a.batch <= 0 || a.H <= 0 || a.H_p <= 0 || a.P <= 0)
    return fail(TG_ERR_INVALID_ARG, "%s: batch=%d, H=%d, H_p=%d, P=%d", fn, a.batch, a.H, a.H_p, a.P);
  if (d != 128 && d != 256) return fail(TG_ERR_SHAPE, "%s: d=%d (128 or 256)", fn, d);
  if (a.H % a.H_p || a.P % 16) return fail(TG_ERR_SHAPE, "%s: H=%d of H_p=%d, P=%d (a multiple of 16)", fn, a.H, a.H_p, a.P);
  if ((int64_t)a.batch * a.H > INT32_MAX - kThreads)
    return fail(TG_ERR_SHAPE, "%s: batch=%d times H=%d heads", fn, a.batch, a.H);
  if (a.plus < 0 || a.reserve < 0 || a.plus > a.reserve)
    return fail(TG_ERR_INVALID_ARG, "%s: plus=%d, reserve=%d (0 <= plus <= reserve)", fn, a.plus, a.reserve);
  if (!unit_ok(a.k_unit) || !unit_ok(a.v_unit))
    return fail(TG_ERR_INVALID_ARG, "%s: k_unit=%g, v_unit=%g (powers of two in [2^-60, 2^60])", fn, (double)a.k_unit,
                (double)a.v_unit);
  if (a.src_pages <= 0 || a.src_pages > INT32_MAX || a.dst_pages <= 0 || a.dst_pages > INT32_MAX)
    return fail(TG_ERR_CAPACITY, "%s: pools of %lld and %lld pages (1..2^31-1)", fn, (long long)a.src_pages,
                (long long)a.dst_pages);
  if (!a.head_order || !a.ntok || !a.src_off || !a.src_ids || !a.src || !a.dst_off || !a.dst_ids || !a.dst)
    return fail(TG_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if ((reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst)) & 15)
    return fail(TG_ERR_INVALID_ARG, "%s: pools must be 16-byte aligned", fn);
  PagesArgs b = a;
  if (to4) b.k_unit = 1.f / a.k_unit, b.v_unit = 1.f / a.v_unit;  // exact
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms * kBlocksPerSm);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (d == 128)
    e = to4 ? cudaLaunchKernelEx(&cfg, convert_pages_kernel<128, true>, b) : cudaLaunchKernelEx(&cfg, convert_pages_kernel<128, false>, b);
  else
    e = to4 ? cudaLaunchKernelEx(&cfg, convert_pages_kernel<256, true>, b) : cudaLaunchKernelEx(&cfg, convert_pages_kernel<256, false>, b);
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return tgi::ok();
}

}  // namespace

extern "C" int tg_quant_pages(tg_stream_t stream, int batch, int H, int H_p, int P, int d, const int32_t *head_order,
                              const int32_t *ntok, const int64_t *src_off, const int32_t *src_ids, const uint16_t *src,
                              int64_t src_pages, const int64_t *dst_off, const int32_t *dst_ids, void *dst,
                              int64_t dst_pages, float k_unit, float v_unit, int32_t *dev_status) {
  PagesArgs a = {};
  a.head_order = head_order, a.ntok = ntok, a.src_off = src_off, a.src_ids = src_ids, a.dst_off = dst_off, a.dst_ids = dst_ids;
  a.src = reinterpret_cast<const uint8_t *>(src), a.dst = static_cast<uint8_t *>(dst), a.src_pages = src_pages;
  a.dst_pages = dst_pages, a.status = dev_status, a.batch = batch, a.H = H, a.H_p = H_p, a.P = P;
  a.k_unit = k_unit, a.v_unit = v_unit;
  return convert("tg_quant_pages", true, stream, d, a);
}

extern "C" int tg_dequant_pages(tg_stream_t stream, int batch, int H, int H_p, int P, int d, const int32_t *head_order,
                                const int32_t *ntok, const int32_t *added, int plus, int reserve, const int64_t *src_off,
                                const int32_t *src_ids, const void *src, int64_t src_pages, const int64_t *dst_off,
                                const int32_t *dst_ids, uint16_t *dst, int64_t dst_pages, float k_unit, float v_unit,
                                int32_t *dev_status) {
  PagesArgs a = {};
  a.head_order = head_order, a.ntok = ntok, a.added = added, a.plus = plus, a.reserve = reserve, a.src_off = src_off;
  a.src_ids = src_ids, a.dst_off = dst_off, a.dst_ids = dst_ids, a.src = static_cast<const uint8_t *>(src);
  a.dst = reinterpret_cast<uint8_t *>(dst), a.src_pages = src_pages, a.dst_pages = dst_pages, a.status = dev_status;
  a.batch = batch, a.H = H, a.H_p = H_p, a.P = P, a.k_unit = k_unit, a.v_unit = v_unit;
  return convert("tg_dequant_pages", false, stream, d, a);
}
