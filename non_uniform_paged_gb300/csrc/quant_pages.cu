// bf16 pages into 4-bit pages and back (tg_quant_pages, tg_dequant_pages).
//
// Mathematics: tg.h, page formats.  A value is 2 bytes on one side and 9/16 on the other, read once and written once:
// bound by memory.
//
// The work is tiles of 16 tokens of every (request, place in the groups); their number is known on the device
// alone.  Each block of threads adds up the tiles of all heads; each warp takes an even share of them, one after the
// other in the lists, and looks up 32 of them at a time, a tile by each lane, so that the chain counts -> list -> page
// is waited for once in 32 tiles.  A tile's 4-bit side passes through shared memory, because its 16-byte pieces (V by blocks
// of values, scales) are not the pieces of 8 values that a lane has of a bf16 row.
#include "page4.cuh"
#include "ptx.cuh"
#include "tg_internal.h"

#include <cuda_runtime.h>

namespace {

using namespace tgk;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
// Blocks to an SM, of 80 registers (1.26M rows of 128: into 4 bits 136 us, with 4 blocks of 64 registers 150; out of them 140 and 146).
constexpr int kBlocksPerSm = 3;
constexpr int kEntries = 1024;  // heads whose first tile shared memory keeps; of more it is counted again

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
  __shared__ int64_t s_first[kEntries + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, sub = lane % LANES, side = lane / LANES;
  const int entries = a.batch * a.H;
  const bool kept = entries <= kEntries;
  griddep_wait();
  // tiles of an entry (request, place): of 16 tokens that are there, or of all pages that hold one
  auto tiles_of = [&](int e) -> int64_t {
    const int64_t n = tokens_of(a, e / a.H, e % a.H);
    return TO4 ? (n + 15) / 16 : (n + a.P - 1) / a.P * (a.P / 16);
  };
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
  for (int e = 0; e < entries; e += kThreads) {
    const int64_t total = block_scan(e + tid < entries ? tiles_of(e + tid) : 0, before);
    if (kept && e + tid < entries) s_first[e + tid] = all + before;
    all += total;
  }
  // this block's tiles [lo, hi), and this warp's [from, to) of them
  const int64_t lo = all / gridDim.x * blockIdx.x + min((int64_t)blockIdx.x, all % gridDim.x);
  const int64_t hi = lo + all / gridDim.x + (blockIdx.x < all % gridDim.x);
  if (lo >= hi) return;
  if (!kept) {
    int64_t sum = 0;
    for (int e = 0; e < entries; e += kThreads) {
      const int64_t n = e + tid < entries ? tiles_of(e + tid) : 0;
      const int64_t total = block_scan(n, before);
      if (sum + before <= lo && lo < sum + before + n) s_at[0] = e + tid, s_at[1] = sum + before;
      sum += total;
    }
  }
  __syncthreads();
  const int64_t mine_lo = lo + (hi - lo) * warp / kWarps, mine_hi = lo + (hi - lo) * (warp + 1) / kWarps;
  uint8_t *mine = tiles[warp];
  // the entry of tile n and the entry's first tile
  auto entry_of = [&](int64_t n, int64_t &begin) -> int {
    if (kept) {  // the last entry that begins at or before n
      int l = 0, h = entries;
      while (h - l > 1) {
        const int m = (l + h) / 2;
        if (s_first[m] <= n) l = m;
        else h = m;
      }
      begin = s_first[l];
      return l;
    }
    int e = (int)s_at[0];
    begin = s_at[1];
    for (int64_t count = tiles_of(e); n >= begin + count; count = tiles_of(e)) begin += count, ++e;
    return e;
  };

  for (int64_t n0 = mine_lo; n0 < mine_hi; n0 += 32) {
    // lane's tile n0 + lane: its pages (-1: none), its place in them and its tokens
    int l_from = -1, l_to = -1, l_in = 0, l_left = 0;
    if (n0 + lane < mine_hi) {
      int64_t begin;
      const int e = entry_of(n0 + lane, begin);
      const int b = e / a.H, p = e - b * a.H, group = p / a.H_p;
      const int64_t list = (int64_t)b * (a.H / a.H_p) + group, token = (n0 + lane - begin) * 16;
      l_from = (int)page_of(a, a.src_off, a.src_ids, a.src_pages, list, token);
      l_to = (int)page_of(a, a.dst_off, a.dst_ids, a.dst_pages, list, token);
      l_in = (p - group * a.H_p) * (a.P / 16) + (int)(token % a.P / 16);  // tile of the page
      l_left = (int)min(max(tokens_of(a, b, p) - token, (int64_t)0), (int64_t)16);
      if (l_from < 0 || l_to < 0) report(a.status, TG_STATUS_BAD_PAGE);
    }
    const int here = (int)min((int64_t)32, mine_hi - n0);
    const int p16 = a.P / 16;
    if (TO4) {
      // groups of 4 rows to a lane (K's, then V's), the next one, of the next tile too, on its way while one is encoded
      constexpr int GROUP = 4, GROUPS = 2 * 16 / PER / GROUP;
      auto fetch = [&](uint4(&v)[GROUP], int j, int g) {
        const int from = __shfl_sync(0xffffffffu, l_from, j), in = __shfl_sync(0xffffffffu, l_in, j);
        const int left = from < 0 ? 0 : __shfl_sync(0xffffffffu, l_left, j);
        const int hp = p16 == 1 ? in : in / p16, r0 = (in - hp * p16) * 16, kv = g / (GROUPS / 2);
        const uint16_t *src = reinterpret_cast<const uint16_t *>(a.src) + (((int64_t)from * a.H_p + hp) * 2 * a.P + kv * a.P + r0) * D;
#pragma unroll
        for (int s = 0; s < GROUP; ++s) {
          const int r = (g % (GROUPS / 2) * GROUP + s) * PER + side;
          v[s] = r < left ? __ldcs(reinterpret_cast<const uint4 *>(src + r * D + sub * 8)) : make_uint4(0, 0, 0, 0);
        }
      };
      uint4 v[2][GROUP];
      fetch(v[0], 0, 0);
      for (int j = 0; j < here; ++j) {
        const int from = __shfl_sync(0xffffffffu, l_from, j), to = __shfl_sync(0xffffffffu, l_to, j);
        const int in = __shfl_sync(0xffffffffu, l_in, j);
        bool odd = false;
        __syncwarp();
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          if (g + 1 < GROUPS) fetch(v[(g + 1) & 1], j, g + 1);
          else if (j + 1 < here) fetch(v[0], j + 1, 0);
          const int kv = g / (GROUPS / 2);
#pragma unroll
          for (int s = 0; s < GROUP; ++s) {
            const int r = (g % (GROUPS / 2) * GROUP + s) * PER + side, c = sub % 16;
            const uint32_t w[4] = {v[g & 1][s].x, v[g & 1][s].y, v[g & 1][s].z, v[g & 1][s].w};
            float2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            const Code8 o = encode_exact(x, kv ? a.v_unit : a.k_unit, odd);  // (the units' reciprocals)
            uint8_t *tile = mine + sub / 16 * kTile4;
            *reinterpret_cast<uint32_t *>(tile + (kv ? v_codes4(r, c) : k_codes4(r, c))) = o.codes;
            if (!(c & 1)) tile[kv ? v_scale4(r, c / 2) : k_scale4(r, c / 2)] = (uint8_t)o.scale;
          }
        }
        __syncwarp();
        if (from < 0 || to < 0) continue;
        if (odd) report(a.status, TG_STATUS_NONFINITE);
        uint8_t *dst = a.dst + ((int64_t)to * a.H_p * p16 + in) * TILE;
        for (int i = lane; i < CHUNKS; i += 32)
          *reinterpret_cast<uint4 *>(dst + 16 * i) = *reinterpret_cast<const uint4 *>(mine + 16 * i);
      }
    } else {
      // a tile's pieces, the next tile's on their way while one is written out
      constexpr int PIECES = (CHUNKS + 31) / 32;
      auto fetch = [&](uint4(&v)[PIECES], int j) {
        const int from = __shfl_sync(0xffffffffu, l_from, j), in = __shfl_sync(0xffffffffu, l_in, j);
        if (from < 0) return;
        const uint8_t *src = a.src + ((int64_t)from * a.H_p * p16 + in) * TILE + 16 * lane;
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          if (32 * i + lane < CHUNKS) v[i] = __ldcs(reinterpret_cast<const uint4 *>(src + 512 * i));
      };
      uint4 v[PIECES];
      fetch(v, 0);
      for (int j = 0; j < here; ++j) {
        const int from = __shfl_sync(0xffffffffu, l_from, j), to = __shfl_sync(0xffffffffu, l_to, j);
        const int in = __shfl_sync(0xffffffffu, l_in, j), left = __shfl_sync(0xffffffffu, l_left, j);
        const int hp = p16 == 1 ? in : in / p16, r0 = (in - hp * p16) * 16;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          if (32 * i + lane < CHUNKS) *reinterpret_cast<uint4 *>(mine + 16 * (32 * i + lane)) = v[i];
        __syncwarp();
        if (j + 1 < here) fetch(v, j + 1);
        if (from < 0 || to < 0) continue;
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.dst) + (((int64_t)to * a.H_p + hp) * 2 * a.P + r0) * D + sub * 8;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll 4
          for (int s = 0; s < 16 / PER; ++s) {
            const int r = s * PER + side, c = sub % 16;
            const uint8_t *tile = mine + sub / 16 * kTile4;
            Code8 o;
            o.codes = *reinterpret_cast<const uint32_t *>(tile + (kv ? v_codes4(r, c) : k_codes4(r, c)));
            o.scale = tile[kv ? v_scale4(r, c / 2) : k_scale4(r, c / 2)];
            uint4 x = held8(o, kv ? a.v_unit : a.k_unit);
            if (r >= left) x = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(dst + ((int64_t)kv * a.P + r) * D) = x;
          }
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
