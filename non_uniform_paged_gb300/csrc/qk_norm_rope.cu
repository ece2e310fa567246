// Query/key RMS norm, position rotation and placement of the context rows (tg_qk_norm_rope).
//
// Mathematics: y = x * rsqrt(mean(x^2) + eps) * w per head, then the plane rotation of each
// pair by the table's (cos, sin).  Every value is read once and written once: the kernel is
// bound by memory, and for a decode step by its own latency.
//
// A head is d / 8 lanes of 8 values (16 bytes each way): half a warp at d = 128, a warp at
// d = 256.  A warp takes one token and 8 steps of heads, with all 8 loads in flight before
// the first is used, so its table row (up to 64 bytes per lane) and the norm weights are
// loaded once per 8 (d = 256) or 16 (d = 128) heads.  Pairs (i, i + rot/2) sit rot/16 lanes
// apart and are exchanged by shuffles; pairs (2i, 2i+1) lie in one lane.
#include "ptx.cuh"
#include "tg_internal.h"

#include <cuda_runtime.h>

#include <cmath>

namespace {

using namespace tgk;

constexpr int kSteps = 8;     // heads in flight per lane group
constexpr int kWarps = 4;

struct RopeArgs {
  const int32_t *cu_q, *start, *positions;
  const uint16_t *qkv;
  int64_t stride;
  const float *qw, *kw;
  const float *table;
  uint16_t *q, *K, *V;
  int32_t *status;
  int batch, T, H_q, H, Nmax, rot, max_pos, chunks;
  float eps;
};

template <int D, bool PAIRS>
__global__ void __launch_bounds__(kWarps * 32) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES;  // lanes of a head, heads side by side
  const int lane = threadIdx.x & 31, sub = lane % LANES, side = lane / LANES;
  const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(task / a.chunks);
  const int head0 = (int)(task - (int64_t)t * a.chunks) * kSteps * PER + side;
  if (t >= a.T) return;
  const int heads = a.H_q + 2 * a.H;
  // the loads do not wait for the request's lookup
  uint4 raw[kSteps];
  const uint16_t *src = a.qkv + (int64_t)t * a.stride + sub * 8;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = head0 + s * PER;
    raw[s] = h < heads ? __ldcs(reinterpret_cast<const uint4 *>(src + h * D)) : make_uint4(0, 0, 0, 0);
  }
  // the request: how many end at or before t
  int b = 0;
  for (int i = 0; i < a.batch; i += 32) {
    const int32_t end = i + lane < a.batch ? __ldg(a.cu_q + i + lane + 1) : INT32_MAX;
    const unsigned m = __ballot_sync(0xffffffffu, end <= t);
    b += __popc(m);
    if (m != 0xffffffffu) break;
  }
  if (b >= a.batch) return;  // behind the last request
  const int64_t row = (int64_t)__ldg(a.start + b) + (t - __ldg(a.cu_q + b));
  const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + t) : row;
  if (row < 0 || row >= a.Nmax || (a.rot > 0 && (pos < 0 || pos >= a.max_pos))) {
    if (lane == 0) report(a.status, TG_STATUS_BAD_INPUT);
    return;
  }
  // this lane's rotation: pair indices [i0, i0 + 8) (or 4 pairs), identity behind rot
  const bool turned = sub * 8 < a.rot;
  float c[8], sn[8];
  int partner = lane;
  if (turned) {
    const float *tb = a.table + pos * a.rot;  // [rot/2][2]
    if (PAIRS) {
      const float4 *p = reinterpret_cast<const float4 *>(tb + sub * 8);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = __ldg(p + i);
        c[4 * i] = c[4 * i + 1] = v.x, c[4 * i + 2] = c[4 * i + 3] = v.z;
        sn[4 * i] = -v.y, sn[4 * i + 1] = v.y, sn[4 * i + 2] = -v.w, sn[4 * i + 3] = v.w;
      }
    } else {
      const int half = a.rot / 16;  // lanes of half a rotation
      const bool low = sub < half;
      partner = low ? lane + half : lane - half;
      const float4 *p = reinterpret_cast<const float4 *>(tb + (low ? sub : sub - half) * 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = __ldg(p + i);
        c[2 * i] = v.x, c[2 * i + 1] = v.z;
        sn[2 * i] = low ? -v.y : v.y, sn[2 * i + 1] = low ? -v.w : v.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, sn[i] = 0.f;
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int h = head0 + s * PER;
    const bool is_q = h < a.H_q, is_v = h >= a.H_q + a.H;
    const float *w = is_q ? a.qw : a.kw;
    const uint32_t in[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(in[i] << 16), x[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
    if (a.qw || a.kw) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      if (w && !is_v) {
        const float f = rsqrtf(ss * (1.f / D) + a.eps);
        const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + sub * 8));
        const float4 w1 = __ldg(reinterpret_cast<const float4 *>(w + sub * 8 + 4));
        x[0] *= f * w0.x, x[1] *= f * w0.y, x[2] *= f * w0.z, x[3] *= f * w0.w;
        x[4] *= f * w1.x, x[5] *= f * w1.y, x[6] *= f * w1.z, x[7] *= f * w1.w;
      }
    }
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = PAIRS ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], partner);
      z[i] = turned ? fmaf(other, sn[i], x[i] * c[i]) : x[i];
    }
    if (h >= heads) continue;
    uint4 v = make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
    uint16_t *dst;
    if (is_q) {
      dst = a.q + ((int64_t)t * a.H_q + h) * D;
    } else {
      const int hk = is_v ? h - a.H_q - a.H : h - a.H_q;
      dst = (is_v ? a.V : a.K) + (((int64_t)b * a.H + hk) * a.Nmax + row) * D;
      if (is_v) v = raw[s];
    }
    *reinterpret_cast<uint4 *>(dst + sub * 8) = v;
  }
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace

extern "C" int tg_qk_norm_rope(tg_stream_t stream, int batch, int T, int H_q, int H, int d, int Nmax, int rot,
                               int max_pos, uint32_t flags, const int32_t *cu_q, const int32_t *start,
                               const uint16_t *qkv, int64_t qkv_stride, const float *q_weight, const float *k_weight,
                               float eps, const int32_t *positions, const float *cos_sin, uint16_t *q, uint16_t *K,
                               uint16_t *V, int32_t *dev_status) {
  const char *fn = "tg_qk_norm_rope";
  using tgi::fail;
  if (batch <= 0 || T < 0 || H_q <= 0 || H <= 0 || Nmax <= 0)
    return fail(TG_ERR_INVALID_ARG, "%s: batch=%d, T=%d, H_q=%d, H=%d, Nmax=%d", fn, batch, T, H_q, H, Nmax);
  if (d != 128 && d != 256) return fail(TG_ERR_SHAPE, "%s: d=%d (128 or 256)", fn, d);
  if (rot < 0 || rot > d || rot % 16) return fail(TG_ERR_SHAPE, "%s: rot=%d (a multiple of 16 in [0, d])", fn, rot);
  if (flags & ~TG_ROPE_PAIRS) return fail(TG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
  const int64_t heads = (int64_t)H_q + 2 * (int64_t)H;
  if (heads * d > INT32_MAX) return fail(TG_ERR_SHAPE, "%s: H_q + 2 H = %lld heads", fn, (long long)heads);
  if (qkv_stride < heads * d || qkv_stride % 8)
    return fail(TG_ERR_SHAPE, "%s: qkv_stride=%lld (a multiple of 8, at least %lld)", fn, (long long)qkv_stride,
                (long long)(heads * d));
  if (!std::isfinite(eps)) return fail(TG_ERR_NONFINITE, "%s: eps is not finite", fn);
  if (eps < 0.f) return fail(TG_ERR_INVALID_ARG, "%s: eps=%g < 0", fn, (double)eps);
  if (T == 0) return tgi::ok();
  if (!cu_q || !start || !qkv || !q || !K || !V) return fail(TG_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (rot > 0 && (!cos_sin || max_pos <= 0)) return fail(TG_ERR_INVALID_ARG, "%s: rot=%d without a table", fn, rot);
  if (misaligned(qkv, 16) || misaligned(q, 16) || misaligned(K, 16) || misaligned(V, 16) || misaligned(cos_sin, 16) ||
      misaligned(q_weight, 16) || misaligned(k_weight, 16))
    return fail(TG_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
  RopeArgs a;
  a.cu_q = cu_q, a.start = start, a.positions = positions, a.qkv = qkv, a.stride = qkv_stride;
  a.qw = q_weight, a.kw = k_weight, a.table = cos_sin, a.q = q, a.K = K, a.V = V, a.status = dev_status;
  a.batch = batch, a.T = T, a.H_q = H_q, a.H = H, a.Nmax = Nmax, a.rot = rot, a.max_pos = max_pos, a.eps = eps;
  const int per = kSteps * (d == 128 ? 2 : 1);
  a.chunks = (int)((heads + per - 1) / per);
  const int64_t blocks = ((int64_t)T * a.chunks + kWarps - 1) / kWarps;
  if (blocks > INT32_MAX) return fail(TG_ERR_SHAPE, "%s: T=%d with %lld heads", fn, T, (long long)heads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool pairs = flags & TG_ROPE_PAIRS;
  const dim3 grid((unsigned)blocks), block(kWarps * 32);
  if (d == 128) {
    if (pairs) qk_norm_rope_kernel<128, true><<<grid, block, 0, s>>>(a);
    else qk_norm_rope_kernel<128, false><<<grid, block, 0, s>>>(a);
  } else {
    if (pairs) qk_norm_rope_kernel<256, true><<<grid, block, 0, s>>>(a);
    else qk_norm_rope_kernel<256, false><<<grid, block, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return tgi::ok();
}
