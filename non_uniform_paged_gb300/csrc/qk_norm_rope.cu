// Query/key RMS norm, position rotation and placement of the context rows (tg_qk_norm_rope).
//
// Mathematics: y = x * rsqrt(mean(x^2) + eps) * w per head, then the plane rotation of each
// pair by the table's (cos, sin).  Every value is read once and written once: the kernel is
// bound by memory, and for a decode step by its own latency.
//
// A head is d / 8 lanes: half a warp at d = 128, a warp at d = 256.  A lane has two groups of 4
// values: of the pairs (i, i + rot/2), 4 first and the 4 second values, so that a rotation needs
// no exchange between lanes (a group of 4 is still 128 contiguous bytes over half a warp); of
// the pairs (2i, 2i+1) and behind rot, 8 consecutive ones.  A warp takes one token and walks over
// its heads in batches of 4 loads, each batch queries, keys or values only, the next one in
// flight while one is worked on; the request's row and the table row are looked up once.
// What bounds it beside memory is instructions (at 4400 a token the issue slots would take as
// long as the bytes): the weights are multiplied into the token's rotation once a batch, and
// the arithmetic is two values an instruction.  Where there are few tokens, a token's batches
// go to different warps.
#include "packed.cuh"
#include "ptx.cuh"
#include "tg_internal.h"

#include <cuda_runtime.h>

#include <cmath>

namespace {

using namespace tgk;

constexpr int kSteps = 4;  // loads of a batch: heads at d = 256, pairs of heads at d = 128
// Blocks of one warp, 24 to an SM: a block's place is free when its token is done.  For 20000 tokens
// of 32 + 16 heads of 128, blocks of 4 warps took 92 us, of one 88; batches of 4 instead of 8 loads,
// with 24 instead of 16 warps to an SM, 81.  (At 80 registers the d = 128 forms spill 8 and 20 bytes.)
constexpr int kBlocks = 24;

struct RopeArgs {
  const int32_t *cu_q, *start, *positions;
  const uint16_t *qkv;
  int64_t stride;
  const float *qw, *kw;
  const float *table;
  uint16_t *q, *K, *V;
  int32_t *status;
  int batch, T, H_q, H, Nmax, rot, max_pos;
  int q_batches, kv_batches;  // batches of the query heads, and of the key (and of the value) heads
  int parts;                  // warps of a token: one, or one for each of its batches
  float eps;
};

struct Head8 {  // a lane's 8 values of a head
  uint2 a, b;
};

__device__ __forceinline__ float2 unpack2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(32, kBlocks) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES;  // lanes of a head, heads side by side
  const int lane = threadIdx.x, sub = lane % LANES, side = lane / LANES;
  const int all = a.q_batches + 2 * a.kv_batches;
  const int t = blockIdx.x / a.parts, part = blockIdx.x - t * a.parts;
  const int first = part, last = a.parts == 1 ? all : part + 1;
  // the two groups of this lane
  const bool turned = sub * 8 < a.rot;
  const int ga = !PAIRS && turned ? sub * 4 : sub * 8, gb = !PAIRS && turned ? sub * 4 + a.rot / 2 : sub * 8 + 4;
  const uint16_t *src = a.qkv + (int64_t)t * a.stride;
  // batch k: kind (0 queries, 1 keys, 2 values), first head of its kind, heads of its kind
  auto kind_of = [&](int k) { return k < a.q_batches ? 0 : k < a.q_batches + a.kv_batches ? 1 : 2; };
  auto head_of = [&](int k, int kind) {
    return (k - (kind == 0 ? 0 : kind == 1 ? a.q_batches : a.q_batches + a.kv_batches)) * kSteps * PER;
  };
  auto load = [&](Head8 *x, int k) {
    const int kind = kind_of(k), h0 = head_of(k, kind) + side, n = kind == 0 ? a.H_q : a.H;
    const uint16_t *p = src + ((kind == 0 ? 0 : kind == 1 ? a.H_q : a.H_q + a.H) + h0) * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (h0 + s * PER < n) {
        x[s].a = __ldcs(reinterpret_cast<const uint2 *>(p + s * PER * D + ga));
        x[s].b = __ldcs(reinterpret_cast<const uint2 *>(p + s * PER * D + gb));
      }
    }
  };
  griddep_wait();  // a programmatic dependent of the kernel before it: set up while that one ends
  Head8 x0[kSteps] = {}, x1[kSteps] = {};
  load(x0, first);  // does not wait for the request's lookup
  // The request: how many end at or before t, 32 at a time.  (4096 requests of one token take 34 us,
  // 4096 tokens of one request 16.)
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
  // this lane's four pairs
  float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (turned) {
    const float4 *p = reinterpret_cast<const float4 *>(a.table + pos * a.rot + sub * 8);  // [rot/2][2]
    const float4 u = __ldg(p), v = __ldg(p + 1);
    c[0] = u.x, sn[0] = u.y, c[1] = u.z, sn[1] = u.w, c[2] = v.x, sn[2] = v.y, c[3] = v.z, sn[3] = v.w;
  }
  const int64_t kv_row = ((int64_t)b * a.H * a.Nmax + row) * D, kv_head = (int64_t)a.Nmax * D;

  auto work = [&](const Head8 *in, int k) {
    const int kind = kind_of(k), h0 = head_of(k, kind) + side, n = kind == 0 ? a.H_q : a.H;
    const int64_t step = kind == 0 ? PER * D : PER * kv_head;
    uint16_t *dst = kind == 0 ? a.q + ((int64_t)t * a.H_q + h0) * D : (kind == 1 ? a.K : a.V) + kv_row + h0 * kv_head;
    if (kind == 2) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s, dst += step) {
        if (h0 + s * PER < n) {
          *reinterpret_cast<uint2 *>(dst + ga) = in[s].a;
          *reinterpret_cast<uint2 *>(dst + gb) = in[s].b;
        }
      }
      return;
    }
    // z_u = uc x_u - vs x_v, z_v = vc x_v + us x_u, the weights multiplied in; u, v: a lane's first and
    // second values of its pairs
    const float *w = kind == 0 ? a.qw : a.kw;
    float wu[4] = {1.f, 1.f, 1.f, 1.f}, wv[4] = {1.f, 1.f, 1.f, 1.f};
    if (w) {
      const float4 p = __ldg(reinterpret_cast<const float4 *>(w + ga)), q = __ldg(reinterpret_cast<const float4 *>(w + gb));
      const float e[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) wu[i] = e[PAIRS ? 2 * i : i], wv[i] = e[PAIRS ? 2 * i + 1 : i + 4];
    }
    float2 uc[2], us[2], vc[2], vs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 cc = {c[2 * i], c[2 * i + 1]}, ss = {sn[2 * i], sn[2 * i + 1]};
      const float2 u = {wu[2 * i], wu[2 * i + 1]}, v = {wv[2 * i], wv[2 * i + 1]};
      uc[i] = mul2(u, cc), us[i] = mul2(u, ss), vc[i] = mul2(v, cc), vs[i] = mul2(v, make_float2(-ss.x, -ss.y));
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s, dst += step) {
      if (h0 - side + s * PER >= n) break;
      const float2 x[4] = {unpack2(in[s].a.x), unpack2(in[s].a.y), unpack2(in[s].b.x), unpack2(in[s].b.y)};
      float2 xu[2], xv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xu[i] = PAIRS ? make_float2(x[2 * i].x, x[2 * i + 1].x) : x[i];
        xv[i] = PAIRS ? make_float2(x[2 * i].y, x[2 * i + 1].y) : x[i + 2];
      }
      float2 zu[2], zv[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) zu[i] = mul2(uc[i], xu[i]), zv[i] = mul2(vc[i], xv[i]);
      if (turned) {  // behind rot a value meets no other: 0 times an infinite one would be NaN
#pragma unroll
        for (int i = 0; i < 2; ++i) zu[i] = fma2(vs[i], xv[i], zu[i]), zv[i] = fma2(us[i], xu[i], zv[i]);
      }
      if (w) {
        float2 sq = mul2(xu[0], xu[0]);
        sq = fma2(xu[1], xu[1], sq), sq = fma2(xv[0], xv[0], sq), sq = fma2(xv[1], xv[1], sq);
        float ss = sq.x + sq.y;
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float f = rsqrtf(fmaf(ss, 1.f / D, a.eps));
        const float2 ff = {f, f};
#pragma unroll
        for (int i = 0; i < 2; ++i) zu[i] = mul2(zu[i], ff), zv[i] = mul2(zv[i], ff);
      }
      if (h0 + s * PER >= n) continue;
      Head8 o;
      if (PAIRS) {
        o.a = make_uint2(pack_bf16x2(zu[0].x, zv[0].x), pack_bf16x2(zu[0].y, zv[0].y));
        o.b = make_uint2(pack_bf16x2(zu[1].x, zv[1].x), pack_bf16x2(zu[1].y, zv[1].y));
      } else {
        o.a = make_uint2(pack_bf16x2(zu[0].x, zu[0].y), pack_bf16x2(zu[1].x, zu[1].y));
        o.b = make_uint2(pack_bf16x2(zv[0].x, zv[0].y), pack_bf16x2(zv[1].x, zv[1].y));
      }
      *reinterpret_cast<uint2 *>(dst + ga) = o.a;
      *reinterpret_cast<uint2 *>(dst + gb) = o.b;
    }
  };
  for (int k = first; k < last; k += 2) {
    if (k + 1 < last) load(x1, k + 1);
    work(x0, k);
    if (k + 1 >= last) break;
    if (k + 2 < last) load(x0, k + 2);
    work(x1, k + 1);
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
  // A warp a token, or, below 2048 tokens, one for each of its batches: 256 tokens of 32 + 16 heads of
  // 128 take 6.6 us one way and 3.2 the other, 2048 tokens 10.3 and 10.0, 4096 tokens 15.0 and 18.7.
  // (Other head counts were not measured; with more heads a token's warp has more batches in a row.)
  const int per = kSteps * (d == 128 ? 2 : 1);
  a.q_batches = (H_q + per - 1) / per;
  a.kv_batches = (H + per - 1) / per;
  a.parts = T < 2048 ? a.q_batches + 2 * a.kv_batches : 1;
  const int64_t blocks = (int64_t)T * a.parts;
  if (blocks > INT32_MAX) return fail(TG_ERR_SHAPE, "%s: T=%d with %lld heads", fn, T, (long long)heads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool pairs = flags & TG_ROPE_PAIRS;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = d == 128 ? (pairs ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<128, true>, a)
                                          : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<128, false>, a))
                                 : (pairs ? cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<256, true>, a)
                                          : cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<256, false>, a));
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return tgi::ok();
}
