// Query/key RMS norm, position rotation and the new tokens' rows behind the retained ones in the pages
// (tg_append_rope): bf16 pages, or 4-bit pages with the rounding done on the way.
//
// Mathematics: norm and rotation as tg_qk_norm_rope; the row of token i of request b in head h is token
// ntok[b][h] + added[b] + i of the head's page list.  Every projection is read once and written once: bound by
// memory, and for a decode step by the chain request -> its tokens' count -> page id -> store.
//
// A block is a warp: one token, or one batch of a token's heads where there are few tokens.  A head is d / 8
// lanes; a lane's 8 values are 4 first and the 4 second ones of its pairs (i, i + rot/2), so that the rotation
// exchanges nothing, or 8 consecutive ones (pairs (2i, 2i + 1), values behind rot, V).  Each batch's heads have
// their rows looked up by as many lanes at once, before their values are needed.
//
// 4-bit pages.  A head's rotated values go through shared memory, so that a lane has 8 consecutive ones and a pair
// of lanes a block of 16.  float32 leaves a value z off by some 2^-20 of the row's largest, which decides a
// code or a scale wrongly where z / s comes that close to the border of two.  So both are taken of the value moved
// down and up by 2^-18 of the row's largest; where they differ (a row in a hundred) the row is computed
// again in float64, from the projections in registers.  V is exact and needs none of this.
#include "page4.cuh"
#include "ptx.cuh"
#include "tg_internal.h"

#include <cuda_runtime.h>

#include <cmath>

namespace {

using namespace tgk;

constexpr int kSteps = 4;  // loads of a batch: heads at d = 256, pairs of heads at d = 128

struct AppendArgs {
  const int32_t *cu_q, *positions, *origin, *head_order, *ntok, *added, *pt_ids, *start;
  const int64_t *pt_off;
  const uint16_t *qkv;
  int64_t stride, pool_pages;
  const float *qw, *kw, *table;
  uint8_t *pool;
  uint16_t *q, *K, *V;
  int32_t *status;
  int batch, H_q, H, H_p, P, Nmax, rot, max_pos, axes, reserve;
  int q_batches, kv_batches;  // batches of the query heads, and of the key (and of the value) heads
  int parts;                  // warps of a token: one, or one for each of its batches
  float eps, k_unit, v_unit;
  uint32_t axis[8];  // two bits for each pair
};

struct Head8 {  // a lane's 8 values of a head
  uint2 a, b;
};

__device__ __forceinline__ float2 unpack2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void unpack8(const Head8 &h, float (&x)[8]) {
  const uint32_t w[4] = {h.a.x, h.a.y, h.b.x, h.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(w[i]);
    x[2 * i] = f.x, x[2 * i + 1] = f.y;
  }
}
// a float64 value in float32 for a rounding to a few bits: cut off, the last bit set where something was
__device__ __forceinline__ float sticky(double v) {
  float f = __double2float_rz(v);
  if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

template <int D, bool PAIRS, bool E2M1>
__global__ void __launch_bounds__(32, E2M1 ? 20 : 24) append_rope_kernel(const AppendArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES;  // lanes of a head, heads side by side
  constexpr int BATCH = kSteps * PER;             // heads of a batch
  __shared__ __align__(16) float zs[E2M1 ? PER * D : 1];
  __shared__ __align__(16) double zd[E2M1 ? PER * D : 1];
  const int lane = threadIdx.x, sub = lane % LANES, side = lane / LANES;
  const int all = a.q_batches + 2 * a.kv_batches;
  const int t = blockIdx.x / a.parts, part = blockIdx.x - t * a.parts;
  const int first = part, last = a.parts == 1 ? all : part + 1;
  // the two groups of this lane in a query or key head; of a value head they are 8 consecutive values
  const bool turned = sub * 8 < a.rot;
  const int ga = !PAIRS && turned ? sub * 4 : sub * 8, gb = !PAIRS && turned ? sub * 4 + a.rot / 2 : sub * 8 + 4;
  const uint16_t *src = a.qkv + (int64_t)t * a.stride;
  auto kind_of = [&](int k) { return k < a.q_batches ? 0 : k < a.q_batches + a.kv_batches ? 1 : 2; };
  auto head_of = [&](int k, int kind) {  // first head, or place in the groups, of batch k
    return (k - (kind == 0 ? 0 : kind == 1 ? a.q_batches : a.q_batches + a.kv_batches)) * BATCH;
  };
  griddep_wait();  // a programmatic dependent of the kernel before it: set up while that one ends

  // the request: how many end at or before t, 32 at a time
  int b = 0;
  for (int i = 0; i < a.batch; i += 32) {
    const int32_t end = i + lane < a.batch ? __ldg(a.cu_q + i + lane + 1) : INT32_MAX;
    const unsigned m = __ballot_sync(0xffffffffu, end <= t);
    b += __popc(m);
    if (m != 0xffffffffu) break;
  }
  if (b >= a.batch) return;  // behind the last request
  const int i = t - __ldg(a.cu_q + b);
  const int64_t grown = a.added ? __ldg(a.added + b) : 0;
  const int64_t row = a.K ? (int64_t)__ldg(a.start + b) + i : 0;
  bool bad = grown < 0 || grown + i >= a.reserve || (a.K && (row < 0 || row >= a.Nmax));
  // this lane's four pairs
  float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.rot > 0) {
    const int64_t half = a.rot / 2;
    if (a.axes == 1) {
      const int64_t pos = a.positions ? (int64_t)__ldg(a.positions + t) : (int64_t)__ldg(a.origin + b) + grown + i;
      bad = bad || pos < 0 || pos >= a.max_pos;
      if (turned && !bad) {
        const float4 *p = reinterpret_cast<const float4 *>(a.table + (pos * half + sub * 4) * 2);  // [rot/2][2]
        const float4 u = __ldg(p), v = __ldg(p + 1);
        c[0] = u.x, sn[0] = u.y, c[1] = u.z, sn[1] = u.w, c[2] = v.x, sn[2] = v.y, c[3] = v.z, sn[3] = v.w;
      }
    } else if (turned) {
      const uint32_t ax = a.axis[sub / 4] >> (8 * (sub & 3));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t pos = __ldg(a.positions + (int64_t)t * a.axes + (ax >> (2 * j) & 3));
        const bool out = pos < 0 || pos >= a.max_pos;
        bad = bad || out;
        if (!out) {
          const float2 u = __ldg(reinterpret_cast<const float2 *>(a.table + (pos * half + sub * 4 + j) * 2));
          c[j] = u.x, sn[j] = u.y;
        }
      }
    }
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) report(a.status, TG_STATUS_BAD_INPUT);
    return;
  }

  // Lane j < BATCH looks up place p0 + j of the groups: its head, and the token's row in its pages: of bf16 pages a row
  // number (K; V is P behind it), of 4-bit pages the byte of its tile times 16 plus its row there; -1: none.
  auto look_up = [&](int p0, int &head, int64_t &at) {
    head = -1, at = -1;
    const int p = p0 + lane;
    if (lane >= BATCH || p >= a.H) return;
    head = __ldg(a.head_order + p);
    if (head < 0 || head >= a.H) {
      head = -1;
      report(a.status, TG_STATUS_BAD_INPUT);
      return;
    }
    const int64_t slot = __ldg(a.ntok + (int64_t)b * a.H + head) + grown + i;
    const int64_t *off = a.pt_off + (int64_t)b * (a.H / a.H_p) + p / a.H_p;
    const int64_t at0 = __ldg(off), at1 = __ldg(off + 1), pg = slot / a.P;
    const int r = (int)(slot - pg * a.P), hp = p % a.H_p;
    const int32_t page = slot >= 0 && at0 + pg < at1 ? __ldg(a.pt_ids + at0 + pg) : -1;
    if (page < 0 || page >= a.pool_pages) {
      report(a.status, TG_STATUS_BAD_PAGE);
      return;
    }
    const int64_t in = (int64_t)page * a.H_p + hp;
    at = E2M1 ? (in * (a.P / 16) + r / 16) * (D / 128 * kTile4) * 16 + r % 16 : in * 2 * a.P + r;
  };
  auto load = [&](Head8 *x, int kind, int h0, int head) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = kind == 0 ? h0 + s * PER + side : __shfl_sync(0xffffffffu, head, s * PER + side);
      if (h < 0 || (kind == 0 && h >= a.H_q)) continue;
      const uint16_t *p = src + ((kind == 0 ? 0 : kind == 1 ? a.H_q : a.H_q + a.H) + h) * D;
      x[s].a = __ldcs(reinterpret_cast<const uint2 *>(p + (kind == 2 ? sub * 8 : ga)));
      x[s].b = __ldcs(reinterpret_cast<const uint2 *>(p + (kind == 2 ? sub * 8 + 4 : gb)));
    }
  };
  auto store4 = [&](const Code8 &o, int64_t at, int kind) {
    uint8_t *tile = a.pool + (at >> 4) + sub / 16 * kTile4;
    const int r = (int)(at & 15), e = sub % 16;
    *reinterpret_cast<uint32_t *>(tile + (kind == 1 ? k_codes4(r, e) : v_codes4(r, e))) = o.codes;
    if (!(e & 1)) tile[kind == 1 ? k_scale4(r, e / 2) : v_scale4(r, e / 2)] = (uint8_t)o.scale;
  };
  auto dense = [&](int kind, int h) { return (kind == 1 ? a.K : a.V) + (((int64_t)b * a.H + h) * a.Nmax + row) * D; };

  for (int k = first; k < last; ++k) {
    const int kind = kind_of(k), h0 = head_of(k, kind);
    int head = -1;
    int64_t at = -1;
    if (kind != 0) look_up(h0, head, at);
    Head8 in[kSteps] = {};
    load(in, kind, h0, head);
    if (kind == 2) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int h = __shfl_sync(0xffffffffu, head, s * PER + side);
        const int64_t to = __shfl_sync(0xffffffffu, at, s * PER + side);
        const uint4 raw = make_uint4(in[s].a.x, in[s].a.y, in[s].b.x, in[s].b.y);
        if (!E2M1) {
          if (to >= 0) *reinterpret_cast<uint4 *>(a.pool + ((to + a.P) * D + sub * 8) * 2) = raw;
          if (a.V && h >= 0 && to >= 0) *reinterpret_cast<uint4 *>(dense(2, h) + sub * 8) = raw;
          continue;
        }
        float x[8];
        unpack8(in[s], x);
        bool odd = false;
        const Code8 o = encode_exact(x, a.v_unit, odd);
        if (odd) report(a.status, TG_STATUS_NONFINITE);
        if (h < 0 || to < 0) continue;
        store4(o, to, 2);
        if (a.V) *reinterpret_cast<uint4 *>(dense(2, h) + sub * 8) = held8(o, a.v_unit);
      }
      continue;
    }
    const float *w = kind == 0 ? a.qw : a.kw;
    float wu[4] = {1.f, 1.f, 1.f, 1.f}, wv[4] = {1.f, 1.f, 1.f, 1.f};
    if (w) {
      const float4 p = __ldg(reinterpret_cast<const float4 *>(w + ga)), q = __ldg(reinterpret_cast<const float4 *>(w + gb));
      const float e[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) wu[j] = e[PAIRS ? 2 * j : j], wv[j] = e[PAIRS ? 2 * j + 1 : j + 4];
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = kind == 0 ? (h0 + s * PER + side < a.H_q ? h0 + s * PER + side : -1)
                              : __shfl_sync(0xffffffffu, head, s * PER + side);
      const int64_t to = kind == 0 ? 0 : __shfl_sync(0xffffffffu, at, s * PER + side);
      if (h0 + s * PER >= (kind == 0 ? a.H_q : a.H)) break;
      float x[8], xu[4], xv[4], zu[4], zv[4];
      unpack8(in[s], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xu[j] = x[PAIRS ? 2 * j : j], xv[j] = x[PAIRS ? 2 * j + 1 : j + 4];
        zu[j] = wu[j] * c[j] * xu[j], zv[j] = wv[j] * c[j] * xv[j];
        if (turned) {  // behind rot a value meets no other: 0 times an infinite one would be NaN
          zu[j] = fmaf(-sn[j] * wv[j], xv[j], zu[j]);
          zv[j] = fmaf(sn[j] * wu[j], xu[j], zv[j]);
        }
      }
      if (w) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        const float f = rsqrtf(fmaf(ss, 1.f / D, a.eps));
#pragma unroll
        for (int j = 0; j < 4; ++j) zu[j] *= f, zv[j] *= f;
      }
      if (kind == 0 || !E2M1) {
        if (h < 0 || to < 0) continue;
        Head8 o;
        if (PAIRS) {
          o.a = make_uint2(pack_bf16x2(zu[0], zv[0]), pack_bf16x2(zu[1], zv[1]));
          o.b = make_uint2(pack_bf16x2(zu[2], zv[2]), pack_bf16x2(zu[3], zv[3]));
        } else {
          o.a = make_uint2(pack_bf16x2(zu[0], zu[1]), pack_bf16x2(zu[2], zu[3]));
          o.b = make_uint2(pack_bf16x2(zv[0], zv[1]), pack_bf16x2(zv[2], zv[3]));
        }
        uint16_t *dst = kind == 0 ? a.q + ((int64_t)t * a.H_q + h) * D : reinterpret_cast<uint16_t *>(a.pool) + to * D;
        *reinterpret_cast<uint2 *>(dst + ga) = o.a;
        *reinterpret_cast<uint2 *>(dst + gb) = o.b;
        if (kind == 1 && a.K) {
          dst = dense(1, h);
          *reinterpret_cast<uint2 *>(dst + ga) = o.a;
          *reinterpret_cast<uint2 *>(dst + gb) = o.b;
        }
        continue;
      }
      // ---- 4-bit K
      float z[8];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        zs[side * D + ga + (PAIRS ? 2 * j : j)] = zu[j];
        zs[side * D + (PAIRS ? ga + 2 * j + 1 : gb + j)] = zv[j];
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = zs[side * D + sub * 8 + j];
      Code8 o;
      if (!w && a.rot == 0) {  // the projections themselves
        bool odd = false;
        o = encode_exact(z, a.k_unit, odd);
        if (odd) report(a.status, TG_STATUS_NONFINITE);
      } else {
        const float to_unit = 1.f / a.k_unit;  // exact
        float top = 0.f;
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(z[j])), odd = odd || not_finite(z[j]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        float most = top;
#pragma unroll
        for (int d = 2; d < LANES; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        // (values that only passed through, behind rot without a norm, are exact: their ties are no doubt)
        const bool passed = !w && sub * 8 >= a.rot;
        const float off = passed ? 0.f : most * 0x1p-18f;
        o.scale = max(e4m3_of(__fdiv_rn(fmaxf(top - off, 0.f) * to_unit, 6.f)), 1u);
        bool near = o.scale != max(e4m3_of(__fdiv_rn((top + off) * to_unit, 6.f)), 1u);
        const float inv = 1.f / e4m3_to_float(o.scale) * to_unit, move = off * inv;
        o.codes = 0;
        uint32_t up = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float r0 = passed ? over_scale_exact(z[2 * j], inv) : z[2 * j] * inv;
          const float r1 = passed ? over_scale_exact(z[2 * j + 1], inv) : z[2 * j + 1] * inv;
          o.codes |= e2m1x2_of(r0 - move, r1 - move) << (8 * j);
          up |= e2m1x2_of(r0 + move, r1 + move) << (8 * j);
        }
        near = near || o.codes != up;
        if (odd) report(a.status, TG_STATUS_NONFINITE);
        if (__any_sync(0xffffffffu, near)) {
          // the row again in float64
          double f = 1.0;
          if (w) {
            double ss = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += (double)x[j] * (double)x[j];
#pragma unroll
            for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            f = 1.0 / sqrt(ss / D + (double)a.eps);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const double yu = (double)xu[j] * f * wu[j], yv = (double)xv[j] * f * wv[j];
            const double u = turned ? yu * c[j] - yv * sn[j] : yu, v = turned ? yv * c[j] + yu * sn[j] : yv;
            zd[side * D + ga + (PAIRS ? 2 * j : j)] = u;
            zd[side * D + (PAIRS ? ga + 2 * j + 1 : gb + j)] = v;
          }
          __syncwarp();
          double zz[8], dt = 0.0;
#pragma unroll
          for (int j = 0; j < 8; ++j) zz[j] = zd[side * D + sub * 8 + j], dt = fmax(dt, fabs(zz[j]));
          dt = fmax(dt, __shfl_xor_sync(0xffffffffu, dt, 1));
          o.scale = max(e4m3_of(sticky(dt / (6.0 * a.k_unit))), 1u);
          const double sc = (double)e4m3_to_float(o.scale) * a.k_unit;
          o.codes = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) o.codes |= e2m1x2_of(sticky(zz[2 * j] / sc), sticky(zz[2 * j + 1] / sc)) << (8 * j);
        }
      }
      if (h < 0 || to < 0) continue;
      store4(o, to, 1);
      if (a.K) *reinterpret_cast<uint4 *>(dense(1, h) + sub * 8) = held8(o, a.k_unit);
    }
  }
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

template <int D>
cudaError_t launch(const cudaLaunchConfig_t &cfg, bool pairs, bool e2m1, const AppendArgs &a) {
  if (e2m1)
    return pairs ? cudaLaunchKernelEx(&cfg, append_rope_kernel<D, true, true>, a)
                 : cudaLaunchKernelEx(&cfg, append_rope_kernel<D, false, true>, a);
  return pairs ? cudaLaunchKernelEx(&cfg, append_rope_kernel<D, true, false>, a)
               : cudaLaunchKernelEx(&cfg, append_rope_kernel<D, false, false>, a);
}

}  // namespace

extern "C" int tg_append_rope(tg_stream_t stream, int batch, int T, int H_q, int H, int H_p, int P, int d, int rot,
                              int max_pos, uint32_t flags, const int32_t *cu_q, const uint16_t *qkv, int64_t qkv_stride,
                              const float *q_weight, const float *k_weight, float eps, int axes, const int32_t *positions,
                              const uint8_t *axis_of, const int32_t *origin, const float *cos_sin,
                              const int32_t *head_order, const int32_t *ntok, const int32_t *added, int reserve,
                              const int64_t *pt_off, const int32_t *pt_ids, int format, float k_unit, float v_unit,
                              void *pool, int64_t pool_pages, uint16_t *q, uint16_t *K, uint16_t *V, int Nmax,
                              const int32_t *start, int32_t *dev_status) {
  const char *fn = "tg_append_rope";
  using tgi::fail;
  if (batch <= 0 || T < 0 || H_q <= 0 || H <= 0 || H_p <= 0 || P <= 0 || reserve < 0)
    return fail(TG_ERR_INVALID_ARG, "%s: batch=%d, T=%d, H_q=%d, H=%d, H_p=%d, P=%d, reserve=%d", fn, batch, T, H_q, H,
                H_p, P, reserve);
  if (d != 128 && d != 256) return fail(TG_ERR_SHAPE, "%s: d=%d (128 or 256)", fn, d);
  if (H % H_p || P % 16) return fail(TG_ERR_SHAPE, "%s: H=%d of H_p=%d, P=%d (a multiple of 16)", fn, H, H_p, P);
  if (rot < 0 || rot > d || rot % 16) return fail(TG_ERR_SHAPE, "%s: rot=%d (a multiple of 16 in [0, d])", fn, rot);
  if (flags & ~TG_ROPE_PAIRS) return fail(TG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", fn, flags);
  if (format != TG_PAGES_BF16 && format != TG_PAGES_E2M1) return fail(TG_ERR_INVALID_ARG, "%s: format=%d", fn, format);
  const bool e2m1 = format == TG_PAGES_E2M1;
  if (e2m1 && (!unit_ok(k_unit) || !unit_ok(v_unit)))
    return fail(TG_ERR_INVALID_ARG, "%s: k_unit=%g, v_unit=%g (powers of two in [2^-60, 2^60])", fn, (double)k_unit,
                (double)v_unit);
  if (axes < 1 || axes > 4) return fail(TG_ERR_SHAPE, "%s: axes=%d (1..4)", fn, axes);
  const int64_t heads = (int64_t)H_q + 2 * (int64_t)H;
  if (heads * d > INT32_MAX) return fail(TG_ERR_SHAPE, "%s: H_q + 2 H = %lld heads", fn, (long long)heads);
  if (qkv_stride < heads * d || qkv_stride % 8)
    return fail(TG_ERR_SHAPE, "%s: qkv_stride=%lld (a multiple of 8, at least %lld)", fn, (long long)qkv_stride,
                (long long)(heads * d));
  if (!std::isfinite(eps)) return fail(TG_ERR_NONFINITE, "%s: eps is not finite", fn);
  if (eps < 0.f) return fail(TG_ERR_INVALID_ARG, "%s: eps=%g < 0", fn, (double)eps);
  if (pool_pages <= 0 || pool_pages > INT32_MAX)
    return fail(TG_ERR_CAPACITY, "%s: pool_pages=%lld (1..2^31-1)", fn, (long long)pool_pages);
  if (!K != !V) return fail(TG_ERR_INVALID_ARG, "%s: K and V go together", fn);
  if (K && (Nmax <= 0 || !start)) return fail(TG_ERR_INVALID_ARG, "%s: dense rows without Nmax and start", fn);
  AppendArgs a = {};
  if (rot > 0) {
    if (!cos_sin || max_pos <= 0) return fail(TG_ERR_INVALID_ARG, "%s: rot=%d without a table", fn, rot);
    if (axes == 1 ? !positions && !origin : !positions || !axis_of)
      return fail(TG_ERR_INVALID_ARG, "%s: %d axes without their positions", fn, axes);
    for (int i = 0; axes > 1 && i < rot / 2; ++i) {
      if (axis_of[i] >= axes) return fail(TG_ERR_INVALID_ARG, "%s: axis_of[%d]=%d of %d", fn, i, axis_of[i], axes);
      a.axis[i / 16] |= (uint32_t)axis_of[i] << (2 * (i % 16));
    }
  }
  if (T == 0) return tgi::ok();
  if (!cu_q || !qkv || !q || !pool || !head_order || !ntok || !pt_off || !pt_ids)
    return fail(TG_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (misaligned(qkv, 16) || misaligned(q, 16) || misaligned(K, 16) || misaligned(V, 16) || misaligned(cos_sin, 16) ||
      misaligned(q_weight, 16) || misaligned(k_weight, 16) || misaligned(pool, 16))
    return fail(TG_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", fn);
  a.cu_q = cu_q, a.positions = positions, a.origin = origin, a.head_order = head_order, a.ntok = ntok, a.added = added;
  a.pt_ids = pt_ids, a.start = start, a.pt_off = pt_off, a.qkv = qkv, a.stride = qkv_stride, a.pool_pages = pool_pages;
  a.qw = q_weight, a.kw = k_weight, a.table = cos_sin, a.pool = static_cast<uint8_t *>(pool), a.q = q, a.K = K, a.V = V;
  a.status = dev_status, a.batch = batch, a.H_q = H_q, a.H = H, a.H_p = H_p, a.P = P, a.Nmax = Nmax, a.rot = rot;
  a.max_pos = max_pos, a.axes = axes, a.reserve = reserve, a.eps = eps, a.k_unit = k_unit, a.v_unit = v_unit;
  // a warp a token, or, below 2048 tokens, one for each of its batches, as in tg_qk_norm_rope
  const int per = kSteps * (d == 128 ? 2 : 1);
  a.q_batches = (H_q + per - 1) / per;
  a.kv_batches = (H + per - 1) / per;
  a.parts = T < 2048 ? a.q_batches + 2 * a.kv_batches : 1;
  const int64_t blocks = (int64_t)T * a.parts;
  if (blocks > INT32_MAX) return fail(TG_ERR_SHAPE, "%s: T=%d with %lld heads", fn, T, (long long)heads);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool pairs = flags & TG_ROPE_PAIRS;
  const cudaError_t e = d == 128 ? launch<128>(cfg, pairs, e2m1, a) : launch<256>(cfg, pairs, e2m1, a);
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return tgi::ok();
}
