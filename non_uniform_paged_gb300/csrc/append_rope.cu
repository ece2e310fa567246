// Query/key RMS norm, position rotation and the new tokens' rows behind the retained ones in the pages
// (tg_append_rope): bf16 pages, or 4-bit pages with the rounding done on the way.
//
// Mathematics: norm and rotation as tg_qk_norm_rope; the row of token i of request b in head h is token
// ntok[b][h] + added[b] + i of the head's page list.  Every projection is read once and written once: bound by
// memory, and for a decode step by the chain request -> its tokens' count -> page id -> store.
//
// A block is a warp: a share of a token's batches of heads (which share: tg_append_rope below).  A head is d / 8
// lanes; a lane's 8 values are 4 first and the 4 second ones of its pairs (i, i + rot/2), so that the rotation
// exchanges nothing, or 8 consecutive ones (pairs (2i, 2i + 1), values behind rot, V).  Where the heads' rows lie is
// looked up once, for 32 places of the groups at a time, each by a lane; K and V lie side by side.  Queries, keys and
// values have a loop each; a batch of queries (a unit of 4-bit keys) is on its way while the one before it is worked
// on.  15000 tokens of 32 + 8 + 8 heads of 128 into bf16 pages, 372 MB: 68 us, 5.5 TB/s (71.5 with one loop for all
// three; 70.1 with 24 blocks to an SM and 72.9 with 20, for 28; 72.6 with batches of 2 loads for 4; one warp a token).
// The 72 registers of 28 blocks do not hold two batches of queries: 144 to 188 bytes a thread are spilled (64 to 136 read
// back), 4% of that call's instructions.
//
// 4-bit pages.  A head's rotated values go through shared memory, so that a lane has 8 consecutive ones and a pair
// of lanes a block of 16.  float32 leaves a value z = f (u c x_u - v s x_v) off by at most 15 2^-24 t,
// t = f (|u c x_u| + |v s x_v|): 11 in f (13 additions of squares halved by the root, 4 in rsqrtf), four roundings in the
// rest; z / s adds three, and two are to spare.  That decides a code or a scale wrongly where z / s comes so close
// to the border of two.  So both are taken of the value moved down and up by as much, with the block's
// largest t; where they differ (a row in some hundred) the row is computed again in float64, from the projections in
// registers, and what was open is taken from that.  V is exact and needs none of this.  (2500 tokens of 16 + 8 + 8 heads
// of 256: 30.5 us.  A bound by the row's largest value with float64 divisions costs 23 more; the keys'
// loop unrolled 16 more, waiting for instructions.)
#include "packed.cuh"
#include "page4.cuh"
#include "ptx.cuh"
#include "tg_internal.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

namespace {

using namespace tgk;

constexpr int kSteps = 4;  // loads of a batch: heads at d = 256, pairs of heads at d = 128
constexpr int kBlocksPerSm = 28, kBlocksPerSm4 = 20;  // of 72 and, for 4-bit pages, 96 registers
constexpr int kMaxParts = 512;                        // warps of a token
// A row whose mean square and eps together are below this is normalised as 2^100 times itself, with 2^200 eps: float32 loses squares
// of values below 2^-63.  The factor takes such a row to 2^54 at most.  Only an eps below it lets a row be one, and such calls run
// kernels of their own (SMALL): in the others the test alone costs 1% (68.0 and 68.7 us, 30.3 and 30.9).
constexpr float kSmallMean = 0x1p-100f, kSmallUp = 0x1p100f;

struct AppendArgs {
  const int32_t *cu_q, *positions, *origin, *head_order, *ntok, *added, *pt_ids, *start;
  const int64_t *pt_off;
  const uint16_t *qkv;
  int64_t stride, pool_pages;
  const float *qw, *kw, *table;
  uint8_t *pool;
  uint16_t *q, *K, *V;
  int32_t *status;
  int batch, H_q, H, H_p, G, P, Nmax, rot, max_pos, axes, reserve;
  // shares of work: batches of the query heads, of the key heads (4-bit pages: units, heads side by side) and of the value heads
  int q_batches, k_batches, v_batches;
  unsigned parts;             // warps of a token, each with an even share of its batches
  float eps, k_unit, v_unit, k_to_unit, v_to_unit;  // to: the reciprocals
  uint32_t axis[8];  // two bits for each pair
};

struct Head8 {  // a lane's 8 values of a head
  uint2 a, b;
};

__device__ __forceinline__ float2 unpack2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// A float64 value in float32 for a rounding to a few bits: cut off, the last bit set where something was, so that the
// rounding knows a tie.
__device__ __forceinline__ float sticky(double v) {
  float f = __double2float_rz(v);
  if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

template <int D, bool PAIRS, bool E2M1, bool SMALL>
__global__ void __launch_bounds__(32, E2M1 ? kBlocksPerSm4 : kBlocksPerSm) append_rope_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LANES = D / 8, PER = 32 / LANES;  // lanes of a head, heads side by side
  constexpr int BATCH = kSteps * PER;             // heads of a batch: divides 32
  __shared__ __align__(16) float zs[E2M1 ? PER * D : 1], ts[E2M1 ? PER * D / 4 : 1];
  __shared__ __align__(16) double zd[E2M1 ? PER * D : 1];
  const int lane = threadIdx.x, sub = lane % LANES, side = lane / LANES;
  const int t = (int)(blockIdx.x / a.parts);
  const unsigned part = blockIdx.x - t * a.parts;
  // the token's batches [first, last) of this warp: queries, then keys, then values
  const int k_first = a.q_batches, v_first = k_first + a.k_batches, all = v_first + a.v_batches;
  // (the product fits: at most 2^24 heads, and kMaxParts)
  const int first = (unsigned)all * part / a.parts, last = (unsigned)all * (part + 1) / a.parts;
  // the two groups of this lane in a query or key head; of a value head they are 8 consecutive values
  const bool turned = sub * 8 < a.rot;
  const int ga = !PAIRS && turned ? sub * 4 : sub * 8, gb = !PAIRS && turned ? sub * 4 + a.rot / 2 : sub * 8 + 4;
  const uint16_t *src = a.qkv + (int64_t)t * a.stride;
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
  const int grown = a.added ? __ldg(a.added + b) : 0;
  const int64_t row = a.K ? (int64_t)__ldg(a.start + b) + i : 0;

  // 32 places of the groups from p0 on, lane j's p0 + j: the head there (-1: none), and the number of the token's row in its
  // pages, counting rows of d values (bf16: K's; V's is P behind) or tokens of a head (4 bits); -1: none.
  int p0 = 0, head = -1, rows = -1;
  auto places = [&](int from, bool quiet) {
    p0 = from, head = rows = -1;
    const int p = p0 + lane;
    if (p >= a.H) return;
    const int h = __ldg(a.head_order + p);
    if (h < 0 || h >= a.H) {
      report(a.status, TG_STATUS_BAD_INPUT);
      return;
    }
    head = h;
    const int64_t far = (int64_t)__ldg(a.ntok + (int64_t)b * a.H + h) + grown + i;
    const unsigned group = (unsigned)p / (unsigned)a.H_p, hp = p - group * a.H_p;
    const int64_t *off = a.pt_off + (int64_t)b * a.G + group;
    const int64_t at0 = __ldg(off), at1 = __ldg(off + 1);
    const unsigned slot = (unsigned)far, pg = slot / (unsigned)a.P, r = slot - pg * a.P;
    const int32_t page = far >= 0 && far <= INT32_MAX && at0 + pg < at1 ? __ldg(a.pt_ids + at0 + pg) : -1;
    if (page < 0 || page >= a.pool_pages) {
      if (!quiet) report(a.status, TG_STATUS_BAD_PAGE);
      return;
    }
    rows = (page * a.H_p + (int)hp) * (E2M1 ? a.P : 2 * a.P) + (int)r;
  };
  bool bad = i < 0 || grown < 0 || (int64_t)grown + i >= a.reserve || (a.K && (row < 0 || row >= a.Nmax));
  // (a token that is refused below reports nothing of its pages)
  if (last > k_first)
    places(first <= k_first ? 0 : first >= v_first ? (first - v_first) * BATCH & ~31 : (first - k_first) * (E2M1 ? PER : BATCH) & ~31, bad);
  // this lane's four pairs
  float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.rot > 0) {
    const int half = a.rot / 2;
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
      int pos[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) pos[j] = __ldg(a.positions + (int64_t)t * a.axes + (ax >> (2 * j) & 3));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool out = pos[j] < 0 || pos[j] >= a.max_pos;
        bad = bad || out;
        const float2 u = __ldg(reinterpret_cast<const float2 *>(a.table + ((int64_t)(out ? 0 : pos[j]) * half + sub * 4 + j) * 2));
        c[j] = u.x, sn[j] = u.y;
      }
    }
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) report(a.status, TG_STATUS_BAD_INPUT);
    return;
  }
  // a lane's values of a query or key head
  auto load_turned = [&](Head8 &x, const uint16_t *from, int h) {
    x.a = __ldcs(reinterpret_cast<const uint2 *>(from + h * D + ga));
    x.b = __ldcs(reinterpret_cast<const uint2 *>(from + h * D + gb));
  };
  auto dense = [&](uint16_t *base, int h) { return base + (((int64_t)b * a.H + h) * a.Nmax + row) * D; };

  // The rotation with the weights multiplied in: z_u = uc x_u + vs x_v, z_v = vc x_v + us x_u; u, v: a lane's first and
  // second values of its pairs
  float2 uc[2], us[2], vc[2], vs[2];
  auto weigh = [&](const float *w) {
    float wu[4] = {1.f, 1.f, 1.f, 1.f}, wv[4] = {1.f, 1.f, 1.f, 1.f};
    if (w) {
      const float4 p = __ldg(reinterpret_cast<const float4 *>(w + ga)), q = __ldg(reinterpret_cast<const float4 *>(w + gb));
      const float e[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) wu[j] = e[PAIRS ? 2 * j : j], wv[j] = e[PAIRS ? 2 * j + 1 : j + 4];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 cc = {c[2 * j], c[2 * j + 1]}, ss = {sn[2 * j], sn[2 * j + 1]};
      const float2 u = {wu[2 * j], wu[2 * j + 1]}, v = {wv[2 * j], wv[2 * j + 1]};
      uc[j] = mul2(u, cc), us[j] = mul2(u, ss), vc[j] = mul2(v, cc), vs[j] = mul2(v, make_float2(-ss.x, -ss.y));
    }
  };
  auto split = [&](const Head8 &in, float2(&xu)[2], float2(&xv)[2]) {
    const float2 x[4] = {unpack2(in.a.x), unpack2(in.a.y), unpack2(in.b.x), unpack2(in.b.y)};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      xu[j] = PAIRS ? make_float2(x[2 * j].x, x[2 * j + 1].x) : x[j];
      xv[j] = PAIRS ? make_float2(x[2 * j].y, x[2 * j + 1].y) : x[j + 2];
    }
  };
  // what the norm multiplies the head's values by; those of a small row are scaled up here, by `lift`
  auto root = [&](float2(&xu)[2], float2(&xv)[2], float &lift) {
    auto mean = [&](float eps) {
      float2 sq = mul2(xu[0], xu[0]);
      sq = fma2(xu[1], xu[1], sq), sq = fma2(xv[0], xv[0], sq), sq = fma2(xv[1], xv[1], sq);
      float ss = sq.x + sq.y;
#pragma unroll
      for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      return fmaf(ss, 1.f / D, eps);
    };
    float m = mean(a.eps);
    if (SMALL) {
      lift = m < kSmallMean ? kSmallUp : 1.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) xu[j] = mul2(xu[j], make_float2(lift, lift)), xv[j] = mul2(xv[j], make_float2(lift, lift));
      m = mean(a.eps * lift * lift);
    }
    return rsqrtf(m);
  };

  // a lane's rotated values of a head, as bf16
  auto turn = [&](const Head8 &in, bool norm, uint2 &oa, uint2 &ob) {
    float2 xu[2], xv[2], zu[2], zv[2];
    split(in, xu, xv);
    float f, lift;
    if (SMALL && norm) f = root(xu, xv, lift);
#pragma unroll
    for (int j = 0; j < 2; ++j) zu[j] = mul2(uc[j], xu[j]), zv[j] = mul2(vc[j], xv[j]);
    if (turned) {  // behind rot a value meets no other: 0 times an infinite one would be NaN
#pragma unroll
      for (int j = 0; j < 2; ++j) zu[j] = fma2(vs[j], xv[j], zu[j]), zv[j] = fma2(us[j], xu[j], zv[j]);
    }
    if (norm) {
      if (!SMALL) f = root(xu, xv, lift);
#pragma unroll
      for (int j = 0; j < 2; ++j) zu[j] = mul2(zu[j], make_float2(f, f)), zv[j] = mul2(zv[j], make_float2(f, f));
    }
    if (PAIRS) {
      oa = make_uint2(pack_bf16x2(zu[0].x, zv[0].x), pack_bf16x2(zu[0].y, zv[0].y));
      ob = make_uint2(pack_bf16x2(zu[1].x, zv[1].x), pack_bf16x2(zu[1].y, zv[1].y));
    } else {
      oa = make_uint2(pack_bf16x2(zu[0].x, zu[0].y), pack_bf16x2(zu[1].x, zu[1].y));
      ob = make_uint2(pack_bf16x2(zv[0].x, zv[0].y), pack_bf16x2(zv[1].x, zv[1].y));
    }
  };

  // ---- queries: a batch is loaded while the one ahead of it is worked on
  if (first < k_first) {
    const int end = min(last, k_first);
    auto load = [&](Head8(&x)[kSteps], int k) {
      const int h0 = k * BATCH + side;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (h0 + s * PER < a.H_q) load_turned(x[s], src + s * PER * D, h0);
    };
    auto work = [&](const Head8(&x)[kSteps], int k) {
      uint16_t *dst = a.q + ((int64_t)t * a.H_q + k * BATCH + side) * D;
#pragma unroll
      for (int s = 0; s < kSteps; ++s, dst += PER * D) {
        if (k * BATCH + s * PER >= a.H_q) break;
        uint2 oa, ob;
        turn(x[s], a.qw != nullptr, oa, ob);
        if (k * BATCH + s * PER + side >= a.H_q) continue;
        *reinterpret_cast<uint2 *>(dst + ga) = oa;
        *reinterpret_cast<uint2 *>(dst + gb) = ob;
      }
    };
    Head8 x0[kSteps] = {}, x1[kSteps] = {};
    load(x0, first);
    weigh(a.qw);
    for (int k = first; k < end; k += 2) {
      if (k + 1 < end) load(x1, k + 1);
      work(x0, k);
      if (k + 1 >= end) break;
      if (k + 2 < end) load(x0, k + 2);
      work(x1, k + 1);
    }
  }
  // ---- keys of bf16 pages
  if (!E2M1) {
    const int begin = max(first, k_first), end = min(last, v_first);
    if (begin < end) weigh(a.kw);
    for (int k = begin; k < end; ++k) {
      const int h0 = (k - k_first) * BATCH;
      if ((h0 & ~31) != p0) places(h0 & ~31, false);
      Head8 x[kSteps] = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int h = __shfl_sync(0xffffffffu, head, (h0 + s * PER + side) & 31);
        if (h >= 0) load_turned(x[s], src + a.H_q * D, h);
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (h0 + s * PER >= a.H) break;
        uint2 oa, ob;
        turn(x[s], a.kw != nullptr, oa, ob);
        const int to = __shfl_sync(0xffffffffu, rows, (h0 + s * PER + side) & 31);
        const int h = __shfl_sync(0xffffffffu, head, (h0 + s * PER + side) & 31);
        if (to < 0) continue;
        uint16_t *dst = reinterpret_cast<uint16_t *>(a.pool) + (int64_t)to * D;
        *reinterpret_cast<uint2 *>(dst + ga) = oa;
        *reinterpret_cast<uint2 *>(dst + gb) = ob;
        if (a.K) {
          dst = dense(a.K, h);
          *reinterpret_cast<uint2 *>(dst + ga) = oa;
          *reinterpret_cast<uint2 *>(dst + gb) = ob;
        }
      }
    }
  }
  // ---- keys of 4-bit pages: one unit in a turn of the loop (what unrolling it adds to the code costs more than it hides)
  if (E2M1) {
    const int end = min(last, v_first) - k_first;  // units
    auto load = [&](Head8 &x, int u) {
      const int h = __shfl_sync(0xffffffffu, head, (u * PER + side) & 31);
      if (h >= 0) load_turned(x, src + a.H_q * D, h);
    };
    if (first < v_first && last > k_first) weigh(a.kw);
    Head8 nx = {};
    int loaded = -1;  // the unit in nx
    for (int u = max(first - k_first, 0); u < end; ++u) {
      if ((u * PER & ~31) != p0) places(u * PER & ~31, false);
      if (loaded != u) load(nx, u);
      const Head8 in = nx;
      if (u + 1 < end && ((u + 1) * PER & ~31) == p0) load(nx, loaded = u + 1);  // on its way meanwhile
      const int to = __shfl_sync(0xffffffffu, rows, (u * PER + side) & 31);
      const int h = __shfl_sync(0xffffffffu, head, (u * PER + side) & 31);
      const bool w = a.kw != nullptr;
      float2 xu[2], xv[2], zu[2], zv[2];
      split(in, xu, xv);
      float f = 1.f, lift = 1.f;
      if (SMALL && w) f = root(xu, xv, lift);
      float ta, tb;  // the largest |first product| + |second one| of the first and of the second group
#pragma unroll
      for (int j = 0; j < 2; ++j) zu[j] = mul2(uc[j], xu[j]), zv[j] = mul2(vc[j], xv[j]);
      if (turned) {  // behind rot a value meets no other: 0 times an infinite one would be NaN
        float2 tu[2], tv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 su = mul2(vs[j], xv[j]), sv = mul2(us[j], xu[j]);
          tu[j] = make_float2(fabsf(zu[j].x) + fabsf(su.x), fabsf(zu[j].y) + fabsf(su.y));
          tv[j] = make_float2(fabsf(zv[j].x) + fabsf(sv.x), fabsf(zv[j].y) + fabsf(sv.y));
          zu[j] = fma2(vs[j], xv[j], zu[j]), zv[j] = fma2(us[j], xu[j], zv[j]);
        }
        ta = fmaxf(fmaxf(tu[0].x, tu[0].y), fmaxf(tu[1].x, tu[1].y));
        tb = fmaxf(fmaxf(tv[0].x, tv[0].y), fmaxf(tv[1].x, tv[1].y));
        if (PAIRS) ta = tb = fmaxf(ta, tb);
      } else {
        ta = tb = fmaxf(fmaxf(fmaxf(fabsf(zu[0].x), fabsf(zu[0].y)), fmaxf(fabsf(zu[1].x), fabsf(zu[1].y))),
                        fmaxf(fmaxf(fabsf(zv[0].x), fabsf(zv[0].y)), fmaxf(fabsf(zv[1].x), fabsf(zv[1].y))));
      }
      if (w) {
        if (!SMALL) f = root(xu, xv, lift);
        const float2 ff = {f, f};
#pragma unroll
        for (int j = 0; j < 2; ++j) zu[j] = mul2(zu[j], ff), zv[j] = mul2(zv[j], ff);
        ta *= f, tb *= f;
      }
      // the values in order, 8 consecutive ones to a lane
      __syncwarp();
      {
        float4 *p = reinterpret_cast<float4 *>(zs + side * D + ga), *q = reinterpret_cast<float4 *>(zs + side * D + gb);
        *p = PAIRS ? make_float4(zu[0].x, zv[0].x, zu[0].y, zv[0].y) : make_float4(zu[0].x, zu[0].y, zu[1].x, zu[1].y);
        *q = PAIRS ? make_float4(zu[1].x, zv[1].x, zu[1].y, zv[1].y) : make_float4(zv[0].x, zv[0].y, zv[1].x, zv[1].y);
        ts[(side * D + ga) / 4] = ta, ts[(side * D + gb) / 4] = tb;
      }
      __syncwarp();
      float z[8];
      float most;  // how far a value of the block may be off
      // (values that only passed through, behind rot without a norm, are exact: their ties are no doubt)
      const bool passed = !w && sub * 8 >= a.rot;
      {
        const float4 *p = reinterpret_cast<const float4 *>(zs + side * D + sub * 8);
        const float4 p1 = p[0], p2 = p[1], q = *reinterpret_cast<const float4 *>(ts + side * D / 4 + (sub & ~1) * 2);
        z[0] = p1.x, z[1] = p1.y, z[2] = p1.z, z[3] = p1.w, z[4] = p2.x, z[5] = p2.y, z[6] = p2.z, z[7] = p2.w;
        most = passed ? 0.f : fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)) * (20.f * 0x1p-24f);
      }
      float top = max_abs_nan(max_abs_nan(max_abs_nan(z[0], z[1]), max_abs_nan(z[2], z[3])),
                              max_abs_nan(max_abs_nan(z[4], z[5]), max_abs_nan(z[6], z[7])));
      bool odd = false;
      if (!(top < __uint_as_float(0x7f800000u))) {  // infinite, or a NaN, which counts for nothing in the scale
        odd = true;
        top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(z[j]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      Code8 o;
      o.scale = scale_of(fmaxf(top - most, 0.f) * a.k_to_unit);
      const uint32_t scale_up = scale_of((top + most) * a.k_to_unit);
      uint32_t up;
      auto codes = [&]() {  // of the scale, with the values moved down and up
        const float inv = rcp(e4m3_to_float(o.scale)) * a.k_to_unit;
        const float2 move = {most * inv, most * inv};
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 zj = {z[2 * j], z[2 * j + 1]};
          float2 r = mul2(zj, make_float2(inv, inv));
          if (!w && passed) r = over_scale_exact(zj, inv);
          const float2 u = add2(r, move), d = add2(r, make_float2(-move.x, -move.y));
          lo[2 * j] = d.x, lo[2 * j + 1] = d.y, hi[2 * j] = u.x, hi[2 * j + 1] = u.y;
        }
        o.codes = e2m1x8_of(lo), up = e2m1x8_of(hi);
      };
      codes();
      if (__any_sync(0xffffffffu, o.scale != scale_up || o.codes != up)) {
        // the row again in float64; the root's reciprocal by a Newton step from float32's (2^-43 off at most)
        double f64 = 1.0;
        if (w) {
          double ss = 0.0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            ss = fma((double)xu[j].x, (double)xu[j].x, ss), ss = fma((double)xu[j].y, (double)xu[j].y, ss);
            ss = fma((double)xv[j].x, (double)xv[j].x, ss), ss = fma((double)xv[j].y, (double)xv[j].y, ss);
          }
#pragma unroll
          for (int e = LANES / 2; e; e >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, e);
          const double mean = fma(ss, 1.0 / D, (double)a.eps * lift * lift);
          f64 = (double)rsqrtf((float)mean);
          f64 = f64 * fma(-0.5 * mean, f64 * f64, 1.5);
        }
        double *zp = zd + side * D;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int iu = PAIRS ? ga + 2 * j : ga + j, iv = PAIRS ? ga + 2 * j + 1 : gb + j;
          const double yu = (double)(j & 1 ? xu[j / 2].y : xu[j / 2].x) * f64 * (w ? a.kw[iu] : 1.f);
          const double yv = (double)(j & 1 ? xv[j / 2].y : xv[j / 2].x) * f64 * (w ? a.kw[iv] : 1.f);
          zp[iu] = turned ? yu * c[j] - yv * sn[j] : yu;
          zp[iv] = turned ? yv * c[j] + yu * sn[j] : yv;
        }
        __syncwarp();
        if (o.scale != scale_up) {  // the scale first (its block's two lanes agree), then the codes over it
          const double *block = zp + (sub & ~1) * 8;
          double dt = 0.0;
          for (int j = 0; j < 16; ++j) dt = fmax(dt, fabs(block[j]));
          o.scale = max(e4m3_of(sticky(dt / (6.0 * a.k_unit))), 1u);
          codes();
        }
        uint32_t differ = o.codes ^ up;
        const double unit_s = (double)e4m3_to_float(o.scale) * a.k_unit;
        while (differ) {
          const int j = (__ffs(differ) - 1) >> 2;
          o.codes = (o.codes & ~(15u << (4 * j))) | e2m1_of(sticky(zp[sub * 8 + j] / unit_s)) << (4 * j);
          differ &= ~(15u << (4 * j));
        }
      }
      if (to < 0) continue;
      if (odd) report(a.status, TG_STATUS_NONFINITE);
      uint8_t *tile = a.pool + ((int64_t)(to >> 4) * (D / 128) + sub / 16) * kTile4;
      const int r = to & 15, e = sub % 16;
      *reinterpret_cast<uint32_t *>(tile + k_codes4(r, e)) = o.codes;
      if (!(e & 1)) tile[k_scale4(r, e / 2)] = (uint8_t)o.scale;
      if (a.K) *reinterpret_cast<uint4 *>(dense(a.K, h) + sub * 8) = held8(o, a.k_unit);
    }
  }
  // ---- values
  const uint16_t *from = src + (a.H_q + a.H) * D + sub * 8;
  for (int k = max(first, v_first); k < last; ++k) {
    const int h0 = (k - v_first) * BATCH;
    if ((h0 & ~31) != p0) places(h0 & ~31, false);
    uint4 x[kSteps] = {};
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int h = __shfl_sync(0xffffffffu, head, (h0 + s * PER + side) & 31);
      if (h >= 0) x[s] = __ldcs(reinterpret_cast<const uint4 *>(from + h * D));
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int to = __shfl_sync(0xffffffffu, rows, (h0 + s * PER + side) & 31);
      const int h = __shfl_sync(0xffffffffu, head, (h0 + s * PER + side) & 31);
      uint4 held = x[s];
      if (!E2M1) {
        if (to < 0) continue;
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.pool) + (int64_t)(to + a.P) * D + sub * 8) = held;
      } else {
        const uint32_t v[4] = {held.x, held.y, held.z, held.w};
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = unpack2(v[j]);
        bool odd = false;
        const Code8 o = encode_exact(f, a.v_to_unit, odd);
        if (to < 0) continue;
        if (odd) report(a.status, TG_STATUS_NONFINITE);
        uint8_t *tile = a.pool + ((int64_t)(to >> 4) * (D / 128) + sub / 16) * kTile4;
        const int r = to & 15, e = sub % 16;
        *reinterpret_cast<uint32_t *>(tile + v_codes4(r, e)) = o.codes;
        if (!(e & 1)) tile[v_scale4(r, e / 2)] = (uint8_t)o.scale;
        if (a.V) held = held8(o, a.v_unit);
      }
      if (a.V) *reinterpret_cast<uint4 *>(dense(a.V, h) + sub * 8) = held;
    }
  }
}

bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

template <int D, bool SMALL>
cudaError_t launch(const cudaLaunchConfig_t &cfg, bool pairs, bool e2m1, const AppendArgs &a) {
  if (e2m1)
    return pairs ? cudaLaunchKernelEx(&cfg, append_rope_kernel<D, true, true, SMALL>, a)
                 : cudaLaunchKernelEx(&cfg, append_rope_kernel<D, false, true, SMALL>, a);
  return pairs ? cudaLaunchKernelEx(&cfg, append_rope_kernel<D, true, false, SMALL>, a)
               : cudaLaunchKernelEx(&cfg, append_rope_kernel<D, false, false, SMALL>, a);
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
  if (pool_pages <= 0 || pool_pages > INT32_MAX / H_p / (e2m1 ? P : 2 * (int64_t)P))
    return fail(TG_ERR_CAPACITY, "%s: pool_pages=%lld gives more than 2^31-1 rows, or none", fn, (long long)pool_pages);
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
  a.status = dev_status, a.batch = batch, a.H_q = H_q, a.H = H, a.H_p = H_p, a.G = H / H_p, a.P = P, a.Nmax = Nmax, a.rot = rot;
  a.max_pos = max_pos, a.axes = axes, a.reserve = reserve, a.eps = eps, a.k_unit = k_unit, a.v_unit = v_unit;
  if (e2m1) a.k_to_unit = 1.f / k_unit, a.v_to_unit = 1.f / v_unit;  // exact
  // As many warps a token as let about all of them be on the card at once, up to one for each of its batches.  More tokens
  // than that: two for bf16 pages, which ends the call more evenly, one for 4-bit pages, where each more looks up places
  // and weights anew beside arithmetic that already counts.  us of 1, 2, 3, 5 (4 bits) and all warps a token, bf16: 512
  // tokens of 32 + 8 + 8 heads of 128: 9.1, 6.4, 5.7, 5.8; 1024: 10.7, 8.1, 7.2, 9.6; 2048: 14.9, 12.6, 13.8, 15.6; 9000:
  // 46.3, 43.7, 45.0, 54.7; 9000 of 16 + 8 + 8 heads of 256: 69.8, 63.8, 63.9, 72.3.  4 bits, of those: 16: 14.8, 9.6, 8.2, 6.9,
  // 5.0; 512: 21.0, 15.4, 13.1, 11.4, 13.4; 1024: 24.5, 18.1, 16.1, 18.2, 20.9; 3000: 31.3, 33.9, 35.2, 43.1, 49.9.
  const int per = kSteps * (d == 128 ? 2 : 1);
  a.q_batches = (H_q + per - 1) / per;
  a.v_batches = (H + per - 1) / per;
  a.k_batches = e2m1 ? (H + per / kSteps - 1) / (per / kSteps) : a.v_batches;
  const int all = a.q_batches + a.k_batches + a.v_batches;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  // (4 bits: the number nearest to 18 of the 20 an SM: a few warps behind the others cost less than longer shares)
  const int fit = e2m1 ? (sms * (kBlocksPerSm4 - 2) + T / 2) / T : sms * kBlocksPerSm / T;
  int parts = std::min({std::max(fit, e2m1 ? 1 : 2), all, kMaxParts});
  if (!e2m1) {  // batches weigh alike: no more warps than the longest share needs
    const int share = (all + parts - 1) / parts;
    parts = (all + share - 1) / share;
  }
  a.parts = parts;
  const int64_t blocks = (int64_t)T * parts;
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
  if (eps < kSmallMean && (q_weight || k_weight))
    e = d == 128 ? launch<128, true>(cfg, pairs, e2m1, a) : launch<256, true>(cfg, pairs, e2m1, a);
  else
    e = d == 128 ? launch<128, false>(cfg, pairs, e2m1, a) : launch<256, false>(cfg, pairs, e2m1, a);
  if (e != cudaSuccess) return fail(TG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return tgi::ok();
}
