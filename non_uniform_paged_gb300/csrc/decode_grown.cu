// Decode attention over runs that grow, of bf16 pages and of 4-bit pages (tg_decode_grown).
//
// bf16 pages: the body of tg_decode_attn (decode_body.cuh) over the pieces that grown_item gives.
//
// 4-bit pages.  Mathematics: out = sum_t softmax_t(scale q . k_t) v_t with k, v = code * block scale * unit.
// A token is 9/16 of a byte a value, so that the same bytes hold 3.6 times the tokens of bf16 pages and
// arithmetic comes near to bounding the kernel: at the copy rate an SM gets 24 bytes a clock, 43 values
// to turn into f16 and multiply.
//  * Roles, hand-off, merge and plan are decode_body's.  A tile of 16 tokens (x 128 values) is 2304
//    contiguous bytes, one bulk copy (two at d = 256).
//  * Codes become f16 pairs by the hardware's conversion (eight values are four conversions of a register's
//    bytes; measured above 80 values a clock and SM with their consumer), times the scale, which is exact: a code
//    has 2 significant bits, a scale 4.
//  * S^T = K Q^T as m16n8k16 f16 MMAs.  The order of the contraction is free, so a lane takes 32 consecutive values of
//    a token: one 16-byte load, two scales.  q is f16 too: scaled by a power of two to a maximum in [1, 2),
//    which costs nothing that bf16 has but what is 2^-14 of the maximum and below.
//  * O^T += V^T P^T: a lane takes one block of 16 values of four tokens.  A pair of tokens' codes are brought
//    side by side in their bytes before the conversion, so that the pair of their scales multiplies them.
//  * Weights are f16, 2^15 times as large as the softmax's: what a weight of f16 loses is then below 2^-39 of the largest.
#include "decode_body.cuh"
#include "page4.cuh"

#include <cuda_runtime.h>

#include <cmath>

namespace {

using namespace tgk;

template <int D>
__global__ void __launch_bounds__(Layout<D>::THREADS, 1)
    grown_decode_kernel(const __grid_constant__ CUtensorMap pool_map, const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  decode_body<D, true>(&pool_map, a, smem_raw);
}

// NW streaming warps, each with an R-stage ring of tiles, and NE epilogue warps
template <int D>
struct Cfg4;
template <>
struct Cfg4<128> {
  static constexpr int NW = 12, R = 4, NE = 4;
};
template <>
struct Cfg4<256> {
  static constexpr int NW = 6, R = 4, NE = 4;
};

template <int D>
struct Layout4 {
  static constexpr int NW = Cfg4<D>::NW, R = Cfg4<D>::R, NE = Cfg4<D>::NE;
  static constexpr int THREADS = (NW + NE) * 32;
  static constexpr int STAGE = D / 128 * kTile4;  // 16 tokens
  static constexpr int RING = NW * R * STAGE;
  // as Layout: barriers, start time, items and their page-table bases and order, hand-off (m, l), merged (M, L), flags
  static constexpr int SMALL = NW * R * 8 + 4 * 8 + 8 + kMaxItems * (8 + (int)sizeof(tg_work_item)) +
                               kMaxItems * 4 + 2 * NW * 8 * 4 * 2 + 8 * 4 * 2 + 16;
  __host__ __device__ static int ostride(int g) { return g <= 4 ? D + 4 : D; }
  __host__ __device__ static int comb_floats(int g) { return NW * g * ostride(g); }
  static int smem_bytes(int g) { return SMALL + 128 + RING + 2 * comb_floats(g) * 4 + kFacMax * 4; }
};

constexpr float kWeightLog2 = 15.f;  // weights are 2^15 times the softmax's

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}

struct Pool4 {
  const uint8_t *base;
  int64_t head_bytes;  // of a head in a page
  float v_unit;
};

template <int D>
__global__ void __launch_bounds__(Layout4<D>::THREADS, 1) decode4_kernel(const DecodeArgs a, const Pool4 pool) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using LY = Layout4<D>;
  constexpr int NW = LY::NW, R = LY::R, NE = LY::NE, NT = LY::THREADS, C = D / 128;  // C: tiles side by side
  constexpr int NS = NW * 32, NET = NE * 32;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw);                 // [NW][R] copy stages
  uint64_t *full = bars + NW * R;                                          // [2] hand-off buffer written
  uint64_t *empty = full + 2;                                              // [2] hand-off buffer read
  uint64_t *s_t0 = empty + 2;                                              // CTA start (globaltimer)
  int64_t *s_base = reinterpret_cast<int64_t *>(s_t0 + 1);                 // [kMaxItems]
  tg_work_item *s_items = reinterpret_cast<tg_work_item *>(s_base + kMaxItems);
  int *s_order = reinterpret_cast<int *>(s_items + kMaxItems);             // [kMaxItems] processing order
  float *comb_m = reinterpret_cast<float *>(s_order + kMaxItems);          // [2][NW][8]
  float *comb_l = comb_m + 2 * NW * 8;                                     // [2][NW][8]
  float *s_mm = comb_l + 2 * NW * 8;                                       // [8]
  float *s_ll = s_mm + 8;                                                  // [8]
  int *flag = reinterpret_cast<int *>(s_ll + 8);                           // last CTA of a shared run
  volatile int *s_dead = flag + 1;                                         // a hand-off wait gave up
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + LY::SMALL + 127) & ~uintptr_t(127));
  const int ostride = LY::ostride(a.g), cfl = LY::comb_floats(a.g);
  float *comb_o = reinterpret_cast<float *>(ring + LY::RING);              // [2][NW][g][ostride]
  float *fac = comb_o + 2 * cfl;                                           // [kFacMax]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  if (tid == 0) *s_t0 = globaltimer_ns();

  // the plan does not change: read ahead of the kernel before this one
  const tg_work_item lead = a.lead[blockIdx.x];
  const int n_items = lead.reserved[0], i_begin = lead.reserved[1];
  const bool items_in_smem = n_items <= kMaxItems;
  if (items_in_smem) {
    tg_work_item first = lead;
    first.reserved[0] = first.reserved[1] = 0;
    for (int i = tid; i < n_items; i += NT) s_items[i] = i == 0 ? first : a.items[i_begin + i];
  }
  if (warp < NW && lane == 0)
    for (int s = 0; s < R; ++s) mbar_init(&bars[warp * R + s], 1);
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&full[b], NS);
      mbar_init(&empty[b], NET);
    }
    *s_dead = 0;
  }
  fence_barrier_init();
  griddep_wait();
  griddep_launch_dependents();
  if (items_in_smem)
    for (int i = tid; i < n_items; i += NT) {
      s_items[i] = grown_item(a, s_items[i]);
      s_base[i] = __ldcg(a.pt_off + s_items[i].b * a.G + s_items[i].g);
    }
  __syncthreads();
  if (tid == 0 && items_in_smem) {  // shared-run pieces first, then owned runs, each in plan order
    int c = 0;
    for (int i = 0; i < n_items; ++i)
      if (s_items[i].nparts > 1) s_order[c++] = i;
    for (int i = 0; i < n_items; ++i)
      if (s_items[i].nparts <= 1) s_order[c++] = i;
  }
  __syncthreads();
  auto get_item = [&](int k) -> tg_work_item {
    return items_in_smem ? s_items[s_order[k]] : grown_item(a, a.items[i_begin + k]);
  };
  auto get_base = [&](int k, const tg_work_item &it) -> int64_t {
    return items_in_smem ? s_base[s_order[k]] : __ldcg(a.pt_off + it.b * a.G + it.g);
  };

  if (warp < NW) {
    // ================================================================ streaming warps
    auto warp_tiles = [&](const tg_work_item &it, int &lo) -> int {
      int hi;
      item_tiles(it, lo, hi);
      return hi - lo > warp ? (hi - lo - warp + NW - 1) / NW : 0;
    };
    int total_tiles = 0;
    for (int k = 0; k < n_items; ++k) {
      int lo;
      total_tiles += warp_tiles(get_item(k), lo);
    }
    // where a tile of this warp lies: 32 of them looked up at a time, one by each lane, a batch ahead
    auto tile_at = [&](int n) -> int64_t {
      if (n >= total_tiles) return -1;
      int rem = n;
      for (int k = 0; k < n_items; ++k) {
        const tg_work_item it = get_item(k);
        int lo;
        const int cnt = warp_tiles(it, lo);
        if (rem < cnt) {
          const int tok = 16 * (lo + warp + NW * rem);
          const int64_t at = get_base(k, it) + tok / a.P;
          if (at >= __ldcg(a.pt_off + it.b * a.G + it.g + 1)) return -1;  // a list too short
          const int32_t page = __ldcg(a.pt_ids + at);
          if (page < 0 || page >= a.pool_pages) return -1;
          return ((int64_t)page * a.H_p + it.hpos) * pool.head_bytes + (tok % a.P / 16) * LY::STAGE;
        }
        rem -= cnt;
      }
      return -1;
    };
    int64_t at_cur = tile_at(lane), at_nxt = tile_at(32 + lane);
    int issued = 0, consumed = 0;
    auto issue = [&]() {  // whole warp: tile number `issued` of this warp into stage issued % R
      const int64_t at = __shfl_sync(0xffffffffu, at_cur, issued & 31);
      if (lane == 0) {
        const int s = issued % R;
        uint64_t *bar = &bars[warp * R + s];
        if (at < 0) {
          report(a.status, TG_STATUS_BAD_PAGE);
          mbar_arrive(bar);  // complete the phase without data
        } else {
          mbar_arrive_expect_tx(bar, LY::STAGE);
          bulk_load(ring + (warp * R + s) * LY::STAGE, pool.base + at, LY::STAGE, bar);
        }
      }
      ++issued;
      if ((issued & 31) == 0) {
        at_cur = at_nxt;
        at_nxt = tile_at(issued + 32 + lane);
      }
    };
    for (int s = 0; s < R && issued < total_tiles; ++s) issue();

    bool dead = false;  // a copy wait timed out: skip all further tiles, keep handing off
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[C][8][4];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[c][i][0] = o[c][i][1] = o[c][i][2] = o[c][i][3] = 0.f;

    for (int k = 0; k < n_items; ++k) {
      const tg_work_item it = get_item(k);
      int k_lo, k_hi;
      item_tiles(it, k_lo, k_hi);
      if (k_hi - k_lo > warp && !dead) {
        // Query fragments, B of S^T = K Q^T: head gid, values 32 tig .. 32 tig + 31 of each 128, as f16 times
        // 2^-e, e the exponent of the head's largest; z0, z1: what that and the softmax scale give the scores of
        // the heads 2 tig and 2 tig + 1 that this lane holds
        uint32_t qf[C][8][2];
        float z0, z1;
        {
          uint4 raw[C][4];
          const uint16_t *qrow = a.q + ((size_t)it.b * a.H_q + (size_t)it.h * a.g + gid) * D + 32 * tig;
          uint32_t top = 0;  // magnitude bits
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              raw[c][i] = gid < a.g ? __ldcg(reinterpret_cast<const uint4 *>(qrow + 128 * c + 8 * i)) : make_uint4(0, 0, 0, 0);
              const uint32_t w[4] = {raw[c][i].x, raw[c][i].y, raw[c][i].z, raw[c][i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) top = max(top, max(w[j] << 16 & 0x7fffffffu, w[j] & 0x7fff0000u));
            }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const uint32_t e = min(max(top >> 23, 1u), 253u);  // biased
          const float down = __uint_as_float((254 - e) << 23), up = __uint_as_float(e << 23) * a.scale_log2;
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w[4] = {raw[c][i].x, raw[c][i].y, raw[c][i].z, raw[c][i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                qf[c][2 * i + j / 2][j & 1] =
                    pack_f16x2(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xffff0000u) * down);
            }
          z0 = __shfl_sync(0xffffffffu, up, 8 * tig);
          z1 = __shfl_sync(0xffffffffu, up, 8 * tig + 4);
        }
        for (int kk = k_lo + warp; kk < k_hi; kk += NW) {
          const int s = consumed % R;
          bool ok = mbar_wait(&bars[warp * R + s], (uint32_t)((consumed / R) & 1), kWaitLimitNs);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (lane == 0) report(a.status, TG_STATUS_TIMEOUT);
            dead = true;
            break;
          }
          const uint32_t tile = smem_addr(ring + (warp * R + s) * LY::STAGE);
          const int r0 = it.t0 - kk * 16, r1 = it.t1 - kk * 16;  // valid rows [r0, r1) of the tile

          // S^T = K Q^T (rows: tokens gid and gid + 8, columns: heads 2 tig and 2 tig + 1)
          float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const uint32_t kt = tile + c * kTile4;
            const uint4 x = lds128(kt + 64 * gid + 16 * tig), y = lds128(kt + 64 * (gid + 8) + 16 * tig);
            const uint32_t sx = e4m3x2_to_f16x2(lds16(kt + kKScales4 + 8 * gid + 2 * tig));
            const uint32_t sy = e4m3x2_to_f16x2(lds16(kt + kKScales4 + 8 * (gid + 8) + 2 * tig));
            const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // eight values of each row; the first 16 have one scale, the others the next
              const uint32_t fx = __byte_perm(sx, 0, i < 2 ? 0x1010 : 0x3232), fy = __byte_perm(sy, 0, i < 2 ? 0x1010 : 0x3232);
              uint32_t hx[4], hy[4];
              e2m1x8_to_f16x2(wx[i], hx);
              e2m1x8_to_f16x2(wy[i], hy);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_f16(sc, mul_f16x2(hx[2 * j], fx), mul_f16x2(hy[2 * j], fy), mul_f16x2(hx[2 * j + 1], fx),
                        mul_f16x2(hy[2 * j + 1], fy), qf[c][2 * i + j][0], qf[c][2 * i + j][1]);
            }
          }
          // online softmax, base 2
          const bool v0 = gid >= r0 && gid < r1, v1 = gid + 8 >= r0 && gid + 8 < r1;
          const float x0 = v0 ? sc[0] * z0 : -INFINITY, x1 = v0 ? sc[1] * z1 : -INFINITY;
          const float x2 = v1 ? sc[2] * z0 : -INFINITY, x3 = v1 ? sc[3] * z1 : -INFINITY;
          float mx0 = fmaxf(x0, x2), mx1 = fmaxf(x1, x3);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
          }
          const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
          const float c0 = ex2(m0 - mn0), c1 = ex2(m1 - mn1);
          // (15 comes last: added to a maximum of 2^28 it would be rounded to 16 or 32)
          const float p0 = ex2(x0 - mn0 + kWeightLog2), p1 = ex2(x1 - mn1 + kWeightLog2);
          const float p2 = ex2(x2 - mn0 + kWeightLog2), p3 = ex2(x3 - mn1 + kWeightLog2);
          l0 = l0 * c0 + p0 + p2;
          l1 = l1 * c1 + p1 + p3;
          m0 = mn0;
          m1 = mn1;
          const uint32_t w0 = movmatrix_t(pack_f16x2(p0, p1)), w1 = movmatrix_t(pack_f16x2(p2, p3));
          // O^T += V^T P^T (rows: values 16 gid + 2 i and one on, columns: heads); this lane's tokens: 2 tig, 2 tig + 1
          // and the two 8 behind them
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const uint32_t vt = tile + c * kTile4 + kVCodes4;
            const uint4 x = lds128(vt + 64 * gid + 16 * tig), y = lds128(vt + 512 + 64 * gid + 16 * tig);
            uint32_t sx = e4m3x2_to_f16x2(lds16(tile + c * kTile4 + kVScales4 + 16 * gid + 2 * tig));
            uint32_t sy = e4m3x2_to_f16x2(lds16(tile + c * kTile4 + kVScales4 + 16 * gid + 2 * tig + 8));
            if (r0 > 0 || r1 < 16) {  // rows that are no token of this piece may hold anything: 0 times a code is 0
              auto kept = [&](int t) {
                return (t >= r0 && t < r1 ? 0xffffu : 0u) | (t + 1 >= r0 && t + 1 < r1 ? 0xffff0000u : 0u);
              };
              sx &= kept(2 * tig);
              sy &= kept(2 * tig + 8);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // values 8 i .. 8 i + 7 of the block
              const uint32_t xa = i ? x.y : x.x, xb = i ? x.w : x.z, ya = i ? y.y : y.x, yb = i ? y.w : y.z;
              // even and odd values, the first token in the lower half of each byte
              uint32_t ex[4], ox[4], ey[4], oy[4];
              e2m1x8_to_f16x2((xa & 0x0f0f0f0fu) | (xb << 4 & 0xf0f0f0f0u), ex);
              e2m1x8_to_f16x2((xa >> 4 & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), ox);
              e2m1x8_to_f16x2((ya & 0x0f0f0f0fu) | (yb << 4 & 0xf0f0f0f0u), ey);
              e2m1x8_to_f16x2((ya >> 4 & 0x0f0f0f0fu) | (yb & 0xf0f0f0f0u), oy);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float(&oo)[4] = o[c][4 * i + j];
                oo[0] *= c0;
                oo[1] *= c1;
                oo[2] *= c0;
                oo[3] *= c1;
                mma_f16(oo, mul_f16x2(ex[j], sx), mul_f16x2(ox[j], sx), mul_f16x2(ey[j], sy), mul_f16x2(oy[j], sy), w0, w1);
              }
            }
          }
          ++consumed;
          __syncwarp();
          if (issued < total_tiles) {
            if (lane == 0) fence_proxy_async_smem();  // our reads of this stage come before the refill
            issue();
          }
        }
      }

      // ---- hand this warp's state of item k to the epilogue (buffer k & 1, its use k >> 1)
      const int hb = k & 1, use = k >> 1;
      if (use > 0 && !*s_dead && !mbar_wait(&empty[hb], (uint32_t)((use - 1) & 1), kWaitLimitNs)) {
        if (lane == 0) report(a.status, TG_STATUS_TIMEOUT);
        *s_dead = 1;
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
      }
      // the epilogue knows weights that are 1 at the maximum, and V without its unit
      constexpr float kBack = 1.f / 32768.f;
      const float back = kBack * pool.v_unit;
      float *cm = comb_m + (hb * NW + warp) * 8, *cl = comb_l + (hb * NW + warp) * 8;
      if (gid == 0) {
        cm[2 * tig] = m0;
        cm[2 * tig + 1] = m1;
        cl[2 * tig] = l0 * kBack;
        cl[2 * tig + 1] = l1 * kBack;
      }
      float *co = comb_o + hb * cfl + warp * a.g * ostride;  // [g][ostride] of this warp
      const int h0 = 2 * tig, h1 = 2 * tig + 1;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float(&oo)[4] = o[c][i];
          const int at = 128 * c + 16 * gid + 2 * i;
          if (h0 < a.g) *reinterpret_cast<float2 *>(co + h0 * ostride + at) = make_float2(oo[0] * back, oo[2] * back);
          if (h1 < a.g) *reinterpret_cast<float2 *>(co + h1 * ostride + at) = make_float2(oo[1] * back, oo[3] * back);
          oo[0] = oo[1] = oo[2] = oo[3] = 0.f;
        }
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
      mbar_arrive(&full[hb]);  // (release: this thread's hand-off writes come first)
    }
    // drain copies still in flight (only after a timeout; otherwise issued == consumed)
    if (lane == 0) {
      for (int t = consumed; t < issued; ++t)
        if (!mbar_wait(&bars[warp * R + t % R], (uint32_t)((t / R) & 1), kWaitLimitNs)) break;
    }
    __syncwarp();
    return;
  }
  decode_epilogue<D, NW, NE, true>(a, get_item, n_items, comb_m, comb_l, comb_o, cfl, ostride, fac, s_mm, s_ll, flag,
                                   s_dead, full, empty, s_t0);
}

template <int D>
int launch(cudaStream_t stream, int format, const void *map, const DecodeArgs &args, const Pool4 &pool, int N_CTA) {
  const char *name = "tg_decode_grown";
  void *fn;
  int threads, smem;
  if (format == TG_PAGES_BF16) {
    fn = reinterpret_cast<void *>(&grown_decode_kernel<D>);
    threads = Layout<D>::THREADS, smem = Layout<D>::smem_bytes(args.g);
  } else {
    fn = reinterpret_cast<void *>(&decode4_kernel<D>);
    threads = Layout4<D>::THREADS, smem = Layout4<D>::smem_bytes(args.g);
  }
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return tgi::fail(TG_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", name, cudaGetErrorString(e));
  void *bf16[] = {const_cast<void *>(map), const_cast<DecodeArgs *>(&args)};
  void *e2m1[] = {const_cast<DecodeArgs *>(&args), const_cast<Pool4 *>(&pool)};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(N_CTA);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelExC(&cfg, fn, format == TG_PAGES_BF16 ? bf16 : e2m1);
  if (e != cudaSuccess) return tgi::fail(TG_ERR_CUDA, "%s: launch failed: %s", name, cudaGetErrorString(e));
  return tgi::ok();
}

}  // namespace

extern "C" int tg_decode_grown(tg_stream_t stream, const void *plan_host, const void *plan_dev, int layer, int format,
                               const uint16_t *q, const void *pool, int64_t pool_pages, const int64_t *pt_off,
                               const int32_t *pt_ids, const int32_t *ntok, const int32_t *added, int plus, int reserve,
                               float scale, float k_unit, float v_unit, void *workspace, int64_t workspace_bytes,
                               uint16_t *out, float *lse, int32_t *dev_status, int64_t *cta_time) {
  const char *fn = "tg_decode_grown";
  using tgi::fail;
  if (!plan_host || !plan_dev || !q || !pool || !pt_off || !pt_ids || !ntok || !workspace || !out)
    return fail(TG_ERR_INVALID_ARG, "%s: NULL pointer argument", fn);
  if (format != TG_PAGES_BF16 && format != TG_PAGES_E2M1) return fail(TG_ERR_INVALID_ARG, "%s: format=%d", fn, format);
  if (plus < 0 || reserve < 0 || plus > reserve)
    return fail(TG_ERR_INVALID_ARG, "%s: plus=%d, reserve=%d (0 <= plus <= reserve)", fn, plus, reserve);
  const tg_plan_header *hd;
  const tg_plan_layer *lt;
  int rc = check_decode_call(fn, plan_host, plan_dev, layer, q, static_cast<const uint16_t *>(pool), scale, &hd, &lt);
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(q) & 15) return fail(TG_ERR_INVALID_ARG, "%s: q must be 16-byte aligned", fn);
  if (workspace_bytes < hd->workspace_bytes)
    return fail(TG_ERR_CAPACITY, "%s: workspace %lld < %lld bytes", fn, (long long)workspace_bytes,
                (long long)hd->workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(TG_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  DecodeArgs args = decode_args(hd, lt, plan_dev, static_cast<uint8_t *>(workspace), q, out, lse, pt_off, pt_ids,
                                pool_pages, scale, dev_status, cta_time);
  args.ntok = ntok, args.added = added, args.plus = plus, args.reserve = reserve;
  args.wait_tables = 1;  // the kernel before it may have written pages, queries and added
  CUtensorMap map;
  Pool4 p4 = {static_cast<const uint8_t *>(pool), (int64_t)(hd->P / 16) * (hd->d / 128) * kTile4, v_unit};
  if (format == TG_PAGES_BF16) {
    rc = make_pool_map(&map, static_cast<const uint16_t *>(pool), pool_pages, hd, fn);
    if (rc) return rc;
  } else {
    if (!unit_ok(k_unit) || !unit_ok(v_unit))
      return fail(TG_ERR_INVALID_ARG, "%s: k_unit=%g, v_unit=%g (powers of two in [2^-60, 2^60])", fn, (double)k_unit,
                  (double)v_unit);
    if (pool_pages <= 0 || pool_pages > INT32_MAX)
      return fail(TG_ERR_CAPACITY, "%s: pool_pages=%lld (1..2^31-1)", fn, (long long)pool_pages);
    args.scale_log2 *= k_unit;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return hd->d == 128 ? launch<128>(s, format, &map, args, p4, hd->N_CTA) : launch<256>(s, format, &map, args, p4, hd->N_CTA);
}
