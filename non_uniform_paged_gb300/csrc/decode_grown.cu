// Decode attention over runs that grow, of bf16 pages and of 4-bit pages (tg_decode_grown).
//
// bf16 pages: the body of tg_decode_attn (decode_body.cuh) over the pieces that grown_item gives.  1.35 M rows of 128 (691 MB, 101.7
// us at the copy rate) 109 us; 1.32 M rows of 256 under 2 query heads (1355 MB, 199.6 us) 204, tg_decode_attn over the same rows 187.
//
// 4-bit pages.  Mathematics: out = sum_t softmax_t(scale q . k_t) v_t with k, v = code * block scale * unit.
// A token is 9/16 of a byte a value, so that the same bytes hold 3.6 times the tokens of bf16 pages and
// arithmetic bounds the kernel before memory does: at the copy rate an SM gets 24 bytes a clock, 43 values
// to turn into f16 and multiply.
//  * Roles, hand-off, merge and plan are decode_body's.  A warp's step is 32 tokens: two tiles of 16 tokens (x 128
//    values) of 2304 contiguous bytes, a bulk copy each (two each at d = 256), issued by a lane for each tile.
//  * Codes become f16 pairs by the hardware's conversion (eight values are four conversions of a register's
//    bytes; measured above 80 values a clock and SM with their consumer), times the scale, which is exact: a code
//    has 2 significant bits, a scale 4.
//  * S^T = K Q^T as m16n8k16 f16 MMAs.  The order of the contraction is free, so a lane takes 32 consecutive values of
//    a token: one 16-byte load, two scales.  q is f16 too: scaled by a power of two to a maximum in [1, 2),
//    which costs nothing that bf16 has but what is 2^-14 of the maximum and below.
//  * O^T += V^T P^T: a lane takes one block of 16 values of four tokens.  A pair of tokens' codes are brought
//    side by side in their bytes before the conversion, so that the pair of their scales multiplies them.
//  * Weights are f16, 2^8 times the softmax's against a maximum that moves only when a score passes it by 7
//    (kWeightLog2 below): at most 2^15, and what f16 loses of a weight is below 2^-24 / 2^8 of the maximum's.
// Measured: 2.7 M rows of 128 under 4 query heads a KV head (389 MB, 57.3 us at the copy rate) 72.7 us, 1.9 M rows of
// 256 under 2 (545 MB, 80.2 us) 98.  No unit is at its limit: of the active clocks ALU (conversions, byte moves) 52%, FMA (with the
// f16 products) 34, HMMA 26, issue 58; DRAM 64% of all (48, 32, 27, 51 and 68 at d = 256).  Three (two) streaming warps a
// scheduler do not cover the chains of dependent instructions of a step.  Steps of 16 tokens with a maximum in each took
// 106.9 and 165; warps that only load, 87 us and more where this took 81; 16 streaming warps spill; three stages, no gain.
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

// NW streaming warps, each with an R-stage ring of steps of 32 tokens, and NE epilogue warps
template <int D>
struct Cfg4;
template <>
struct Cfg4<128> {
  static constexpr int NW = 12, R = 2, NE = 4;
};
template <>
struct Cfg4<256> {
  static constexpr int NW = 8, R = 2, NE = 4;
};

template <int D>
struct Layout4 {
  static constexpr int NW = Cfg4<D>::NW, R = Cfg4<D>::R, NE = Cfg4<D>::NE;
  static_assert(R < 16, "the second batch of tiles is looked up behind the first copies");
  static constexpr int THREADS = (NW + NE) * 32;
  static constexpr int TILE = D / 128 * kTile4;  // 16 tokens
  static constexpr int STAGE = 2 * TILE;
  static constexpr int RING = NW * R * STAGE;
  // as Layout: barriers, start time, items and the bounds of their page lists, hand-off (m, l), merged (M, L), flags
  static constexpr int SMALL = NW * R * 8 + 4 * 8 + 8 + kMaxItems * (16 + (int)sizeof(tg_work_item)) +
                               2 * NW * 8 * 4 * 2 + 8 * 4 * 2 + 16;
  static constexpr int MOST = 227 * 1024;
  __host__ __device__ static int ostride(int g) { return g <= 4 ? D + 4 : D; }
  __host__ __device__ static int comb_floats(int g) { return NW * g * ostride(g); }
  // two hand-off buffers, or one where two do not fit (d = 256 with more than four query heads)
  static int buffers(int g) { return bytes(g, 2) <= MOST ? 2 : 1; }
  static int bytes(int g, int nb) { return SMALL + 128 + RING + nb * comb_floats(g) * 4 + kFacMax * 4; }
  static int bytes_most() {  // as Layout::smem_most
    int most = 0;
    for (int g = 1; g <= 8; ++g) most = std::max(most, bytes(g, buffers(g)));
    return most;
  }
};

// A weight is 2^(x - m), with m a reference 8 below the largest score when it was taken, which moves only when a weight
// would pass 2^15: all are in reach of f16, and a step that moves nothing neither reduces a maximum over lanes nor
// rescales O.  m is that difference rounded up, and scores are rounded before m is taken off them, as m's own was: then
// the largest score's weight is between 1 and 2^8 whatever their magnitude (past 2^27 m is the score itself; one fma of
// product and reference would leave the product's rounding, which passes 2^5 there, in the exponent).
constexpr float kWeightLog2 = 8.f, kWeightMost = 15.f;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
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

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void arrive_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load_at(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

struct Pool4 {
  const uint8_t *base;
  int p16;  // tiles of a head in a page
  float v_unit;
  int buffers;  // hand-off buffers
};

template <int D>
__global__ void __launch_bounds__(Layout4<D>::THREADS, 1) decode4_kernel(const DecodeArgs a, const Pool4 pool) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using LY = Layout4<D>;
  constexpr int NW = LY::NW, R = LY::R, NE = LY::NE, C = D / 128;  // C: tiles side by side
  constexpr int NS = NW * 32, NET = NE * 32;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw);                 // [NW][R] copy stages
  uint64_t *full = bars + NW * R;                                          // [2] hand-off buffer written
  uint64_t *empty = full + 2;                                              // [2] hand-off buffer read
  uint64_t *s_t0 = empty + 2;                                              // CTA start (globaltimer)
  int64_t *s_base = reinterpret_cast<int64_t *>(s_t0 + 1);                 // [kMaxItems] first entry of the page list
  int64_t *s_end = s_base + kMaxItems;                                     // [kMaxItems] and behind its last
  tg_work_item *s_items = reinterpret_cast<tg_work_item *>(s_end + kMaxItems);  // [kMaxItems] in processing order
  float *comb_m = reinterpret_cast<float *>(s_items + kMaxItems);          // [2][NW][8]
  float *comb_l = comb_m + 2 * NW * 8;                                     // [2][NW][8]
  float *s_mm = comb_l + 2 * NW * 8;                                       // [8]
  float *s_ll = s_mm + 8;                                                  // [8]
  int *flag = reinterpret_cast<int *>(s_ll + 8);
  volatile int *s_dead = flag + 1;                                         // a hand-off wait gave up
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + LY::SMALL + 127) & ~uintptr_t(127));
  const int ostride = LY::ostride(a.g), cfl = LY::comb_floats(a.g);
  float *comb_o = reinterpret_cast<float *>(ring + LY::RING);              // [2][NW][g][ostride]
  float *fac = comb_o + pool.buffers * cfl;                                // [kFacMax]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  if (tid == 0) *s_t0 = globaltimer_ns();

  // the plan does not change: read ahead of the kernel before this one
  const tg_work_item lead = a.lead[blockIdx.x];
  const int n_items = lead.reserved[0], i_begin = lead.reserved[1];
  const bool items_in_smem = n_items <= kMaxItems;
  tg_work_item mine = lead;  // of warp 0's lanes: item `lane`
  if (items_in_smem && warp == 0 && lane > 0 && lane < n_items) mine = a.items[i_begin + lane];
  if (warp < NW && lane == 0)
    for (int s = 0; s < R; ++s) mbar_init(&bars[warp * R + s], 2);  // (a lane for each half)
  if (tid == NS) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&full[b], NS);
      mbar_init(&empty[b], NET);
    }
    *s_dead = 0;
  }
  fence_barrier_init();
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 0 && items_in_smem) {
    // shared-run pieces first, then owned runs, each in plan order
    const bool have = lane < n_items;
    const unsigned all = __ballot_sync(0xffffffffu, have), shared = __ballot_sync(0xffffffffu, have && mine.nparts > 1);
    const unsigned before = (1u << lane) - 1;
    const int at = shared >> lane & 1 ? __popc(shared & before) : __popc(shared) + __popc(all & ~shared & before);
    if (have) {
      const int64_t *off = a.pt_off + (int64_t)mine.b * a.G + mine.g;
      const int64_t base = __ldcg(off), end = __ldcg(off + 1);
      s_items[at] = grown_item(a, mine);
      s_base[at] = base;
      s_end[at] = end;
    }
  }
  __syncthreads();
  auto get_item = [&](int k) -> tg_work_item { return items_in_smem ? s_items[k] : grown_item(a, a.items[i_begin + k]); };

  if (warp < NW) {
    // ================================================================ streaming warps
    // steps of 32 tokens of item `it` that this warp takes: lo + warp, lo + warp + NW, ...
    auto warp_steps = [&](const tg_work_item &it, int &lo) -> int {
      lo = it.t0 >> 5;
      const int n = it.t1 > it.t0 ? ((it.t1 + 31) >> 5) - lo : 0;
      return n > warp ? (n - warp + NW - 1) / NW : 0;
    };
    // where a warp's steps of item k end: of up to 16 items in lane k, of more they are counted again
    int total = 0, ends = 0;
    if (items_in_smem) {
      int lo;
      ends = lane < n_items ? warp_steps(s_items[lane], lo) : 0;
#pragma unroll
      for (int d = 1; d < kMaxItems; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, ends, d);
        if (lane >= d) ends += v;
      }
      total = __shfl_sync(0xffffffffu, ends, kMaxItems - 1);
    } else {
      for (int k = 0; k < n_items; ++k) {
        int lo;
        total += warp_steps(get_item(k), lo);
      }
    }
    // The two tiles of a step of this warp, by their number in the pool: sixteen steps looked up at a time by the whole
    // warp, a tile by each lane, a batch ahead.  kNone: no token of the item in it.
    constexpr int kBad = -1, kNone = -2;
    auto tile_at = [&](int n) -> int {
      int step = n >> 1, lo;
      tg_work_item it;
      int64_t base, end;
      if (items_in_smem) {
        int k = 0;
        for (int i = 0; i < n_items - 1; ++i) k += step >= __shfl_sync(0xffffffffu, ends, i);
        const int first = __shfl_sync(0xffffffffu, ends, max(k - 1, 0));
        if (n >= 2 * total) return kNone;
        step -= k > 0 ? first : 0;
        it = s_items[k], base = s_base[k], end = s_end[k];
      } else {
        if (n >= 2 * total) return kNone;
        for (int k = 0; k < n_items; ++k) {
          it = get_item(k);
          const int cnt = warp_steps(it, lo);
          if (step < cnt) break;
          step -= cnt;
        }
        base = __ldcg(a.pt_off + it.b * a.G + it.g), end = __ldcg(a.pt_off + it.b * a.G + it.g + 1);
      }
      const int tok = 32 * ((it.t0 >> 5) + warp + NW * step) + 16 * (n & 1);
      if (tok + 16 <= it.t0 || tok >= it.t1) return kNone;
      const int t = tok >> 4, in_list = pool.p16 == 1 ? t : t / pool.p16;
      if (base + in_list >= end) return kBad;  // a list too short
      const int32_t page = __ldcg(a.pt_ids + base + in_list);
      if (page < 0 || page >= a.pool_pages) return kBad;
      return (page * a.H_p + it.hpos) * pool.p16 + t - in_list * pool.p16;
    };
    int at_cur = tile_at(lane), at_nxt = 0;
    int issued = 0, consumed = 0;
    const uint32_t stage0 = smem_addr(ring + warp * R * LY::STAGE);
    // lanes 0 and 1 copy a tile each into their half of the stage
    const uint32_t bar0 = smem_addr(&bars[warp * R]), to0 = stage0 + (lane & 1) * LY::TILE;
    auto issue = [&]() {  // whole warp: step number `issued` of this warp into stage issued % R
      const int at = __shfl_sync(0xffffffffu, at_cur, 2 * (issued & 15) + (lane & 1));
      if (lane < 2) {
        fence_proxy_async_smem();  // what was read of this stage comes before the refill
        const int s = issued % R;
        if (at == kBad) report(a.status, TG_STATUS_BAD_PAGE);
        // (an arrival without data)
        arrive_expect(bar0 + 8 * s, at >= 0 ? LY::TILE : 0);
        if (at >= 0) bulk_load_at(to0 + s * LY::STAGE, pool.base + (int64_t)at * LY::TILE, LY::TILE, bar0 + 8 * s);
      }
      ++issued;
      if ((issued & 15) == 0) {
        at_cur = at_nxt;
        at_nxt = tile_at(2 * issued + 32 + lane);
      }
    };
    for (int s = 0; s < R && issued < total; ++s) issue();
    at_nxt = tile_at(32 + lane);  // (looked up behind the first copies, which are fewer than sixteen steps)

    bool dead = false;  // a copy wait timed out: skip all further tiles, keep handing off
    // the reference of each head's weights, and their sum
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[C][8][4];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) o[c][i][0] = o[c][i][1] = o[c][i][2] = o[c][i][3] = 0.f;

    for (int k = 0; k < n_items; ++k) {
      const tg_work_item it = get_item(k);
      int lo;
      const int steps = warp_steps(it, lo);
      if (steps > 0 && !dead) {
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
        for (int i = 0; i < steps; ++i) {
          const int kk = lo + warp + i * NW;
          const int s = consumed % R;
          if (!__all_sync(0xffffffffu, mbar_wait_suspended(&bars[warp * R + s], (uint32_t)((consumed / R) & 1), kWaitLimitNs))) {
            if (lane == 0) report(a.status, TG_STATUS_TIMEOUT);
            dead = true;
            break;
          }
          const uint32_t stage = stage0 + s * LY::STAGE;
          const int r0 = it.t0 - kk * 32, r1 = it.t1 - kk * 32;  // valid rows [r0, r1) of the step
          const bool part = r0 > 0 || r1 < 32;

          // S^T = K Q^T (rows: tokens gid and gid + 8 of each half, columns: heads 2 tig and 2 tig + 1)
          float sc[2][4];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            sc[hf][0] = sc[hf][1] = sc[hf][2] = sc[hf][3] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const uint32_t kt = stage + hf * LY::TILE + c * kTile4;
              const uint4 x = lds128(kt + 64 * gid + 16 * tig), y = lds128(kt + 64 * (gid + 8) + 16 * tig);
              const uint32_t sx = e4m3x2_to_f16x2(lds16(kt + kKScales4 + 8 * gid + 2 * tig));
              const uint32_t sy = e4m3x2_to_f16x2(lds16(kt + kKScales4 + 8 * (gid + 8) + 2 * tig));
              const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int w = 0; w < 4; ++w) {  // eight values of each row; the first 16 have one scale, the others the next
                const uint32_t fx = __byte_perm(sx, 0, w < 2 ? 0x1010 : 0x3232), fy = __byte_perm(sy, 0, w < 2 ? 0x1010 : 0x3232);
                uint32_t hx[4], hy[4];
                e2m1x8_to_f16x2(wx[w], hx);
                e2m1x8_to_f16x2(wy[w], hy);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  mma_f16(sc[hf], mul_f16x2(hx[2 * j], fx), mul_f16x2(hy[2 * j], fy), mul_f16x2(hx[2 * j + 1], fx),
                          mul_f16x2(hy[2 * j + 1], fy), qf[c][2 * w + j][0], qf[c][2 * w + j][1]);
              }
            }
          }
          if (part) {
            // Rows that are no token of this piece may hold anything.  Their scores are replaced below; their V's scales
            // are cleared here, for a weight of 0 times a code times 0 is 0.
            if (lane < r0 || lane >= r1) {
#pragma unroll
              for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  asm volatile("st.shared.u8 [%0], %1;" ::"r"(stage + (lane >> 4) * LY::TILE + c * kTile4 + v_scale4(lane & 15, j)),
                               "r"(0) : "memory");
            }
            __syncwarp();
          }
          // the codes of V (of the first 128 values: of 256 they would spill), on their way during the softmax
          uint4 vx[2], vy[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t vt = stage + hf * LY::TILE + kVCodes4;
            vx[hf] = lds128(vt + 64 * gid + 16 * tig), vy[hf] = lds128(vt + 512 + 64 * gid + 16 * tig);
          }
          // online softmax, base 2; y = x - m
          auto logits = [&](float(&y)[2][4]) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                const float2 v = add2(mul2(make_float2(sc[hf][j], sc[hf][j + 1]), make_float2(z0, z1)), make_float2(-m0, -m1));
                y[hf][j] = v.x, y[hf][j + 1] = v.y;
              }
            if (part) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int t = 16 * hf + gid + (j & 2 ? 8 : 0);
                  if (t < r0 || t >= r1) y[hf][j] = -INFINITY;
                }
            }
          };
          float y[2][4];
          logits(y);
          const float top = max3(max3(y[0][0], y[0][1], y[0][2]), max3(y[0][3], y[1][0], y[1][1]), fmaxf(y[1][2], y[1][3]));
          if (__any_sync(0xffffffffu, top > kWeightMost)) {
            // the reference moves to 8 below the maximum so far
            float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int j = 0; j < 4; j += 2) {
                const int t = 16 * hf + gid + 4 * j;
                if (t < r0 || t >= r1) continue;
                x0 = fmaxf(x0, sc[hf][j] * z0);
                x1 = fmaxf(x1, sc[hf][j + 1] * z1);
              }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
              x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            }
            const float n0 = fmaxf(m0, __fadd_ru(x0, -kWeightLog2)), n1 = fmaxf(m1, __fadd_ru(x1, -kWeightLog2));
            const float c0 = n0 == m0 ? 1.f : ex2(m0 - n0), c1 = n1 == m1 ? 1.f : ex2(m1 - n1);
            m0 = n0, m1 = n1;
            l0 *= c0, l1 *= c1;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
              for (int j = 0; j < 8; ++j) o[c][j][0] *= c0, o[c][j][1] *= c1, o[c][j][2] *= c0, o[c][j][3] *= c1;
            logits(y);
          }
          uint32_t wt[2][2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float p0 = ex2(y[hf][0]), p1 = ex2(y[hf][1]), p2 = ex2(y[hf][2]), p3 = ex2(y[hf][3]);
            const float2 l = add2(make_float2(l0, l1), add2(make_float2(p0, p1), make_float2(p2, p3)));
            l0 = l.x, l1 = l.y;
            wt[hf][0] = movmatrix_t(pack_f16x2(p0, p1));
            wt[hf][1] = movmatrix_t(pack_f16x2(p2, p3));
          }
          // O^T += V^T P^T (rows: values 16 gid + 2 i and one on, columns: heads); this lane's tokens: 2 tig, 2 tig + 1
          // and the two 8 behind them, of each half
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t tile = stage + hf * LY::TILE + c * kTile4;
              const uint4 x = c == 0 ? vx[hf] : lds128(tile + kVCodes4 + 64 * gid + 16 * tig);
              const uint4 yv = c == 0 ? vy[hf] : lds128(tile + kVCodes4 + 512 + 64 * gid + 16 * tig);
              const uint32_t sx = e4m3x2_to_f16x2(lds16(tile + kVScales4 + 16 * gid + 2 * tig));
              const uint32_t sy = e4m3x2_to_f16x2(lds16(tile + kVScales4 + 16 * gid + 2 * tig + 8));
#pragma unroll
              for (int w = 0; w < 2; ++w) {  // values 8 w .. 8 w + 7 of the block
                const uint32_t xa = w ? x.y : x.x, xb = w ? x.w : x.z, ya = w ? yv.y : yv.x, yb = w ? yv.w : yv.z;
                // even and odd values, the first token in the lower half of each byte
                uint32_t ex[4], ox[4], ey[4], oy[4];
                e2m1x8_to_f16x2((xa & 0x0f0f0f0fu) | (xb << 4 & 0xf0f0f0f0u), ex);
                e2m1x8_to_f16x2((xa >> 4 & 0x0f0f0f0fu) | (xb & 0xf0f0f0f0u), ox);
                e2m1x8_to_f16x2((ya & 0x0f0f0f0fu) | (yb << 4 & 0xf0f0f0f0u), ey);
                e2m1x8_to_f16x2((ya >> 4 & 0x0f0f0f0fu) | (yb & 0xf0f0f0f0u), oy);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  mma_f16(o[c][4 * w + j], mul_f16x2(ex[j], sx), mul_f16x2(ox[j], sx), mul_f16x2(ey[j], sy),
                          mul_f16x2(oy[j], sy), wt[hf][0], wt[hf][1]);
              }
            }
          ++consumed;
          __syncwarp();
          if (issued < total) issue();
        }
      }

      // ---- hand this warp's state of item k to the epilogue (of two buffers: k & 1, its use k >> 1)
      const int hb = pool.buffers == 2 ? k & 1 : 0, use = pool.buffers == 2 ? k >> 1 : k;
      if (use > 0 && !*s_dead && !mbar_wait(&empty[hb], (uint32_t)((use - 1) & 1), kWaitLimitNs)) {
        if (lane == 0) report(a.status, TG_STATUS_TIMEOUT);
        *s_dead = 1;
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, off);
        l1 += __shfl_xor_sync(0xffffffffu, l1, off);
      }
      const float unit = pool.v_unit;
      float *cm = comb_m + (hb * NW + warp) * 8, *cl = comb_l + (hb * NW + warp) * 8;
      if (gid == 0) {
        cm[2 * tig] = m0;
        cm[2 * tig + 1] = m1;
        cl[2 * tig] = l0;
        cl[2 * tig + 1] = l1;
      }
      float *co = comb_o + hb * cfl + warp * a.g * ostride;  // [g][ostride] of this warp
      const int h0 = 2 * tig, h1 = 2 * tig + 1;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float(&oo)[4] = o[c][i];
          const int at = 128 * c + 16 * gid + 2 * i;
          if (h0 < a.g) *reinterpret_cast<float2 *>(co + h0 * ostride + at) = make_float2(oo[0] * unit, oo[2] * unit);
          if (h1 < a.g) *reinterpret_cast<float2 *>(co + h1 * ostride + at) = make_float2(oo[1] * unit, oo[3] * unit);
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
  grown_epilogue<D, NW, NE>(a, get_item, n_items, pool.buffers, comb_m, comb_l, comb_o, cfl, ostride, fac, s_mm, s_ll, flag,
                            s_dead, full, empty, s_t0);
}

struct Kernel {
  void *fn;
  int threads, smem, buffers;
};

// The kernel of a call with g query heads a KV head, ready to launch.  It comes ahead of the tensor map: a host thread's first
// call into the runtime makes the context current that the driver's encoder needs.
template <int D>
int kernel_of(const char *name, int format, int g, Kernel &k) {
  k.buffers = Layout4<D>::buffers(g);
  int most;
  if (format == TG_PAGES_BF16) {
    k.fn = reinterpret_cast<void *>(&grown_decode_kernel<D>);
    k.threads = Layout<D>::THREADS, k.smem = Layout<D>::smem_bytes(g), most = Layout<D>::smem_most();
  } else {
    k.fn = reinterpret_cast<void *>(&decode4_kernel<D>);
    k.threads = Layout4<D>::THREADS, k.smem = Layout4<D>::bytes(g, k.buffers), most = Layout4<D>::bytes_most();
  }
  cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return tgi::fail(TG_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", name, cudaGetErrorString(e));
  return TG_OK;
}

int launch(const char *name, cudaStream_t stream, int format, const Kernel &k, const void *map, const DecodeArgs &args, const Pool4 &pool,
           int N_CTA) {
  void *bf16[] = {const_cast<void *>(map), const_cast<DecodeArgs *>(&args)};
  void *e2m1[] = {const_cast<DecodeArgs *>(&args), const_cast<Pool4 *>(&pool)};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(N_CTA);
  cfg.blockDim = dim3(k.threads);
  cfg.dynamicSmemBytes = (size_t)k.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, k.fn, format == TG_PAGES_BF16 ? bf16 : e2m1);
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
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15)
    return fail(TG_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", fn);
  if (workspace_bytes < hd->workspace_bytes)
    return fail(TG_ERR_CAPACITY, "%s: workspace %lld < %lld bytes", fn, (long long)workspace_bytes,
                (long long)hd->workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(TG_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", fn);
  DecodeArgs args = decode_args(hd, lt, plan_dev, static_cast<uint8_t *>(workspace), q, out, lse, pt_off, pt_ids,
                                pool_pages, scale, dev_status, cta_time);
  args.ntok = ntok, args.added = added, args.plus = plus, args.reserve = reserve;
  args.wait_tables = 1;  // the kernel before it may have written pages, queries and added
  const int p16 = hd->P / 16;
  if (format == TG_PAGES_BF16) {
    if ((rc = check_pool(pool_pages, hd, fn))) return rc;
  } else {
    if (!unit_ok(k_unit) || !unit_ok(v_unit))
      return fail(TG_ERR_INVALID_ARG, "%s: k_unit=%g, v_unit=%g (powers of two in [2^-60, 2^60])", fn, (double)k_unit,
                  (double)v_unit);
    if (pool_pages <= 0 || pool_pages > INT32_MAX / hd->H_p / p16)
      return fail(TG_ERR_CAPACITY, "%s: pool_pages=%lld gives more than 2^31-1 tiles, or none", fn, (long long)pool_pages);
    args.scale_log2 *= k_unit;
  }
  Kernel k;
  rc = hd->d == 128 ? kernel_of<128>(fn, format, args.g, k) : kernel_of<256>(fn, format, args.g, k);
  if (rc) return rc;
  CUtensorMap map;
  if (format == TG_PAGES_BF16 && (rc = make_pool_map(&map, static_cast<const uint16_t *>(pool), pool_pages, hd, fn))) return rc;
  const Pool4 p4 = {static_cast<const uint8_t *>(pool), p16, v_unit, k.buffers};
  return launch(fn, reinterpret_cast<cudaStream_t>(stream), format, k, &map, args, p4, hd->N_CTA);
}
