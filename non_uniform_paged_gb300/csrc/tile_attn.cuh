// Attention of tiles of query rows over runs of keys on the fifth-generation tensor cores:
// the kernel behind tg_prefill_attn (contexts [batch][H][Nmax][d], causal) and
// tg_prefix_attn (page lists, every row sees every key), and the kernel that merges the
// pieces of cut runs.
//
// Mathematics.  For a row q and keys t in blocks of 128, with base-2 logits
// x_t = scale * log2(e) * q . k_t, a reference m and running l, O:
//     l += sum_t 2^(x_t - m),   O += sum_t 2^(x_t - m) v_t,
// and out = O / l, lse = ln 2 * (m + log2 l).  m follows the row's maximum lazily: it moves
// (and l, O are scaled by 2^(m_old - m_new)) only when the maximum has risen by more than 8,
// so weights stay below 2^8 and float32 sums lose nothing.  The weights are rounded to bf16
// for the product with V (at most 2^-8 relative each, both signs); l sums them unrounded.
//
// Layout.  A tile is 128 rows: tile_tokens(g) consecutive tokens (or requests) x the g query
// heads of one KV head, so a key is read once for all heads that share it, and one query
// token still fills g rows.  A thread block (one per SM, 227 KB of shared memory) works on
// two tiles at d = 128 and one at d = 256: S (128 x 128 float32) twice and O (256 columns
// in all) fill the 512 columns of tensor memory.
//   warps 0-3 (4-7): softmax and output of tile 0 (1), one row per thread;
//   then a warp whose elected lane issues the MMAs, one that streams Q, K and V by TMA, and one
//   that clears the V rows behind the end of a context.
// K and V go through a ring of five 32 KB stages (128 keys x 128 columns each; d = 256
// takes two per block).  P overwrites S in tensor memory and is the A operand of P V.
// At d = 128 the two tiles alternate: while one is in softmax the tensor cores run
// P V and the next Q K^T of the other; at d = 256 the two S buffers alternate over blocks.
// Items of the plan follow one another without a break: the loader runs ahead into the next.
#pragma once

#include "tcgen05.cuh"
#include "tg_internal.h"
#include "tile_common.h"

namespace tgk {

constexpr int kStages = 5;
constexpr uint32_t kStageBytes = 32768;       // 128 rows x 128 bf16, two 64-column halves
constexpr uint32_t kHalfBytes = 16384;
constexpr uint32_t kQBytes = 65536;           // 256 x 128 or 128 x 256
constexpr uint32_t kTileSmem = kQBytes + kStages * kStageBytes + 1024 + 1024;  // + barriers, + alignment
constexpr uint64_t kTileWaitNs = 2000000000ull;
constexpr float kTileLn2 = 0.69314718055994531f;
constexpr float kTileLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;  // the reference moves when the maximum has risen by 2^8

struct TileArgs {
  const tg_tile_item *items, *lead;
  uint16_t *out;
  float *lse;
  const uint16_t *own_out;
  const float *own_lse;
  float *ws_ml, *ws_o;
  const int64_t *pt_off;
  const int32_t *pt_ids;
  int64_t pool_pages;
  int32_t *status;
  int H, H_q, g, tq, window;
  int P, H_p, R;  // paged: R keys per TMA box, a divisor of P and of 128
  int signal;     // a dependent kernel follows: let it start early
  float scale_log2;
};

struct TileBars {
  // pv_done: each P V of a tile (d = 128) or of the tile (d = 256, [0]); there [1] is the last one
  // of an item, because an S of d = 256 is issued ahead of the P V before it, so that [0] may lag
  // two phases behind when an item ends
  // p_half: the first 64 keys' weights are in tensor memory; p_ready: all 128
  uint64_t q_full, q_empty, full[kStages], empty[kStages], s_full[2], p_half[2], p_ready[2], pv_done[2], to_clear, cleared, drain;
  uint32_t tmem;
  int32_t abort;
};

// Wait for a phase; false when this block gave up (here or elsewhere).  Every lane of the warp
// gets the same answer.
__device__ __forceinline__ bool tile_wait_slow(uint64_t *bar, uint32_t parity, volatile int32_t *abort,
                                              int32_t *status) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kTileWaitNs) {
      *abort = 1;
      report(status, TG_STATUS_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool tile_wait(uint64_t *bar, uint32_t parity, TileBars *b, int32_t *status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = tile_wait_slow(bar, parity, &b->abort, status);
  return __all_sync(0xffffffffu, ok);
}

// the same for a role that one lane plays
__device__ __forceinline__ bool lane_wait(uint64_t *bar, uint32_t parity, TileBars *b, int32_t *status) {
  if (mbar_try_wait(bar, parity)) return true;
  return tile_wait_slow(bar, parity, &b->abort, status);
}

// The items of a thread block; the next one's line is fetched ahead into L1.
struct ItemList {
  const tg_tile_item *at;
  tg_tile_item cur;
  int left;
  __device__ __forceinline__ void fetch(const tg_tile_item *p) {
    const int4 *s = reinterpret_cast<const int4 *>(p);
    int4 *d = reinterpret_cast<int4 *>(&cur);
    d[0] = __ldg(s), d[1] = __ldg(s + 1), d[2] = __ldg(s + 2);
  }
  __device__ __forceinline__ void start(const TileArgs &a) {
    const tg_tile_item *lead = a.lead + blockIdx.x;
    const int2 v = __ldg(reinterpret_cast<const int2 *>(lead->reserved));
    left = v.x;
    at = a.items + v.y;
  }
  __device__ __forceinline__ bool advance() {
    if (left <= 0) return false;
    fetch(at++);
    if (--left > 0) asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
    return true;
  }
};

// ------------------------------------------------------------------ softmax and output warps
template <int D, bool PAGED>
__device__ __forceinline__ void softmax_role(const TileArgs &a, TileBars *bar, int tile) {
  const int r = threadIdx.x & 127;             // row of the tile = lane of tensor memory
  const int tok = r / a.g, head = r - tok * a.g;
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t o_base = 256 + (D == 128 ? tile * 128 : 0) + lanes;
  const float sl2 = a.scale_log2;
  uint32_t s_count = 0, pv_count = 0, item_count = 0;
  ItemList list;
  list.start(a);
  while (list.advance()) {
    const tg_tile_item &it = list.cur;
    const tgi::TileRange rg = tgi::tile_range(it, tile, a.tq, a.window, !PAGED);
    const int first = tile * a.tq;
    const int n = min(it.nrow - first, a.tq);
    if (n <= 0) continue;
    int lo = 0, hi = it.kv_len;            // keys [lo, hi) that this row sees
    int lo_last = 0, hi_first = it.kv_len; // ... that every row of the tile sees
    if (!PAGED) {
      const int pos = it.pos0 + first;
      hi = min(hi, pos + tok + 1);
      hi_first = min(hi_first, pos + 1);
      if (a.window > 0) {
        lo = max(0, pos + tok - a.window + 1);
        lo_last = max(0, pos + n - a.window);
      }
    }
    float m = -INFINITY, l = 0.f;
    for (int j = rg.b; j < rg.e; ++j) {
      const int buf = D == 128 ? tile : (int)(s_count & 1);
      const uint32_t phase = (D == 128 ? s_count : s_count >> 1) & 1;
      ++s_count;
      const uint32_t s_addr = buf * 128 + lanes;
      if (!tile_wait(&bar->s_full[buf], phase, bar, a.status)) return;
      tc_fence_after();
      float s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, reinterpret_cast<uint32_t *>(s) + c * 32);
      tmem_wait_ld();
      const int k0 = j * 128;
      if (k0 + 128 > hi_first || k0 < lo_last) {
        const int h1 = hi - k0, l1 = lo - k0;
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = (c < h1 && c >= l1) ? s[c] : -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 128; c += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[c + k]), c + 4 + k < 128 ? s[c + 4 + k] : s[c + k]);
      }
      const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
      if (j == rg.b) {
        m = m_new;
      } else if (__any_sync(0xffffffffu, (m_new - m) * sl2 > kLazy)) {
        // the block before has been added to O: at d = 128 this S was issued after it
        if (D == 256) {
          if (!tile_wait(&bar->pv_done[0], (pv_count - 1) & 1, bar, a.status)) return;
          tc_fence_after();
        }
        const float f = m_new == -INFINITY ? 1.f : ex2((m - m_new) * sl2);
        m = m_new;
        l *= f;
#pragma unroll 1
        for (int c = 0; c < (D == 128 ? 4 : 8); ++c) {
          uint32_t o[32];
          tmem_ld32(o_base + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          tmem_st32(o_base + c * 32, o);
        }
      }
      const float neg = m == -INFINITY ? 0.f : -m * sl2;
      float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float2 x = fma2(make_float2(s[c * 32 + 2 * k], s[c * 32 + 2 * k + 1]), make_float2(sl2, sl2),
                          make_float2(neg, neg));
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          sum[k & 1] = add2(sum[k & 1], x);
          p[k] = pack_bf16x2(x.x, x.y);
        }
        tmem_st16(s_addr + c * 16, p);
        if (c == 1) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if ((threadIdx.x & 31) == 0) mbar_arrive(&bar->p_half[buf]);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&bar->p_ready[buf]);
      ++pv_count;
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }

    // output: this row's O / l, or the piece's (m, l, O)
    const bool mine = tok < n && r < a.tq * a.g;
    const int64_t row = ((int64_t)(it.row0 + first + tok)) * a.H_q + it.h * a.g + head;
    const bool some = rg.b < rg.e;
    if (some) {
      const uint32_t done = D == 128 ? pv_count - 1 : item_count++;
      if (!tile_wait(&bar->pv_done[D == 128 ? tile : 1], done & 1, bar, a.status)) return;
      tc_fence_after();
    }
    float mo = m == -INFINITY ? -INFINITY : m * sl2;  // base-2 reference
    if (it.slot >= 0) {
      const int64_t at = (int64_t)it.slot * 256 + tile * 128 + r;
      if (mine) *reinterpret_cast<float2 *>(a.ws_ml + at * 2) = make_float2(mo, l);
      float *dst = a.ws_o + (int64_t)it.slot * 32768 + (int64_t)(tile * 128 + r) * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (some) {
          tmem_ld32(o_base + c * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (mine) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(dst + c * 32 + k * 4) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
    } else {
      float f1, f2 = 0.f, total = l, top = mo;
      if (PAGED && a.own_lse && mine) {
        const float w = a.own_lse[row] * kTileLog2e;
        top = fmaxf(mo, w);
        const float e1 = mo == -INFINITY ? 0.f : ex2(mo - top);
        const float e2 = w == -INFINITY ? 0.f : ex2(w - top);
        total = l * e1 + e2;
        f1 = total == 0.f ? 0.f : e1 / total;
        f2 = total == 0.f ? 0.f : e2 / total;
      } else {
        f1 = total == 0.f ? 0.f : 1.f / total;
      }
      if (mine && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kTileLn2;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (some) {
          tmem_ld32(o_base + c * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (mine) {
          uint16_t *dst = a.out + row * D + c * 32;
          const uint4 *src = PAGED && f2 != 0.f ? reinterpret_cast<const uint4 *>(a.own_out + row * D + c * 32) : nullptr;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[8 * k + e]) * f1;
            if (src) {
              const uint4 w = src[k];
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[2 * e] += f2 * __uint_as_float(ww[e] << 16);
                v[2 * e + 1] += f2 * __uint_as_float(ww[e] & 0xffff0000u);
              }
            }
            *reinterpret_cast<uint4 *>(dst + 8 * k) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          }
        }
      }
    }
    tc_fence_before();  // the next item's first P V overwrites O after this warp's next arrival
  }
}

// ------------------------------------------------------------------ MMA lane
struct RingPos {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) stage = 0, phase ^= 1;
  }
  __device__ __forceinline__ void skip(uint32_t n) {
    const uint32_t s = stage + n;
    phase ^= (s / kStages) & 1;
    stage = s % kStages;
  }
};

// the key blocks [b, e) that an item's tiles need together (empty: none)
template <int D, bool PAGED>
__device__ __forceinline__ tgi::TileRange item_range(const tg_tile_item &it, const TileArgs &a, tgi::TileRange *r0,
                                                     tgi::TileRange *r1) {
  *r0 = tgi::tile_range(it, 0, a.tq, a.window, !PAGED);
  *r1 = {0, 0};
  if (D == 128) *r1 = tgi::tile_range(it, 1, a.tq, a.window, !PAGED);
  if (r1->b >= r1->e) return *r0;
  if (r0->b >= r0->e) return *r1;
  return {min(r0->b, r1->b), max(r0->e, r1->e)};
}
// rows of the last block behind the context's end have to be cleared (pages hold finite rows)
template <bool PAGED>
__device__ __forceinline__ bool has_tail(const tg_tile_item &it, int j1) {
  return !PAGED && j1 * 128 > it.kv_len;
}

// S = Q K^T over one 128-column piece
__device__ __forceinline__ void issue_qk(uint32_t s, uint32_t q, uint32_t k, bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, 128, false);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t at = (i >> 2) * kHalfBytes + (i & 3) * 32;
    mma_ss(s, smem_desc(q + at, 16, 1024), smem_desc(k + at, 16, 1024), idesc, accumulate || i > 0);
  }
}
// O += P V over 64 of a stage's 128 keys x 128 columns
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint32_t v, int half, bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, 128, true);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = half * 4 + i;
    mma_ts(o, p + k * 8, smem_desc(v + k * 2048, kHalfBytes, 1024), idesc, accumulate || i > 0);
  }
}

template <int D, bool PAGED>
__device__ __forceinline__ bool mma_items(const TileArgs &a, TileBars *bar, uint32_t q_at, uint32_t ring_at) {
  RingPos rp;
  uint32_t q_phase = 0, p_count[2] = {0, 0}, c_phase = 0;
  ItemList list;
  list.start(a);
  while (list.advance()) {
    const tg_tile_item &it = list.cur;
    tgi::TileRange r0, r1;
    const tgi::TileRange rg = item_range<D, PAGED>(it, a, &r0, &r1);
    const int j0 = rg.b, j1 = rg.e;
    if (j0 >= j1) continue;
    const bool tail = has_tail<PAGED>(it, j1);
    if (!lane_wait(&bar->q_full, q_phase, bar, a.status)) return false;
    q_phase ^= 1;
    if (D == 128) {
      // K of the first block for both tiles, then per block and tile: P V, next Q K^T
      if (!lane_wait(&bar->full[rp.stage], rp.phase, bar, a.status)) return false;
      const uint32_t k = ring_at + rp.stage * kStageBytes;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const tgi::TileRange r = i ? r1 : r0;
        if (r.b == j0 && r.b < r.e) issue_qk(i * 128, q_at + i * kStageBytes, k, false), mma_commit(&bar->s_full[i]);
      }
      mma_commit(&bar->empty[rp.stage]);
      if (j1 - j0 == 1) mma_commit(&bar->q_empty);
      rp.next();
      for (int j = j0; j < j1; ++j) {
        const RingPos vp = rp;
        rp.next();
        const RingPos kp = rp;
        const bool more = j + 1 < j1;
        if (more) rp.next();
        const uint32_t v = ring_at + vp.stage * kStageBytes, kn = ring_at + kp.stage * kStageBytes;
        if (!lane_wait(&bar->full[vp.stage], vp.phase, bar, a.status)) return false;
        if (!more && tail) {
          mbar_arrive(&bar->to_clear);
          if (!lane_wait(&bar->cleared, c_phase, bar, a.status)) return false;
          c_phase ^= 1;
        }
        bool k_there = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const tgi::TileRange r = i ? r1 : r0;
          if (j >= r.b && j < r.e) {
            const uint32_t o = 256 + i * 128, p = i * 128;
            if (!lane_wait(&bar->p_half[i], p_count[i] & 1, bar, a.status)) return false;
            tc_fence_after();
            issue_pv(o, p, v, 0, j > r.b);
            if (!lane_wait(&bar->p_ready[i], p_count[i] & 1, bar, a.status)) return false;
            ++p_count[i];
            tc_fence_after();
            issue_pv(o, p, v, 1, true);
            mma_commit(&bar->pv_done[i]);
          }
          if (more && j + 1 >= r.b && j + 1 < r.e) {
            if (!k_there && !lane_wait(&bar->full[kp.stage], kp.phase, bar, a.status)) return false;
            k_there = true;
            issue_qk(i * 128, q_at + i * kStageBytes, kn, false);
            mma_commit(&bar->s_full[i]);
          }
        }
        mma_commit(&bar->empty[vp.stage]);
        if (more) mma_commit(&bar->empty[kp.stage]);
        if (j + 2 == j1) mma_commit(&bar->q_empty);
      }
    } else {
      // ring order: K(j0), K(j0+1), V(j0), K(j0+2), V(j0+1), ...
      for (int j = j0 - 1; j < j1; ++j) {
        if (j + 1 < j1) {
          const uint32_t buf = p_count[1] & 1;  // p_count[1] counts the S buffers issued
          ++p_count[1];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!lane_wait(&bar->full[rp.stage], rp.phase, bar, a.status)) return false;
            issue_qk(buf * 128, q_at + c * kStageBytes, ring_at + rp.stage * kStageBytes, c > 0);
            mma_commit(&bar->empty[rp.stage]);
            rp.next();
          }
          mma_commit(&bar->s_full[buf]);
          if (j + 2 == j1) mma_commit(&bar->q_empty);
        }
        if (j >= j0) {
          const uint32_t buf = p_count[0] & 1, phase = (p_count[0] >> 1) & 1;
          ++p_count[0];
          const RingPos v0 = rp;
          rp.next();
          const RingPos v1 = rp;
          rp.next();
          const uint32_t s0 = ring_at + v0.stage * kStageBytes, s1 = ring_at + v1.stage * kStageBytes;
          if (!lane_wait(&bar->full[v0.stage], v0.phase, bar, a.status)) return false;
          if (!lane_wait(&bar->full[v1.stage], v1.phase, bar, a.status)) return false;
          if (j + 1 == j1 && tail) {
            mbar_arrive(&bar->to_clear);
          if (!lane_wait(&bar->cleared, c_phase, bar, a.status)) return false;
            c_phase ^= 1;
          }
          if (!lane_wait(&bar->p_half[buf], phase, bar, a.status)) return false;
          tc_fence_after();
          issue_pv(256, buf * 128, s0, 0, j > j0);
          issue_pv(384, buf * 128, s1, 0, j > j0);
          if (!lane_wait(&bar->p_ready[buf], phase, bar, a.status)) return false;
          tc_fence_after();
          issue_pv(256, buf * 128, s0, 1, true);
          mma_commit(&bar->empty[v0.stage]);
          issue_pv(384, buf * 128, s1, 1, true);
          mma_commit(&bar->empty[v1.stage]);
          mma_commit(&bar->pv_done[0]);
          if (j + 1 == j1) mma_commit(&bar->pv_done[1]);
        }
      }
    }
  }
  return true;
}

// ------------------------------------------------------------------ clearing warp
// Zeroes the rows of an item's last V block that lie behind the context: P is 0 there, and must
// meet 0 whatever memory holds.  It finds the block's stages by counting the ring; the MMA lane
// tells it that they have landed and waits for it.
template <int D>
__device__ __forceinline__ void clear_tails(const TileArgs &a, TileBars *bar, uint32_t ring_at) {
  constexpr int NP = D / 128;
  const int lane = threadIdx.x & 31;
  uint32_t phase = 0;
  RingPos rp;
  ItemList list;
  list.start(a);
  while (list.advance()) {
    tgi::TileRange r0, r1;
    const tgi::TileRange rg = item_range<D, false>(list.cur, a, &r0, &r1);
    if (rg.b >= rg.e) continue;
    rp.skip((rg.e - rg.b) * 2 * NP - NP);  // the item's last V block ends its stages
    if (!has_tail<false>(list.cur, rg.e)) {
      rp.skip(NP);
      continue;
    }
    const int from = list.cur.kv_len - (rg.e - 1) * 128;
    if (!tile_wait(&bar->to_clear, phase, bar, a.status)) return;
    phase ^= 1;
    for (int c = 0; c < NP; ++c) {
      for (int i = from * 8 + lane; i < 128 * 8; i += 32) {
        const uint32_t at = ring_at + rp.stage * kStageBytes + (uint32_t)i * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + kHalfBytes), "r"(0) : "memory");
      }
      rp.next();
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->cleared);
  }
}

// ------------------------------------------------------------------ loader warp
// The lanes look up the pages of a block's boxes, one block ahead; an elected lane issues the copies.
template <int D, bool PAGED>
__device__ __forceinline__ void load_items(const CUtensorMap *qm, const CUtensorMap *km, const CUtensorMap *vm,
                                           const TileArgs &a, TileBars *bar, uint32_t q_at, uint32_t ring_at) {
  constexpr int NP = D / 128;  // stages per K or V block
  const int lane = threadIdx.x & 31;
  RingPos rp;
  uint32_t filled = 0, q_count = 0;  // stages filled, Q loads
  bool ok = true;
  const uint32_t q_box = (uint32_t)a.tq * a.g * 128;  // bytes of one 64-column box of Q
  const int outside = PAGED ? (int)(a.pool_pages * a.H_p * 2) : 0;  // a block past the pool: reads as zeros
  const int boxes = PAGED ? 128 / a.R : 0;
  ItemList list;
  list.start(a);
  while (ok && list.advance()) {
    const tg_tile_item &it = list.cur;
    tgi::TileRange r0, r1;
    const tgi::TileRange rg = item_range<D, PAGED>(it, a, &r0, &r1);
    const int j0 = rg.b, j1 = rg.e;
    if (j0 >= j1) continue;
    int64_t off0 = 0;
    int lists = 0;  // pages of the list
    if (PAGED) {
      off0 = a.pt_off[it.src];
      lists = (int)(a.pt_off[it.src + 1] - off0);
    }
    // lane i: the page block (K's; V's is the next) and first row of box i of block j
    auto place = [&](int j, int *row) -> int {
      const int t = j * 128 + lane * a.R;
      const int pg = t / a.P;
      *row = t - pg * a.P;
      if (lane >= boxes || t >= it.kv_len || j >= j1) return outside;
      const int32_t id = pg < lists ? __ldg(a.pt_ids + off0 + pg) : -1;
      if (id < 0 || id >= a.pool_pages) {
        report(a.status, TG_STATUS_BAD_PAGE);
        return outside;
      }
      return (id * a.H_p + it.hpos) * 2;
    };
    // one block of K (kv 0) or V (kv 1) into the ring
    auto fill = [&](int j, int kv, int z, int row) -> bool {
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        if (filled >= kStages && !tile_wait(&bar->empty[rp.stage], rp.phase ^ 1, bar, a.status)) return false;
        const uint32_t dst = ring_at + rp.stage * kStageBytes;
        uint64_t *full = &bar->full[rp.stage];
        if (PAGED) {
          int zs[8], rows[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int zi = __shfl_sync(0xffffffffu, z, i);
            zs[i] = zi == outside ? zi : zi + kv;
            rows[i] = __shfl_sync(0xffffffffu, row, i);
          }
          if (elect_one()) {
            mbar_arrive_expect_tx(full, kStageBytes);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (i < boxes) {
                const uint32_t to = dst + i * a.R * 128;
                tma_load_3d(to, km, full, c * 128, rows[i], zs[i]);
                tma_load_3d(to + kHalfBytes, km, full, c * 128 + 64, rows[i], zs[i]);
              }
            }
          }
        } else if (elect_one()) {
          const CUtensorMap *m = kv ? vm : km;
          const int context = it.src * a.H + it.h;
          mbar_arrive_expect_tx(full, kStageBytes);
          tma_load_3d(dst, m, full, c * 128, j * 128, context);
          tma_load_3d(dst + kHalfBytes, m, full, c * 128 + 64, j * 128, context);
        }
        __syncwarp();
        ++filled;
        rp.next();
      }
      return true;
    };
    int z = 0, row = 0, z_next = 0, row_next = 0, z_before = 0, row_before = 0;
    if (PAGED) z = place(j0, &row);
    if (q_count > 0 && !tile_wait(&bar->q_empty, (q_count - 1) & 1, bar, a.status)) {
      ok = false;
      break;
    }
    ++q_count;
    if (elect_one()) {
      if (D == 128) {
        const bool has0 = r0.b < r0.e, has1 = r1.b < r1.e;
        mbar_arrive_expect_tx(&bar->q_full, ((has0 ? 2 : 0) + (has1 ? 2 : 0)) * q_box);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((c >> 1) ? has1 : has0)
            tma_load_3d(q_at + c * kHalfBytes, qm, &bar->q_full, (c & 1) * 64, it.h * a.g, it.row0 + (c >> 1) * a.tq);
      } else {
        mbar_arrive_expect_tx(&bar->q_full, 4 * q_box);
#pragma unroll
        for (int c = 0; c < 4; ++c) tma_load_3d(q_at + c * kHalfBytes, qm, &bar->q_full, c * 64, it.h * a.g, it.row0);
      }
    }
    __syncwarp();
    for (int j = j0; ok && j < j1; ++j) {
      if (PAGED) z_next = place(j + 1, &row_next);
      ok = fill(j, 0, z, row);
      if (D == 128) {
        if (ok) ok = fill(j, 1, z, row);
      } else {
        if (ok && j > j0) ok = fill(j - 1, 1, z_before, row_before);
        if (ok && j + 1 == j1) ok = fill(j, 1, z, row);
        z_before = z, row_before = row;
      }
      z = z_next, row = row_next;
    }
  }
  // leave nothing in flight: every stage used and Q must have been consumed, or, after a
  // give-up, at least have landed
  for (uint32_t i = 0; ok && i < kStages && i < filled; ++i)
    ok = tile_wait(&bar->empty[i], ((filled - 1 - i) / kStages) & 1, bar, a.status);
  if (ok && q_count) ok = tile_wait(&bar->q_empty, (q_count - 1) & 1, bar, a.status);
  if (!ok) {
    for (uint32_t i = 0; i < kStages && i < filled; ++i)
      mbar_wait(&bar->full[i], ((filled - 1 - i) / kStages) & 1, 100000000ull);
    if (q_count) mbar_wait(&bar->q_full, (q_count - 1) & 1, 100000000ull);
    __syncwarp();
  }
}

// d = 128: two softmax warpgroups and a third of the MMA, loader and clearing warps and an idle
// one, so that registers can move from the third to the first two (168 each at launch: 384 x 168
// = 256 x 216 + 128 x 72); d = 256: seven warps, 255 registers each at most.
template <int D>
constexpr int tile_threads() {
  return D == 128 ? 384 : 224;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(tile_threads<D>(), 1)
    tile_attn_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                     const __grid_constant__ CUtensorMap vm, const TileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int SW = D == 128 ? 8 : 4;  // softmax warps
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  TileBars *bar = reinterpret_cast<TileBars *>(base + kQBytes + kStages * kStageBytes);
  const uint32_t q_at = smem_addr(base), ring_at = q_at + kQBytes;
  const int warp = threadIdx.x >> 5;
  if (warp == SW) tmem_alloc(&bar->tmem, 512);
  if (threadIdx.x == 0) {
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->q_empty, 1);
    for (int i = 0; i < kStages; ++i) mbar_init(&bar->full[i], 1), mbar_init(&bar->empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->s_full[i], 1), mbar_init(&bar->pv_done[i], 1);
      mbar_init(&bar->p_half[i], 4), mbar_init(&bar->p_ready[i], 4);
    }
    mbar_init(&bar->to_clear, 1);
    mbar_init(&bar->cleared, 1);
    mbar_init(&bar->drain, 1);
    bar->abort = 0;
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this block's, so they start at column 0: the MMAs and the softmax
  // address them by constants
  if (warp < SW) {
    if (D == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    softmax_role<D, PAGED>(a, bar, warp >> 2);
  } else {
    if (D == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == SW) {
      if (elect_one() && !mma_items<D, PAGED>(a, bar, q_at, ring_at)) {
        // gave up: what was issued must finish before tensor memory is freed
        mma_commit(&bar->drain);
        mbar_wait(&bar->drain, 0, 100000000ull);
      }
    } else if (warp == SW + 1) {
      if (elect_one()) prefetch_tensormap(&qm), prefetch_tensormap(&km), prefetch_tensormap(&vm);
      __syncwarp();
      load_items<D, PAGED>(&qm, &km, &vm, a, bar, q_at, ring_at);
    } else if (warp == SW + 2) {
      if (!PAGED) clear_tails<D>(a, bar, ring_at);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (a.signal) griddep_launch_dependents();
  tc_fence_after();
  if (warp == SW) tmem_free(bar->tmem, 512);
}

// ------------------------------------------------------------------ merge of cut runs
struct MergeArgs {
  const tg_tile_merge *merges;
  const float *ws_ml, *ws_o;
  uint16_t *out;
  float *lse;
  const uint16_t *own_out;
  const float *own_lse;
  int H_q, g, tq;
};

constexpr int kMergeWarps = 8;

// One warp per output row: sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p over the pieces (and
// the request's own result).  grid = merges x 256 / kMergeWarps.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tile_merge_kernel(const MergeArgs a) {
  constexpr int PER = 256 / kMergeWarps, E = D / 32;
  const tg_tile_merge mg = a.merges[blockIdx.x / PER];
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int k = (blockIdx.x % PER) * kMergeWarps + (threadIdx.x >> 5);  // row among the item's rows
  if (k >= mg.nrow * a.g) return;
  const int tok = k / a.g, head = k - tok * a.g;
  const int tile = tok / a.tq;
  const int r = tile * 128 + (tok - tile * a.tq) * a.g + head;
  const int64_t row = (int64_t)(mg.row0 + tok) * a.H_q + mg.h * a.g + head;
  const float2 *ml = reinterpret_cast<const float2 *>(a.ws_ml) + (int64_t)mg.slot0 * 256 + r;
  const float *po = a.ws_o + (int64_t)mg.slot0 * 32768 + (int64_t)r * D + lane * E;
  float M = -INFINITY;
  for (int p = lane; p < mg.nparts; p += 32) M = fmaxf(M, ml[(int64_t)p * 256].x);
  const float w = a.own_lse ? a.own_lse[row] * kTileLog2e : -INFINITY;
  M = fmaxf(M, w);
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float o[E] = {}, total = 0.f;
  for (int p0 = 0; p0 < mg.nparts; p0 += 32) {
    float f = 0.f, part = 0.f;
    if (p0 + lane < mg.nparts) {
      const float2 v = ml[(int64_t)(p0 + lane) * 256];
      f = v.x == -INFINITY ? 0.f : ex2(v.x - M);
      part = f * v.y;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
    total += part;
    const int n = min(32, mg.nparts - p0);
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
      const float fp = __shfl_sync(0xffffffffu, f, p);
      const float4 *src = reinterpret_cast<const float4 *>(po + (int64_t)(p0 + p) * 32768);
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        const float4 v = src[e];
        o[4 * e] += fp * v.x, o[4 * e + 1] += fp * v.y, o[4 * e + 2] += fp * v.z, o[4 * e + 3] += fp * v.w;
      }
    }
  }
  const float e2 = w == -INFINITY ? 0.f : ex2(w - M);
  total += e2;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  if (e2 != 0.f) {
    const uint32_t *src = reinterpret_cast<const uint32_t *>(a.own_out + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const uint32_t v = src[e];
      o[2 * e] += e2 * __uint_as_float(v << 16);
      o[2 * e + 1] += e2 * __uint_as_float(v & 0xffff0000u);
    }
  }
  uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E / 2; ++e) dst[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (lane == 0 && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (M + log2f(total)) * kTileLn2;
}

}  // namespace tgk
