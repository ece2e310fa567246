// Attention of tiles of query rows over runs of keys on the fifth-generation tensor cores:
// the kernel behind tg_prefill_attn (contexts [batch][H][Nmax][d], causal) and
// tg_prefix_attn (page lists, every row sees every key), and the kernel that merges the
// pieces of cut runs.
//
// Mathematics.  For a row q and keys t in blocks of 80, with base-2 logits
// x_t = scale * log2(e) * q . k_t, a reference m and running l, O:
//     l += sum_t 2^(x_t - m),   O += sum_t 2^(x_t - m) v_t,
// and out = O / l, lse = ln 2 * (m + log2 l).  m is the maximum of the row's first block with a
// key and moves (l and O scaled by 2^(m_old - m_new)) only when a later block's weights sum to more
// than 2^16: bf16 and float32 share their exponent range, so weights above 1 are as exact as
// those below, and the hot loop has no maximum to find.  The weights are rounded to bf16 for the
// product with V (at most 2^-8 relative each, both signs); l sums them unrounded.
//
// Layout.  A tile is 128 rows: tile_tokens(g) consecutive tokens (or requests) x the g query
// heads of one KV head, so a key is read once for all heads that share it, and one query
// token still fills g rows.  A thread block (one per SM, 227 KB of shared memory) works on
// two tiles at d = 128 and one at d = 256.
//   warps 0-7: softmax and output, a thread per row at d = 128, two at d = 256;
//   then two warps whose elected lanes issue the MMAs, one that streams Q, K and V by TMA, and
//   one that clears the V rows that no row sees.
// K and V go through a ring of eight 20 KB stages (80 keys x 128 columns each; d = 256
// takes two per block).
//
// Why 80 keys: O takes 256 of the 512 columns of tensor memory; two S of 80 columns and two P of
// 40 (bf16, the A operand of P V) fit in the rest.
//
// Who waits for whom.  At d = 128 each tile has an S and a P and goes in steps: in step t the lanes
// issue Q K^T of block t and P V of block t - 2, and the softmax, which has the weights of block
// t - 1 in registers by then, waits for both products at once, stores P(t - 1), reads S(t) and
// says so; then it computes on while the products of step t + 1 run.  One wait and one arrival a
// block: each costs 60 to 200 clocks on an SM whose special-function queue is full.  At d = 256 the
// blocks of the one tile alternate between two S and two P, each with barriers of its own, because
// a step would leave the tensor cores idle while the softmax turns round.
// With S of 128 columns and P in their place the softmax and both products alternated: 3100 clocks
// for 2048 of MMAs.
// Items of the plan follow one another without a break: the loader runs ahead into the next.
#pragma once

#include "tcgen05.cuh"
#include "tg_internal.h"
#include "tile_common.h"

namespace tgk {

constexpr int kKeys = tgi::kTileKeys;
constexpr int kStages = 8;
constexpr uint32_t kHalfBytes = kKeys * 128;      // 64 columns of a block
constexpr uint32_t kStageBytes = 2 * kHalfBytes;  // 80 rows x 128 bf16
constexpr uint32_t kQPiece = 32768;               // 128 rows x 128 columns
constexpr uint32_t kQBytes = 2 * kQPiece;         // 256 x 128 or 128 x 256
constexpr uint32_t kTileSmem = kQBytes + kStages * kStageBytes + 1024 + 1024;  // + barriers, + alignment
constexpr uint32_t kWeights = 160;  // first column of P (S: 0 and 80)
constexpr uint32_t kSwap = 240;    // columns through which two warps exchange row values
constexpr uint32_t kOut = 256;     // first column of O
// A wait gives up when its block has loaded nothing for this long, looked at every so many polls.  (The
// short form is for the test of giving up: there nearly every wait does.)
#ifdef TG_TILE_SHORT_WAIT
constexpr uint64_t kTileWaitNs = 0;
constexpr uint32_t kTilePolls = 1;
#else
constexpr uint64_t kTileWaitNs = 2000000000ull;
constexpr uint32_t kTilePolls = 64;
#endif
constexpr float kTileLn2 = 0.69314718055994531f;
constexpr float kTileLog2e = 1.4426950408889634f;
constexpr float kMost = 65536.f;  // the reference moves when a block's weights sum to more

struct TileArgs {
  const tg_tile_item *items, *lead;
  uint16_t *out;
  float *lse;
  const uint16_t *own_out;
  const float *own_lse;
  float *ws_ml, *ws_own, *ws_o;
  const int64_t *pt_off;
  const int32_t *pt_ids;
  int64_t pool_pages;
  int32_t *status;
  int H, H_q, g, tq, window;
  int P, H_p;  // paged
  int signal;  // a dependent kernel follows: let it start early
  float scale_log2;
};

// Barriers and flags, by byte offset from their shared-memory address (32-bit addresses keep the
// MMA lanes' code short: one lane runs an instruction every few clocks only).
//   d = 128, by tile -- made: a step's products are done (both lanes arrive); taken: P stored and S
//   read (the four softmax warps).  d = 256, by S and P buffer -- s_full: S written; s_free: read;
//   p_ready: P written; pv_done: multiplied with V and added to O.  Whoever waits for a phase of one
//   of them takes part in the next, so none is overtaken.
constexpr uint32_t kQFull = 0, kQEmpty = 8, kFull = 16, kEmpty = kFull + 8 * kStages, kSFull = kEmpty + 8 * kStages,
                   kPvDone = kSFull + 16, kToClear = kPvDone + 16, kCleared = kToClear + 8, kDrain = kCleared + 8,
                   kSFree = kDrain + 16, kPReady = kSFree + 16, kTmemSlot = kPReady + 16, kAbort = kTmemSlot + 4,
                   kProgress = kAbort + 4;  // stages filled, by the loader at every block of K
constexpr uint32_t kMade = kSFull, kTaken = kSFree;  // d = 128

__device__ __forceinline__ void bar_init(uint32_t at, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(at), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t at) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(at) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t at, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(at), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t at, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(at), "r"(parity)
      : "memory");
  return done != 0;
}

// Whether to give up: because another warp did, or because the loader has filled no stage for the time
// above.  How long one wait lasts says nothing: the clearing warp waits while every item that needs no
// clearing goes by, and a second tile's warps while items leave theirs empty.  Every other warp feeds on
// the loader's stages or frees them, so a block in which any of them moves fills the next one soon.
struct Patience {
  uint64_t since;
  uint32_t seen;
};
static __device__ __noinline__ bool tile_give_up(uint32_t bars, Patience *p, int32_t *status) {
  int32_t abort;
  uint32_t progress;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(abort) : "r"(bars + kAbort) : "memory");
  if (abort) return true;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(progress) : "r"(bars + kProgress) : "memory");
  const uint64_t now = globaltimer_ns();
  if (p->since == 0 || progress != p->seen) {
    p->since = now, p->seen = progress;
    return false;
  }
  if (now - p->since < kTileWaitNs) return false;
  asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(bars + kAbort), "r"(1) : "memory");
  report(status, TG_STATUS_TIMEOUT);
  return true;
}
// Wait for a phase of the barrier at bars + at; false when this block gave up.
__device__ __forceinline__ bool lane_wait(uint32_t bars, uint32_t at, uint32_t parity, int32_t *status) {
  if (bar_try(bars + at, parity)) return true;
  Patience p = {0, 0};
  for (uint32_t n = 1; !bar_try(bars + at, parity); ++n)
    if (!(n & (kTilePolls - 1)) && tile_give_up(bars, &p, status)) return false;
  return true;
}
// the last wait of a block that gave up: at most 0.1 s
__device__ __forceinline__ void bar_wait_ns(uint32_t at, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!bar_try(at, parity) && globaltimer_ns() - t0 < 100000000ull) {
  }
}
// for a whole warp: every lane gets the same answer
__device__ __forceinline__ bool tile_wait(uint32_t bars, uint32_t at, uint32_t parity, int32_t *status) {
  return __all_sync(0xffffffffu, lane_wait(bars, at, parity, status));
}

// The items of a thread block; the first comes with their count, the next one's line is fetched
// ahead into L1.
struct ItemList {
  const tg_tile_item *at;
  tg_tile_item cur;
  int left;
  bool first;
  __device__ __forceinline__ void fetch(const tg_tile_item *p) {
    const int4 *s = reinterpret_cast<const int4 *>(p);
    int4 *d = reinterpret_cast<int4 *>(&cur);
    d[0] = __ldg(s), d[1] = __ldg(s + 1), d[2] = __ldg(s + 2);
  }
  __device__ __forceinline__ void start(const TileArgs &a) {
    fetch(a.lead + blockIdx.x);
    left = cur.reserved[0];
    at = a.items + cur.reserved[1] + 1;
    first = true;
  }
  __device__ __forceinline__ bool advance() {
    if (left <= 0) return false;
    if (!first) fetch(at++);
    first = false;
    if (--left > 0) asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
    return true;
  }
};

// a position in a cycle of N barriers, and its phase
template <uint32_t N>
struct Cycle {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) at = 0, phase ^= 1;
  }
  __device__ __forceinline__ void skip(uint32_t n) {
    const uint32_t s = at + n;
    phase ^= (s / N) & 1;
    at = s % N;
  }
};

// the key blocks that the tiles of an item need, one by one and together (empty: b >= e)
struct ItemRange {
  tgi::TileRange tile[2];
  int b, e;
};
template <int D, bool PAGED>
__device__ __forceinline__ ItemRange item_range(const tg_tile_item &it, const TileArgs &a) {
  ItemRange r;
  r.tile[0] = tgi::tile_range(it, 0, a.tq, a.window, !PAGED);
  r.tile[1] = {0, 0};
  if (D == 128) r.tile[1] = tgi::tile_range(it, 1, a.tq, a.window, !PAGED);
  const bool has0 = r.tile[0].b < r.tile[0].e, has1 = r.tile[1].b < r.tile[1].e;
  r.b = !has1 ? r.tile[0].b : !has0 ? r.tile[1].b : min(r.tile[0].b, r.tile[1].b);
  r.e = !has1 ? r.tile[0].e : !has0 ? r.tile[1].e : max(r.tile[0].e, r.tile[1].e);
  return r;
}

// ------------------------------------------------------------------ softmax and output warps
__device__ __forceinline__ void store_v8(uint16_t *to, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// d = 128: a warp has 32 rows of its tile.  d = 256, one tile: two warps share 32 rows, each with 40
// of a block's 80 keys and half of the output's columns; a row's reference is common to both, its
// sum l is joined at the end, and a warp that gave up waiting goes on without waiting, so that its
// partner finds it at their barrier.  (Two warps at d = 128 as well would be sixteen: what a block costs a
// warp beside its keys then weighs more than the keys, 1.71 against 1.38 ms for 16384 tokens; at
// d = 256, 0.34 against 0.36 ms for 8192.)
template <int D>
constexpr int halves() {
  return D == 128 ? 1 : 2;
}
template <int D, bool PAGED>
__device__ __forceinline__ void softmax_role(const TileArgs &a, uint32_t bars, int tile, int half) {
  constexpr int HALVES = halves<D>(), ROWS = D == 128 ? 256 : 128, N = kKeys / HALVES, COLS = D / HALVES;
  const int r = threadIdx.x & 127;             // row of the tile = lane of tensor memory
  const int pair = 1 + (r >> 5);               // named barrier of two warps that share rows
  const int tok = r / a.g, head = r - tok * a.g;
  const uint32_t lanes = (uint32_t)(r & ~31) << 16;
  const uint32_t o_base = kOut + (D == 128 ? tile * 128 : 0) + half * COLS + lanes;
  const uint32_t swap = kSwap + lanes;
  const float sl2 = a.scale_log2;
  bool alive = true;
  auto wait = [&](uint32_t at, uint32_t parity) -> bool {
    bool ok = true;
    if (HALVES == 1) ok = tile_wait(bars, at, parity, a.status);
    if (HALVES == 2 && alive) alive = tile_wait(bars, at, parity, a.status);
    tc_fence_after();
    return ok;
  };
  // Both warps' values of a row, through tensor memory: two pairs of columns in turn, so that a
  // value is overwritten only behind the barrier after the one ahead of its reading.
  uint32_t turn = 0;
  auto exchange = [&](float v) -> float {
    const uint32_t column = turn;
    turn ^= 2;
    tmem_st1(swap + column + half, v);
    tmem_wait_st();
    tc_fence_before();
    pair_sync(pair);
    tc_fence_after();
    const float other = tmem_ld1(swap + column + 1 - half);
    tmem_wait_ld();
    return other;
  };
  uint32_t count = 0;  // d = 128: steps done; d = 256: blocks done
  // block n uses buffer slot_of(n), at d = 256 in the phase_of(n) of its barriers
  auto slot_of = [&](uint32_t n) -> uint32_t { return D == 128 ? (uint32_t)tile : n & 1; };
  auto phase_of = [&](uint32_t n) -> uint32_t { return (n >> 1) & 1; };
  ItemList list;
  list.start(a);
  while (list.advance()) {
    const tg_tile_item &it = list.cur;
    const tgi::TileRange rg = tgi::tile_range(it, tile, a.tq, a.window, !PAGED);
    const int first = tile * a.tq;
    const int n = min(it.nrow - first, a.tq);
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
    const bool some = rg.b < rg.e;
    float s[N];
    auto read_s = [&](uint32_t slot) {
      const uint32_t at = slot * kKeys + half * N + lanes;
      uint32_t *sr = reinterpret_cast<uint32_t *>(s);
      tmem_ld32(at, sr);
      if (HALVES == 1) tmem_ld32(at + 32, sr + 32), tmem_ld16(at + 64, sr + 64);
      if (HALVES == 2) tmem_ld8(at + 32, sr + 32);
    };
    // what this warp read and wrote in tensor memory is done
    auto arrive = [&](uint32_t at) {
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) bar_arrive(bars + at);
    };
    if (HALVES == 1 && some) {  // step 0: the first S
      if (!wait(kMade + 8 * tile, count++ & 1)) return;
      read_s(tile);
      tmem_wait_ld();
      if (rg.e - rg.b > 1) arrive(kTaken + 8 * tile);
    }
    for (int j = rg.b; j < rg.e; ++j, ++count) {
      const uint32_t slot = slot_of(count);
      if (HALVES == 2) {
        wait(kSFull + 8 * slot, phase_of(count));
        read_s(slot);
        tmem_wait_ld();
        arrive(kSFree + 8 * slot);
      }
      const int k0 = j * kKeys;
      if (k0 + kKeys > hi_first || k0 < lo_last) {
        const int h1 = hi - k0 - half * N, l1 = lo - k0 - half * N;
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = (c < h1 && c >= l1) ? s[c] : -INFINITY;
      }
      // A row's reference is the maximum of the first block in which it sees a key.  Later blocks are
      // weighted by it as it stands; only where a half block's weights sum to more than kMost is the
      // block's maximum taken and the block done again.
      auto find_max = [&]() -> float {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < N; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[c + k]), s[c + 4 + k]);
        const float v = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        return HALVES == 1 ? v : fmaxf(v, exchange(v));
      };
      if (__any_sync(0xffffffffu, m == -INFINITY)) {  // the same rows, so the same answer, in both warps
        const float mx = find_max();
        if (m == -INFINITY) m = mx;
      }
      float part;
      uint32_t p[N / 2];
#pragma unroll 1
      for (bool again = false;; again = true) {
        const float neg = m == -INFINITY ? 0.f : -m * sl2;
        float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          float2 x = fma2(make_float2(s[2 * k], s[2 * k + 1]), make_float2(sl2, sl2), make_float2(neg, neg));
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          sum[k & 1] = add2(sum[k & 1], x);
          p[k] = pack_bf16x2(x.x, x.y);
        }
        part = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (again || !(HALVES == 1 ? __any_sync(0xffffffffu, part > kMost) : pair_any(pair, part > kMost))) break;
        const float m_new = fmaxf(m, find_max());
        const float f = m_new == -INFINITY ? 1.f : ex2((m - m_new) * sl2);
        m = m_new;
        l *= f;
        if (j > rg.b) {  // scale O, once the block before has been added to it
          if (HALVES == 1 && !wait(kMade + 8 * tile, count & 1)) return;
          if (HALVES == 2) wait(kPvDone + 8 * slot_of(count - 1), phase_of(count - 1));
#pragma unroll 1
          for (int c = 0; c < COLS / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_base + c * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(o_base + c * 32, o);
          }
        }
      }
      l += part;
      const uint32_t p_addr = kWeights + slot * (kKeys / 2) + half * (N / 2) + lanes;
      if (HALVES == 1) {
        // the step after: S of the next block is there, P of the block before has been multiplied
        if (rg.e - rg.b == 1)
          --count;  // there is none: P goes with the step before
        else if (!wait(kMade + 8 * tile, count & 1))
          return;
        if (j + 1 < rg.e) read_s(tile);
        tmem_st32(p_addr, p), tmem_st8(p_addr + 32, p + 32);
        tmem_wait_ld();
        tmem_wait_st();
        arrive(kTaken + 8 * tile);
      } else {
        // P of this buffer's block before has been multiplied
        if (count >= 2) wait(kPvDone + 8 * slot, phase_of(count - 2));
        tmem_st16(p_addr, p), tmem_st4(p_addr + 16, p + 16);
        tmem_wait_st();
        arrive(kPReady + 8 * slot);
      }
    }
    if (HALVES == 1 && some) {  // the step that adds the last block; the next item's first Q K^T may follow
      if (!wait(kMade + 8 * tile, count++ & 1)) return;
      arrive(kTaken + 8 * tile);
    }
    if (n <= 0) continue;

    // output: this row's O / l, or the piece's (m, l, O); half of the columns each
    const bool mine = tok < n && r < a.tq * a.g;
    const int64_t row = ((int64_t)(it.row0 + first + tok)) * a.H_q + it.h * a.g + head;
    if (HALVES == 2 && some) {
      l += exchange(l);
      wait(kPvDone + 8 * slot_of(count - 1), phase_of(count - 1));
    }
    const float mo = m == -INFINITY ? -INFINITY : m * sl2;  // base-2 reference
    if (it.slot >= 0) {
      // [D / 4][ROWS][4]: a warp stores 512 contiguous bytes at a time
      const int at = tile * 128 + r;
      if (mine && half == 0) {
        *reinterpret_cast<float2 *>(a.ws_ml + ((int64_t)it.slot * 256 + at) * 2) = make_float2(mo, l);
        // kept for the merge, whose blocks may write lse over own_lse
        if (PAGED && a.own_lse) a.ws_own[(int64_t)it.slot * 256 + at] = a.own_lse[row];
      }
      float *dst = a.ws_o + (int64_t)it.slot * 32768 + half * COLS * ROWS + at * 4;
#pragma unroll 1
      for (int c = 0; c < COLS / 32; ++c) {
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
            *reinterpret_cast<uint4 *>(dst + (c * 8 + k) * (ROWS * 4)) =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
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
      // own_lse may be lse itself: both warps read it before one writes
      if (HALVES == 2 && PAGED && a.own_lse) pair_sync(pair);
      if (mine && half == 0 && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (top + log2f(total)) * kTileLn2;
      // A prompt's rows: two lanes exchange 16 of 32 columns, so that a store touches 16 lines of 128 bytes,
      // not 32 (16 prompts of 64 to 4096 tokens, the same inputs again at 2070 MHz: 178 -> 172 us).  A
      // decode batch's rows go out as they are.
      const int odd = threadIdx.x & 1;
      int even_row = -1, odd_row = -1;  // of the two lanes, from the tile's first
      uint16_t *to = nullptr;
      if (!PAGED) {
        const int here = mine ? tok * a.H_q + head : -1, there = __shfl_xor_sync(0xffffffffu, here, 1);
        even_row = odd ? there : here, odd_row = odd ? here : there;
        to = a.out + ((int64_t)(it.row0 + first) * a.H_q + it.h * a.g) * D + half * COLS + odd * 16;
      }
#pragma unroll 1
      for (int c = 0; c < COLS / 32; ++c) {
        uint32_t o[32];
        if (some) {
          tmem_ld32(o_base + c * 32, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (!PAGED) {  // paired
          uint32_t w[2][8];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[k >> 3][k & 7] = pack_bf16x2(__uint_as_float(o[2 * k]) * f1, __uint_as_float(o[2 * k + 1]) * f1);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[0][e] : w[1][e], 1);
            if (odd) w[0][e] = got;
            else w[1][e] = got;
          }
          if (even_row >= 0) store_v8(to + (int64_t)even_row * D + c * 32, w[0]);
          if (odd_row >= 0) store_v8(to + (int64_t)odd_row * D + c * 32, w[1]);
        } else if (mine) {
          const int64_t at = row * D + half * COLS + c * 32;
          uint16_t *dst = a.out + at;
          const uint4 *src = f2 != 0.f ? reinterpret_cast<const uint4 *>(a.own_out + at) : nullptr;
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // 16 columns: a whole 32-byte sector of a lane's row
            uint32_t w[8];
            if (src) {
              const uint4 x = src[2 * k], y = src[2 * k + 1];
              w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float v0 = __uint_as_float(o[16 * k + 2 * e]) * f1, v1 = __uint_as_float(o[16 * k + 2 * e + 1]) * f1;
              if (src) v0 += f2 * __uint_as_float(w[e] << 16), v1 += f2 * __uint_as_float(w[e] & 0xffff0000u);
              w[e] = pack_bf16x2(v0, v1);
            }
            store_v8(dst + 16 * k, w);
          }
        }
      }
    }
    tc_fence_before();  // the next item's first P V overwrites O after this warp's next arrival
  }
}

// ------------------------------------------------------------------ MMA lanes
// Rows of V that no row of the item sees lie in its first block, ahead of the window, and in its
// last, behind the run's end: those blocks' rows [from, to) are kept, the others cleared.
template <bool PAGED>
__device__ __forceinline__ tgi::TileRange kept_rows(const tg_tile_item &it, const ItemRange &rg, int j, const TileArgs &a) {
  const int first = !PAGED && a.window > 0 ? it.pos0 - a.window + 1 : 0;
  tgi::TileRange k = {0, kKeys};
  if (j == rg.b) k.b = max(0, first - j * kKeys);
  if (j + 1 == rg.e) k.e = min(kKeys, it.kv_len - j * kKeys);
  return k;
}
__device__ __forceinline__ bool cleared(const tgi::TileRange &k) { return k.b > 0 || k.e < kKeys; }

// S = Q K^T over one 128-column piece
__device__ __forceinline__ void issue_qk(uint32_t s, uint32_t q, uint32_t k, bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, kKeys, false);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mma_ss(s, smem_desc(q + (i >> 2) * 16384 + (i & 3) * 32, 16, 1024),
           smem_desc(k + (i >> 2) * kHalfBytes + (i & 3) * 32, 16, 1024), idesc, accumulate || i > 0);
}
// O += P V over one stage of 80 keys x 128 columns
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint32_t v, bool accumulate) {
  constexpr uint32_t idesc = mma_desc(128, 128, true);
#pragma unroll
  for (int i = 0; i < kKeys / 16; ++i)
    mma_ts(o, p + i * 8, smem_desc(v + i * 2048, kHalfBytes, 1024), idesc, accumulate || i > 0);
}

// d = 128: a tile with blocks [b, e) has the steps b .. e + 1, Q K^T of block j in step j and P V in
// step j + 2; a lane takes part in every step, with its products or by arriving for nothing.  Of
// a single block the step without either is left out.
__device__ __forceinline__ bool in_steps(const tgi::TileRange &r, int j) {
  return r.b < r.e && j >= r.b && j < r.e + 2 && !(r.e - r.b == 1 && j == r.e);
}
// the softmax has taken what the step before made (n: steps of the tile so far)
__device__ __forceinline__ bool next_step(uint32_t bars, int tile, uint32_t n, int32_t *status) {
  if (n > 0 && !lane_wait(bars, kTaken + 8 * tile, (n - 1) & 1, status)) return false;
  tc_fence_after();
  return true;
}

// Two lanes issue: one the Q K^T, the other the P V.  The tensor pipe takes a few MMAs ahead only,
// about 200 clocks of work; a lane alone left it empty while it waited for the next barrier
// (2390 clocks a block of both tiles against 1800 with two, 1456 of MMAs).
template <int D, bool PAGED>
__device__ __forceinline__ void qk_items(const TileArgs &a, uint32_t bars, uint32_t q_at, uint32_t ring_at) {
  constexpr int NP = D / 128;
  Cycle<kStages> ring;
  uint32_t q_phase = 0, count[2] = {0, 0};
  ItemList list;
  list.start(a);
  while (list.advance()) {
    const tg_tile_item &it = list.cur;
    const ItemRange rg = item_range<D, PAGED>(it, a);
    if (rg.b >= rg.e) continue;
    if (!lane_wait(bars, kQFull, q_phase, a.status)) return;
    q_phase ^= 1;
    // ring order: K(b), K(b+1), V(b), K(b+2), V(b+1), ...
    for (int j = rg.b; j < rg.e; ++j) {
      Cycle<kStages> ks[NP];
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        ks[c] = ring;
        ring.next();
        if (!lane_wait(bars, kFull + 8 * ks[c].at, ks[c].phase, a.status)) return;
      }
      if (D == 128) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!in_steps(rg.tile[i], j)) continue;
          if (!next_step(bars, i, count[i]++, a.status)) return;
          if (j < rg.tile[i].e) {
            issue_qk(i * kKeys, q_at + i * kQPiece, ring_at + ks[0].at * kStageBytes, false);
            mma_commit(bars + kMade + 8 * i);
          } else {
            bar_arrive(bars + kMade + 8 * i);
          }
        }
      } else {
        const uint32_t slot = count[0] & 1, uses = count[0] >> 1;
        if (uses > 0 && !lane_wait(bars, kSFree + 8 * slot, (uses - 1) & 1, a.status)) return;
        tc_fence_after();
        ++count[0];
#pragma unroll
        for (int c = 0; c < NP; ++c) issue_qk(slot * kKeys, q_at + c * kQPiece, ring_at + ks[c].at * kStageBytes, c > 0);
        mma_commit(bars + kSFull + 8 * slot);
      }
#pragma unroll
      for (int c = 0; c < NP; ++c) mma_commit(bars + kEmpty + 8 * ks[c].at);
      if (j > rg.b) ring.skip(NP);  // V(j-1)
    }
    mma_commit(bars + kQEmpty);
    ring.skip(NP);  // V(e-1)
    if (D == 128) {  // the two steps that only P V takes part in
      for (int j = rg.e; j < rg.e + 2; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!in_steps(rg.tile[i], j)) continue;
          if (!next_step(bars, i, count[i]++, a.status)) return;
          bar_arrive(bars + kMade + 8 * i);
        }
      }
    }
  }
}

template <int D, bool PAGED>
__device__ __forceinline__ void pv_items(const TileArgs &a, uint32_t bars, uint32_t ring_at) {
  constexpr int NP = D / 128;
  Cycle<kStages> ring;
  uint32_t c_phase = 0, count[2] = {0, 0};
  ItemList list;
  list.start(a);
  while (list.advance()) {
    const tg_tile_item &it = list.cur;
    const ItemRange rg = item_range<D, PAGED>(it, a);
    if (rg.b >= rg.e) continue;
    ring.skip(NP);  // K(b)
    const bool clear_first = cleared(kept_rows<PAGED>(it, rg, rg.b, a));
    const bool clear_last = cleared(kept_rows<PAGED>(it, rg, rg.e - 1, a));
    if (D == 128) {  // the two steps ahead of a tile's first P V
      for (int j = rg.b; j < rg.b + 2; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!in_steps(rg.tile[i], j)) continue;
          if (!next_step(bars, i, count[i]++, a.status)) return;
          bar_arrive(bars + kMade + 8 * i);
        }
      }
    }
    for (int j = rg.b; j < rg.e; ++j) {
      if (j + 1 < rg.e) ring.skip(NP);  // K(j+1)
      Cycle<kStages> vs[NP];
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        vs[c] = ring;
        ring.next();
        if (!lane_wait(bars, kFull + 8 * vs[c].at, vs[c].phase, a.status)) return;
      }
      if ((j == rg.b && clear_first) || (j + 1 == rg.e && clear_last)) {
        bar_arrive(bars + kToClear);
        if (!lane_wait(bars, kCleared, c_phase, a.status)) return;
        c_phase ^= 1;
      }
      if (D == 128) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!in_steps(rg.tile[i], j + 2)) continue;
          if (!next_step(bars, i, count[i]++, a.status)) return;
          if (j >= rg.tile[i].b) {
            issue_pv(kOut + i * 128, kWeights + i * (kKeys / 2), ring_at + vs[0].at * kStageBytes, j > rg.tile[i].b);
            mma_commit(bars + kMade + 8 * i);
          } else {
            bar_arrive(bars + kMade + 8 * i);
          }
        }
      } else {
        const uint32_t slot = count[0] & 1, uses = count[0] >> 1;
        if (!lane_wait(bars, kPReady + 8 * slot, uses & 1, a.status)) return;
        tc_fence_after();
        ++count[0];
#pragma unroll
        for (int c = 0; c < NP; ++c)
          issue_pv(kOut + c * 128, kWeights + slot * (kKeys / 2), ring_at + vs[c].at * kStageBytes, j > rg.b);
        mma_commit(bars + kPvDone + 8 * slot);
      }
#pragma unroll
      for (int c = 0; c < NP; ++c) mma_commit(bars + kEmpty + 8 * vs[c].at);
    }
  }
}

// ------------------------------------------------------------------ clearing warp
// Zeroes the rows of an item's first and last V block that none of its rows sees: P is 0 there, and
// must meet 0 whatever memory holds.  It finds the blocks' stages by counting the ring; the P V lane
// tells it that they have landed and waits for it.
template <int D, bool PAGED>
__device__ __forceinline__ void clear_rows(const TileArgs &a, uint32_t bars, uint32_t ring_at) {
  constexpr int NP = D / 128;
  const int lane = threadIdx.x & 31;
  uint32_t phase = 0;
  Cycle<kStages> ring;
  ItemList list;
  list.start(a);
  while (list.advance()) {
    const ItemRange rg = item_range<D, PAGED>(list.cur, a);
    if (rg.b >= rg.e) continue;
    const int n = rg.e - rg.b;
    for (int i = 0; i < n; i = max(i + 1, n - 1)) {  // the first and the last block
      const tgi::TileRange keep = kept_rows<PAGED>(list.cur, rg, rg.b + i, a);
      if (!cleared(keep)) continue;
      if (!tile_wait(bars, kToClear, phase, a.status)) return;
      phase ^= 1;
      Cycle<kStages> at = ring;
      at.skip((i + 1 == n ? 2 * n - 1 : 2) * NP);  // ring order: K(b), K(b+1), V(b), ..., V(e-1)
      for (int c = 0; c < NP; ++c) {
        for (int k = lane; k < kKeys * 8; k += 32) {
          if ((k >> 3) >= keep.b && (k >> 3) < keep.e) continue;
          const uint32_t to = ring_at + at.at * kStageBytes + (uint32_t)k * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + kHalfBytes), "r"(0) : "memory");
        }
        at.next();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(bars + kCleared);
    }
    ring.skip(2 * n * NP);
  }
}

// ------------------------------------------------------------------ loader warp
// The lanes look up the pages of a block's boxes of 16 rows, one block ahead; an elected lane
// issues the copies.
template <int D, bool PAGED>
__device__ __forceinline__ void load_items(const CUtensorMap *qm, const CUtensorMap *km, const CUtensorMap *vm,
                                           const TileArgs &a, uint32_t bars, uint32_t q_at, uint32_t ring_at) {
  constexpr int NP = D / 128, BOXES = kKeys / 16;
  const int lane = threadIdx.x & 31;
  Cycle<kStages> ring;
  uint32_t filled = 0, q_count = 0;  // stages filled, Q loads
  bool ok = true;
  const uint32_t q_box = (uint32_t)a.tq * a.g * 128;  // bytes of one 64-column box of Q
  const int outside = PAGED ? (int)(a.pool_pages * a.H_p * 2) : 0;  // a block past the pool: reads as zeros
  ItemList list;
  list.start(a);
  while (ok && list.advance()) {
    const tg_tile_item &it = list.cur;
    const ItemRange rg = item_range<D, PAGED>(it, a);
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
      const int t = j * kKeys + lane * 16;
      const int pg = t / a.P;
      *row = t - pg * a.P;
      if (lane >= BOXES || t >= it.kv_len || j >= j1) return outside;
      const int32_t id = pg < lists ? __ldg(a.pt_ids + off0 + pg) : -1;
      if (id < 0 || id >= a.pool_pages) {
        report(a.status, TG_STATUS_BAD_PAGE);
        return outside;
      }
      return (id * a.H_p + it.hpos) * 2;
    };
    auto progress = [&] {
      asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(bars + kProgress), "r"(filled + 1) : "memory");
    };
    // one block of K (kv 0) or V (kv 1) into the ring
    auto fill = [&](int j, int kv, int z, int row) -> bool {
#pragma unroll
      for (int c = 0; c < NP; ++c) {
        if (filled >= kStages && !tile_wait(bars, kEmpty + 8 * (ring.at), ring.phase ^ 1, a.status)) return false;
        const uint32_t dst = ring_at + ring.at * kStageBytes;
        const uint32_t full = bars + kFull + 8 * ring.at;
        if (PAGED) {
          int zs[BOXES], rows[BOXES];
#pragma unroll
          for (int i = 0; i < BOXES; ++i) {
            const int zi = __shfl_sync(0xffffffffu, z, i);
            zs[i] = zi == outside ? zi : zi + kv;
            rows[i] = __shfl_sync(0xffffffffu, row, i);
          }
          if (elect_one()) {
            if (!kv) progress();
            bar_expect(full, kStageBytes);
#pragma unroll
            for (int i = 0; i < BOXES; ++i) {
              tma_load_3d(dst + i * 2048, km, full, c * 128, rows[i], zs[i]);
              tma_load_3d(dst + i * 2048 + kHalfBytes, km, full, c * 128 + 64, rows[i], zs[i]);
            }
          }
        } else if (elect_one()) {
          const CUtensorMap *m = kv ? vm : km;
          const int context = it.src * a.H + it.h;
          if (!kv) progress();
          bar_expect(full, kStageBytes);
          tma_load_3d(dst, m, full, c * 128, j * kKeys, context);
          tma_load_3d(dst + kHalfBytes, m, full, c * 128 + 64, j * kKeys, context);
        }
        __syncwarp();
        ++filled;
        ring.next();
      }
      return true;
    };
    int z = 0, row = 0, z_next = 0, row_next = 0, z_before = 0, row_before = 0;
    if (PAGED) z = place(j0, &row);
    if (q_count > 0 && !tile_wait(bars, kQEmpty, (q_count - 1) & 1, a.status)) {
      ok = false;
      break;
    }
    ++q_count;
    if (elect_one()) {
      if (D == 128) {
        const bool has0 = rg.tile[0].b < rg.tile[0].e, has1 = rg.tile[1].b < rg.tile[1].e;
        bar_expect(bars + kQFull, ((has0 ? 2 : 0) + (has1 ? 2 : 0)) * q_box);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((c >> 1) ? has1 : has0)
            tma_load_3d(q_at + c * 16384, qm, bars + kQFull, (c & 1) * 64, it.h * a.g, it.row0 + (c >> 1) * a.tq);
      } else {
        bar_expect(bars + kQFull, 4 * q_box);
#pragma unroll
        for (int c = 0; c < 4; ++c) tma_load_3d(q_at + c * 16384, qm, bars + kQFull, c * 64, it.h * a.g, it.row0);
      }
    }
    __syncwarp();
    for (int j = j0; ok && j <= j1; ++j) {
      if (PAGED) z_next = place(j + 1, &row_next);
      if (j < j1) ok = fill(j, 0, z, row);
      if (ok && j > j0) ok = fill(j - 1, 1, z_before, row_before);
      z_before = z, row_before = row;
      z = z_next, row = row_next;
    }
  }
  // leave nothing in flight: every stage used and Q must have been consumed, or, after a
  // give-up, at least have landed
  for (uint32_t i = 0; ok && i < kStages && i < filled; ++i)
    ok = tile_wait(bars, kEmpty + 8 * (i), ((filled - 1 - i) / kStages) & 1, a.status);
  if (ok && q_count) ok = tile_wait(bars, kQEmpty, (q_count - 1) & 1, a.status);
  if (!ok) {
    for (uint32_t i = 0; i < kStages && i < filled; ++i)
      bar_wait_ns(bars + kFull + 8 * i, ((filled - 1 - i) / kStages) & 1);
    if (q_count) bar_wait_ns(bars + kQFull, (q_count - 1) & 1);
    __syncwarp();
  }
}

// twelve warps, 168 registers each at launch; at d = 128 they move to the eight softmax warps
// (384 x 168 = 256 x 208 + 128 x 88).  What does not fit is spilled: 12 bytes stored and 92 loaded in the
// prompts' form, 16 and 260 in the pages'; at d = 256 nothing.
constexpr int kTileThreads = 384;

template <int D, bool PAGED>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_attn_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                     const __grid_constant__ CUtensorMap vm, const TileArgs a) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int SW = 8;  // softmax warps
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_at = smem_addr(base), ring_at = q_at + kQBytes, bars = ring_at + kStages * kStageBytes;
  const int warp = threadIdx.x >> 5;
  if (warp == SW) tmem_alloc(reinterpret_cast<uint32_t *>(base + kQBytes + kStages * kStageBytes + kTmemSlot), 512);
  if (warp == SW + 2 && elect_one()) prefetch_tensormap(&qm), prefetch_tensormap(&km), prefetch_tensormap(&vm);
  if (threadIdx.x == 0) {
    for (uint32_t at = 0; at < kTmemSlot; at += 8) bar_init(bars + at, at >= kSFree ? SW * D / 256 : D == 128 && at >= kMade && at < kMade + 16 ? 2 : 1);
    asm volatile("st.volatile.shared.s32 [%0], %1;" ::"r"(bars + kAbort), "r"(0) : "memory");
    asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(bars + kProgress), "r"(0) : "memory");
    fence_barrier_init();
  }
  // rows behind the last whole group of heads get no query: zeros, once
  const int spare = 128 - a.tq * a.g;
  for (int i = threadIdx.x; i < 4 * spare * 8; i += kTileThreads) {
    const int box = i / (spare * 8), k = i - box * spare * 8;
    *reinterpret_cast<uint4 *>(base + box * 16384 + (128 - spare) * 128 + k * 16) = make_uint4(0, 0, 0, 0);
  }
  if (spare) fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Launched as the programmatic dependent of the kernel before it: what came so far overlapped that
  // kernel's end; everything from here may read what it wrote.
  griddep_wait();
  // the merge may be set up from now on; its blocks find room when this kernel's leave
  if (a.signal) griddep_launch_dependents();
  // all 512 columns are this block's, so they start at column 0: the MMAs and the softmax
  // address them by constants
  if (D == 128 && warp < SW) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  if (D == 128 && warp >= SW) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  if (warp < SW) {
    softmax_role<D, PAGED>(a, bars, D == 128 ? warp >> 2 : 0, D == 128 ? 0 : warp >> 2);
  } else if (warp <= SW + 1) {
    if (elect_one()) {
      if (warp == SW) qk_items<D, PAGED>(a, bars, q_at, ring_at);
      else pv_items<D, PAGED>(a, bars, ring_at);
      // What was issued must finish before tensor memory is freed and the block's shared memory goes to
      // another.  The softmax waits for the last P V and the loader for every stage, but neither does
      // where the block gave up, perhaps after this lane had issued its last.
      mma_commit(bars + kDrain + 8 * (warp - SW));
      bar_wait_ns(bars + kDrain + 8 * (warp - SW), 0);
    }
    __syncwarp();
  } else if (warp == SW + 2) {
    load_items<D, PAGED>(&qm, &km, &vm, a, bars, q_at, ring_at);
  } else {
    clear_rows<D, PAGED>(a, bars, ring_at);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == SW) tmem_free(0, 512);
}

// ------------------------------------------------------------------ merge of cut runs
struct MergeArgs {
  const tg_tile_merge *merges;
  const float *ws_ml, *ws_own, *ws_o;
  uint16_t *out;
  float *lse;
  const uint16_t *own_out;  // NULL: nothing to merge with
  int H_q, g, tq;
};

constexpr int kMergeThreads = 128;
// blocks of one merge: 16 rows x 16 columns each
constexpr int merge_blocks(int d) { return (32768 / d / 16) * (d / 16); }

// out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p over the pieces (and the request's own result).
// A warp has 4 columns of 16 rows, its halves the even and the odd pieces: a piece's loads are 256
// contiguous bytes.  What counts is latency: ten pieces' (m, l) and O are loaded together and
// joined to what came before by their own maximum, so that a run of up to twenty pieces, the
// usual cut over an idle device, waits for memory once.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tile_merge_kernel(const MergeArgs a) {
  constexpr int ROWS = 32768 / D, COLS = D / 16, AT_ONCE = 10;
  // the plan is there: the kernel before let this one start after it had waited for its own
  const tg_tile_merge mg = a.merges[blockIdx.x / merge_blocks(D)];
  const int chunk = blockIdx.x % merge_blocks(D);
  const int lane = threadIdx.x & 31, odd = lane >> 4;
  const int at = (chunk / COLS) * 16 + (lane & 15);                   // row of the slot
  const int c4 = (chunk % COLS) * 4 + (threadIdx.x >> 5);             // which 4 columns
  const int tile = at >> 7, r = at & 127, tok = r / a.g, head = r - tok * a.g;
  const int n = min(mg.nrow - tile * a.tq, a.tq);
  const bool mine = tok < n && r < a.tq * a.g;
  if (!__any_sync(0xffffffffu, mine)) return;
  const int64_t row = (int64_t)(mg.row0 + tile * a.tq + tok) * a.H_q + mg.h * a.g + head;
  griddep_wait();
  const float2 *ml = reinterpret_cast<const float2 *>(a.ws_ml) + (int64_t)mg.slot0 * 256 + at;
  const float4 *po = reinterpret_cast<const float4 *>(a.ws_o) + (int64_t)mg.slot0 * 8192 + c4 * ROWS + at;
  float M = -INFINITY, total = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine && !odd && a.own_out) {
    const float w = __ldcg(a.ws_own + (int64_t)mg.slot0 * 256 + at) * kTileLog2e;
    const uint2 own = *reinterpret_cast<const uint2 *>(a.own_out + row * D + c4 * 4);
    if (w != -INFINITY) {
      M = w, total = 1.f;
      o = make_float4(__uint_as_float(own.x << 16), __uint_as_float(own.x & 0xffff0000u),
                      __uint_as_float(own.y << 16), __uint_as_float(own.y & 0xffff0000u));
    }
  }
  // a state (M, total, o) scaled to another maximum
  auto scale_to = [&](float top) {
    const float f = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    total *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
  };
  for (int p0 = odd; p0 < mg.nparts; p0 += 2 * AT_ONCE) {
    float2 v[AT_ONCE];
    float4 x[AT_ONCE];
#pragma unroll
    for (int p = 0; p < AT_ONCE; ++p) {
      const int k = p0 + 2 * p;
      v[p] = make_float2(-INFINITY, 0.f);
      if (mine && k < mg.nparts) {
        v[p] = __ldcg(ml + k * 256);
        x[p] = __ldcg(po + (int64_t)k * 8192);
      }
    }
    float top = M;
#pragma unroll
    for (int p = 0; p < AT_ONCE; ++p) top = fmaxf(top, v[p].x);
    scale_to(top);
#pragma unroll
    for (int p = 0; p < AT_ONCE; ++p) {
      if (v[p].x == -INFINITY) continue;
      const float f = ex2(v[p].x - top);
      total += f * v[p].y, o.x += f * x[p].x, o.y += f * x[p].y, o.z += f * x[p].z, o.w += f * x[p].w;
    }
  }
  // the even pieces' state and the odd ones', in that order in both halves
  scale_to(fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16)));
  total += __shfl_xor_sync(0xffffffffu, total, 16);
  o.x += __shfl_xor_sync(0xffffffffu, o.x, 16), o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
  o.z += __shfl_xor_sync(0xffffffffu, o.z, 16), o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
  if (!mine || odd) return;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  *reinterpret_cast<uint2 *>(a.out + row * D + c4 * 4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (c4 == 0 && a.lse) a.lse[row] = total == 0.f ? -INFINITY : (M + log2f(total)) * kTileLn2;
}

}  // namespace tgk
