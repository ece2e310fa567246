// Tile plans shared by their host builder and the kernels that run them (not installed).
#pragma once

#include "../../include/tg.h"

#include <cstdint>

namespace tgi {

constexpr int kTileRows = 128;  // rows of one MMA tile: tokens (or requests) x the g heads of a KV head
// keys of one block: two S of 80 columns, two P of 40 and 4 columns of exchange fit in the 256 of tensor
// memory beside O
constexpr int kTileKeys = 80;
constexpr int kPrefillPlan = 0, kPrefixPlan = 1;

// tiles of one item: two at d = 128, one at d = 256 (their outputs fill tensor memory)
constexpr int tiles_per_item(int d) { return d == 128 ? 2 : 1; }
// tokens (requests) of one tile: whole groups of g rows
constexpr int tile_tokens(int g) { return kTileRows / g; }

struct TileRange {
  int32_t b, e;
};
// key blocks that tile i of an item needs: an empty range has b >= e
#ifdef __CUDACC__
__host__ __device__ __forceinline__
#else
inline
#endif
    TileRange
    tile_range(const tg_tile_item &it, int i, int tq, int window, bool causal) {
  const int first = i * tq;
  const int n = it.nrow - first < tq ? it.nrow - first : tq;
  TileRange r = {it.blk0, it.blk0};
  if (n <= 0) return r;
  r.e = it.blk1;
  if (!causal) return r;
  int hi = it.pos0 + first + n;  // keys below hi are seen by the tile's last row
  if (hi > it.kv_len) hi = it.kv_len;
  const int e = hi <= 0 ? 0 : (hi + kTileKeys - 1) / kTileKeys;
  if (e < r.e) r.e = e;
  if (window > 0) {
    const int lo = it.pos0 + first - window + 1;  // the first row's first key
    if (lo > 0 && lo / kTileKeys > r.b) r.b = lo / kTileKeys;
  }
  return r;
}

// workspace: m, l float32 [slots][256][2] | own lse float32 [slots][256] |
// o float32 [slots][d / 4][32768 / d rows][4]
constexpr int64_t kSlotMl = 256 * 3 * 4;
constexpr int64_t kSlotO = 32768 * 4;

}  // namespace tgi
