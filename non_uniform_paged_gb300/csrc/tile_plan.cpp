// Tile plans: the static work lists of tg_prefill_attn and tg_prefix_attn.
//
// The same idea as the decode plan ([Tangram] "Tangram: Unlocking Non-Uniform KV Cache
// Compression for Efficient Multi-turn LLM Serving", paper-review page, 3.3: the split of
// the work over the thread blocks is fixed ahead of the calls): here the unit is a tile of
// query rows against a range of 80-key blocks, because many rows share each key.
//
// Items are sorted by cost and given, longest first, to the block with the least work.  Where
// that leaves blocks idle -- an item is longer than an even share, or each block gets so few
// items that they do not divide evenly -- runs of keys are cut: all of them, or only those of
// the items that are left over when every block has had the same number; a few lengths of
// piece are tried, and the one whose longest block is shortest under the cost model is kept.
#include "tile_common.h"

#include "tg_internal.h"

#include <algorithm>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <vector>

namespace {

using tgi::fail;

// Cost model in units of one 80-key block of an item (about 0.85 us): an item's start and end, a
// piece's partial, and the second kernel of a plan that has any, alone and for each full piece it
// reads.
constexpr double kItemCost = 3.0, kPieceCost = 1.0, kMergeCost = 2.5, kMergePiece = 0.025;

double item_cost(const tg_tile_item &it, bool piece) {
  return (it.blk1 - it.blk0) + kItemCost + (piece ? kPieceCost : 0.0);
}

int64_t pieces_of(int nblk, int cut) { return nblk <= cut ? 1 : (nblk + cut - 1) / cut; }

// how runs are cut: of the items behind the first `whole`, to at most `length` blocks
struct Cut {
  int length = INT32_MAX;
  size_t whole = 0;
  int64_t pieces(const std::vector<tg_tile_item> &sorted, size_t k) const {
    return k < whole ? 1 : pieces_of(sorted[k].blk1 - sorted[k].blk0, length);
  }
};

// longest block's work
double makespan(const std::vector<tg_tile_item> &sorted, const Cut &cut, int n_cta, int full_rows) {
  std::vector<double> cost;
  double pieces = 0;  // in full ones
  for (size_t k = 0; k < sorted.size(); ++k) {
    const int n = sorted[k].blk1 - sorted[k].blk0;
    const int64_t p = cut.pieces(sorted, k);
    if (p > 1) pieces += (double)p * sorted[k].nrow / full_rows;
    for (int64_t i = 0; i < p; ++i)
      cost.push_back((double)((i + 1) * n / p - i * n / p) + kItemCost + (p > 1 ? kPieceCost : 0.0));
  }
  if (pieces > 0) std::sort(cost.begin(), cost.end(), std::greater<double>());
  std::priority_queue<double, std::vector<double>, std::greater<double>> load;
  for (size_t c = 0; c < cost.size() && c < (size_t)n_cta; ++c) load.push(0.0);
  double worst = 0;
  for (double c : cost) {
    const double l = load.top() + c;
    load.pop();
    load.push(l);
    worst = std::max(worst, l);
  }
  return worst + (pieces > 0 ? kMergeCost + kMergePiece * pieces : 0.0);
}

Cut choose_cut(const std::vector<tg_tile_item> &sorted, int n_cta, int full_rows) {
  Cut best;
  double total = 0;
  for (const tg_tile_item &it : sorted) total += item_cost(it, false);
  const double share = total / n_cta;
  double least = makespan(sorted, best, n_cta, full_rows);
  const int most = sorted[0].blk1 - sorted[0].blk0;
  if (most <= 1 || least <= 1.03 * share) return best;
  auto attempt = [&](int length, size_t whole) {
    if (length < 1 || whole >= sorted.size() || length >= sorted[whole].blk1 - sorted[whole].blk0) return;
    Cut c;
    c.length = length, c.whole = whole;
    const double m = makespan(sorted, c, n_cta, full_rows);
    if (m < least - 1e-9) least = m, best = c;
  };
  // every run to a fraction of the even share
  for (double f : {0.25, 0.34, 0.42, 0.5, 0.6, 0.7, 0.85, 1.0, 1.25, 1.6, 2.0, 3.0}) attempt((int)std::min(1e9, std::max(1.0, f * share)), 0);
  // the shortest pieces that still start all at once, one per block
  if ((int64_t)sorted.size() <= n_cta) {
    int lo = 1, hi = most;
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      int64_t n = 0;
      for (const tg_tile_item &it : sorted) n += pieces_of(it.blk1 - it.blk0, mid);
      if (n <= n_cta) hi = mid; else lo = mid + 1;
    }
    attempt(lo, 0);
  }
  // only the items left over when every block has had as many
  const size_t whole = sorted.size() / n_cta * n_cta;
  if (whole > 0 && whole < sorted.size()) {
    const int n = sorted[whole].blk1 - sorted[whole].blk0;
    for (int k = 2; k <= 16; ++k) attempt((n + k - 1) / k, whole);
  }
  return best;
}

// cut, order and serialise; hd carries the sizes
int finish(const char *fn, tg_tile_header hd, std::vector<tg_tile_item> &base, void *plan, int64_t plan_cap,
           int64_t *plan_bytes, int64_t *workspace_bytes) {
  auto longer = [](const tg_tile_item &a, const tg_tile_item &b) { return a.blk1 - a.blk0 > b.blk1 - b.blk0; };
  std::stable_sort(base.begin(), base.end(), longer);
  const int full_rows = tgi::tile_tokens(hd.H_q / hd.H) * tgi::tiles_per_item(hd.d);
  const Cut cut = base.empty() ? Cut() : choose_cut(base, hd.N_CTA, full_rows);
  std::vector<tg_tile_item> items;
  std::vector<tg_tile_merge> merges;
  int64_t slots = 0;
  for (size_t at = 0; at < base.size(); ++at) {
    const tg_tile_item &it = base[at];
    const int n = it.blk1 - it.blk0;
    const int64_t p = cut.pieces(base, at);
    if (p == 1) {
      items.push_back(it);
      continue;
    }
    tg_tile_merge m = {it.row0, it.nrow, it.h, (int32_t)slots, (int32_t)p, {0, 0, 0}};
    merges.push_back(m);
    for (int64_t k = 0; k < p; ++k) {
      tg_tile_item piece = it;
      piece.blk0 = it.blk0 + (int32_t)(k * n / p);
      piece.blk1 = it.blk0 + (int32_t)((k + 1) * n / p);
      piece.slot = (int32_t)slots++;
      items.push_back(piece);
    }
  }
  // (the merge's grid is 128 blocks a merge)
  if (items.size() > INT32_MAX || slots > INT32_MAX || merges.size() > (1u << 23))
    return fail(TG_ERR_SHAPE, "%s: too many work items", fn);
  std::stable_sort(items.begin(), items.end(), longer);
  const int n_cta = (int)std::max<int64_t>(1, std::min<int64_t>(hd.N_CTA, (int64_t)items.size()));
  using Load = std::pair<double, int>;
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> load;
  for (int c = 0; c < n_cta; ++c) load.push({0.0, c});
  std::vector<std::vector<int32_t>> of(n_cta);
  for (size_t k = 0; k < items.size(); ++k) {
    Load l = load.top();
    load.pop();
    of[l.second].push_back((int32_t)k);
    l.first += item_cost(items[k], items[k].slot >= 0);
    load.push(l);
  }

  hd.N_CTA = n_cta;
  hd.n_items = (int32_t)items.size();
  hd.n_merge = (int32_t)merges.size();
  hd.n_slots = (int32_t)slots;
  hd.lead = tgi::align_up(sizeof(tg_tile_header), 16);
  hd.items = hd.lead + (int64_t)n_cta * sizeof(tg_tile_item);
  hd.merges = hd.items + (int64_t)items.size() * sizeof(tg_tile_item);
  hd.plan_bytes = hd.merges + (int64_t)merges.size() * sizeof(tg_tile_merge);
  hd.block = tgi::kTileKeys;
  hd.workspace_bytes = slots * (tgi::kSlotMl + tgi::kSlotO);
  if (plan_bytes) *plan_bytes = hd.plan_bytes;
  if (workspace_bytes) *workspace_bytes = hd.workspace_bytes;
  if (!plan) return tgi::ok();
  if (plan_cap < hd.plan_bytes)
    return fail(TG_ERR_CAPACITY, "%s: plan_cap=%lld < %lld", fn, (long long)plan_cap, (long long)hd.plan_bytes);
  uint8_t *out = static_cast<uint8_t *>(plan);
  std::memset(out, 0, (size_t)hd.plan_bytes);
  std::memcpy(out, &hd, sizeof hd);
  tg_tile_item *lead = reinterpret_cast<tg_tile_item *>(out + hd.lead);
  tg_tile_item *list = reinterpret_cast<tg_tile_item *>(out + hd.items);
  int32_t at = 0;
  for (int c = 0; c < n_cta; ++c) {
    if (!of[c].empty()) lead[c] = items[of[c][0]];
    lead[c].reserved[0] = (int32_t)of[c].size();
    lead[c].reserved[1] = at;
    for (int32_t k : of[c]) list[at++] = items[k];
  }
  if (!merges.empty()) std::memcpy(out + hd.merges, merges.data(), merges.size() * sizeof(tg_tile_merge));
  return tgi::ok();
}

int check_heads(const char *fn, int H, int H_q, int d, int N_CTA) {
  if (H <= 0 || H_q <= 0 || N_CTA <= 0) return fail(TG_ERR_INVALID_ARG, "%s: sizes must be positive", fn);
  if (N_CTA > 65536) return fail(TG_ERR_INVALID_ARG, "%s: N_CTA=%d (1..65536; one per SM)", fn, N_CTA);
  if (H_q % H) return fail(TG_ERR_SHAPE, "%s: H_q=%d %% H=%d is not 0", fn, H_q, H);
  if (H_q / H > 8) return fail(TG_ERR_SHAPE, "%s: g=%d > 8 query heads per KV head", fn, H_q / H);
  if (d != 128 && d != 256) return fail(TG_ERR_SHAPE, "%s: d=%d (128 or 256)", fn, d);
  return TG_OK;
}

int plan_prefill(int batch, int H, int H_q, int d, int N_CTA, const int32_t *q_len, const int32_t *kv_len, int window,
                 void *plan, int64_t plan_cap, int64_t *plan_bytes, int64_t *workspace_bytes) {
  const char *fn = "tg_plan_prefill";
  if (int rc = check_heads(fn, H, H_q, d, N_CTA)) return rc;
  if (batch <= 0 || window < 0) return fail(TG_ERR_INVALID_ARG, "%s: batch=%d, window=%d", fn, batch, window);
  if (!q_len || !kv_len) return fail(TG_ERR_INVALID_ARG, "%s: NULL q_len/kv_len", fn);
  const int tq = tgi::tile_tokens(H_q / H), step = tq * tgi::tiles_per_item(d);
  int64_t rows = 0, count = 0;
  int32_t max_kv = 0;
  for (int b = 0; b < batch; ++b) {
    if (q_len[b] < 0 || kv_len[b] < 0)
      return fail(TG_ERR_INVALID_ARG, "%s: request %d has q_len=%d, kv_len=%d", fn, b, q_len[b], kv_len[b]);
    if (q_len[b] > (1 << 30) || kv_len[b] > (1 << 30))
      return fail(TG_ERR_SHAPE, "%s: request %d is longer than 2^30 tokens", fn, b);
    rows += q_len[b];
    count += (int64_t)((q_len[b] + step - 1) / step) * H;
    max_kv = std::max(max_kv, kv_len[b]);
  }
  if (rows > INT32_MAX || count > (1 << 24))
    return fail(TG_ERR_SHAPE, "%s: %lld query tokens, %lld work items", fn, (long long)rows, (long long)count);
  if (window >= max_kv) window = 0;  // reaches back to every first key (and differences stay in int32)
  std::vector<tg_tile_item> base;
  base.reserve((size_t)count);
  int64_t row0 = 0;
  for (int b = 0; b < batch; ++b) {
    // the request's last tiles are its longest; the heads of a tile go to different blocks
    for (int t = (q_len[b] + step - 1) / step - 1; t >= 0; --t)
      for (int h = 0; h < H; ++h) {
        tg_tile_item it;
        std::memset(&it, 0, sizeof it);
        it.row0 = (int32_t)(row0 + (int64_t)t * step);
        it.nrow = std::min(step, q_len[b] - t * step);
        it.h = h;
        it.src = b;
        it.pos0 = kv_len[b] - q_len[b] + t * step;
        it.kv_len = kv_len[b];
        it.slot = -1;
        it.blk1 = (kv_len[b] + tgi::kTileKeys - 1) / tgi::kTileKeys;
        int lo = INT32_MAX, hi = 0;
        for (int i = 0; i < tgi::tiles_per_item(d); ++i) {
          const tgi::TileRange r = tgi::tile_range(it, i, tq, window, true);
          if (r.b < r.e) lo = std::min(lo, r.b), hi = std::max(hi, r.e);
        }
        it.blk0 = hi ? lo : 0;
        it.blk1 = hi;
        base.push_back(it);
      }
    row0 += q_len[b];
  }
  tg_tile_header hd;
  std::memset(&hd, 0, sizeof hd);
  hd.magic = TG_TILE_MAGIC;
  hd.version = TG_TILE_VERSION;
  hd.kind = tgi::kPrefillPlan;
  hd.batch = hd.groups = batch;
  hd.rows = (int32_t)rows;
  hd.H = H, hd.H_q = H_q, hd.d = d, hd.window = window, hd.max_kv = max_kv, hd.N_CTA = N_CTA;
  return finish(fn, hd, base, plan, plan_cap, plan_bytes, workspace_bytes);
}

int plan_prefix(int groups, int H, int H_q, int H_p, int P, int d, int N_CTA, const int32_t *req_off,
                const int32_t *head_order, const int32_t *ntok, void *plan, int64_t plan_cap, int64_t *plan_bytes,
                int64_t *workspace_bytes) {
  const char *fn = "tg_plan_prefix";
  if (int rc = check_heads(fn, H, H_q, d, N_CTA)) return rc;
  if (groups <= 0 || H_p <= 0 || P <= 0) return fail(TG_ERR_INVALID_ARG, "%s: sizes must be positive", fn);
  if (H % H_p) return fail(TG_ERR_SHAPE, "%s: H=%d %% H_p=%d is not 0", fn, H, H_p);
  if (P % 16) return fail(TG_ERR_SHAPE, "%s: P=%d must be a multiple of 16", fn, P);
  if (!req_off || !head_order || !ntok) return fail(TG_ERR_INVALID_ARG, "%s: NULL req_off/head_order/ntok", fn);
  const int tq = tgi::tile_tokens(H_q / H), step = tq * tgi::tiles_per_item(d);
  if (req_off[0] != 0) return fail(TG_ERR_INVALID_ARG, "%s: req_off[0]=%d", fn, req_off[0]);
  int64_t count = 0;
  for (int r = 0; r < groups; ++r) {
    if (req_off[r + 1] < req_off[r]) return fail(TG_ERR_INVALID_ARG, "%s: req_off is not ascending at %d", fn, r + 1);
    count += ((int64_t)(req_off[r + 1] - req_off[r]) + step - 1) / step * H;
  }
  if (count > (1 << 24)) return fail(TG_ERR_SHAPE, "%s: %lld work items", fn, (long long)count);
  if (req_off[groups] > (1 << 30) || (int64_t)groups * (H / H_p) >= INT32_MAX)
    return fail(TG_ERR_SHAPE, "%s: %d requests, %d groups of %d page lists", fn, req_off[groups], groups, H / H_p);
  std::vector<int32_t> place(H, -1);
  for (int i = 0; i < H; ++i) {
    const int32_t h = head_order[i];
    if (h < 0 || h >= H || place[h] >= 0) return fail(TG_ERR_INVALID_ARG, "%s: head_order is not a permutation", fn);
    place[h] = i;
  }
  int32_t max_kv = 0;
  std::vector<tg_tile_item> base;
  base.reserve((size_t)count);
  for (int r = 0; r < groups; ++r)
    for (int t = 0; t < (req_off[r + 1] - req_off[r] + step - 1) / step; ++t)
      for (int h = 0; h < H; ++h) {
        const int32_t n = ntok[(size_t)r * H + h];
        if (n < 0) return fail(TG_ERR_INVALID_ARG, "%s: ntok[%d][%d]=%d", fn, r, h, n);
        if (n > (1 << 30)) return fail(TG_ERR_SHAPE, "%s: ntok[%d][%d] is over 2^30 tokens", fn, r, h);
        tg_tile_item it;
        std::memset(&it, 0, sizeof it);
        it.row0 = req_off[r] + t * step;
        it.nrow = std::min(step, req_off[r + 1] - it.row0);
        it.h = h;
        it.src = r * (H / H_p) + place[h] / H_p;
        it.hpos = place[h] % H_p;
        it.kv_len = n;
        it.blk1 = (n + tgi::kTileKeys - 1) / tgi::kTileKeys;
        it.slot = -1;
        max_kv = std::max(max_kv, n);
        base.push_back(it);
      }
  tg_tile_header hd;
  std::memset(&hd, 0, sizeof hd);
  hd.magic = TG_TILE_MAGIC;
  hd.version = TG_TILE_VERSION;
  hd.kind = tgi::kPrefixPlan;
  hd.batch = hd.rows = req_off[groups];
  hd.groups = groups;
  hd.H = H, hd.H_q = H_q, hd.H_p = H_p, hd.P = P, hd.d = d, hd.max_kv = max_kv, hd.N_CTA = N_CTA;
  return finish(fn, hd, base, plan, plan_cap, plan_bytes, workspace_bytes);
}

}  // namespace

extern "C" int tg_plan_prefill(int batch, int H, int H_q, int d, int N_CTA, const int32_t *q_len,
                               const int32_t *kv_len, int window, void *plan, int64_t plan_cap, int64_t *plan_bytes,
                               int64_t *workspace_bytes) {
  try {
    return plan_prefill(batch, H, H_q, d, N_CTA, q_len, kv_len, window, plan, plan_cap, plan_bytes, workspace_bytes);
  } catch (const std::bad_alloc &) {
    return fail(TG_ERR_CAPACITY, "tg_plan_prefill: out of host memory");
  }
}

extern "C" int tg_plan_prefix(int groups, int H, int H_q, int H_p, int P, int d, int N_CTA, const int32_t *req_off,
                              const int32_t *head_order, const int32_t *ntok, void *plan, int64_t plan_cap,
                              int64_t *plan_bytes, int64_t *workspace_bytes) {
  try {
    return plan_prefix(groups, H, H_q, H_p, P, d, N_CTA, req_off, head_order, ntok, plan, plan_cap, plan_bytes,
                       workspace_bytes);
  } catch (const std::bad_alloc &) {
    return fail(TG_ERR_CAPACITY, "tg_plan_prefix: out of host memory");
  }
}
