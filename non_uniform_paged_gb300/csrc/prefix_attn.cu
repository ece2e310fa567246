// Decode attention of a batch over retained tokens that its requests share (tg_prefix_attn).
//
// [Tangram] "Tangram: Unlocking Non-Uniform KV Cache Compression for Efficient Multi-turn LLM
// Serving" (paper-review page), 3.2 Ragged Paging: the shared tokens lie in group pages of
// H_p x 2 x P x d elements, each head with its own count.  tg_decode_attn would read them once
// per request; here the requests of a group are the rows of one tile, so a key crosses the
// memory bus once for all of them.  The kernel is tile_attn.cuh.
#include "tile_launch.cuh"

using namespace tgk;

extern "C" int tg_prefix_attn(tg_stream_t stream, const void *plan_host, const void *plan_dev, const uint16_t *q,
                              const uint16_t *pool, int64_t pool_pages, const int64_t *pt_off, const int32_t *pt_ids,
                              float scale, const uint16_t *own_out, const float *own_lse, void *workspace,
                              int64_t workspace_bytes, uint16_t *out, float *lse, int32_t *dev_status) {
  const char *fn = "tg_prefix_attn";
  const tg_tile_header *hd;
  int rc = check_tile_call(fn, tgi::kPrefixPlan, plan_host, plan_dev, q, out, lse, scale, workspace, workspace_bytes,
                           &hd);
  if (rc) return rc;
  if (!own_out != !own_lse) return tgi::fail(TG_ERR_INVALID_ARG, "%s: own_out and own_lse go together", fn);
  if (misaligned(own_out, 16) || misaligned(pool, 16))
    return tgi::fail(TG_ERR_INVALID_ARG, "%s: pool and own_out must be 16-byte aligned", fn);
  if (!hd->n_items) return tgi::ok();  // no request
  if (hd->max_kv > 0) {
    if (!pool || !pt_off || !pt_ids) return tgi::fail(TG_ERR_INVALID_ARG, "%s: NULL pool or page table", fn);
    if (pool_pages <= 0 || pool_pages > INT32_MAX / (2 * hd->H_p) - 1)
      return tgi::fail(TG_ERR_CAPACITY, "%s: pool_pages=%lld", fn, (long long)pool_pages);
  }
  TileArgs a = tile_args(hd, plan_dev, scale, workspace, out, lse, dev_status);
  CUtensorMap qm, pm;
  rc = ready_tiles<true>(fn, hd->d);
  if (!rc) rc = tile_map(&qm, fn, "q", q, hd->d, hd->H_q, hd->rows, a.g, a.tq);
  if (rc) return rc;
  a.P = hd->P;
  a.H_p = hd->H_p;
  if (hd->max_kv > 0) {
    rc = tile_map(&pm, fn, "pool", pool, hd->d, hd->P, pool_pages * hd->H_p * 2, 16, 1);
    if (rc) return rc;
  } else {
    pm = qm;  // nothing is shared: never read
  }
  a.pt_off = pt_off;
  a.pt_ids = pt_ids;
  a.pool_pages = pool_pages;
  a.own_out = own_out;
  a.own_lse = own_lse;
  return hd->d == 128 ? launch_tiles<128, true>(fn, stream, hd, plan_dev, qm, pm, pm, a)
                      : launch_tiles<256, true>(fn, stream, hd, plan_dev, qm, pm, pm, a);
}
