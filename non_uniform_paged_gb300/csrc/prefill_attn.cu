// Causal attention of a packed prefill pass over its contexts (tg_prefill_attn).
//
// [Tangram] "Tangram: Unlocking Non-Uniform KV Cache Compression for Efficient Multi-turn LLM
// Serving" (paper-review page), 3.1: compression runs inside (chunked) prefill, after a
// chunk's keys and values exist; this is the attention of that chunk, over the same
// [batch][H][Nmax][d] rows that tg_compact_topk retains from.  The kernel is tile_attn.cuh.
#include "tile_launch.cuh"

using namespace tgk;

extern "C" int tg_prefill_attn(tg_stream_t stream, const void *plan_host, const void *plan_dev, const uint16_t *q,
                               const uint16_t *K, const uint16_t *V, int Nmax, float scale, void *workspace,
                               int64_t workspace_bytes, uint16_t *out, float *lse, int32_t *dev_status) {
  const char *fn = "tg_prefill_attn";
  const tg_tile_header *hd;
  int rc = check_tile_call(fn, tgi::kPrefillPlan, plan_host, plan_dev, q, out, lse, scale, workspace, workspace_bytes,
                           &hd);
  if (rc) return rc;
  if (Nmax < hd->max_kv) return tgi::fail(TG_ERR_SHAPE, "%s: Nmax=%d < the plan's longest context %d", fn, Nmax, hd->max_kv);
  if (!hd->n_items) return tgi::ok();  // no query token
  const int64_t lists = (int64_t)hd->batch * hd->H;
  if (lists > INT32_MAX || Nmax < 0) return tgi::fail(TG_ERR_SHAPE, "%s: batch * H or Nmax leaves int32", fn);
  if (hd->max_kv > 0 && (!K || !V)) return tgi::fail(TG_ERR_INVALID_ARG, "%s: NULL K or V", fn);
  if (misaligned(K, 16) || misaligned(V, 16)) return tgi::fail(TG_ERR_INVALID_ARG, "%s: K and V must be 16-byte aligned", fn);
  const TileArgs a = tile_args(hd, plan_dev, scale, workspace, out, lse, dev_status);
  CUtensorMap qm, km, vm;
  rc = ready_tiles<false>(fn, hd->d);
  if (!rc) rc = tile_map(&qm, fn, "q", q, hd->d, hd->H_q, hd->rows, a.g, a.tq);
  if (rc) return rc;
  if (hd->max_kv > 0) {
    rc = tile_map(&km, fn, "K", K, hd->d, Nmax, lists, tgi::kTileKeys, 1);
    if (!rc) rc = tile_map(&vm, fn, "V", V, hd->d, Nmax, lists, tgi::kTileKeys, 1);
    if (rc) return rc;
  } else {
    km = vm = qm;  // no context holds a key: never read
  }
  return hd->d == 128 ? launch_tiles<128, false>(fn, stream, hd, plan_dev, qm, km, vm, a)
                      : launch_tiles<256, false>(fn, stream, hd, plan_dev, qm, km, vm, a);
}
