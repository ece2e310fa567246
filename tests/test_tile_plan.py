"""Tile plans of tg_prefill_attn and tg_prefix_attn (host only): every needed (tile, key block)
is covered once, pieces and slots add up, and bad arguments are refused."""
import ctypes

import numpy as np
import pytest


def _needed(row0, nrow, pos0, kv_len, tq, tiles, window, causal, block):
    """Key blocks that each 128-row tile of an item needs, by brute force over its rows."""
    out = []
    for i in range(tiles):
        rows = range(i * tq, min(nrow, (i + 1) * tq))
        blocks = set()
        for r in rows:
            hi = min(kv_len, pos0 + r + 1) if causal else kv_len
            lo = max(0, pos0 + r - window + 1) if causal and window else 0
            if hi > lo:
                blocks.update(range(lo // block, (hi - 1) // block + 1))
        out.append(blocks)
    return out


def _check_plan(lib, plan, ws, want, tq, tiles, window, causal):
    """want: {(h, src, row0): (nrow, pos0, kv_len, hpos)}"""
    hd = lib.tile_header(plan)
    lead, items = lib.tile_items(plan)
    assert hd["plan_bytes"] == plan.size and hd["workspace_bytes"] == ws
    assert 1 <= hd["N_CTA"] <= max(1, hd["n_items"]) and items.size == hd["n_items"]
    assert ws == hd["n_slots"] * (256 * 12 + 32768 * 4)
    at = 0
    for c in range(hd["N_CTA"]):
        assert tuple(lead[c]["reserved"]) [1] == at
        at += int(lead[c]["reserved"][0])
    assert at == items.size
    got, slots = {}, []
    for it in items:
        key = (int(it["h"]), int(it["src"]), int(it["row0"]))
        got.setdefault(key, []).append(it)
        if it["slot"] >= 0:
            slots.append(int(it["slot"]))
    assert sorted(slots) == list(range(hd["n_slots"]))
    assert set(got) == set(want)
    for key, (nrow, pos0, kv_len, hpos) in want.items():
        parts = sorted(got[key], key=lambda it: int(it["blk0"]))
        assert all((int(p["nrow"]), int(p["kv_len"]), int(p["hpos"])) == (nrow, kv_len, hpos) for p in parts)
        if causal:
            assert all(int(p["pos0"]) == pos0 for p in parts)
        need = _needed(key[2], nrow, pos0, kv_len, tq, tiles, window, causal, hd["block"])
        every = set().union(*need)
        covered = [b for p in parts for b in range(int(p["blk0"]), int(p["blk1"]))]
        assert len(covered) == len(set(covered)) and every <= set(covered)
        if every:
            assert min(covered) == min(every) and max(covered) == max(every)
        else:
            assert not covered
        if len(parts) > 1:
            s = [int(p["slot"]) for p in parts]
            assert s == list(range(s[0], s[0] + len(s)))
        else:
            assert int(parts[0]["slot"]) == -1
    assert hd["n_merge"] == sum(len(p) > 1 for p in got.values())
    return hd


@pytest.mark.parametrize("seed", range(12))
def test_prefill_plan_covers_every_block_once(lib, seed):
    r = np.random.default_rng(seed)
    batch, H, g = int(r.integers(1, 7)), int(r.integers(1, 4)), int(r.integers(1, 9))
    d, window = int(r.choice([128, 256])), int(r.choice([0, 0, 1, 100, 700]))
    q_len = r.integers(0, 700, batch) * (r.random(batch) < 0.8)
    kv_len = np.maximum(0, q_len + r.choice([-50, 0, 0, 300, 5000], batch))
    n_cta = int(r.choice([1, 7, 152, 1000]))
    plan, ws = lib.tg_plan_prefill(q_len, kv_len, H, H * g, d, n_cta, window)
    tq, tiles = 128 // g, 2 if d == 128 else 1
    want, row = {}, 0
    for b in range(batch):
        for t in range(0, int(q_len[b]), tq * tiles):
            for h in range(H):
                want[(h, b, row + t)] = (min(tq * tiles, int(q_len[b]) - t), int(kv_len[b] - q_len[b]) + t, int(kv_len[b]), 0)
        row += int(q_len[b])
    hd = _check_plan(lib, plan, ws, want, tq, tiles, window, True)
    assert (hd["rows"], hd["batch"], hd["max_kv"]) == (row, batch, kv_len.max())


@pytest.mark.parametrize("seed", range(8))
def test_prefix_plan_covers_every_block_once(lib, seed):
    r = np.random.default_rng(100 + seed)
    groups, H_p, G, g = int(r.integers(1, 4)), int(r.choice([1, 2, 4])), int(r.integers(1, 4)), int(r.integers(1, 9))
    H, d = H_p * G, int(r.choice([128, 256]))
    off = np.concatenate([[0], np.cumsum(r.integers(0, 90, groups))])
    ntok = r.integers(0, 9000, (groups, H)) * (r.random((groups, H)) < 0.9)
    order = r.permutation(H)
    plan, ws = lib.tg_plan_prefix(off, order, ntok, H * g, H_p, 16, d, int(r.choice([1, 20, 152])))
    tq, tiles = 128 // g, 2 if d == 128 else 1
    want = {}
    place = np.argsort(order)
    for q in range(groups):
        for t in range(int(off[q]), int(off[q + 1]), tq * tiles):
            for h in range(H):
                want[(h, q * G + int(place[h]) // H_p, t)] = (min(tq * tiles, int(off[q + 1]) - t), 0, int(ntok[q, h]),
                                                              int(place[h]) % H_p)
    _check_plan(lib, plan, ws, want, tq, tiles, 0, False)


def test_one_long_run_is_cut_over_the_blocks(lib):
    """One request, one KV head, 100000 keys: the run is cut so that no block holds much more than
    its share; many equal tiles are not cut."""
    plan, ws = lib.tg_plan_prefill([1], [100000], 1, 8, 128, 152)
    hd = lib.tile_header(plan)
    _, items = lib.tile_items(plan)
    assert hd["n_merge"] == 1 and 100 <= hd["n_items"] <= 152 and ws > 0
    assert (items["blk1"] - items["blk0"]).max() <= 2 * (100000 // hd["block"]) // 152 + 1
    plan, ws = lib.tg_plan_prefill([16384], [16384], 8, 32, 128, 152)
    assert lib.tile_header(plan)["n_merge"] == 0 and ws == 0


def test_left_over_items_are_cut(lib):
    """512 equal items on 152 blocks: three each, and the 56 left over are cut over all blocks."""
    plan, ws = lib.tg_plan_prefill([4096], [100000], 8, 32, 128, 152)
    hd = lib.tile_header(plan)
    lead, items = lib.tile_items(plan)
    load = [sum(int(it["blk1"] - it["blk0"]) for it in items[int(l["reserved"][1]):][:int(l["reserved"][0])]) for l in lead]
    assert 0 < hd["n_merge"] <= 64 and ws > 0
    assert max(load) <= 1.05 * sum(load) / len(load)


def test_windows_that_reach_past_every_context_are_none(lib):
    """A window of at least the longest context hides nothing, up to the largest int32."""
    ref, _ = lib.tg_plan_prefill([300, 40], [300, 20], 2, 4, 128, 152)
    for window in (300, 301, 2**31 - 1):
        plan, _ = lib.tg_plan_prefill([300, 40], [300, 20], 2, 4, 128, 152, window)
        assert plan.tobytes() == ref.tobytes()
    plan, _ = lib.tg_plan_prefill([300, 40], [300, 20], 2, 4, 128, 152, 299)
    assert lib.tile_header(plan)["window"] == 299


def test_more_blocks_than_items(lib):
    plan, _ = lib.tg_plan_prefill([5], [5], 1, 1, 128, 65536)
    assert lib.tile_header(plan)["N_CTA"] == 1


def test_longest_first_keeps_the_blocks_even(lib):
    plan, _ = lib.tg_plan_prefill([4096, 300, 17, 2000], [4096, 300, 17, 2000], 8, 32, 128, 152)
    lead, items = lib.tile_items(plan)
    load = [sum(int(it["blk1"] - it["blk0"]) for it in items[int(l["reserved"][1]):][:int(l["reserved"][0])]) for l in lead]
    assert max(load) <= 1.25 * (sum(load) / len(load)) + 2


def test_plan_refusals(lib):
    def code(call):
        with pytest.raises(lib.TGError) as e:
            call()
        return e.value.code

    assert code(lambda: lib.tg_plan_prefill([], [], 1, 1, 128, 1)) == lib.ERR_INVALID_ARG
    assert code(lambda: lib.tg_plan_prefill([-1], [4], 1, 1, 128, 1)) == lib.ERR_INVALID_ARG
    assert code(lambda: lib.tg_plan_prefill([1], [-4], 1, 1, 128, 1)) == lib.ERR_INVALID_ARG
    assert code(lambda: lib.tg_plan_prefill([1], [4], 1, 1, 128, 0)) == lib.ERR_INVALID_ARG
    assert code(lambda: lib.tg_plan_prefill([1], [4], 1, 1, 128, 65537)) == lib.ERR_INVALID_ARG
    assert code(lambda: lib.tg_plan_prefill([1], [4], 1, 1, 128, 1, -1)) == lib.ERR_INVALID_ARG
    assert code(lambda: lib.tg_plan_prefill([1], [4], 1, 1, 64, 1)) == lib.ERR_SHAPE
    assert code(lambda: lib.tg_plan_prefill([1], [4], 2, 3, 128, 1)) == lib.ERR_SHAPE
    assert code(lambda: lib.tg_plan_prefill([1], [4], 1, 9, 128, 1)) == lib.ERR_SHAPE
    assert code(lambda: lib.tg_plan_prefill([2**30 + 1], [4], 1, 1, 128, 1)) == lib.ERR_SHAPE
    assert code(lambda: lib.tg_plan_prefill([2**30] * 2, [4] * 2, 1, 1, 128, 1)) == lib.ERR_SHAPE
    ok = dict(req_off=[0, 2], head_order=[0, 1], ntok=[[5, 6]], H_q=4, H_p=2, P=16, d=128, N_CTA=4)

    def bad(**kw):
        return code(lambda: lib.tg_plan_prefix(**dict(ok, **kw)))

    lib.tg_plan_prefix(**ok)
    assert bad(req_off=[1, 2]) == lib.ERR_INVALID_ARG
    assert bad(req_off=[0, -1]) == lib.ERR_INVALID_ARG
    assert bad(head_order=[0, 0]) == lib.ERR_INVALID_ARG
    assert bad(head_order=[0, 2]) == lib.ERR_INVALID_ARG
    assert bad(ntok=[[5, -1]]) == lib.ERR_INVALID_ARG
    assert bad(P=24) == lib.ERR_SHAPE
    assert bad(H_p=3) == lib.ERR_SHAPE
    assert bad(H_q=5) == lib.ERR_SHAPE
    assert bad(d=64) == lib.ERR_SHAPE
    with pytest.raises(ValueError):
        lib.tg_plan_prefix([0, 1, 2], [0], [[5]], 1, 1, 16, 128, 1)
    # a buffer one byte short
    so, n, w = lib.load(), ctypes.c_int64(0), ctypes.c_int64(0)
    one = np.ones(1, np.int32)
    args = (1, 1, 1, 128, 1, one.ctypes.data, one.ctypes.data, 0)
    assert so.tg_plan_prefill(*args, None, 0, ctypes.addressof(n), ctypes.addressof(w)) == 0
    buf = np.zeros(n.value, np.uint8)
    assert so.tg_plan_prefill(*args, buf.ctypes.data, n.value - 1, ctypes.addressof(n), ctypes.addressof(w)) == lib.ERR_CAPACITY
    assert so.tg_plan_prefill(1, 1, 1, 128, 1, None, one.ctypes.data, 0, None, 0, None, None) == lib.ERR_INVALID_ARG


def test_struct_sizes(lib):
    assert lib.TILE_ITEM_DTYPE.itemsize == 48 and lib._TILE_HEADER_DTYPE.itemsize == 112


def test_calls_refuse_on_the_host(lib):
    """Arguments the C entries refuse before any launch; the fake pointers are never read."""
    so = lib.load()
    fake, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4098)
    plan, _ = lib.tg_plan_prefill([4], [4], 1, 2, 128, 1)
    cut, ws = lib.tg_plan_prefill([1], [100000], 1, 8, 128, 152)
    pre, _ = lib.tg_plan_prefix([0, 2], [0], [[40]], 2, 1, 16, 128, 1)

    def prefill(p=plan, dev=fake, q=fake, K=fake, V=fake, Nmax=4, scale=1.0, w=None, wb=0, out=fake, lse=None):
        return so.tg_prefill_attn(None, p.ctypes.data if p is not None else None, dev, q, K, V, Nmax, scale, w, wb, out,
                                  lse, None)

    assert prefill(p=None) == lib.ERR_INVALID_ARG
    assert prefill(dev=None) == lib.ERR_INVALID_ARG
    assert prefill(p=pre) == lib.ERR_INVALID_ARG
    assert prefill(p=np.zeros(200, np.uint8)) == lib.ERR_INVALID_ARG
    assert prefill(q=None) == lib.ERR_INVALID_ARG
    assert prefill(K=None) == lib.ERR_INVALID_ARG
    assert prefill(out=None) == lib.ERR_INVALID_ARG
    assert prefill(q=odd) == lib.ERR_INVALID_ARG
    assert prefill(V=odd) == lib.ERR_INVALID_ARG
    assert prefill(Nmax=3) == lib.ERR_SHAPE
    assert prefill(scale=float("nan")) == lib.ERR_NONFINITE
    assert prefill(scale=0.0) == lib.ERR_INVALID_ARG
    assert prefill(scale=-1.0) == lib.ERR_INVALID_ARG
    assert prefill(p=cut, Nmax=100000) == lib.ERR_INVALID_ARG
    assert prefill(p=cut, Nmax=100000, w=fake, wb=ws - 1) == lib.ERR_CAPACITY
    assert prefill(p=cut, Nmax=100000, w=odd, wb=ws) == lib.ERR_INVALID_ARG

    def prefix(p=pre, q=fake, pool=fake, pages=3, off=fake, ids=fake, scale=1.0, oo=None, ol=None, out=fake):
        return so.tg_prefix_attn(None, p.ctypes.data, fake, q, pool, pages, off, ids, scale, oo, ol, None, 0, out, None, None)

    assert prefix(p=plan) == lib.ERR_INVALID_ARG
    assert prefix(oo=fake) == lib.ERR_INVALID_ARG
    assert prefix(ol=fake) == lib.ERR_INVALID_ARG
    assert prefix(oo=odd, ol=fake) == lib.ERR_INVALID_ARG
    assert prefix(scale=float("inf")) == lib.ERR_NONFINITE

    def rope(batch=1, T=3, H_q=2, H=1, d=128, Nmax=8, rot=128, max_pos=8, flags=0, cu=fake, start=fake, qkv=fake,
             stride=512, qw=None, kw=None, eps=1e-6, tab=fake, q=fake, K=fake, V=fake):
        return so.tg_qk_norm_rope(None, batch, T, H_q, H, d, Nmax, rot, max_pos, flags, cu, start, qkv, stride, qw, kw, eps,
                                  None, tab, q, K, V, None)

    assert rope(T=0) == 0
    assert rope(batch=0) == lib.ERR_INVALID_ARG
    assert rope(T=-1) == lib.ERR_INVALID_ARG
    assert rope(d=64, rot=64) == lib.ERR_SHAPE
    assert rope(rot=24) == lib.ERR_SHAPE
    assert rope(rot=144) == lib.ERR_SHAPE
    assert rope(flags=2) == lib.ERR_INVALID_ARG
    assert rope(stride=511) == lib.ERR_SHAPE
    assert rope(stride=504) == lib.ERR_SHAPE
    assert rope(eps=-1.0) == lib.ERR_INVALID_ARG
    assert rope(eps=float("nan")) == lib.ERR_NONFINITE
    assert rope(tab=None) == lib.ERR_INVALID_ARG
    assert rope(max_pos=0) == lib.ERR_INVALID_ARG
    assert rope(K=None) == lib.ERR_INVALID_ARG
    assert rope(qkv=odd) == lib.ERR_INVALID_ARG
    assert rope(qw=odd) == lib.ERR_INVALID_ARG


def test_prefix_sizes_past_32_bits_are_refused(lib):
    """As many requests as int32 holds, and more page lists: refused, not planned without work."""
    one = np.zeros(1, np.int32)
    for batch in (2**31 - 1, 2**30 + 1):
        with pytest.raises(lib.TGError) as e:
            lib.tg_plan_prefix([0, batch], one, one[None], 1, 1, 16, 128, 152)
        assert e.value.code == -2
    lib.tg_plan_prefix([0, 70000], one, one[None], 1, 1, 16, 128, 152)
