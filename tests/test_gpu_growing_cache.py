"""GrowingCache as it is used: retention, steps that append and attend, and a turn over what was generated."""
import math

import numpy as np
import pytest
import torch

import synth
from pages4_helpers import attend64, hold, rows_of
from prompt_helpers import merge64, rope64

pytestmark = pytest.mark.gpu


def _table(max_pos, rot, cuda):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=cuda) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=cuda)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _cache(w, cuda, pages, reserve, allocator=None):
    from non_uniform_paged_gb300.ragged import GrowingCache
    N = synth.contexts(w)
    return GrowingCache(w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, synth.budgets_hat(w), N, reserve, pages=pages,
                        cluster=w.cluster, n_cta=24, device=cuda, allocator=allocator), N


def _retained(cache, layer, K, V, kept):
    """What the pages hold of each head's retained rows, in token order."""
    rows = {}
    for b in range(cache.batch):
        for h in range(cache.H):
            n = int(cache.pages["ntok"][layer, b, h])
            at = kept[b, h, :n].long()
            rows[b, h] = [hold(x[b, h, at].double())[0] if cache.four else x[b, h, at].double() for x in (K, V)]
    return rows


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
@pytest.mark.parametrize("d,H,H_q,H_p,cluster", [(128, 4, 8, 2, True), (256, 2, 4, 1, False)])
def test_retention_then_steps_that_see_their_own_tokens(lib, cuda, pages, d, H, H_q, H_p, cluster):
    w = synth.small(d=d, H=H, H_q=H_q, H_p=H_p, cluster=cluster, L=2, batch=3, N=400)
    alloc = None
    if pages == "bf16":  # scattered pages out of an allocator
        alloc = lib.PageAllocator(2000)
        hold_pages = [alloc.admit([7 + i]) for i in range(9)]
        for i in (1, 4, 7):
            alloc.release(hold_pages[i])
    cache, N = _cache(w, cuda, pages, 12, alloc)
    g, table = H_q // H, _table(1000, d, cuda)
    weight = torch.rand(d, device=cuda) + 0.5
    origin = torch.from_numpy(np.asarray(N, np.int32)).to(cuda)
    seen = []
    for layer in range(w.L):
        s = synth.scores(w, layer, cuda)
        K, V = synth.keys_values(w, layer, cuda)
        kept = torch.full((w.batch, H, w.N), -1, dtype=torch.int32, device=cuda)
        cache.compact_layer(layer, s, K, V, kept_idx=kept)
        seen.append(_retained(cache, layer, K, V, kept))
    for step in range(5):
        for layer in range(w.L):
            gen = torch.Generator(device=cuda).manual_seed(100 * step + layer)
            qkv = torch.randn((w.batch, H_q + 2 * H, d), generator=gen, device=cuda).to(torch.bfloat16)
            q = torch.empty((w.batch, H_q, d), dtype=torch.bfloat16, device=cuda)
            out, lse = torch.empty_like(q), torch.empty((w.batch, H_q), device=cuda)
            cache.append_layer(layer, qkv, table, q, origin=origin, q_weight=weight, k_weight=weight)
            cache.decode_layer(layer, q, out, lse)
            torch.cuda.synchronize()
            assert lib.tg_check_status(cache.status) == 0
            cs = table[(origin + step).long()]
            ref, tol = rope64(qkv, cs, H_q, H, weight, weight, 1e-6, False, d)
            assert bool(((q.double() - ref[:, :H_q]).abs() <= tol[:, :H_q]).all())
            for b in range(w.batch):
                for h in range(H):
                    k, v = ref[b, H_q + h], ref[b, H_q + H + h]
                    if cache.four:
                        k, v = hold(k)[0], hold(v)[0]
                    else:  # the key as it is in the page, within the rounding that the append test checks
                        p = int(np.where(cache.pages["order"][layer] == h)[0][0])
                        lst = (layer * w.batch + b) * cache.G + p // H_p
                        ids = cache.pages["pt_ids"][cache.pages["pt_off"][lst]:cache.pages["pt_off"][lst + 1]]
                        n = int(cache.pages["ntok"][layer, b, h]) + step + 1
                        k = rows_of(cache.pool.view(-1, H_p, 2, w.P, d), torch.from_numpy(ids).to(cuda), H_p, w.P, d, p % H_p, n, False)[-1]
                        assert bool(((k - ref[b, H_q + h]).abs() <= tol[b, H_q + h]).all())
                    rows = seen[layer][b, h]
                    rows[0], rows[1] = torch.cat([rows[0], k[None]]), torch.cat([rows[1], v[None]])
                    at = slice(h * g, (h + 1) * g)
                    o, le, t, lt = attend64(q[b, at], rows[0], rows[1], cache.scale, cache.four)
                    assert bool(((out[b, at].double() - o).abs() <= t).all()), (step, layer, b, h)
                    assert bool(((lse[b, at].double() - le).abs() <= lt).all())
        cache.advance()
    assert cache.lists.added.tolist() == [5] * 3


def test_chunked_retention_into_4_bits(lib, cuda):
    """Retention chunk by chunk goes through the same bf16 pages: a layer's held rows, whatever their slots."""
    w = synth.small(L=2, batch=2, N=300)
    cache, N = _cache(w, cuda, "e2m1", 4)
    for layer in range(w.L):
        s = synth.scores(w, layer, cuda)
        K, V = synth.keys_values(w, layer, cuda)
        slots = cache.compact_layer_chunked(layer, s, K, V, 64)
        pool, pages, off, ids = cache.dequantize_layer(layer)
        torch.cuda.synchronize()
        assert lib.tg_check_status(cache.status) == 0
        for b in range(w.batch):
            for p in range(w.H):
                h = int(cache.pages["order"][layer, p])
                n = int(cache.pages["ntok"][layer, b, h])
                l = b * cache.G + p // w.H_p
                for i, x in enumerate((K, V)):
                    got = rows_of(pool.view(-1, w.H_p, 2, w.P, w.d), ids[off[l]:off[l + 1]], w.H_p, w.P, w.d, p % w.H_p, n, bool(i))
                    assert torch.equal(got, hold(x[b, h, slots[b, h, :n].long()].double())[0])


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_a_turn_appends_its_tokens_and_attends_to_all(lib, cuda, pages):
    """A turn over retained and generated tokens: append with dense rows, attention of the pass over those, and the
    cache's tokens from before it as each request's shared prefix."""
    from non_uniform_paged_gb300.ragged import PrefillPass, SharedPrefix
    w = synth.small(L=1, batch=3, N=300, H=4, H_q=8, H_p=2)
    cache, N = _cache(w, cuda, pages, 40)
    H, H_q, d, g = w.H, w.H_q, w.d, 2
    s = synth.scores(w, 0, cuda)
    K, V = synth.keys_values(w, 0, cuda)
    kept = torch.full((w.batch, H, w.N), -1, dtype=torch.int32, device=cuda)
    cache.compact_layer(0, s, K, V, kept_idx=kept)
    rows = _retained(cache, 0, K, V, kept)
    new = [9, 1, 25]
    p = PrefillPass(H, H_q, d, new, new, device=cuda)
    T = sum(new)
    qkv = torch.randn((T, H_q + 2 * H, d), device=cuda, generator=torch.Generator(device=cuda).manual_seed(5)).to(torch.bfloat16)
    q, out = (torch.empty((T, H_q, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    lse = torch.empty((T, H_q), device=cuda)
    nK, nV = (torch.empty((3, H, 25, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    positions = torch.randint(0, 900, (T, 3), device=cuda, generator=torch.Generator(device=cuda).manual_seed(6)).to(torch.int32)
    axis_of = [i % 3 for i in range(d // 2)]
    # what the cache held before the turn
    old, old_pages, old_off, old_ids = cache.dequantize_layer(0)
    cache.append_layer(0, qkv, _table(900, d, cuda), q, cu_q=p.cu_q, positions=positions, axis_of=axis_of, K=nK, V=nV, start=p.start)
    p.attend(q, nK, nV, out, lse)
    shared = SharedPrefix.of_cache(cache, np.concatenate([[0], np.cumsum(new)]))
    own_out, own_lse = out.clone(), lse.clone()
    shared.attend(0, q, old, old_pages, old_off, old_ids, out, lse, own_out=own_out, own_lse=own_lse)
    cache.advance(torch.tensor(new, dtype=torch.int32, device=cuda))
    torch.cuda.synchronize()
    for x in (cache, p, shared):
        assert lib.tg_check_status(x.status) == 0
    at = 0
    for b, n in enumerate(new):
        for h in range(H):
            head = slice(h * g, (h + 1) * g)
            for i in range(n):
                t = at + i
                r = attend64(q[t, head], rows[b, h][0], rows[b, h][1], cache.scale, False)
                m, both, tol, ltol = merge64(*r, own_out[t, head], own_lse[t, head])
                assert bool(((out[t, head].double() - m).abs() <= tol).all()), (b, h, i)
                assert bool(((lse[t, head].double() - both).abs() <= ltol).all())
            for i, x in enumerate((nK, nV)):
                rows[b, h][i] = torch.cat([rows[b, h][i], x[b, h, :n].double()])
        at += n
    # a decode step after the turn sees retained, appended and its own tokens
    qkv = torch.randn((3, H_q + 2 * H, d), device=cuda, generator=torch.Generator(device=cuda).manual_seed(7)).to(torch.bfloat16)
    q, out = (torch.empty((3, H_q, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    lse = torch.empty((3, H_q), device=cuda)
    nK, nV = (torch.empty((3, H, 1, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    cache.append_layer(0, qkv, None, q, K=nK, V=nV, start=torch.zeros(3, dtype=torch.int32, device=cuda))
    cache.decode_layer(0, q, out, lse)
    for b in range(3):
        for h in range(H):
            k, v = (torch.cat([rows[b, h][i], x[b, h].double()]) for i, x in enumerate((nK, nV)))
            o, le, t, lt = attend64(q[b, h * g:(h + 1) * g], k, v, cache.scale, cache.four)
            assert bool(((out[b, h * g:(h + 1) * g].double() - o).abs() <= t).all())
            assert bool(((lse[b, h * g:(h + 1) * g].double() - le).abs() <= lt).all())


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_made_on_one_stream_run_and_dropped_on_another(lib, cuda, pages):
    """The owner's buffers outlive the calls that are queued when it is dropped."""
    from non_uniform_paged_gb300.ragged import GrowingLists
    ntok, d = np.full((4, 2), 200, np.int32), 128
    order = np.arange(2, dtype=np.int32)
    side = torch.cuda.Stream()
    n = 4 * 2 * 14
    off = torch.arange(0, n + 1, 14, device=cuda)
    ids = torch.arange(n, dtype=torch.int32, device=cuda)
    pool = torch.randn((n, 1, 2, 16, d), device=cuda).to(torch.bfloat16) if pages == "bf16" else \
        torch.randint(0, 64, (n, 1, 1, 2304), device=cuda, dtype=torch.uint8)
    q = torch.randn((4, 4, d), device=cuda).to(torch.bfloat16)
    outs = [torch.zeros_like(q) for _ in range(6)]
    torch.cuda.synchronize()
    for o in outs:
        lists = GrowingLists(4, 1, 16, d, order, ntok, 8, pages=pages, n_cta=30, device=cuda)
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            lists.attend(0, q, pool, n, off, ids, o)
        plan = lists.plan.plan_dev.numel()
        del lists
        torch.full((plan,), 255, dtype=torch.uint8, device=cuda)  # what might take the dropped plan's place
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs) and bool(outs[0].any())


def test_scale_of_a_head_without_tokens(lib, cuda):
    """Nothing retained and nothing appended: out 0 and lse -inf, then one token: its own value."""
    from non_uniform_paged_gb300.ragged import GrowingLists
    for pages in ("bf16", "e2m1"):
        lists = GrowingLists(2, 1, 16, 128, [0], [[0]], 16, pages=pages, n_cta=3, device=cuda)
        off, ids = torch.tensor([0, 1], device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
        pool = torch.full((1, 1, 2, 16, 128), math.nan, dtype=torch.bfloat16, device=cuda) if pages == "bf16" else \
            torch.full((1, 1, 1, 2304), 255, dtype=torch.uint8, device=cuda)
        qkv = torch.randn((1, 4, 128), device=cuda).to(torch.bfloat16)
        q = torch.empty((1, 2, 128), dtype=torch.bfloat16, device=cuda)
        out, lse = torch.full_like(q, 9.0), torch.zeros((1, 2), device=cuda)
        lists.attend(0, qkv[:, :2].contiguous(), pool, 1, off, ids, out, lse=lse, plus=0)
        assert not out.any() and bool(torch.isneginf(lse).all())
        lists.append(0, qkv, None, q, pool, 1, off, ids)
        lists.attend(0, q, pool, 1, off, ids, out, lse=lse)
        v = qkv[0, 3].double()
        want = hold(v)[0] if pages == "e2m1" else v
        assert torch.equal(out[0, 0].double(), want) and torch.equal(out[0, 1].double(), want)


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_retention_on_another_stream_behind_a_busy_one(lib, cuda, pages):
    """The pages that retention goes through are made at its first call: ready for the stream that it runs on."""
    w = synth.small(L=2, batch=2, N=300)
    s, (K, V) = synth.scores(w, 1, cuda), synth.keys_values(w, 1, cuda)
    rows = []
    for busy in (False, True):
        cache, N = _cache(w, cuda, pages, 4)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        if busy:
            torch.cuda._sleep(20_000_000)
        cache.compact_layer(1, s, K, V, stream=side)
        side.synchronize()
        pool, n, off, ids = cache.dequantize_layer(1)
        torch.cuda.synchronize()
        assert lib.tg_check_status(cache.status) == 0
        got = []
        for b in range(w.batch):
            for p in range(w.H):
                l = b * cache.G + p // w.H_p
                mine = ids[int(off[l]):int(off[l + 1])]
                n = int(cache.pages["ntok"][1, b, int(cache.pages["order"][1, p])])
                got += [rows_of(pool.view(-1, w.H_p, 2, w.P, w.d), mine, w.H_p, w.P, w.d, p % w.H_p, n, v) for v in (False, True)]
        rows.append(torch.cat(got))
    assert torch.equal(*rows) and bool(rows[0].any())


def test_a_step_without_a_token_for_each_request_is_refused(lib, cuda):
    from non_uniform_paged_gb300.ragged import GrowingLists
    lists = GrowingLists(2, 1, 16, 128, [0], [[3], [4]], 2, n_cta=3, device=cuda)
    off, ids = torch.tensor([0, 1, 2], device=cuda), torch.arange(2, dtype=torch.int32, device=cuda)
    pool = torch.zeros((2, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda)
    qkv = torch.randn((1, 4, 128), device=cuda).to(torch.bfloat16)
    with pytest.raises(ValueError):
        lists.append(0, qkv, None, torch.empty((1, 2, 128), dtype=torch.bfloat16, device=cuda), pool, 2, off, ids)


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_a_prefix_of_a_cache_that_has_grown_holds_what_was_appended(lib, cuda, pages):
    """SharedPrefix over the cache after steps of uneven counts: every token that advance() counted, and none behind."""
    from non_uniform_paged_gb300.ragged import SharedPrefix
    w = synth.small(L=2, batch=3, N=300, H=4, H_q=8, H_p=2)
    cache, N = _cache(w, cuda, pages, 40)
    g, layer, steps = 2, 1, [18, 0, 5]
    for l in range(2):
        cache.compact_layer(l, synth.scores(w, l, cuda), *synth.keys_values(w, l, cuda))
    gen = torch.Generator(device=cuda).manual_seed(3)
    T = sum(steps) + 6
    cu = torch.tensor(np.concatenate([[0], np.cumsum([n + 2 for n in steps])]), dtype=torch.int32, device=cuda)
    qkv = torch.randn((T, 16, w.d), generator=gen, device=cuda).to(torch.bfloat16)
    q = torch.empty((T, 8, w.d), dtype=torch.bfloat16, device=cuda)
    cache.append_layer(layer, qkv, None, q, cu_q=cu)  # two tokens of each request are not counted
    cache.advance(torch.tensor(steps, dtype=torch.int32, device=cuda))
    want = cache.pages["ntok"] + np.asarray(steps)[None, :, None]
    assert np.array_equal(cache.held_tokens(), want)
    shared = SharedPrefix.of_cache(cache, [0, 1, 2, 3])
    pool, n, off, ids = cache.dequantize_layer(layer)
    q = torch.randn((3, 8, w.d), generator=gen, device=cuda).to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty((3, 8), device=cuda)
    shared.attend(layer, q, pool, n, off, ids, out, lse)
    torch.cuda.synchronize()
    assert lib.tg_check_status(shared.status) == 0 and lib.tg_check_status(cache.status) == 0
    order = cache.pages["order"][layer]
    for b in range(3):
        for p in range(4):
            h, l = int(order[p]), b * cache.G + p // 2
            mine = ids[int(off[l]):int(off[l + 1])]
            k, v = (rows_of(pool.view(-1, 2, 2, w.P, w.d), mine, 2, w.P, w.d, p % 2, int(want[layer, b, h]), i) for i in (False, True))
            o, le, t, lt = attend64(q[b, h * g:(h + 1) * g], k, v, cache.scale, False)
            assert bool(((out[b, h * g:(h + 1) * g].double() - o).abs() <= t).all())
            assert bool(((lse[b, h * g:(h + 1) * g].double() - le).abs() <= lt).all())


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_caches_of_one_allocator_share_a_pool(lib, cuda, pages):
    """Two caches whose pages lie between each other's in one pool: each step's bits are those of caches apart."""
    from non_uniform_paged_gb300.ragged import GrowingCache
    w = synth.small(L=2, batch=2, N=200)
    N, Bhat, g = synth.contexts(w), synth.budgets_hat(w), torch.Generator(device=cuda).manual_seed(9)

    def make(allocator, pool=True):
        return GrowingCache(w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, Bhat, N, 6, pages=pages, n_cta=16, device=cuda,
                            alloc_pool=pool, allocator=allocator)
    apart, alloc = [make(None), make(None)], lib.PageAllocator(3000)
    shared = [make(alloc, False), make(alloc, False)]
    page = lib.tg_page_bytes(shared[0].lists.format, w.H_p, w.P, w.d)
    pool = torch.empty(3000 * page, dtype=torch.uint8, device=cuda)
    for c in shared:
        assert c.pool is None and c.n_pages == 3000
        c.pool = pool if pages == "e2m1" else pool.view(torch.bfloat16)
    data = [(synth.scores(w, l, cuda), *synth.keys_values(w, l, cuda)) for l in range(2)]
    steps = torch.randn((2, 3, 2, w.batch, w.H_q + 2 * w.H, w.d), generator=g, device=cuda).to(torch.bfloat16)  # cache, step, layer
    outs = []
    for caches in (apart, shared):
        out = torch.zeros((2, 3, 2, w.batch, w.H_q, w.d), dtype=torch.bfloat16, device=cuda)
        q = torch.empty((w.batch, w.H_q, w.d), dtype=torch.bfloat16, device=cuda)
        for i, c in enumerate(caches):
            for l in range(2):
                s, K, V = data[(l + i) % 2]
                c.compact_layer(l, s, K, V)
        for n in range(3):
            for i, c in enumerate(caches):
                for l in range(2):
                    c.append_layer(l, steps[i, n, l], None, q)
                    c.decode_layer(l, q, out[i, n, l])
                c.advance()
        torch.cuda.synchronize()
        assert all(lib.tg_check_status(c.status) == 0 for c in caches)
        outs.append(out)
    assert torch.equal(*outs) and not torch.equal(outs[0][0], outs[0][1])
