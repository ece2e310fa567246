"""tg_prefix_attn against its 64-bit definition over ragged pages, alone and merged with the
requests' own attention; bad pages; and the whole path from projections to a decode step."""
import math

import numpy as np
import pytest
import torch

from prompt_helpers import attend64, check, merge64, rope64, seen_keys

pytestmark = pytest.mark.gpu


def _setup(cuda, req_off, ntok, H_p, P, d, g, order=None, seed=0, spare=3):
    groups, H = np.asarray(ntok).shape
    G, batch = H // H_p, req_off[-1]
    order = np.arange(H, dtype=np.int32) if order is None else np.asarray(order, np.int32)
    gen = torch.Generator(device=cuda).manual_seed(seed)
    counts = [-(-max(int(ntok[r][order[i * H_p + j]]) for j in range(H_p)) // P) for r in range(groups) for i in range(G)]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    pages = int(off[-1]) + spare
    ids = torch.randperm(pages, generator=gen, device=cuda)[:max(1, int(off[-1]))].to(torch.int32)
    pool = torch.randn((pages, H_p, 2, P, d), generator=gen, device=cuda).to(torch.bfloat16)
    place = np.argsort(order)
    kv = {}
    for r in range(groups):
        for h in range(H):
            n, lst, j = int(ntok[r][h]), r * G + int(place[h]) // H_p, int(place[h]) % H_p
            own = ids[off[lst]:off[lst + 1]].long()
            full = -(-n // P)
            # what a head's block holds in pages past its last is anybody's
            pool[own[full:], j] = float("nan")
            k = pool[own[:full], j].transpose(0, 1).reshape(2, -1, d)[:, :n] if full else pool.new_zeros((2, 0, d))
            kv[r, h] = (k[0].clone(), k[1].clone())
    q = torch.randn((batch, H * g, d), generator=gen, device=cuda).to(torch.bfloat16)
    return dict(q=q, pool=pool, pages=pages, off=torch.from_numpy(off).to(cuda), ids=ids, order=order, kv=kv, gen=gen)


def _run(lib, cuda, req_off, ntok, H_p, P, d, g, own=True, order=None, n_cta=None, seed=0, inplace=False):
    from non_uniform_paged_gb300.ragged import SharedPrefix
    s = _setup(cuda, req_off, ntok, H_p, P, d, g, order, seed)
    batch, H = req_off[-1], len(ntok[0])
    p = SharedPrefix(H * g, H_p, P, d, req_off, s["order"], np.asarray(ntok, np.int32), n_cta=n_cta, device=cuda)
    own_out = own_lse = None
    if own:
        own_out = torch.randn((batch, H * g, d), generator=s["gen"], device=cuda).to(torch.bfloat16)
        own_lse = 3 * torch.randn((batch, H * g), generator=s["gen"], device=cuda) + 3
        own_lse[::3] = -math.inf  # requests that have nothing of their own
        own_out[::3] = float("nan")
    out, lse = torch.full_like(s["q"], 9.0), torch.full(s["q"].shape[:2], 9.0, device=cuda)
    keep = (own_out, own_lse) if not own else (own_out.clone(), own_lse.clone())
    if inplace:
        out, lse = own_out, own_lse
    p.attend(0, s["q"], s["pool"], s["pages"], s["off"], s["ids"], out, lse, own_out=own_out, own_lse=own_lse)
    torch.cuda.synchronize()
    assert lib.tg_check_status(p.status) == 0
    for r in range(len(ntok)):
        lo, hi = req_off[r], req_off[r + 1]
        for j in range(H * g):
            if hi > lo:
                ref = attend64(s["q"][lo:hi, j], *s["kv"][r, j // g], 1 / math.sqrt(d))
                if own:
                    ref = merge64(*ref, keep[0][lo:hi, j], keep[1][lo:hi, j])
                check(out[lo:hi, j], lse[lo:hi, j], ref, f"group {r} head {j}")
    return p, s, out, lse


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("P", [16, 32, 48, 64, 128, 144, 256])
def test_page_sizes(lib, cuda, d, P):
    _run(lib, cuda, [0, 9], [[700, 1, 129, 128]], 2, P, d, 4, seed=P)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("g", [1, 2, 3, 5, 7, 8])
@pytest.mark.parametrize("own", [False, True])
def test_head_groups(lib, cuda, d, g, own):
    _run(lib, cuda, [0, 50], [[333, 90]], 1, 16, d, g, own=own, seed=g)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("own", [False, True])
def test_groups_empty_heads_and_empty_groups(lib, cuda, d, own):
    ntok = [[0, 40, 1000, 17], [5, 0, 0, 0], [0, 0, 0, 0], [300, 200, 100, 50]]
    for n_cta in (1, 152):
        _run(lib, cuda, [0, 3, 3, 70, 71], ntok, 2, 16, d, 4, own=own, order=[2, 0, 3, 1], n_cta=n_cta)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("batch", [1, 31, 32, 33, 64, 65, 200])
def test_batches(lib, cuda, d, batch):
    _run(lib, cuda, [0, batch], [[260, 1030]], 2, 16, d, 4, seed=batch)


@pytest.mark.parametrize("d", [128, 256])
def test_long_prefix_is_cut_and_merged_in_place(lib, cuda, d):
    p, *_ = _run(lib, cuda, [0, 7], [[20000, 5000, 777, 1]], 4, 16, d, 4, inplace=True)
    assert p.plans[0].header["n_merge"] > 0
    p, *_ = _run(lib, cuda, [0, 7], [[200, 50, 77, 1]], 4, 16, d, 4, inplace=True, n_cta=1)
    assert p.plans[0].header["n_merge"] == 0


@pytest.mark.parametrize("n_cta", [1, 152])
def test_bad_pages_are_reported_and_read_as_zeros(lib, cuda, n_cta):
    """A page id outside the pool, and a list shorter than its tokens: the status says so, and the
    missing keys count as zero vectors."""
    from non_uniform_paged_gb300.ragged import SharedPrefix
    d, P = 128, 16
    s = _setup(cuda, [0, 5], [[600]], 1, P, d, 4)
    p = SharedPrefix(4, 1, P, d, [0, 5], s["order"], np.array([[600]], np.int32), n_cta=n_cta, device=cuda)
    K, V = (t.clone() for t in s["kv"][0, 0])
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device=cuda)
    ids, off = s["ids"].clone(), s["off"].clone()
    ids[3], ids[20] = -1, s["pages"]
    off[1] -= 2
    for t in (K, V):
        t[3 * P:4 * P] = 0
        t[20 * P:21 * P] = 0
        t[36 * P:] = 0
    p.attend(0, s["q"], s["pool"], s["pages"], off, ids, out, lse)
    torch.cuda.synchronize()
    assert int(p.status.item()) == lib.STATUS_BAD_PAGE
    for j in range(4):
        check(out[:, j], lse[:, j], attend64(s["q"][:, j], K, V, 1 / math.sqrt(d)), j)


def test_pool_past_32_bit_offsets(lib, cuda):
    from non_uniform_paged_gb300.ragged import SharedPrefix
    pages, P, d = 560_000, 16, 128
    pool = torch.zeros((pages, 1, 2, P, d), dtype=torch.bfloat16, device=cuda)
    g = torch.Generator(device=cuda).manual_seed(3)
    ids = torch.tensor([pages - 1, 0, pages - 7], dtype=torch.int32, device=cuda)
    pool[ids.long()] = torch.randn((3, 1, 2, P, d), generator=g, device=cuda).to(torch.bfloat16)
    q = torch.randn((2, 4, d), generator=g, device=cuda).to(torch.bfloat16)
    p = SharedPrefix(4, 1, P, d, [0, 2], [0], np.array([[45]], np.int32), device=cuda)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    p.attend(0, q, pool, pages, torch.tensor([0, 3], device=cuda), ids, out, lse)
    kv = pool[ids.long(), 0].transpose(0, 1).reshape(2, 48, d)[:, :45]
    for j in range(4):
        check(out[:, j], lse[:, j], attend64(q[:, j], kv[0], kv[1], 1 / math.sqrt(d)), j)


def test_same_bits_in_a_graph_and_on_two_streams(lib, cuda):
    a = _run(lib, cuda, [0, 30], [[9000, 4000]], 2, 16, 128, 4, own=False, seed=1)
    b = _run(lib, cuda, [0, 12], [[3000, 7000]], 1, 16, 256, 2, own=False, seed=2)
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for (p, s, out, lse), st in zip((a, b), streams):
            o, l = torch.empty_like(out), torch.empty_like(lse)
            with torch.cuda.stream(st):
                p.attend(0, s["q"], s["pool"], s["pages"], s["off"], s["ids"], o, l)
            outs.append((o, l, out, lse))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ro) and torch.equal(l, rl) for o, l, ro, rl in outs)
    p, s, out, lse = a
    o, l = torch.empty_like(out), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        p.attend(0, s["q"], s["pool"], s["pages"], s["off"], s["ids"], o, l)
    for _ in range(2):
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_binding_refusals(lib, cuda):
    p, s, out, lse = _run(lib, cuda, [0, 3], [[50, 60]], 2, 16, 128, 2)
    call = dict(layer=0, q=s["q"], pool=s["pool"], pool_pages=s["pages"], pt_off=s["off"], pt_ids=s["ids"], out=out, lse=lse)
    for bad in (dict(q=s["q"][:2]), dict(pool_pages=s["pages"] + 1), dict(pt_off=s["off"][:1]), dict(own_out=out[:1], own_lse=lse)):
        with pytest.raises(ValueError):
            p.attend(**dict(call, **bad))
    with pytest.raises(lib.TGError):
        p.attend(**dict(call, own_out=out))
    with pytest.raises(TypeError):
        p.attend(**dict(call, pt_ids=s["ids"].long()))


@pytest.mark.parametrize("d,H_q,H", [(128, 8, 4), (256, 4, 2)])
def test_projections_to_decode(lib, cuda, d, H_q, H):
    """The operators in a run, as a serving step uses them.  A shared document is prefilled in two
    chunks (place, attend), compacted into a prefix cache with head-wise budgets; each request
    prefills its own question, compacts it into its own cache; a decode step then places one
    token, attends to the request's own pages (tg_decode_attn) and merges the shared prefix."""
    from non_uniform_paged_gb300.ragged import PrefillPass, RaggedCache, SharedPrefix
    gen = torch.Generator(device=cuda).manual_seed(d)
    batch, doc, own = 5, 900, [40, 7, 130, 64, 1]
    P, H_p, g, eps, scale = 16, 2, H_q // H, 1e-6, 1 / math.sqrt(d)
    heads = H_q + 2 * H
    qw, kw = (torch.rand(d, generator=gen, device=cuda) + 0.5 for _ in range(2))
    f = 1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=cuda) / d)
    ang = torch.arange(doc + 200, dtype=torch.float64, device=cuda)[:, None] * f
    table = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()

    def bf(*shape):
        return torch.randn(shape, generator=gen, device=cuda).to(torch.bfloat16)

    # the document, in chunks of 512 and 388 tokens
    K, V = (torch.full((1, H, doc, d), float("nan"), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    at = 0
    for n in (512, doc - 512):
        x = bf(n, heads, d)
        p = PrefillPass(H, H_q, d, [n], [at + n], device=cuda)
        q, out = torch.empty((n, H_q, d), dtype=torch.bfloat16, device=cuda), torch.empty((n, H_q, d), dtype=torch.bfloat16, device=cuda)
        p.place(x, table, q, K, V, q_weight=qw, k_weight=kw, eps=eps)
        p.attend(q, K, V, out)
        ref, tol = rope64(x, table[at:at + n], H_q, H, qw, kw, eps, False, d)
        assert bool(((q.double() - ref[:, :H_q]).abs() <= tol[:, :H_q]).all())
        for j in range(H_q):
            check(out[:, j], None, attend64(q[:, j], K[0, j // g, :at + n], V[0, j // g, :at + n], scale, seen_keys(n, at + n, 0, cuda)))
        assert lib.tg_check_status(p.status) == 0
        at += n
    budgets = np.linspace(0.2, 1.0, H, dtype=np.float32)[None]
    shared = RaggedCache(1, 1, H, H_q, d, P, H_p, 1.0, budgets, [doc], cluster=True, device=cuda)
    kept = torch.full((1, H, doc), -1, dtype=torch.int32, device=cuda)
    shared.compact_layer(0, torch.randn((1, H, doc), generator=gen, device=cuda), K, V, kept_idx=kept)

    # the requests' own questions, behind the document's positions
    T, Nmax = sum(own), max(own)
    x = bf(T, heads, d)
    Ko, Vo = (torch.zeros((batch, H, Nmax, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    p = PrefillPass(H, H_q, d, own, own, device=cuda)
    pos = torch.cat([torch.arange(doc, doc + n, device=cuda) for n in own]).to(torch.int32)
    q = torch.empty((T, H_q, d), dtype=torch.bfloat16, device=cuda)
    p.place(x, table, q, Ko, Vo, q_weight=qw, k_weight=kw, eps=eps, positions=pos)
    mine = RaggedCache(1, batch, H, H_q, d, P, H_p, 1.0, np.ones((1, H), np.float32), own, device=cuda)
    mine.compact_layer(0, torch.zeros((batch, H, Nmax), device=cuda), Ko, Vo)

    # one decode step; its query is placed, then attends to both parts
    x = bf(batch, heads, d)
    step = PrefillPass(H, H_q, d, [1] * batch, [1] * batch, device=cuda)
    q = torch.empty((batch, H_q, d), dtype=torch.bfloat16, device=cuda)
    Kn, Vn = (torch.empty((batch, H, 1, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    pos = torch.tensor([doc + n for n in own], dtype=torch.int32, device=cuda)
    step.place(x, table, q, Kn, Vn, q_weight=qw, k_weight=kw, eps=eps, positions=pos)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    mine.decode_layer(0, q, out, lse)
    prefix = SharedPrefix.of_cache(shared, [0, batch])
    own_out, own_lse = out.clone(), lse.clone()
    prefix.attend(0, q, shared.pool, shared.n_pages, shared.list_offsets(0), shared.pt_ids_dev, out, lse, own_out=out,
                  own_lse=lse)
    torch.cuda.synchronize()
    for s in (shared, mine, prefix, step):
        assert lib.tg_check_status(s.status) == 0
    for j in range(H_q):
        h = j // g
        n = int(shared.pages["ntok"][0, 0, h])
        idx = kept[0, h, :n].long()
        ref = merge64(*attend64(q[:, j], K[0, h, idx], V[0, h, idx], scale), own_out[:, j], own_lse[:, j])
        check(out[:, j], lse[:, j], ref, j)
        # and as one softmax over everything the request sees (its own part rounded once on the way)
        for b in range(batch):
            k = torch.cat([K[0, h, idx], Ko[b, h, :own[b]]])
            v = torch.cat([V[0, h, idx], Vo[b, h, :own[b]]])
            o, l, t, lt = attend64(q[b:b + 1, j], k, v, scale)
            check(out[b:b + 1, j], lse[b:b + 1, j], (o, l, 2 * t + 2.0 ** -8 * own_out[b, j].double().abs(), 4 * lt + 1e-5), (b, j))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("P", [16, 48, 128])
def test_rows_behind_a_count_hold_anything(lib, cuda, d, P):
    """A head's last page past its count: neither its keys nor its values reach a result."""
    from non_uniform_paged_gb300.ragged import SharedPrefix
    ntok, req_off, g, H_p = [[700, 1, 129, 80], [333, 5000, 79, 81]], [0, 9, 60], 4, 2
    G, H = 2, 4
    s = _setup(cuda, req_off, ntok, H_p, P, d, g, seed=P)
    for r in range(2):
        for h in range(H):
            n, lst = ntok[r][h], r * G + h // H_p
            if n % P:
                page = int(s["ids"][int(s["off"][lst]) + n // P])
                s["pool"][page, h % H_p, 0, n % P:] = float("inf")
                s["pool"][page, h % H_p, 1, n % P:] = float("nan")
    for n_cta in (1, 152):
        p = SharedPrefix(H * g, H_p, P, d, req_off, s["order"], np.array(ntok, np.int32), n_cta=n_cta, device=cuda)
        out, lse = torch.full_like(s["q"], 9.0), torch.full(s["q"].shape[:2], 9.0, device=cuda)
        p.attend(0, s["q"], s["pool"], s["pages"], s["off"], s["ids"], out, lse)
        for r in range(2):
            lo, hi = req_off[r], req_off[r + 1]
            for j in range(H * g):
                check(out[lo:hi, j], lse[lo:hi, j], attend64(s["q"][lo:hi, j], *s["kv"][r, j // g], 1 / math.sqrt(d)),
                      f"group {r} head {j}")


def test_made_on_one_stream_run_on_another(lib, cuda):
    """Workspace, status and plan are there when the constructors return, whatever the current stream
    still had to do: memory it was using a moment ago is not handed out."""
    from non_uniform_paged_gb300.ragged import PrefillPass, SharedPrefix
    ntok, d = np.array([[20000, 9000]], np.int32), 128
    s = _setup(cuda, [0, 7], ntok, 2, 16, d, 4)
    work = torch.zeros(1 << 28, dtype=torch.uint8, device=cuda)
    for make in (lambda: SharedPrefix(8, 2, 16, d, [0, 7], s["order"], ntok, device=cuda),
                 lambda: PrefillPass(2, 8, d, [1, 40], [9000, 4000], device=cuda)):
        torch.cuda.synchronize()
        for _ in range(40):
            work.add_(1)
        made = make()
        assert torch.cuda.current_stream().query()
        assert made.workspace is not None
