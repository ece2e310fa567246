"""What a decode step over a GrowingCache attends to: nothing that no one wrote, and as many tokens as each request brought."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


def _cache(cuda, pages, reserve=6, L=2):
    from non_uniform_paged_gb300.ragged import GrowingCache
    w = synth.small(L=L, batch=3, N=200)
    cache = GrowingCache(w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, synth.budgets_hat(w), synth.contexts(w), reserve,
                         pages=pages, n_cta=16, device=cuda)
    cache.pool.view(torch.uint8).fill_(0xff)  # rows that no one wrote: NaN of either format
    for l in range(L):
        cache.compact_layer(l, synth.scores(w, l, cuda), *synth.keys_values(w, l, cuda))
    g = torch.Generator(device=cuda).manual_seed(4)
    q = torch.randn((w.batch, w.H_q, w.d), generator=g, device=cuda).to(torch.bfloat16)
    qkv = torch.randn((2 * w.batch, w.H_q + 2 * w.H, w.d), generator=g, device=cuda).to(torch.bfloat16)
    return w, cache, q, qkv


def _decode(cache, q, layer=0, **how):
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    cache.decode_layer(layer, q, out, lse, **how)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    return torch.cat([out.float().flatten(), lse.flatten()])


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
@pytest.mark.parametrize("reserve", [0, 6])
def test_a_cache_that_only_retained_decodes_what_it_retained(lib, cuda, pages, reserve):
    w, cache, q, _ = _cache(cuda, pages, reserve)
    for l in range(w.L):
        assert torch.equal(_decode(cache, q, l), _decode(cache, q, l, plus=0))
    assert lib.tg_check_status(cache.status) == 0


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_the_default_follows_the_step(lib, cuda, pages):
    w, cache, q, qkv = _cache(cuda, pages)
    own = torch.empty_like(q)
    old = _decode(cache, q, plus=0)
    cache.append_layer(0, qkv[:3], None, own)
    new = _decode(cache, q)
    assert torch.equal(new, _decode(cache, q, plus=1)) and not torch.equal(new, old)
    assert torch.equal(_decode(cache, q, 1), _decode(cache, q, 1, plus=0))  # this layer brought nothing yet
    cache.advance()
    # between steps nothing tells which tokens are meant: the call says
    with pytest.raises(ValueError):
        _decode(cache, q)
    assert torch.equal(_decode(cache, q, plus=0), new)
    cache.append_layer(0, qkv[3:], None, own)
    assert torch.equal(_decode(cache, q), _decode(cache, q, plus=1))
    assert lib.tg_check_status(cache.status) == 0


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_a_replayed_step_decodes_as_it_was_captured(lib, cuda, pages):
    w, cache, q, qkv = _cache(cuda, pages, L=1)
    w2, eager, _, _ = _cache(cuda, pages, L=1)
    own, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)

    def step(c):
        c.append_layer(0, qkv[:3], None, own)
        c.decode_layer(0, q, out, lse)
        c.advance()

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(cache)
    step(eager)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_a_replayed_append_counts_for_the_calls_behind_it(lib, cuda, pages):
    """Only the append is in the graph; decode_layer and advance() are called between its replays."""
    w, cache, q, qkv = _cache(cuda, pages, L=1)
    w2, eager, _, _ = _cache(cuda, pages, L=1)
    own, side = torch.empty_like(q), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        cache.append_layer(0, qkv[:3], None, own)
    for _ in range(3):
        graph.replay()
        eager.append_layer(0, qkv[:3], None, own)
        assert torch.equal(_decode(cache, q), _decode(eager, q))
        cache.advance(), eager.advance()
    assert lib.tg_check_status(cache.status) == 0


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_requests_that_bring_none_one_or_two_tokens(lib, cuda, pages):
    """Counts of the step's own, in place of added and plus: each request decodes what it would if all had brought as many."""
    w, cache, q, qkv = _cache(cuda, pages)
    brought = [0, 1, 2]
    cu = torch.tensor([0, 0, 1, 3], dtype=torch.int32, device=cuda)
    cache.append_layer(0, qkv[:3], None, torch.empty((3, w.H_q, w.d), dtype=torch.bfloat16, device=cuda), cu_q=cu)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    cache.decode_layer(0, q, out, lse, added=torch.tensor(brought, dtype=torch.int32, device=cuda))
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all()) and lib.tg_check_status(cache.status) == 0
    for b, n in enumerate(brought):
        o, le = torch.empty_like(q), torch.empty_like(lse)
        cache.decode_layer(0, q, o, le, plus=n)
        assert torch.equal(o[b], out[b]) and torch.equal(le[b], lse[b])
    with pytest.raises(ValueError):
        cache.decode_layer(0, q, out, lse, added=torch.zeros(2, dtype=torch.int32, device=cuda))
