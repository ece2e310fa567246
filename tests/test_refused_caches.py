"""A cache that is refused after its pages were reserved leaves none of them taken (host only)."""
import pytest

import synth


@pytest.mark.parametrize("growing", [False, True])
@pytest.mark.parametrize("bad", [dict(n_cta=1), dict(d=96, n_cta=24), dict(H_q=36, n_cta=24)])
def test_pages_go_back(lib, growing, bad):
    from non_uniform_paged_gb300.ragged import GrowingCache, RaggedCache
    w = synth.small(H=4, H_q=8, H_p=1, batch=3)
    alloc = lib.PageAllocator(4000)
    held = alloc.admit([5, 7])
    before = alloc.query()
    a = dict(L=w.L, batch=w.batch, H=w.H, H_q=w.H_q, d=w.d, P=w.P, H_p=w.H_p, alpha=w.alpha, Bhat=synth.budgets_hat(w),
             N=synth.contexts(w), device="cpu", alloc_pool=False, allocator=alloc)
    a.update(bad, **(dict(reserve=4) if growing else {}))
    with pytest.raises(lib.TGError):
        (GrowingCache if growing else RaggedCache)(**a)
    assert alloc.query() == before
    alloc.release(held)
    assert alloc.query()[0] == 4000
