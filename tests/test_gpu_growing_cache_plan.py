"""A GrowingCache plans its own decode; that of its base class, over the retained tokens alone, is there when it is asked for."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


def test_the_static_plan_is_made_on_demand_and_is_a_ragged_caches(lib, cuda):
    from non_uniform_paged_gb300.ragged import GrowingCache, RaggedCache
    w = synth.small(L=2, batch=3, N=300)
    args = (w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, synth.budgets_hat(w), synth.contexts(w))
    grown = GrowingCache(*args, 5, n_cta=24, device=cuda)
    static = RaggedCache(*args, n_cta=24, device=cuda)
    assert not {"S", "plan", "plan_dev", "workspace", "workspace_bytes"} & set(vars(grown))
    q = torch.randn((w.batch, w.H_q, w.d), device=cuda, generator=torch.Generator(device=cuda).manual_seed(2)).to(torch.bfloat16)
    out = [torch.empty_like(q) for _ in range(2)]
    for layer in range(w.L):
        for c in (grown, static):
            c.compact_layer(layer, synth.scores(w, layer, cuda), *synth.keys_values(w, layer, cuda))
        RaggedCache.decode_layer(grown, layer, q, out[0])
        static.decode_layer(layer, q, out[1])
        assert torch.equal(*out) and bool(out[0].any())
    assert grown.plan is grown.plan and (grown.plan == static.plan).all() and (grown.S == static.S).all()
    assert grown.workspace_bytes == static.workspace_bytes == grown.workspace.numel()
    assert lib.tg_check_status(grown.status) == 0
    with pytest.raises(AttributeError):
        grown.plans
