"""New tokens behind a context of which only the retained tokens are left: a turn, and decode steps
that see their own token.  The new rows go to dense contexts (tg_qk_norm_rope), tg_prefill_attn
attends to those, and tg_prefix_attn, with the new tokens of a request as a group, joins the retained
pages."""
import math

import numpy as np
import pytest
import torch

from prompt_helpers import attend64, check, rope64

pytestmark = pytest.mark.gpu


class Retained:
    """A ragged cache of random old contexts, and the rows that each head kept."""

    def __init__(self, cuda, H_q, H, d, old, budgets, seed):
        from non_uniform_paged_gb300.ragged import RaggedCache
        g = torch.Generator(device=cuda).manual_seed(seed)
        batch, Nmax = len(old), max(old)
        self.K, self.V = (torch.randn((batch, H, Nmax, d), generator=g, device=cuda).to(torch.bfloat16) for _ in range(2))
        scores = torch.randn((batch, H, Nmax), generator=g, device=cuda)
        self.cache = RaggedCache(1, batch, H, H_q, d, 16, 2, 1.0, np.asarray([budgets], np.float32), old, cluster=True, device=cuda)
        self.kept = torch.full((batch, H, Nmax), -1, dtype=torch.int32, device=cuda)
        self.cache.compact_layer(0, scores, self.K, self.V, kept_idx=self.kept)

    def rows(self, b, h):
        idx = self.kept[b, h, :int(self.cache.pages["ntok"][0, b, h])].long()
        return self.K[b, h, idx], self.V[b, h, idx]

    def join(self, prefix, q, out, lse):
        c = self.cache
        prefix.attend(0, q, c.pool, c.n_pages, c.list_offsets(0), c.pt_ids_dev, out, lse, own_out=out, own_lse=lse)


def _check_rows(r, q, out, lse, own, at, b, H, g, n, seen_new, K, V, d):
    """Tokens [at, at + n) of request b against one softmax over its retained rows and the new ones each
    sees (seen_new: how many); own: the part rounded on the way."""
    for j in range(H * g):
        h = j // g
        k, v = r.rows(b, h)
        m = int(seen_new.max())
        seen = torch.cat([torch.ones((n, k.shape[0]), dtype=torch.bool, device=q.device),
                          torch.arange(m, device=q.device)[None] < seen_new[:, None]], 1)
        o, l, t, lt = attend64(q[at:at + n, j], torch.cat([k, K[b, h, :m]]), torch.cat([v, V[b, h, :m]]), 1 / math.sqrt(d), seen)
        # the new tokens' part is rounded to bf16 once on the way and weighed by e^own_lse, which is off
        # by its own bound (as in the test of the whole path)
        check(out[at:at + n, j], lse[at:at + n, j], (o, l, 2 * t + 2.0 ** -8 * own[at:at + n, j].double().abs(), 4 * lt + 1e-5), (b, j))


@pytest.mark.parametrize("d,H_q,H", [(128, 8, 2), (256, 4, 2)])
def test_a_turn_over_retained_pages(lib, cuda, d, H_q, H):
    """Turns of 1 to 200 tokens behind retained contexts: packed, every token sees what was kept and the
    new tokens up to itself."""
    from non_uniform_paged_gb300.ragged import PrefillPass, SharedPrefix
    old, new = [3000, 17, 900, 1], [70, 1, 200, 33]
    g, T, Nmax = H_q // H, sum(new), max(new)
    r = Retained(cuda, H_q, H, d, old, np.linspace(0.1, 0.7, H), d)
    gen = torch.Generator(device=cuda).manual_seed(d + 1)
    q = torch.randn((T, H_q, d), generator=gen, device=cuda).to(torch.bfloat16)
    K, V = (torch.randn((len(new), H, Nmax, d), generator=gen, device=cuda).to(torch.bfloat16) for _ in range(2))
    p = PrefillPass(H, H_q, d, new, new, device=cuda)
    cu = np.concatenate([[0], np.cumsum(new)])
    prefix = SharedPrefix.of_cache(r.cache, cu)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    p.attend(q, K, V, out, lse)
    own = out.clone()
    r.join(prefix, q, out, lse)
    torch.cuda.synchronize()
    for s in (r.cache, p, prefix):
        assert int(s.status.item()) == 0
    for b, n in enumerate(new):
        _check_rows(r, q, out, lse, own, int(cu[b]), b, H, g, n, torch.arange(1, n + 1, device=cuda), K, V, d)


@pytest.mark.parametrize("d,H_q,H", [(128, 8, 2), (256, 4, 2)])
def test_decode_steps_that_see_their_own_token(lib, cuda, d, H_q, H):
    """Three decode steps: each step's projections are placed behind the tokens since the retention,
    and its queries see the retained tokens, those and their own."""
    from non_uniform_paged_gb300.ragged import PrefillPass, SharedPrefix
    old, tail, steps, eps = [500, 60, 1200, 9, 77], [0, 3, 81, 0, 16], 3, 1e-6
    batch, g, heads, room = len(old), H_q // H, H_q + 2 * H, 96
    r = Retained(cuda, H_q, H, d, old, np.linspace(0.2, 1.0, H), d + 2)
    gen = torch.Generator(device=cuda).manual_seed(d + 3)
    K, V = (torch.randn((batch, H, room, d), generator=gen, device=cuda).to(torch.bfloat16) for _ in range(2))
    for b in range(batch):  # nothing of what lies behind the tail may count
        K[b, :, tail[b]:], V[b, :, tail[b]:] = float("nan"), float("inf")
    qw, kw = (torch.rand(d, generator=gen, device=cuda) + 0.5 for _ in range(2))
    ang = torch.arange(2000, dtype=torch.float64, device=cuda)[:, None] * \
        1e4 ** (-torch.arange(0, d, 2, dtype=torch.float64, device=cuda) / d)
    table = torch.stack([ang.cos(), ang.sin()], -1).float().contiguous()
    prefix = SharedPrefix.of_cache(r.cache, np.arange(batch + 1))
    q = torch.empty((batch, H_q, d), dtype=torch.bfloat16, device=cuda)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    for step in range(steps):
        x = torch.randn((batch, heads, d), generator=gen, device=cuda).to(torch.bfloat16)
        n = [t + step + 1 for t in tail]
        pos = torch.tensor([o + m - 1 for o, m in zip(old, n)], dtype=torch.int32, device=cuda)
        p = PrefillPass(H, H_q, d, [1] * batch, n, device=cuda)
        p.place(x, table, q, K, V, q_weight=qw, k_weight=kw, eps=eps, positions=pos)
        p.attend(q, K, V, out, lse)
        own = out.clone()
        r.join(prefix, q, out, lse)
        torch.cuda.synchronize()
        for s in (r.cache, p, prefix):
            assert int(s.status.item()) == 0
        ref, tol = rope64(x, table[pos.long()], H_q, H, qw, kw, eps, False, d)
        row = torch.tensor(n, device=cuda) - 1
        got = torch.cat([q, K[torch.arange(batch), :, row], V[torch.arange(batch), :, row]], 1)
        assert bool(((got.double() - ref).abs() <= tol).all())
        for b in range(batch):
            _check_rows(r, q, out, lse, own, b, b, H, g, 1, torch.tensor([n[b]], device=cuda), K, V, d)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_cta", [1, 152])
def test_own_results_of_no_weight(lib, cuda, d, n_cta):
    """own_lse of -inf or near the type's lowest value: own_out, whatever it holds, counts for nothing."""
    from non_uniform_paged_gb300.ragged import SharedPrefix
    H, g, ntok, batch = 2, 4, [5000, 0], 6
    r = Retained(cuda, H * g, H, d, [5000], [1.0, 1.0], d + 4)
    c = r.cache
    q = torch.randn((batch, H * g, d), generator=torch.Generator(device=cuda).manual_seed(9), device=cuda).to(torch.bfloat16)
    p = SharedPrefix(H * g, 2, 16, d, [0, batch], c.pages["order"][0], np.array([ntok], np.int32), n_cta=n_cta, device=cuda)
    own_out = torch.full_like(q, float("nan"))
    own_lse = torch.full(q.shape[:2], float("-inf"), device=cuda)
    own_lse[::2] = torch.finfo(torch.float32).min
    got = []
    for kw in ({}, dict(own_out=own_out, own_lse=own_lse)):
        out, lse = torch.full_like(q, 9.0), torch.full_like(own_lse, 9.0)
        p.attend(0, q, c.pool, c.n_pages, c.list_offsets(0), c.pt_ids_dev, out, lse, **kw)
        got.append((out, lse))
    assert (p.plans[0].header["n_merge"] > 0) == (n_cta > 1)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    # the second head holds nothing: 0 and -inf
    assert bool((got[1][0][:, g:] == 0).all()) and bool(torch.isneginf(got[1][1][:, g:]).all())
    for j in range(g):
        k, v = r.rows(0, 0)
        check(got[1][0][:, j], got[1][1][:, j], attend64(q[:, j], k, v, 1 / math.sqrt(d)), j)
