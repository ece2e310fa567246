"""tg_decode_grown over bf16 pages: the weights that meet V are those whose sum divides the output."""
import numpy as np
import pytest
import torch

from pages4_helpers import U, attend64, rows_of
from test_gpu_grown import Lists

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("g,n_cta,low,high", [(2, 40, 2, 16), (8, 7, 2, 40), (1, 152, 100, 900)])
def test_values_with_a_common_mean_keep_it(lib, cuda, d, g, n_cta, low, high):
    """V = 1 +- 0.05.  Weights are two bf16 terms, the first cut off (2^-7) and the rest rounded (2^-8 of it) 2^-20 above what it is:
    together off by less than 2^-14.  The sum is of the whole weights, so an output is off by its own rounding, 2^-14 A and the
    float32 terms of attend64 (A = sum_t softmax_t |v_t|)."""
    ntok = np.random.default_rng(d + g).integers(low, high + 1, (16, 4))
    x = Lists(cuda, "bf16", ntok, 4 * g, d, H_p=2, reserve=3, n_cta=n_cta, hostile=False, seed=g)
    v = x.pool[:, :, 1]
    x.pool[:, :, 1] = (1 + 0.05 * v.float()).to(torch.bfloat16)
    out, lse, status = x.run([b % 3 for b in range(16)], 1)
    assert status == 0
    for b in range(16):
        for p in range(4):
            h, l = int(x.order[p]), b * 2 + p // 2
            n = x.tokens(b, h, b % 3 + 1)
            K, V = (rows_of(x.pool, x.ids[x.off[l]:x.off[l + 1]], 2, 16, d, p % 2, n, bool(i)) for i in (0, 1))
            at = slice(h * g, (h + 1) * g)
            r, le, _, lt = attend64(x.q[b, at], K, V, x.scale, False)
            A = torch.softmax(x.scale * (x.q[b, at].double() @ K.T), -1) @ V.abs()
            e = (lt - 2.0 ** -20 * (1 + le.abs()))[:, None]
            tol = U * (1 + U) * r.abs() + (2.0 ** -14 + 4 * e) * (1 + U) * A
            off = (out[b, at].double() - r).abs()
            assert bool((off <= tol).all()), (b, h, n, (off / tol).max().item())
            assert bool(((lse[b, at].double() - le).abs() <= lt).all())


def test_an_infinite_value_is_infinite_and_spoils_no_other(lib, cuda):
    """The token with the largest weight (1 at the reference) and others hold +inf and -inf in some places of V."""
    x = Lists(cuda, "bf16", [[40, 9]], 4, 128, reserve=0, n_cta=3, hostile=False)
    ref, _, _ = x.run([0])
    for p in range(2):
        ids = x.ids[x.off[p]:x.off[p + 1]].long()
        rows = x.pool[ids, 0, 1].view(-1, 128)
        n, h = int(x.ntok_h[0, int(x.order[p])]), int(x.order[p])
        rows[:n, 5], rows[n // 2, 7] = float("inf"), -float("inf")
        x.pool[ids, 0, 1] = rows.view(-1, 16, 128)
        out, _, status = x.run([0])
        assert status == 0
        got = out[0, 2 * h:2 * h + 2].float()
        assert bool((got[:, 5] == float("inf")).all()) and bool((got[:, 7] == -float("inf")).all())
        others = [i for i in range(128) if i not in (5, 7)]
        assert torch.equal(out[0, 2 * h:2 * h + 2][:, others], ref[0, 2 * h:2 * h + 2][:, others])
