"""The bounded waits of the tile kernel: work that takes longer than a wait's limit is no reason to
give up."""
import math

import pytest
import torch

from prompt_helpers import attend64, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(128, 131040), (256, 92000)])
def test_a_pass_of_seconds_on_one_block(lib, cuda, d, n):
    """A long prompt and a short one on a single thread block, for more than the 2 s after which a
    block gives up that makes no progress.  The clearing warp has work at the end of the contexts
    only (the long one ends with a block), so it waits for nearly the whole pass."""
    from non_uniform_paged_gb300.ragged import PrefillPass
    assert n % 80 == 0
    short, g = 17, 8
    gen = torch.Generator(device=cuda).manual_seed(d)
    q = torch.randn((n + short, g, d), generator=gen, device=cuda).to(torch.bfloat16)
    K, V = (torch.randn((2, 1, n, d), generator=gen, device=cuda).to(torch.bfloat16) for _ in range(2))
    V[1, :, short:] = float("nan")
    p = PrefillPass(1, g, d, [n, short], [n, short], n_cta=1, device=cuda)
    assert p.plan.header["N_CTA"] == 1
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device=cuda)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    p.attend(q, K, V, out, lse)
    end.record()
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    # (a faster device needs a longer prompt)
    assert start.elapsed_time(end) > 2100
    # rows spread over the long prompt -- the first ones are worked on last -- and the short one
    rows = torch.cat([torch.arange(40, device=cuda), torch.linspace(40, n - 1, 88, device=cuda).long()])
    seen = torch.arange(n, device=cuda)[None] <= rows[:, None]
    few = torch.arange(short, device=cuda)
    for j in (0, 3, g - 1):
        ref = attend64(q[rows, j], K[0, 0], V[0, 0], 1 / math.sqrt(d), seen)
        check(out[rows, j], lse[rows, j], ref, f"long, head {j}")
        ref = attend64(q[n:, j], K[1, 0, :short], V[1, 0, :short], 1 / math.sqrt(d), few[None] <= few[:, None])
        check(out[n:, j], lse[n:, j], ref, f"short, head {j}")
    assert bool((out != 9.0).any(-1).all()) and bool((lse != 9.0).all())
