"""tg_qk_norm_rope with infinities and NaN among a head's values: they reach what the definition says
and nothing else."""
import pytest
import torch

from prompt_helpers import rope64
from test_gpu_rope import _table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("rot_of,pairs", [(0, False), (0, True), (2, False), (2, True), (1, False), (1, True)])
@pytest.mark.parametrize("norm", [False, True])
def test_non_finite_values_stay_where_they_are(lib, cuda, d, rot_of, pairs, norm):
    rot = d // rot_of if rot_of else 0
    T, H_q, H, eps = 40, 5, 2, 1e-6
    g = torch.Generator(device=cuda).manual_seed(d + rot)
    qkv = torch.randn((T, H_q + 2 * H, d), generator=g, device=cuda).to(torch.bfloat16)
    # one value of each of these tokens' heads, at places all over the head
    for t in range(0, T, 2):
        for h in range(H_q + 2 * H):
            qkv[t, h, (37 * t + 11 * h) % d] = (float("inf"), float("-inf"), float("nan"))[(t // 2 + h) % 3]
    w = [torch.randn(d, generator=g, device=cuda) if norm else None for _ in range(2)]
    table = _table(T, rot, cuda) if rot else None
    cu, start = torch.tensor([0, T], dtype=torch.int32, device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    q = torch.empty((T, H_q, d), dtype=torch.bfloat16, device=cuda)
    K, V = (torch.empty((1, H, T, d), dtype=torch.bfloat16, device=cuda) for _ in range(2))
    lib.tg_qk_norm_rope(qkv, cu, start, table, q, K, V, q_weight=w[0], k_weight=w[1], eps=eps, pairs=pairs)
    got = torch.cat([q, K[0].transpose(0, 1), V[0].transpose(0, 1)], 1).double()
    ref, tol = rope64(qkv, table, H_q, H, w[0], w[1], eps, pairs, rot)
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isposinf(), ref.isposinf()) and torch.equal(got.isneginf(), ref.isneginf())
    fin = ref.isfinite()
    assert bool(((got - ref).abs() <= tol)[fin].all())
    assert 0 < int((~fin).sum()) and bool(fin.any())
