"""tg_append_rope without an eps, of rows so small that their squares leave float32: the norm is the formula's all the same."""
import pytest
import torch

from pages4_helpers import hold, read_tiles
from prompt_helpers import rope64
from test_gpu_append import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("d,pairs,rot", [(128, False, 128), (256, True, 64)])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140])
def test_rows_of_every_size(lib, cuda, fmt, d, pairs, rot, eps):
    T, H_q, H = 64, 3, 2
    heads = H_q + 2 * H
    values = torch.randn((T, heads, d), device=cuda, generator=torch.Generator(device=cuda).manual_seed(d)) + 0.01
    # a row's values within a few powers of two of each other, rows from 2^-124 to 2^20
    power = torch.linspace(-124, 20, T, device=cuda).round()[:, None, None]
    values = (values * torch.exp2(power)).to(torch.bfloat16).view(T, heads * d)
    c = Case(cuda, fmt, [T], [[5, 9]], H_q, H, d, rot=rot, pairs=pairs, values=values, positions=list(range(T)))
    assert c.call(lib, eps=eps) in ((0,) if fmt == 0 else (0, lib.STATUS_NONFINITE))
    ref, tol = rope64(c.qkv, c._rows(0, 0, T), H_q, H, c.w[0], c.w[1], eps, pairs, rot)
    assert bool(torch.isfinite(ref).all())
    off = (c.q.double() - ref[:, :H_q]).abs()
    assert bool((off <= tol[:, :H_q]).all()), (off / tol[:, :H_q].clamp_min(1e-300)).max().item()
    for p in range(H):
        h = int(c.order[p])
        slot = int(c.ntok[0, h]) + torch.arange(T, device=cuda)
        page = c.ids[c.off[p] + slot // 16].long()
        if fmt == 0:
            got = c.pool[page, 0, 0, slot % 16].double()
            assert bool(((got - ref[:, H_q + h]).abs() <= tol[:, H_q + h]).all())
        else:
            got = read_tiles(c.pool[page, 0, slot % 16 // 16], d, 1.0, False)[0][torch.arange(T, device=cuda), slot % 16]
            assert torch.equal(got, hold(ref[:, H_q + h])[0])
    assert int(c.status) == 0
