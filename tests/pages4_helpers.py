"""64-bit definitions of 4-bit pages and of attention over grown lists, and their error bounds.

What the pages hold is defined exactly (nearest code, ties to even), so values are compared for equality.
Attention over 4-bit pages rounds its output once to bf16 (2^-8 relative) and each weight once to f16
(2^-11); with A = sum_t softmax_t |v_t| an output is off by at most
    2^-8 |ref| + (2^-11 + 4 e) A   (and their product),
e as in prompt_helpers: (d + 3) 2^-24 scale sum |q_i k_i| from float32 sums, 2^-20 from exponentials, and
2^-25 max|q| scale sum |k_i| from query values that f16 holds as subnormals.  Over bf16 pages the weights are
bf16 (2^-8).  The sum of the weights is of the unrounded ones."""
import math

import torch

U = 2.0 ** -8
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3_grid():
    """Every finite e4m3 number from 0 on, in order of its code."""
    code = torch.arange(127)
    e, m = code // 8, (code % 8).double()
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.double() - 7))


def nearest(x, grid):
    """Index of the grid's number nearest to x >= 0 (float64), ties to the even index; past the end: the last."""
    grid = grid.to(x.device)
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def hold(x, unit=1.0):
    """x [...][d] float64 -> (values that 4-bit pages hold of it, scale codes [...][d/16])."""
    b = x.double().unflatten(-1, (-1, 16))
    finite = torch.where(torch.isnan(b), torch.zeros_like(b), b.abs())
    top = finite.amax(-1) / (6 * unit)
    code = nearest(top.clamp(max=448.0), e4m3_grid()).clamp_min(1)
    s = e4m3_grid().to(x.device)[code][..., None] * unit
    r = (b.abs() / s).clamp(max=6.0)
    v = E2M1.to(x.device)[nearest(torch.where(torch.isnan(r), torch.full_like(r, 6.0), r), E2M1)] * s
    v = torch.where((b < 0) & ~torch.isnan(b), -v, v)
    return v.flatten(-2), code


def tile_bytes(d):
    return d // 128 * 2304


def places(t, e, V):
    """Byte of the code, whether it is the upper half, and byte of the scale of value e of token t (ints)
    in a tile of 16 tokens, spelt out from the header."""
    base, i = e // 128 * 2304, e % 128
    j = i // 16
    if V:
        return base + 1024 + 512 * (t // 8) + 64 * j + 8 * (t % 8) + i % 16 // 2, i % 2, base + 2176 + 16 * j + t
    return base + 64 * t + i // 2, i % 2, base + 2048 + 8 * t + j


def read_tiles(raw, d, unit, V):
    """raw uint8 [n][tile bytes] -> values [n][16][d] float64 and scale codes [n][16][d/16]."""
    at = [[places(t, e, V) for e in range(d)] for t in range(16)]
    code_at = torch.tensor([[p[0] for p in row] for row in at], device=raw.device)
    upper = torch.tensor([[p[1] for p in row] for row in at], device=raw.device)
    scale_at = torch.tensor([[p[2] for p in row] for row in at], device=raw.device)
    byte = raw[:, code_at.flatten()].view(-1, 16, d)
    code = torch.where(upper.bool(), byte >> 4, byte & 15).long()
    sc = raw[:, scale_at.flatten()].view(-1, 16, d).long()
    grid = torch.cat([e4m3_grid(), torch.full((1,), math.nan, dtype=torch.float64)]).to(raw.device)
    v = E2M1.to(raw.device)[code & 7] * grid[sc & 127] * unit
    v = torch.where(code >= 8, -v, v)
    return v, sc[:, :, ::16]


def rows_of(pool, ids, H_p, P, d, hpos, n, V, unit=1.0):
    """Values [n][d] (float64) of the first n tokens of a list (its page ids) at group position hpos, out of a
    pool of either format."""
    ids = ids.long()
    pages = ids[:-(-n // P)] if n else ids[:0]
    if pool.dtype == torch.bfloat16:
        return pool.view(-1, H_p, 2, P, d)[pages, hpos, int(V)].reshape(-1, d)[:n].double()
    raw = pool.view(-1, H_p, P // 16, tile_bytes(d))[pages, hpos].reshape(-1, tile_bytes(d))
    return read_tiles(raw, d, unit, V)[0].reshape(-1, d)[:n]


def attend64(q, K, V, scale, four):
    """q [g][d], K, V [n][d] -> out, lse, their bounds; four: over 4-bit pages, else over bf16 pages."""
    weight = 2.0 ** -11 if four else 2.0 ** -8
    q, K, V = q.double(), K.double(), V.double()
    g, d = q.shape
    if K.shape[0] == 0:
        z = torch.zeros((g, d), dtype=torch.float64, device=q.device)
        return z, torch.full((g,), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    x = scale * (q @ K.T)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    out, A = p @ V, p @ V.abs()
    e = (d + 3) * 2.0 ** -24 * scale * (q.abs() @ K.abs().T).amax(-1) + 2.0 ** -20
    e = e + 2.0 ** -25 * scale * q.abs().amax(-1) * K.abs().sum(-1).amax()
    tol = U * (1 + U) * out.abs() + (weight + 4 * e[:, None]) * (1 + U) * A + 1e-30
    return out, lse, tol, e + 2.0 ** -20 * (1 + lse.abs())
