"""64-bit definitions of the prompt-side and shared-prefix operators, and their error bounds.

A rounding to bf16 is off by at most 2^-8 relative.  Attention rounds its output once and each
softmax weight once, so with A = sum_t softmax_t |v_t| an output is off by at most
    2^-8 |ref| + 2^-8 A   (and their product),
plus what float32 adds: a logit is a sum of d products, off by at most (d + 3) 2^-24 * scale *
sum |q_i k_i| =: e, which moves weights by a factor e^(2e), and sums and exponentials add a few
2^-20.  The bounds below take e from the data.  lse is off by e plus 2^-20 (1 + |lse|)."""
import math

import torch

U = 2.0 ** -8


def attend64(q, K, V, scale, seen=None):
    """q [n][d], K, V [m][d] (any dtype), seen bool [n][m] -> out, lse, out bound, lse bound (float64)."""
    q, K, V = q.double(), K.double(), V.double()
    n, d = q.shape
    if K.shape[0] == 0:
        z = torch.zeros((n, d), dtype=torch.float64, device=q.device)
        return z, torch.full((n,), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros(n, device=q.device)
    x = scale * (q @ K.T)
    if seen is not None:
        x = x.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(x, -1)
    empty = torch.isinf(lse)
    p = torch.exp(x - lse.masked_fill(empty, 0)[:, None]).masked_fill(empty[:, None], 0)
    out, A = p @ V, p @ V.abs()
    size = scale * (q.abs() @ K.abs().T)
    if seen is not None:
        size = size.masked_fill(~seen, 0)
    e = (d + 3) * 2.0 ** -24 * size.amax(-1) + 2.0 ** -20
    tol = U * (1 + U) * out.abs() + (U + 4 * e[:, None]) * (1 + U) * A + 1e-30
    return out, lse, tol, e + 2.0 ** -20 * (1 + lse.masked_fill(empty, 0).abs())


def merge64(out, lse, tol, ltol, own_out, own_lse):
    """out and lse merged with a request's own; its own terms are exact inputs."""
    w = own_lse.double()
    both = torch.logaddexp(lse, w)
    none = torch.isinf(both) & (both < 0)
    a = torch.exp(lse - both.masked_fill(none, 0)).masked_fill(none, 0)
    b = torch.exp(w - both.masked_fill(none, 0)).masked_fill(none, 0)
    o2 = own_out.double().masked_fill((b == 0)[:, None], 0)
    m = out * a[:, None] + o2 * b[:, None]
    # the weights a, b move by a factor e^(2 ltol); the output is rounded once more
    t = tol * a[:, None] + 4 * ltol[:, None] * ((out * a[:, None]).abs() + (o2 * b[:, None]).abs()) + U * (1 + U) * m.abs()
    return m, both, t + 1e-30, ltol + 2.0 ** -20 * (1 + both.masked_fill(none, 0).abs())


def check(out, lse, ref, what=""):
    """out bf16, lse float32 (or None) against (out, lse, out bound, lse bound)."""
    r, l, t, lt = ref
    d = (out.double() - r).abs()
    assert torch.isfinite(out).all(), f"{what}: non-finite output"
    assert bool((d <= t).all()), f"{what}: off by {(d / t).max().item():.3g} of its bound"
    if lse is not None:
        none = torch.isinf(l)
        assert torch.equal(none, torch.isinf(lse)), f"{what}: empty rows differ"
        dl = (lse.double() - l).masked_fill(none, 0).abs()
        assert bool((dl <= lt).all()), f"{what}: lse off by {dl.max().item():.3g}"


def seen_keys(nq, nk, window, device):
    """Causal (and windowed) mask of the last nq of nk positions."""
    pos = torch.arange(nk - nq, nk, device=device)[:, None]
    key = torch.arange(nk, device=device)[None]
    m = key <= pos
    return m & (key > pos - window) if window else m


def rope64(qkv, table_rows, H_q, H, q_weight, k_weight, eps, pairs, rot):
    """qkv [n][H_q + 2H][d], table_rows [n][rot/2][2] -> (heads [n][H_q + 2H][d], bound), float64.
    The norm is off by (d/2 + 8) 2^-24 relative, the turn by two roundings more, then bf16."""
    x = qkv.double().clone()
    d = x.shape[-1]
    for lo, hi, w in ((0, H_q, q_weight), (H_q, H_q + H, k_weight)):
        if w is not None:
            y = x[:, lo:hi]
            x[:, lo:hi] = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    z, size = x.clone(), x.abs()
    if rot:
        c, s = table_rows.double()[:, None, :, 0], table_rows.double()[:, None, :, 1]
        i = torch.arange(rot // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        k = H_q + H
        z[:, :k, a] = x[:, :k, a] * c - x[:, :k, b] * s
        z[:, :k, b] = x[:, :k, b] * c + x[:, :k, a] * s
        both = size[:, :k, a] + size[:, :k, b]
        size[:, :k, a] = both
        size[:, :k, b] = both
    tol = U * z.abs() + (d / 2 + 12) * 2.0 ** -24 * 2 * size * (1 + U) + 1e-38
    tol[:, H_q + H:] = 0
    return z, tol
