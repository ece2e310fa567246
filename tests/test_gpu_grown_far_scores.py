"""tg_decode_grown where scores are so far apart that one token, or two equal ones, take all the weight."""
import numpy as np
import pytest
import torch

from pages4_helpers import rows_of
from test_gpu_grown import Lists

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "e2m1"]


def _rows(x, b, p, n):
    l = b * (x.H // x.H_p) + p // x.H_p
    ids = x.ids[x.off[l]:x.off[l + 1]]
    pool = x.pool.view(x.n, -1) if x.four else x.pool
    return [rows_of(pool, ids, x.H_p, x.P, x.d, p % x.H_p, n, bool(i), x.units[i]) for i in (0, 1)]


def _sure(q, K, scale):
    """Scores [g][n] in 64 bits, and how far float32 (and f16 queries of 4-bit pages) may take each of them."""
    s = scale * (q @ K.T)
    e = (q.shape[1] + 3) * 2.0 ** -24 * scale * (q.abs() @ K.abs().T).amax(-1) + 2.0 ** -22 * s.abs().amax(-1)
    return s, e + 2.0 ** -25 * scale * q.abs().amax(-1) * K.abs().sum(-1).amax()


def _compare(out, lse, want, best, e, four):
    """The output is the value within its rounding and, of 4-bit pages, a weight's to f16."""
    tol = (2.0 ** -8 + (2.0 ** -11 if four else 2.0 ** -14)) * (1 + 2.0 ** -8) * want.abs() + 1e-12
    assert bool(((out.double() - want).abs() <= tol).all())
    assert abs(float(lse) - float(best)) <= float(e) + 2.0 ** -20 * (1 + abs(float(best)))


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("power", [16, 24, 26, 28, 29, 30, 31, 32, 40, 90])
def test_the_winner_takes_all(lib, cuda, pages, d, power):
    g = 8
    x = Lists(cuda, pages, [[200, 77], [33, 600]], 2 * g, d, reserve=0, n_cta=5, hostile=False, seed=power)
    x.q *= 2.0 ** power
    out, lse, status = x.run([0, 0])
    assert status == 0
    clear = 0
    for b in range(2):
        for p in range(2):
            h = int(x.order[p])
            K, V = _rows(x, b, p, x.tokens(b, h, 0))
            s, e = _sure(x.q[b, h * g:(h + 1) * g].double(), K, x.scale)
            top = s.topk(2, -1)
            for i in range(g):
                if float(top.values[i, 0] - top.values[i, 1]) < 4 * float(e[i]) + 40:
                    continue  # too near a tie for float32 to tell
                clear += 1
                _compare(out[b, h * g + i], lse[b, h * g + i], V[top.indices[i, 0]], top.values[i, 0], e[i], x.four)
    assert clear >= 16


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("power", [4, 27, 29, 31, 60])
@pytest.mark.parametrize("apart", [1, 7, 17, 40, 500])
def test_two_equal_winners_share_the_weight(lib, cuda, pages, power, apart):
    """The winner's key twice: in one step, in another warp's, in another block's."""
    n, g, d = 700, 4, 128
    x = Lists(cuda, pages, [[n]], g, d, reserve=0, n_cta=3, hostile=False, seed=power)
    x.q[0] = x.q[0, 0]
    x.q *= 2.0 ** power
    K, V = _rows(x, 0, 0, n)
    s, e = _sure(x.q[0].double(), K, x.scale)
    w = int(s[0].argmax())
    to = (w + apart) % n
    for t in (w, to):  # (page, tile of 16 tokens, row)
        page, r = int(x.ids[t // 16]), t % 16
        if not x.four:
            row = x.pool[page, 0, 0, r]
            kept = row.clone() if t == w else row.copy_(kept)
        else:
            row = x.pool[page, 0, 0, 0]
            if t == w:
                kept = row[64 * r:64 * r + 64].clone(), row[2048 + 8 * r:2056 + 8 * r].clone()
            else:
                row[64 * r:64 * r + 64], row[2048 + 8 * r:2056 + 8 * r] = kept
    s[:, to] = s[:, w]
    third = s[0].sort(descending=True).values[2]
    out, lse, status = x.run([0])
    assert status == 0
    if float(s[0, w] - third) < 4 * float(e[0]) + 40:
        assert power == 4  # (moderate scores: the same inputs, compared with the whole softmax)
        return x.compare(out, lse, [0])
    for i in range(g):
        both = (V[w] + V[to]) / 2
        # (of unlike values the two roundings of weights are of |v|, not of their sum)
        tol = 2.0 ** -8 * both.abs() + (2.0 ** -11 if x.four else 2.0 ** -14) * (V[w].abs() + V[to].abs()) + 1e-12
        assert bool(((out[0, i].double() - both).abs() <= tol).all())
