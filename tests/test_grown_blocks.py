"""How many blocks of threads a decode over grown lists is planned for (host only)."""
import numpy as np
import pytest

FULL = 152


def _items(lib, ntok, H_q, H_p, n_cta):
    """The most items that one block of the plan has."""
    L, batch, H = ntok.shape
    order = np.tile(np.arange(H, dtype=np.int32), (L, 1))
    Phi = ntok.astype(np.int64).sum(1).reshape(L, -1, H_p).sum(2)
    plan, _ = lib.tg_plan_decode(lib.tg_split_map(Phi, n_cta), order, ntok, H_q, H_p, 16, 128)
    return max(int(np.diff(lib.plan_items(plan, l)[0]).max()) for l in range(L))


@pytest.mark.parametrize("batch,low,high,reserve,blocks", [(32, 1, 8, 1, 128), (64, 6, 20, 8, FULL), (32, 5, 16, 8, 128), (32, 64, 64, 16, 128),
                                                           (8, 8, 64, 16, 32), (2, 30, 60, 16, 8), (40, 64, 64, 0, FULL)])
@pytest.mark.parametrize("H_p", [1, 4])
def test_many_short_lists_are_spread(lib, batch, low, high, reserve, blocks, H_p):
    """A block takes its lists one after the other.  It has an even share of a group's tokens, end to end: at most as many
    whole lists of the shortest kind as fit in it, and a piece at either end."""
    from non_uniform_paged_gb300.ragged import _grown_blocks
    most = np.random.default_rng(batch).integers(low, high + 1, (2, batch, 8)).astype(np.int32) + reserve
    n = _grown_blocks(most.astype(np.int64), H_p, FULL)
    assert n == blocks
    share = 1.2 * most.sum((1, 2)).max() / n  # (a group's blocks are a whole number: 1.2 covers that here)
    assert _items(lib, most, 32, H_p, n) <= share / (low + reserve) + 2 <= 2.4 * 8 * batch / n * (high + reserve) / (low + reserve) + 2


def test_few_long_lists_go_by_tokens(lib):
    from non_uniform_paged_gb300.ragged import _grown_blocks
    for tokens, want in ((125, 8), (2500, 79), (9250, FULL), (36250, FULL)):
        assert _grown_blocks(np.full((1, 1, 8), tokens, np.int64), 1, FULL) == want
    assert _grown_blocks(np.zeros((1, 1, 8), np.int64), 4, FULL) == 4
    assert _grown_blocks(np.full((3, 2, 8), 30, np.int64), 2, FULL) == 8
    assert _grown_blocks(np.full((1, 1000, 8), 30, np.int64), 1, FULL) == FULL
