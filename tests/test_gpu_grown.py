"""tg_decode_grown over pages of both formats against the 64-bit definition."""
import math

import numpy as np
import pytest
import torch

from pages4_helpers import attend64, rows_of, tile_bytes

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "e2m1"]


class Lists:
    """Random pages of grown lists and the owner of their plan."""

    def __init__(self, cuda, pages, ntok, H_q, d, H_p=1, P=16, reserve=0, n_cta=None, seed=0, units=(1.0, 1.0), hostile=True):
        from non_uniform_paged_gb300.ragged import GrowingLists
        g = torch.Generator(device=cuda).manual_seed(seed)
        ntok = np.asarray(ntok, np.int32)
        batch, H = ntok.shape
        self.order = np.random.default_rng(seed).permutation(H).astype(np.int32)
        self.ntok_h, self.H, self.H_q, self.d, self.H_p, self.P, self.reserve, self.units = ntok, H, H_q, d, H_p, P, reserve, units
        self.batch, self.cuda, self.four = batch, cuda, pages == "e2m1"
        counts = [-(-(max(int(ntok[b, h]) for h in self.order[i:i + H_p]) + reserve) // P)
                  for b in range(batch) for i in range(0, H, H_p)]
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        self.off, self.n = torch.from_numpy(off).to(cuda), max(1, int(off[-1]))
        self.ids = torch.randperm(self.n, generator=g, device=cuda).to(torch.int32)
        self.lists = GrowingLists(H_q, H_p, P, d, self.order, ntok, reserve, pages=pages, k_unit=units[0], v_unit=units[1],
                                  n_cta=n_cta, device=cuda)
        if self.four:
            self.pool = torch.randint(0, 256, (self.n, H_p, P // 16, d // 128, 2304), generator=g, device=cuda, dtype=torch.uint8)
            self.pool[..., 2048:] = self.pool[..., 2048:] % 0x28 + 0x18
        else:
            self.pool = torch.randn((self.n, H_p, 2, P, d), generator=g, device=cuda).to(torch.bfloat16)
        self.hostile = hostile
        self.q = (torch.randn((batch, H_q, d), generator=g, device=cuda) * 1.5).to(torch.bfloat16)
        self.scale = 1.0 / math.sqrt(d)

    def tokens(self, b, h, extra):
        return int(self.ntok_h[b, h]) + extra

    def _behind(self, extra):
        """A copy of the pool whose rows behind the last token of every head are NaN (4 bits: NaN scales and -6)."""
        pool = self.pool.clone()
        G = self.H // self.H_p
        for b in range(self.batch):
            for p in range(self.H):
                n = self.tokens(b, int(self.order[p]), extra[b])
                l = b * G + p // self.H_p
                ids = self.ids[self.off[l]:self.off[l + 1]].long()
                if not ids.numel():
                    continue
                r = torch.arange(n, ids.numel() * self.P, device=self.cuda)
                page, row = ids[r // self.P], r % self.P
                if not self.four:
                    pool[page, p % self.H_p, :, row] = float("nan")
                    continue
                tile = pool[page, p % self.H_p, row // 16]  # gathered, changed in one row each, and put back one by one
                flat = pool.view(-1)
                base = ((page * self.H_p + p % self.H_p) * (self.P // 16) + row // 16) * tile_bytes(self.d)
                for half in range(self.d // 128):
                    t, j = (row % 16)[:, None], torch.arange(8, device=self.cuda)
                    at = base[:, None] + half * 2304
                    flat[(at + 2048 + 8 * t + j).flatten()] = 0x7f
                    flat[(at + 2176 + 16 * j + t).flatten()] = 0x7f
                    byte = torch.arange(64, device=self.cuda)
                    flat[(at + 64 * t + byte).flatten()] = 0xff
                    flat[(at + 1024 + 512 * (t // 8) + 8 * (t % 8) + 64 * (byte // 8) + byte % 8).flatten()] = 0xff
                del tile
        return pool

    def run(self, added, plus=0, pool=None, stream=None):
        self.lists.added.copy_(torch.tensor(added, dtype=torch.int32))
        out = torch.full((self.batch, self.H_q, self.d), float("nan"), dtype=torch.bfloat16, device=self.cuda)
        lse = torch.full((self.batch, self.H_q), float("nan"), device=self.cuda)
        extra = [a + plus for a in added]
        pool = pool if pool is not None else self._behind(extra) if self.hostile else self.pool
        self.lists.attend(0, self.q, pool, self.n, self.off, self.ids, out, lse=lse, plus=plus, stream=stream)
        torch.cuda.synchronize()
        return out, lse, int(self.lists.status)

    def check(self, lib, added, plus=0):
        out, lse, status = self.run(added, plus)
        assert status == 0
        self.compare(out, lse, [a + plus for a in added])
        return out, lse

    def compare(self, out, lse, extra, requests=None):
        g, G = self.H_q // self.H, self.H // self.H_p
        for b in range(self.batch) if requests is None else requests:
            for p in range(self.H):
                h = int(self.order[p])
                n, l = self.tokens(b, h, extra[b]), b * G + p // self.H_p
                ids = self.ids[self.off[l]:self.off[l + 1]]
                K, V = (rows_of(self.pool.view(self.n, -1) if self.four else self.pool, ids, self.H_p, self.P, self.d, p % self.H_p,
                                n, bool(i), self.units[i]) for i in (0, 1))
                at = slice(h * g, (h + 1) * g)
                r, le, t, lt = attend64(self.q[b, at], K, V, self.scale, self.four)
                if n == 0:
                    assert not out[b, at].any() and bool(torch.isneginf(lse[b, at]).all()), (b, h)
                    continue
                d = (out[b, at].double() - r).abs()
                assert bool(torch.isfinite(out[b, at]).all()) and bool((d <= t).all()), (b, h, (d / t).max().item())
                dl = (lse[b, at].double() - le).abs()
                assert bool((dl <= lt).all()), (b, h, (dl / lt).max().item())


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_cta", [1, 2, 5, 40, 152, 600])
def test_many_splits(lib, cuda, pages, d, n_cta):
    """Pieces of every size, most of them cut inside a tile; rows behind the last token hold NaN."""
    ntok = [[700, 33, 16, 1], [0, 5, 250, 15], [17, 128, 64, 0]]
    x = Lists(cuda, pages, ntok, 8, d, H_p=2 if n_cta > 1 else 4, reserve=40, n_cta=n_cta)
    for added, plus in (([0, 0, 0], 0), ([0, 0, 0], 1), ([7, 39, 20], 1), ([40, 0, 13], 0)):
        x.check(lib, added, plus)


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
def test_query_heads(lib, cuda, pages, d, g):
    x = Lists(cuda, pages, [[300, 90], [64, 47]], 2 * g, d, reserve=9, n_cta=9)
    x.check(lib, [3, 8], 1)


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("P,H_p", [(16, 3), (48, 1), (64, 3), (128, 3)])
def test_page_sizes_and_groups(lib, cuda, pages, P, H_p):
    x = Lists(cuda, pages, [[300, 90, 1], [64, 147, 13]], 6, 128, H_p=H_p, P=P, reserve=30, n_cta=11)
    x.check(lib, [0, 29], 1)


@pytest.mark.parametrize("pages", FORMATS)
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 48])
def test_lengths_about_a_tile(lib, cuda, pages, n):
    x = Lists(cuda, pages, [[0]], 4, 128, reserve=48, n_cta=3)
    x.check(lib, [n])
    if n:
        x.check(lib, [n - 1], 1)


@pytest.mark.parametrize("pages", FORMATS)
def test_a_run_that_grows_from_nothing_far_past_its_start(lib, cuda, pages):
    """A reserve much longer than what was retained: every length is split over all blocks of threads alike."""
    x = Lists(cuda, pages, [[3, 0]], 8, 128, reserve=5000, n_cta=64, hostile=False)
    for n in (0, 1, 64, 100, 1000, 4999, 5000):
        x.check(lib, [n])


@pytest.mark.parametrize("pages", FORMATS)
def test_more_items_than_shared_memory_keeps(lib, cuda, pages):
    x = Lists(cuda, pages, [[(37 * b + 11 * h) % 150 for h in range(4)] for b in range(24)], 8, 128, H_p=2, reserve=3, n_cta=2)
    off, _ = lib.plan_items(x.lists.plan._host, 0)
    assert np.diff(off).max() > 16
    x.check(lib, [b % 3 for b in range(24)], 1)


@pytest.mark.parametrize("pages", FORMATS)
def test_more_parts_than_the_factor_buffer(lib, cuda, pages):
    x = Lists(cuda, pages, [[4000]], 8, 128, reserve=200, n_cta=300, hostile=False)
    x.check(lib, [0])
    x.check(lib, [150], 1)


@pytest.mark.parametrize("d", [128, 256])
def test_extremes_of_queries_and_scales(lib, cuda, d):
    """Queries far outside f16, of one large value, and of zeros; the smallest and largest block scales; units."""
    x = Lists(cuda, "e2m1", [[200, 77]], 16, d, reserve=0, n_cta=5, units=(2.0 ** -9, 2.0 ** 5))
    x.pool[..., 2048:2176] = torch.randint(0, 127, x.pool[..., 2048:2176].shape, device=cuda, dtype=torch.uint8,
                                           generator=torch.Generator(device=cuda).manual_seed(1))
    x.q[0, 1] *= 2.0 ** 30
    x.q[0, 2] *= 2.0 ** -40
    x.q[0, 3] = 0
    x.q[0, 4, 1:] *= 2.0 ** -20
    x.q[0, 5] *= 2.0 ** -126
    x.scale = x.lists.scale = 2.0 ** -4
    q = x.q.clone()
    x.q[0, 1] = q[0, 0]
    x.check(lib, [0])
    # a head of scores far apart: one token takes all the weight
    x.q = q
    out, lse, status = x.run([0])
    assert status == 0 and bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("pages", FORMATS)
def test_weights_far_below_the_largest_still_count(lib, cuda, pages):
    """One token far above 60000 equal ones that together weigh as much: their weights are 2^-16 each."""
    n, d = 60001, 128
    x = Lists(cuda, pages, [[n]], 1, d, n_cta=8, hostile=False)
    x.pool.zero_()
    if pages == "e2m1":
        x.pool[..., 2048:] = 56  # scale 1
        x.pool[..., :1024] = 0
        x.pool[..., 1024:2048] = 0x22  # V = 1
        first = int(x.ids[0])
        x.pool[first, 0, 0, 0, 0] = 0x07  # K of token 0: 6 in value 0
        x.pool[first, 0, 0, 0, 1024:1024 + 512:64] = 0xaa  # V of token 0: -1 in every block's first two values
    else:
        x.pool[:, :, 1] = 1.0
        x.pool[int(x.ids[0]), 0, 0, 0, 0] = 6.0
        x.pool[int(x.ids[0]), 0, 1, 0, ::16] = -1.0
        x.pool[int(x.ids[0]), 0, 1, 0, 1::16] = -1.0
    x.q.zero_()
    x.q[0, 0, 0] = math.log(60000.0) / 6 / x.scale
    out, lse = x.check(lib, [0])
    assert abs(float(out[0, 0, 0])) < 0.02 and abs(float(out[0, 0, 2]) - 1) < 0.01


@pytest.mark.parametrize("pages", FORMATS)
def test_counts_outside_the_reserve_are_reported_and_clamped(lib, cuda, pages):
    x = Lists(cuda, pages, [[20], [30]], 2, 128, reserve=10, n_cta=4, hostile=False)
    for added, plus, extra in (([11, 3], 0, [10, 3]), ([10, 3], 1, [10, 4]), ([-5, 3], 0, [0, 3]), ([2 ** 31 - 1, 3], 7, [10, 10]),
                               ([-2 ** 31, 3], 0, [0, 3])):
        x.lists.status.zero_()
        out, lse, status = x.run(added, plus)
        assert status == lib.STATUS_BAD_INPUT
        x.compare(out, lse, extra)


@pytest.mark.parametrize("pages", FORMATS)
def test_counts_that_are_not_the_plans_stay_in_the_lists(lib, cuda, pages):
    """Device counts other than those planned for: nothing outside the lists is read, the other requests are right."""
    x = Lists(cuda, pages, [[100], [100], [100]], 2, 128, reserve=10, n_cta=5, hostile=False)
    kept = x.lists.ntok[0].clone()
    for wrong, status in ((-7, 0), (2 ** 31 - 1, None), (0, 0), (95, 0)):
        x.lists.status.zero_()
        x.lists.ntok[0][1, 0] = wrong
        out, lse, got = x.run([3, 4, 5])
        assert got in ((0, lib.STATUS_BAD_PAGE) if status is None else (status,))
        x.compare(out, lse, [3, 4, 5], requests=[0, 2])
    x.lists.ntok[0].copy_(kept)
    x.lists.status.zero_()
    x.check(lib, [1, 2, 3])


@pytest.mark.parametrize("pages", FORMATS)
def test_bad_pages_are_reported_and_the_others_are_right(lib, cuda, pages):
    x = Lists(cuda, pages, [[100], [100], [100]], 2, 128, reserve=10, n_cta=5, hostile=False)
    ids = x.ids.clone()
    x.ids = ids.clone()
    x.ids[int(x.off[1]) + 2] = x.n
    out, lse, status = x.run([0, 0, 0])
    assert status == lib.STATUS_BAD_PAGE
    x.ids = ids
    x.compare(out, lse, [0, 0, 0], requests=[0, 2])
    x.lists.status.zero_()
    off = x.off.clone()
    x.off = off.clone()
    x.off[2:] -= 3  # request 1's list is too short, request 2's table begins three pages early
    out, lse, status = x.run([0, 0, 0])
    assert status == lib.STATUS_BAD_PAGE
    x.off = off
    x.compare(out, lse, [0, 0, 0], requests=[0])
    # the workspace is as good as before
    x.lists.status.zero_()
    x.check(lib, [1, 2, 3])


@pytest.mark.parametrize("pages", FORMATS)
def test_pages_past_32_bits(lib, cuda, pages):
    many = 2_000_000 if pages == "e2m1" else 600_000
    x = Lists(cuda, pages, [[40]], 4, 128, reserve=8, n_cta=2, hostile=False)
    pool = torch.empty((many,) + tuple(x.pool.shape[1:]), dtype=x.pool.dtype, device=cuda)
    pool[-x.n:] = x.pool
    out = torch.empty((1, 4, 128), dtype=torch.bfloat16, device=cuda)
    lse = torch.empty((1, 4), device=cuda)
    x.lists.attend(0, x.q, pool, many, x.off, x.ids + (many - x.n), out, lse=lse, plus=5)
    x.compare(out, lse, [5])


@pytest.mark.parametrize("pages", FORMATS)
def test_a_captured_step_grows_with_its_replays_and_two_callers_share_nothing(lib, cuda, pages):
    """attend and advance in one graph, replayed: each replay sees one token more; another caller with a workspace of
    its own runs on a second stream meanwhile; the bits are those of eager calls."""
    x = Lists(cuda, pages, [[50, 3], [0, 200]], 8, 128, H_p=2, reserve=20, n_cta=12, hostile=False)
    y = Lists(cuda, pages, [[150, 31], [10, 20]], 8, 128, H_p=2, reserve=20, n_cta=12, hostile=False, seed=1)
    refs = [x.run([i, i], 1)[:2] for i in range(6)]
    ref_y = y.run([4, 0], 1)[:2]
    out, lse = torch.empty_like(refs[0][0]), torch.empty_like(refs[0][1])
    oy, ly = torch.empty_like(out), torch.empty_like(lse)
    x.lists.added.zero_()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=a):
        x.lists.attend(0, x.q, x.pool, x.n, x.off, x.ids, out, lse=lse)
        x.lists.advance()
    torch.cuda.synchronize()
    x.lists.added.zero_()
    for i in range(6):
        with torch.cuda.stream(a):
            graph.replay()
        for _ in range(3):
            y.lists.attend(0, y.q, y.pool, y.n, y.off, y.ids, oy, lse=ly, stream=b)
        torch.cuda.synchronize()
        assert torch.equal(out, refs[i][0]) and torch.equal(lse, refs[i][1]), i
        assert torch.equal(oy, ref_y[0]) and torch.equal(ly, ref_y[1])
    assert x.lists.added.tolist() == [6, 6]


@pytest.mark.parametrize("pages", FORMATS)
def test_calls_one_after_the_other_reuse_the_workspace(lib, cuda, pages):
    x = Lists(cuda, pages, [[900, 33], [5, 250]], 8, 128, H_p=1, reserve=40, n_cta=60, hostile=False)
    ref = x.run([11, 12], 1)
    x.run([0, 40])
    for _ in range(5):
        out, lse, status = x.run([11, 12], 1)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1]) and status == 0


def test_binding_refusals(lib, cuda):
    from non_uniform_paged_gb300.ragged import GrowingLists
    x = Lists(cuda, "e2m1", [[20, 3], [30, 1]], 4, 128, H_p=2, reserve=10, n_cta=4, hostile=False)
    out = torch.zeros_like(x.q)
    args = dict(layer=0, q=x.q, pool=x.pool, pool_pages=x.n, pt_off=x.off, pt_ids=x.ids, out=out)
    for bad in (dict(q=x.q[:1]), dict(out=out[:, :1].contiguous()), dict(pool_pages=x.n + 1), dict(pt_off=x.off[:1]),
                dict(lse=torch.zeros(3, device=cuda)), dict(pool=x.pool.transpose(0, 1)), dict(cta_time=torch.zeros(2, dtype=torch.int64, device=cuda))):
        with pytest.raises(ValueError):
            x.lists.attend(**dict(args, **bad))
    for bad in (dict(q=x.q.float()), dict(pool=x.pool.view(torch.int8)), dict(pt_ids=x.ids.long()), dict(out=out.cpu())):
        with pytest.raises(TypeError):
            x.lists.attend(**dict(args, **bad))
    for bad in (dict(plus=-1), dict(plus=11), dict(scale=float("inf"))):
        with pytest.raises(lib.TGError):
            x.lists.attend(**dict(args, **bad))
    with pytest.raises(IndexError):
        x.lists.attend(**dict(args, layer=1))
    assert not out.any()
    with pytest.raises(ValueError):
        GrowingLists(4, 2, 16, 128, x.order, x.ntok_h, 10, pages="int4", device=cuda)
    with pytest.raises(ValueError):
        GrowingLists(4, 2, 16, 128, x.order, x.ntok_h, 2 ** 31 - 20, device=cuda)
    plan = x.lists.plan
    with pytest.raises(ValueError):
        lib.DecodePlan(plan._host[:100].copy(), plan.plan_dev[:100])
    with pytest.raises(ValueError):
        lib.DecodePlan(plan._host, plan.plan_dev[:-1])
