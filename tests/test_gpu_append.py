"""tg_append_rope against its 64-bit definition, over pages of both formats, and what it leaves alone."""
import numpy as np
import pytest
import torch

from pages4_helpers import hold, read_tiles, tile_bytes
from prompt_helpers import rope64

pytestmark = pytest.mark.gpu


def _table(max_pos, rot, cuda, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=cuda) / max(rot, 1))
    a = torch.arange(max_pos, dtype=torch.float64, device=cuda)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


class Case:
    """Inputs of one call, the call, and the comparison with the definition."""

    def __init__(self, cuda, fmt, lens, kept, H_q, H, d, H_p=1, P=16, rot=None, pairs=False, qw=True, kw=True, axes=1, added=None,
                 reserve=None, dense=False, pad=0, extra=0, units=(1.0, 1.0), positions=None, max_pos=600, seed=0, values=None):
        g = torch.Generator(device=cuda).manual_seed(seed)
        self.cuda, self.fmt, self.lens, self.H_q, self.H, self.d, self.H_p, self.P = cuda, fmt, lens, H_q, H, d, H_p, P
        self.rot, self.pairs, self.axes, self.pad, self.units = d if rot is None else rot, pairs, axes, pad, units
        batch, T, heads = len(lens), sum(lens) + pad, H_q + 2 * H
        wide = torch.randn((T, heads * d + extra), generator=g, device=cuda).to(torch.bfloat16) if values is None else values
        self.qkv = wide[:, :heads * d].view(T, heads, d)
        self.w = [torch.randn(d, generator=g, device=cuda) if on else None for on in (qw, kw)]
        self.cu = torch.tensor([sum(lens[:i]) for i in range(batch + 1)], dtype=torch.int32, device=cuda)
        self.added = torch.tensor([0] * batch if added is None else added, dtype=torch.int32, device=cuda)
        self.reserve = (max(self.added.tolist()) + max(lens + [1])) if reserve is None else reserve
        self.order = torch.randperm(H, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        kept = np.asarray(kept, np.int32).reshape(batch, H)
        self.ntok = torch.from_numpy(kept).to(cuda)
        counts = [-(-(max(int(kept[b, h]) for h in self.order[i:i + H_p]) + self.reserve) // P)
                  for b in range(batch) for i in range(0, H, H_p)]
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int64, device=cuda)
        self.pages = int(self.off[-1])
        self.ids = torch.randperm(self.pages, generator=g, device=cuda).to(torch.int32)
        self.table = _table(max_pos, self.rot, cuda) if self.rot else None
        self.origin = torch.randint(0, 300, (batch,), generator=g, device=cuda).to(torch.int32)
        self.axis_of = torch.randint(0, axes, (self.rot // 2,), generator=torch.Generator().manual_seed(seed)).tolist()
        self.positions = torch.randint(0, max_pos, (T, axes), generator=g, device=cuda).to(torch.int32) if axes > 1 else \
            None if positions is None else torch.tensor(positions, dtype=torch.int32, device=cuda)
        self.mark = 7.0
        self.q = torch.full((T, H_q, d), self.mark, dtype=torch.bfloat16, device=cuda)
        self.pool = torch.full((self.pages, H_p, 2, P, d), self.mark, dtype=torch.bfloat16, device=cuda) if fmt == 0 else \
            torch.full((self.pages, H_p, P // 16, tile_bytes(d)), 0x5b, dtype=torch.uint8, device=cuda)
        self.start = torch.randint(0, 5, (batch,), generator=g, device=cuda).to(torch.int32) if dense else None
        self.Nmax = max(lens + [1]) + 5
        self.K = torch.full((batch, H, self.Nmax, d), self.mark, dtype=torch.bfloat16, device=cuda) if dense else None
        self.V = self.K.clone() if dense else None
        self.status = torch.zeros(1, dtype=torch.int32, device=cuda)

    def call(self, lib, **change):
        a = dict(qkv=self.qkv, cu_q=self.cu, cos_sin=self.table, q=self.q, pool=self.pool, pool_pages=self.pages,
                 head_order=self.order.to(self.cuda), ntok=self.ntok, added=self.added, reserve=self.reserve, pt_off=self.off,
                 pt_ids=self.ids, H_p=self.H_p, P=self.P, fmt=self.fmt, k_unit=self.units[0], v_unit=self.units[1],
                 q_weight=self.w[0], k_weight=self.w[1], pairs=self.pairs, positions=self.positions,
                 axis_of=self.axis_of if self.axes > 1 else None, origin=self.origin, K=self.K, V=self.V, start=self.start,
                 dev_status=self.status)
        a.update(change)
        lib.tg_append_rope(**a)
        torch.cuda.synchronize()
        return int(self.status)

    def call_and_verify(self, lib):
        assert self.call(lib) == 0
        self.verify()

    def _rows(self, b, at, n):
        """Table rows [n][rot/2][2] of request b's tokens."""
        if not self.rot:
            return None
        pair = torch.arange(self.rot // 2, device=self.cuda)
        if self.axes > 1:
            pos = self.positions[at:at + n].long()[:, torch.tensor(self.axis_of, device=self.cuda)]
        elif self.positions is not None:
            pos = self.positions[at:at + n].long()[:, None].expand(n, pair.numel())
        else:
            pos = (int(self.origin[b]) + int(self.added[b]) + torch.arange(n, device=self.cuda))[:, None].expand(n, pair.numel())
        return self.table[pos, pair]

    def verify(self):
        H_q, H, d, H_p, P, G = self.H_q, self.H, self.d, self.H_p, self.P, self.H // self.H_p
        before = 0x5b if self.fmt else self.mark
        touched = torch.zeros((self.pages, H_p, P), dtype=torch.bool, device=self.cuda)
        at = 0
        for b, n in enumerate(self.lens):
            if not n:
                continue
            ref, tol = rope64(self.qkv[at:at + n], self._rows(b, at, n), H_q, H, self.w[0], self.w[1], 1e-6, self.pairs, self.rot)
            dq = (self.q[at:at + n].double() - ref[:, :H_q]).abs()
            assert bool((dq <= tol[:, :H_q]).all()), (b, (dq / tol[:, :H_q].clamp_min(1e-30)).max().item())
            for p in range(H):
                h = int(self.order[p])
                slot = int(self.ntok[b, h]) + int(self.added[b]) + torch.arange(n, device=self.cuda)
                page = self.ids[self.off[b * G + p // H_p] + slot // P].long()
                touched[page, p % H_p, slot % P] = True
                for i in (0, 1):
                    col = H_q + i * H + h
                    if self.fmt == 0:
                        got = self.pool[page, p % H_p, i, slot % P].double()
                        err = (got - ref[:, col]).abs()
                        assert bool((err <= tol[:, col]).all()), (b, h, i, (err / tol[:, col].clamp_min(1e-30)).max().item())
                    else:
                        raw = self.pool[page, p % H_p, slot % P // 16]
                        got = read_tiles(raw, d, self.units[i], bool(i))[0][torch.arange(n, device=self.cuda), slot % 16]
                        want = hold(ref[:, col], self.units[i])[0]
                        assert torch.equal(got, want), (b, h, i, int((got != want).sum()))
                    if self.K is not None:
                        row = (self.K, self.V)[i][b, h, int(self.start[b]):int(self.start[b]) + n].double()
                        assert torch.equal(row, got), (b, h, i)
            at += n
        assert bool((self.q[at:] == self.mark).all())
        if self.fmt == 0:
            assert bool((self.pool[~touched[:, :, None, :, None].expand_as(self.pool)] == before).all())
        else:
            for V in (False, True):  # the codes and scales of rows that no token is
                raw = self.pool.view(-1, tile_bytes(self.d))
                free = ~touched.view(-1, 16)
                was, sc = read_tiles(torch.full((1, tile_bytes(self.d)), 0x5b, dtype=torch.uint8, device=self.cuda), self.d, 1.0, V)
                now, sn = read_tiles(raw, self.d, 1.0, V)
                assert torch.equal(now[free], was.expand_as(now)[free]) and torch.equal(sn[free], sc.expand_as(sn)[free])
        if self.K is not None:
            for b, n in enumerate(self.lens):
                s = int(self.start[b])
                for x in (self.K, self.V):
                    assert bool((x[b, :, :s] == self.mark).all()) and bool((x[b, :, s + n:] == self.mark).all())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("H_q,H,H_p", [(8, 2, 2), (5, 1, 1), (6, 6, 3), (32, 8, 4)])
@pytest.mark.parametrize("rot_of,pairs", [(1, False), (1, True), (2, False), (2, True), (0, False)])
def test_against_definition(lib, cuda, fmt, d, H_q, H, H_p, rot_of, pairs):
    kept = [[(13 * b + 29 * h) % 70 for h in range(H)] for b in range(4)]
    c = Case(cuda, fmt, [1, 0, 37, 90], kept, H_q, H, d, H_p=H_p, rot=d // rot_of if rot_of else 0, pairs=pairs, pad=3,
             added=[5, 0, 0, 40], dense=True)
    assert c.call(lib) == 0
    c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("rot", [16, 48, 112])
@pytest.mark.parametrize("pairs", [False, True])
def test_odd_rotations_and_pages(lib, cuda, fmt, rot, pairs):
    c = Case(cuda, fmt, [9, 40], [[3], [100]], 3, 1, 128, rot=rot, pairs=pairs, P=48)
    assert c.call(lib) == 0
    c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("qw,kw,rot", [(False, False, 128), (False, False, 64), (True, False, 0), (False, True, 32)])
def test_norm_of_one_side_or_none(lib, cuda, fmt, qw, kw, rot):
    """Without a norm, values behind rot and turned by an angle of 0 are bf16 numbers: ties are common."""
    c = Case(cuda, fmt, [64, 19], [[0, 1], [2, 3]], 6, 2, 128, qw=qw, kw=kw, rot=rot, dense=True,
             positions=[0] * 40 + list(range(43)))
    assert c.call(lib) == 0
    c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("d,rot,pairs", [(128, 128, False), (128, 96, True), (256, 256, False), (256, 64, False)])
def test_positions_of_several_axes(lib, cuda, fmt, axes, d, rot, pairs):
    c = Case(cuda, fmt, [33, 2, 1], [[0, 31], [16, 7], [1, 1]], 4, 2, d, H_p=2, rot=rot, pairs=pairs, axes=axes)
    assert c.call(lib) == 0
    c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
def test_one_axis_as_a_column_and_positions_apart_from_slots(lib, cuda, fmt):
    pos = [5, 99, 0, 63, 64, 7]
    c = Case(cuda, fmt, [4, 2], [[10], [0]], 4, 1, 128, positions=pos, max_pos=100)
    assert c.call(lib) == 0
    c.verify()
    other = Case(cuda, fmt, [4, 2], [[10], [0]], 4, 1, 128, positions=pos, max_pos=100)
    other.call(lib, positions=c.positions[:, None].contiguous(), axis_of=None)
    assert torch.equal(c.pool, other.pool) and torch.equal(c.q, other.q)


@pytest.mark.parametrize("fmt", [0, 1])
def test_a_decode_step_of_many_requests_from_strided_rows(lib, cuda, fmt):
    kept = [[(7 * b + h) % 50 for h in range(2)] for b in range(200)]
    c = Case(cuda, fmt, [1] * 200, kept, 8, 2, 128, H_p=2, extra=24, added=[b % 33 for b in range(200)])
    assert c.call(lib) == 0
    c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
def test_more_tokens_than_one_warp_each_covers(lib, cuda, fmt):
    for H_q, H, d, T in ((33, 3, 128, 2100), (9, 1, 256, 2050), (1, 1, 256, 5)):
        c = Case(cuda, fmt, [T], [[17] * H], H_q, H, d, seed=T, max_pos=3000)
        assert c.call(lib) == 0
        c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T", [1, 270, 540, 1100, 1700, 2300, 4500])
def test_every_share_of_a_token_between_warps(lib, cuda, fmt, T):
    """From a warp for each batch of heads down to one or two for a token, over uneven numbers of batches."""
    lens = [T - T // 3, T // 3]
    Case(cuda, fmt, lens, [[1] * 5, [4] * 5], 35, 5, 128, rot=48, max_pos=4000, seed=T).call_and_verify(lib)


def test_units(lib, cuda):
    values = torch.randn((20, 6 * 128), device=cuda).to(torch.bfloat16)
    values[:, 5 * 128:] *= 2.0 ** -14  # V far below the smallest scale
    c = Case(cuda, 1, [20], [[5]], 4, 1, 128, units=(4.0, 2.0 ** -12), values=values, dense=True)
    assert c.call(lib) == 0
    c.verify()
    assert c.V[0, 0, int(c.start[0]):int(c.start[0]) + 20].any()


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("far", [1e2, 1e4, 1e6])
def test_a_pair_of_very_unlike_values(lib, cuda, far, pairs):
    """A value whose partner is far larger: what float32 leaves open is then wide against the block's scale."""
    values = torch.randn((300, 3 * 128), device=cuda, generator=torch.Generator(device=cuda).manual_seed(9)).to(torch.bfloat16)
    values[:, 128 + 64:256] *= far
    values[::3, 128:128 + 16] *= 1 / far
    c = Case(cuda, 1, [300], [[5]], 1, 1, 128, values=values, pairs=pairs, dense=True, qw=False)
    assert c.call(lib) == 0
    c.verify()


def test_values_that_are_not_finite_set_the_status(lib, cuda):
    """An infinite V value is held as the largest, a NaN as the block's +6; neighbours in other blocks are untouched."""
    values = torch.randn((3, 3 * 128), device=cuda).to(torch.bfloat16)
    values[0, 256 + 5], values[1, 256 + 37], values[2, 128 + 3] = float("inf"), float("nan"), float("nan")
    c = Case(cuda, 1, [3], [[0]], 1, 1, 128, rot=0, qw=False, kw=False, values=values, dense=True)
    assert c.call(lib) == lib.STATUS_NONFINITE
    s = int(c.start[0])
    want = hold(c.qkv[:, 1:].double())[0]
    assert torch.equal(c.K[0, 0, s:s + 3].double(), want[:, 0]) and torch.equal(c.V[0, 0, s:s + 3].double(), want[:, 1])
    # turned keys: what is not finite spreads to its pair, the rest of the row is what it is
    values = torch.randn((2, 3 * 128), device=cuda).to(torch.bfloat16)
    values[0, 128 + 3], values[1, 128 + 100] = float("inf"), float("nan")
    c = Case(cuda, 1, [2], [[0]], 1, 1, 128, qw=False, kw=False, values=values, dense=True, positions=[3, 5])
    assert c.call(lib) == lib.STATUS_NONFINITE
    ref, _ = rope64(c.qkv, c._rows(0, 0, 2), 1, 1, None, None, 1e-6, False, 128)
    s = int(c.start[0])
    assert torch.equal(c.K[0, 0, s:s + 2].double(), hold(ref[:, 1])[0])


@pytest.mark.parametrize("fmt", [0, 1])
def test_tokens_outside_the_limits_write_nothing(lib, cuda, fmt):
    def run(**how):
        change = how.pop("change", {})
        c = Case(cuda, fmt, [4], [[6]], 2, 1, 128, **how)
        return c, c.call(lib, **change)

    def written(c):
        return [bool((c.q[i] != c.mark).any()) for i in range(4)]

    c, status = run(reserve=2)  # tokens 2 and 3 pass the reserve
    assert status == lib.STATUS_BAD_INPUT and written(c) == [True, True, False, False]
    c, status = run(added=[-1])
    assert status == lib.STATUS_BAD_INPUT and written(c) == [False] * 4
    assert bool((c.pool == (0x5b if fmt else c.mark)).all())
    c, status = run(positions=[0, -1, 600, 599])
    assert status == lib.STATUS_BAD_INPUT and written(c) == [True, False, False, True]
    # tokens ahead of their request would be rows that it retained
    c, status = run(change={"cu_q": torch.tensor([2, 4], dtype=torch.int32, device=cuda)})
    assert status == lib.STATUS_BAD_INPUT and written(c) == [False, False, True, True]
    c, status = run(change={"cu_q": torch.tensor([4, 4], dtype=torch.int32, device=cuda)})
    assert status == lib.STATUS_BAD_INPUT and written(c) == [False] * 4
    assert bool((c.pool == (0x5b if fmt else c.mark)).all())
    c, status = run(dense=True, change={"start": torch.tensor([6], dtype=torch.int32, device=cuda)})  # rows 6 .. 9 of 9
    assert status == lib.STATUS_BAD_INPUT and written(c) == [True, True, True, False]
    c, status = run(axes=2)
    c = Case(cuda, fmt, [4], [[6]], 2, 1, 128, axes=2)
    c.positions[2, c.axis_of[0]] = 600
    assert c.call(lib) == lib.STATUS_BAD_INPUT and written(c) == [True, True, False, True]


@pytest.mark.parametrize("fmt", [0, 1])
def test_more_heads_than_places_looked_up_at_once(lib, cuda, fmt):
    """70 KV heads in groups of 5 and 14: three lookups of 32 places, with one warp a token and with several."""
    for H_p, T in ((5, 3), (14, 2100)):
        c = Case(cuda, fmt, [T], [[(7 * h) % 40 for h in range(70)]], 3, 70, 128, H_p=H_p, max_pos=3000, dense=T < 10, seed=T)
        assert c.call(lib) == 0
        c.verify()


@pytest.mark.parametrize("fmt", [0, 1])
def test_bad_pages_and_heads_are_reported_and_skipped(lib, cuda, fmt):
    before = 0x5b if fmt else 7.0
    c = Case(cuda, fmt, [2], [[3, 20]], 2, 2, 128)
    ids = c.ids.clone()
    first = int(c.order[0])
    at = int(c.off[0]) + int(c.ntok[0, first]) // 16
    page = int(ids[at])
    for bad in (-1, c.pages, 2 ** 31 - 1):
        ids[at] = bad
        assert c.call(lib, pt_ids=ids) == lib.STATUS_BAD_PAGE
        assert bool((c.pool[page] == before).all()) and bool((c.q != c.mark).any())
        c.status.zero_()
    short = c.off.clone()
    short[1:] = short[0]  # both lists are empty
    c = Case(cuda, fmt, [2], [[3, 20]], 2, 2, 128)
    assert c.call(lib, pt_off=short) == lib.STATUS_BAD_PAGE and bool((c.pool == before).all())
    c.status.zero_()
    assert c.call(lib, head_order=torch.tensor([2, -1], dtype=torch.int32, device=cuda)) == lib.STATUS_BAD_INPUT
    assert bool((c.pool == before).all())


@pytest.mark.parametrize("fmt", [0, 1])
def test_pages_past_32_bits(lib, cuda, fmt):
    many = 2_000_000 if fmt else 600_000
    c = Case(cuda, fmt, [3], [[15]], 1, 1, 128)
    pool = torch.empty((many,) + c.pool.shape[1:], dtype=c.pool.dtype, device=cuda)
    ids = torch.tensor([many - 1, many - 2], dtype=torch.int32, device=cuda)
    assert c.call(lib, pool=pool, pool_pages=many, pt_ids=ids) == 0
    c.pool, c.ids = pool[-2:].clone(), torch.tensor([1, 0], dtype=torch.int32, device=cuda)
    n = 3
    ref, tol = rope64(c.qkv, c._rows(0, 0, n), 1, 1, c.w[0], c.w[1], 1e-6, False, 128)
    for t in range(n):
        page, r = (1, 15) if t == 0 else (0, t - 1)
        for i in (0, 1):
            if fmt == 0:
                assert bool(((c.pool[page, 0, i, r].double() - ref[t, 1 + i]).abs() <= tol[t, 1 + i]).all())
            else:
                got = read_tiles(c.pool[page, 0], 128, 1.0, bool(i))[0][0, r]
                assert torch.equal(got, hold(ref[t, 1 + i])[0])


@pytest.mark.parametrize("T", [16, 3000])
@pytest.mark.parametrize("fmt", [0, 1])
def test_same_bits_in_a_graph_and_on_two_streams(lib, cuda, T, fmt):
    cases = [Case(cuda, fmt, [T], [[9, 50]], 8, 2, 128, seed=s, max_pos=4000) for s in (1, 2)]
    for c in cases:
        assert c.call(lib) == 0
    ref = [(c.q.clone(), c.pool.clone()) for c in cases]
    orders = [c.order.to(cuda) for c in cases]

    def call(i):
        c = cases[i]
        lib.tg_append_rope(c.qkv, c.cu, c.table, c.q, c.pool, c.pages, orders[i], c.ntok, c.added, c.reserve, c.off, c.ids, c.H_p,
                           c.P, fmt=fmt, q_weight=c.w[0], k_weight=c.w[1], origin=c.origin)

    def clear():
        for c in cases:
            c.q.fill_(c.mark)
            c.pool.fill_(0x5b if fmt else c.mark)

    def check():
        torch.cuda.synchronize()
        for c, (q, pool) in zip(cases, ref):
            assert torch.equal(c.q, q) and torch.equal(c.pool, pool)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    clear()
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(i)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        call(0), call(1), call(0)
    clear()
    graph.replay()
    check()


def test_append_to_4_bits_is_append_to_bf16_and_quantisation_of_v(lib, cuda):
    """V goes through both ways alike: appended in 4 bits, or appended in bf16 and quantised."""
    a = Case(cuda, 1, [50], [[0, 0]], 2, 2, 256, H_p=2, seed=5)
    b = Case(cuda, 0, [50], [[0, 0]], 2, 2, 256, H_p=2, seed=5)
    assert a.call(lib) == 0 and b.call(lib) == 0
    four = torch.zeros_like(a.pool)
    n = torch.full((1, 2), 50, dtype=torch.int32, device=cuda)
    lib.tg_quant_pages(a.order.to(cuda), n, 2, 16, 256, a.off, b.ids, b.pool, b.pages, a.off, a.ids, four, a.pages)
    for p in range(2):
        pages = a.ids[:4].long()
        x, y = (read_tiles(t[pages, p].reshape(-1, 4608), 256, 1.0, True)[0].reshape(-1, 256)[:50] for t in (a.pool, four))
        assert torch.equal(x, y)


def test_binding_refusals(lib, cuda):
    c = Case(cuda, 0, [2, 1], [[3, 4], [5, 6]], 2, 2, 128, dense=True)
    three = Case(cuda, 0, [2, 1], [[3, 4], [5, 6]], 2, 2, 128, axes=3)
    for bad in (dict(qkv=c.qkv[:1]), dict(qkv=c.qkv.transpose(1, 2).contiguous().transpose(1, 2)), dict(cu_q=c.cu[:1]),
                dict(added=c.added[:1]), dict(pt_off=c.off[:-1].clone()), dict(pool_pages=c.pages + 1), dict(origin=c.origin[:1]),
                dict(head_order=c.order[:1].to(cuda)), dict(positions=c.origin), dict(V=c.V[:, :, :3].contiguous()), dict(K=c.K[0]),
                dict(start=c.start[:1]), dict(q_weight=torch.ones(64, device=cuda)), dict(ntok=c.ntok[0])):
        with pytest.raises(ValueError):
            c.call(lib, **bad)
    for bad in (dict(axis_of=[0, 1, 2]), dict(axis_of=[256] * 64)):
        with pytest.raises(ValueError):
            three.call(lib, **bad)
    for bad in (dict(fmt=1), dict(qkv=c.qkv.float()), dict(q=c.q.half()), dict(ntok=c.ntok.long()), dict(cu_q=c.cu.cpu()),
                dict(pt_off=c.off.int())):
        with pytest.raises(TypeError):
            c.call(lib, **bad)
    for bad in (dict(V=None), dict(start=None), dict(origin=None), dict(P=24), dict(H_p=3), dict(reserve=-1)):
        with pytest.raises((lib.TGError, ValueError)):
            c.call(lib, **bad)
    with pytest.raises(lib.TGError):
        three.call(lib, axis_of=None)
    with pytest.raises(lib.TGError):
        three.call(lib, axis_of=[3] * 64)
    assert bool((c.q == c.mark).all()) and bool((c.pool == c.mark).all())
