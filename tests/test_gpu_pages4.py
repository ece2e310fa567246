"""tg_quant_pages and tg_dequant_pages: every value of 4-bit pages is the nearest the definition names, and what
is not a token of the lists stays as it was."""
import numpy as np
import pytest
import torch

from pages4_helpers import e4m3_grid, hold, read_tiles, tile_bytes

pytestmark = pytest.mark.gpu


def _lists(lens, H_p, P, cuda, seed=0, extra=0):
    """Tables of [batch][H] token counts with scattered page ids -> (ntok, off, ids, pages)."""
    lens = np.asarray(lens, np.int32)
    batch, H = lens.shape
    counts = [-(-int(lens[b, i:i + H_p].max()) // P) + extra for b in range(batch) for i in range(0, H, H_p)]
    off = np.concatenate([[0], np.cumsum(counts)])
    n = max(1, int(off[-1]))
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).to(torch.int32)[:max(1, int(off[-1]))]
    return torch.from_numpy(lens).to(cuda), torch.from_numpy(off.astype(np.int64)).to(cuda), ids.to(cuda), n


def _order(H, cuda, seed=3):
    return torch.randperm(H, generator=torch.Generator().manual_seed(seed)).to(torch.int32).to(cuda)


def _by_place(lens, order):
    """Counts [batch][H] so that place p of the groups, head order[p], has lens[b][p]."""
    out = np.zeros_like(np.asarray(lens, np.int32))
    out[:, order.cpu().numpy()] = lens
    return out


CASES = [(128, 16, 2, [[37, 16, 1, 700], [0, 5, 31, 33]]), (256, 16, 2, [[37, 16, 1, 300], [0, 5, 31, 33]]),
         (128, 48, 4, [[100, 47, 48, 49], [1, 0, 0, 0], [17, 96, 2, 3]]), (256, 64, 1, [[65, 64, 1], [63, 128, 0]]),
         (128, 16, 1, [[1]]), (128, 16, 1, [[0]])]


def _expected(src, lens, order, off, ids, H_p, P, d, unit):
    """(b, place, n, values [2][n][d] float64) of every list, out of bf16 pages."""
    for b in range(lens.shape[0]):
        for p in range(lens.shape[1]):
            n = int(lens[b, int(order[p])])
            if n:
                l = b * (lens.shape[1] // H_p) + p // H_p
                pages = ids[off[l]:off[l] + -(-n // P)].long()
                rows = src[pages, p % H_p].transpose(0, 1).reshape(2, -1, d)[:, :n].double()
                yield b, p, n, pages, torch.stack([hold(rows[i], unit[i])[0] for i in (0, 1)])


@pytest.mark.parametrize("d,P,H_p,by_place", CASES)
@pytest.mark.parametrize("unit", [(1.0, 1.0), (0.25, 2.0 ** -10)])
def test_values_are_the_nearest_and_the_rest_is_left(lib, cuda, d, P, H_p, by_place, unit):
    by_place = np.asarray(by_place, np.int32)
    H = by_place.shape[1]
    order = _order(H, cuda)
    # page tables go by place, counts by head
    _, off, ids, n_pages = _lists(by_place, H_p, P, cuda)
    ntok = torch.from_numpy(_by_place(by_place, order)).to(cuda)
    g = torch.Generator(device=cuda).manual_seed(d + P)
    src = torch.randn((n_pages, H_p, 2, P, d), generator=g, device=cuda).to(torch.bfloat16)
    src *= torch.exp2(torch.randint(-8, 6, (n_pages, H_p, 2, P, d // 16, 1), generator=g, device=cuda).float()).expand(
        -1, -1, -1, -1, -1, 16).reshape(src.shape).to(torch.bfloat16)
    used = torch.zeros((n_pages, H_p, P), dtype=torch.bool, device=cuda)
    tail = torch.zeros_like(used)
    for b, p, n, pages, _ in _expected(src, ntok, order, off, ids, H_p, P, d, unit):
        row = torch.arange(pages.numel() * P, device=cuda).view(-1, P)
        used[pages, p % H_p] = row < n
        tail[pages, p % H_p] = row >= n
    nan = torch.tensor(float("nan"), dtype=torch.bfloat16, device=cuda)
    src = torch.where(used[:, :, None, :, None], src, nan)  # rows that are no tokens may hold anything
    mark = 0x5b
    dst = torch.full((n_pages, H_p, P // 16, tile_bytes(d)), mark, dtype=torch.uint8, device=cuda)
    back = torch.full((n_pages, H_p, 2, P, d), 7.0, dtype=torch.bfloat16, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    lib.tg_quant_pages(order, ntok, H_p, P, d, off, ids, src, n_pages, off, ids, dst, n_pages, *unit, dev_status=status)
    lib.tg_dequant_pages(order, ntok, H_p, P, d, off, ids, dst, n_pages, off, ids, back, n_pages, k_unit=unit[0],
                         v_unit=unit[1], dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for b, p, n, pages, ref in _expected(src, ntok, order, off, ids, H_p, P, d, unit):
        raw = dst[pages, p % H_p].reshape(-1, tile_bytes(d))
        for i in (0, 1):
            got = read_tiles(raw[:-(-n // 16)], d, unit[i], bool(i))[0].reshape(-1, d)
            assert torch.equal(got[:n], ref[i]), (b, p, i)
            assert not got[n:].any()
            assert torch.equal(back[pages, p % H_p, i].reshape(-1, d)[:n].double(), ref[i])
    assert not back[tail[:, :, None, :, None].expand_as(back)].any()
    assert bool((back[~(used | tail)[:, :, None, :, None].expand_as(back)] == 7.0).all())
    tiles = (used.view(n_pages, H_p, P // 16, 16)).any(-1)
    assert bool((dst[~tiles] == mark).all())


def test_ties_zeros_extremes_and_values_that_are_not_finite(lib, cuda):
    """Every bf16 value over scales of every mantissa: the codes are the definition's, ties included."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    fin = bits[torch.isfinite(bits.float())]
    x = fin[torch.randperm(fin.numel(), generator=torch.Generator().manual_seed(1))][:65024]
    # blocks of 16: fifteen values in reach of a largest one of every mantissa
    top = torch.exp2(torch.randint(-12, 12, (4096, 1), generator=torch.Generator().manual_seed(2)).float()) * \
        (1 + torch.arange(128).repeat(32)[:, None] / 128)
    small = top * torch.randint(-256, 257, (4096, 15), generator=torch.Generator().manual_seed(3)) / 256
    rows = torch.cat([x.float(), torch.cat([top, small], 1).flatten()]).to(torch.bfloat16)
    special = torch.zeros(1024)
    special[0], special[16], special[17], special[33], special[64:80] = float("inf"), float("nan"), 3.0, -float("inf"), -0.0
    rows = torch.cat([rows, special.to(torch.bfloat16)]).view(-1, 128)
    n = rows.shape[0] // 2 // 16 * 16  # K and V halves
    P, H_p, d = 16, 1, 128
    pages = n // 16
    src = rows[:2 * n].view(2, pages, 16, d).transpose(0, 1).reshape(pages, 1, 2, 16, d).contiguous().to(cuda)
    src[-1, 0, 1, -1, :64] = special[:64].to(torch.bfloat16).to(cuda)
    off, ids = torch.tensor([0, pages], device=cuda), torch.arange(pages, dtype=torch.int32, device=cuda)
    order, ntok = torch.zeros(1, dtype=torch.int32, device=cuda), torch.tensor([[n]], dtype=torch.int32, device=cuda)
    dst = torch.zeros((pages, 1, 1, 2304), dtype=torch.uint8, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    lib.tg_quant_pages(order, ntok, H_p, P, d, off, ids, src, pages, off, ids, dst, pages, dev_status=status)
    assert int(status) == lib.STATUS_NONFINITE
    for i in (0, 1):
        want, code = hold(src[:, 0, i].reshape(-1, d).double())
        got, sc = read_tiles(dst.view(-1, 2304), d, 1.0, bool(i))
        assert torch.equal(sc.reshape(-1, 8).cpu(), code.cpu())
        assert torch.equal(got.reshape(-1, d), want)


def test_every_code_and_scale_comes_back(lib, cuda):
    """All 256 bytes with all finite scales, negative zeros too, exactly."""
    raw = torch.zeros((128, 2304), dtype=torch.uint8)
    raw[:, :2048] = torch.randint(0, 256, (128, 2048), generator=torch.Generator().manual_seed(4), dtype=torch.uint8)
    raw[:, 2048:] = (torch.arange(128)[:, None] + torch.arange(256)) % 127
    src = raw.view(128, 1, 1, 2304).to(cuda)
    off, ids = torch.tensor([0, 128], device=cuda), torch.arange(128, dtype=torch.int32, device=cuda)
    order, ntok = torch.zeros(1, dtype=torch.int32, device=cuda), torch.tensor([[2048]], dtype=torch.int32, device=cuda)
    back = torch.zeros((128, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda)
    lib.tg_dequant_pages(order, ntok, 1, 16, 128, off, ids, src, 128, off, ids, back, 128, k_unit=2.0, v_unit=0.5)
    for i, u in ((0, 2.0), (1, 0.5)):
        assert torch.equal(back[:, 0, i].double(), read_tiles(raw.to(cuda), 128, u, bool(i))[0])
    assert e4m3_grid()[126] == 448


def test_grown_lengths_and_other_lists(lib, cuda):
    """Appended tokens are dequantised too; source and destination lists differ in ids and in length."""
    H_p, P, d = 2, 16, 128
    lens = np.array([[20, 3], [0, 40]], np.int32)
    ntok = torch.from_numpy(lens).to(cuda)
    order = torch.arange(2, dtype=torch.int32, device=cuda)
    _, off1, ids1, n1 = _lists(lens + 30, H_p, P, cuda, 1, extra=2)
    _, off2, ids2, n2 = _lists(lens + 30, H_p, P, cuda, 2)
    g = torch.Generator(device=cuda).manual_seed(0)
    src = torch.randint(0, 256, (n1, H_p, 1, 2304), generator=g, device=cuda, dtype=torch.uint8)
    src[..., 2048:] %= 0x70
    added = torch.tensor([7, 29], dtype=torch.int32, device=cuda)
    for plus, want, bad in ((0, (7, 29), 0), (1, (8, 30), 0), (3, (10, 30), lib.STATUS_BAD_INPUT)):
        back = torch.full((n2, H_p, 2, P, d), 7.0, dtype=torch.bfloat16, device=cuda)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        lib.tg_dequant_pages(order, ntok, H_p, P, d, off1, ids1, src, n1, off2, ids2, back, n2, added=added, plus=plus,
                             reserve=30, dev_status=status)
        assert int(status) == bad
        for b in range(2):
            for h in range(2):
                n = int(lens[b, h]) + want[b]
                k = -(-n // P)
                raw = src[ids1[off1[b]:off1[b] + k].long(), h].reshape(-1, 2304)
                got = back[ids2[off2[b]:off2[b] + k].long(), h]
                for i in (0, 1):
                    ref = read_tiles(raw, d, 1.0, bool(i))[0].reshape(-1, d)
                    assert torch.equal(got[:, i].reshape(-1, d)[:n].double(), ref[:n]), (plus, b, h)
                    assert not got[:, i].reshape(-1, d)[n:].any()
    added[0] = -9
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    lib.tg_dequant_pages(order, ntok, H_p, P, d, off1, ids1, src, n1, off2, ids2, back, n2, added=added, reserve=30,
                         dev_status=status)
    assert int(status) == lib.STATUS_BAD_INPUT


def test_bad_pages_and_short_lists_are_skipped(lib, cuda):
    H_p, P, d = 1, 16, 128
    ntok = torch.tensor([[64, 64]], dtype=torch.int32, device=cuda)
    order = torch.arange(2, dtype=torch.int32, device=cuda)
    src = torch.randn((8, 1, 2, P, d), device=cuda).to(torch.bfloat16)
    good = torch.arange(8, dtype=torch.int32, device=cuda)
    off = torch.tensor([0, 4, 8], device=cuda)
    mark = 0x11
    for ids, off2, missing in ((torch.tensor([0, 1, -1, 3, 4, 8, 6, 7]), [0, 4, 8], (2, 5)), (good.cpu(), [0, 3, 7], (3,))):
        dst = torch.full((8, 1, 1, 2304), mark, dtype=torch.uint8, device=cuda)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        lib.tg_quant_pages(order, ntok, H_p, P, d, off, good, src, 8, torch.tensor(off2, device=cuda),
                           ids.to(torch.int32).to(cuda), dst, 8, dev_status=status)
        assert int(status) == lib.STATUS_BAD_PAGE
        left = [i for i in range(8) if bool((dst[i] == mark).all())]
        assert left == ([2, 5] if missing == (2, 5) else [7]), left
    order[1] = 2  # a head that is not there has no tokens
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    lib.tg_quant_pages(order, ntok, H_p, P, d, off, good, src, 8, off, good, dst, 8, dev_status=status)
    assert int(status) == lib.STATUS_BAD_INPUT


def test_many_heads_and_offsets_past_32_bits(lib, cuda):
    """More heads than a block of threads has, most of them empty; then pages behind 2^32 bytes."""
    lens = np.zeros((90, 8), np.int32)
    lens[::7, 3], lens[5, 0], lens[89, 7] = 20, 333, 1
    ntok, off, ids, n = _lists(lens, 1, 16, cuda)
    order = torch.arange(8, dtype=torch.int32, device=cuda)
    src = torch.randn((n, 1, 2, 16, 128), device=cuda).to(torch.bfloat16)
    dst = torch.zeros((n, 1, 1, 2304), dtype=torch.uint8, device=cuda)
    lib.tg_quant_pages(order, ntok, 1, 16, 128, off, ids, src, n, off, ids, dst, n)
    for b, h in ((0, 3), (5, 0), (84, 3), (89, 7)):
        k, l = int(lens[b, h]), b * 8 + h
        pages = ids[off[l]:off[l + 1]].long()
        for i in (0, 1):
            got = read_tiles(dst[pages].view(-1, 2304), 128, 1.0, bool(i))[0].reshape(-1, 128)[:k]
            assert torch.equal(got, hold(src[pages, 0, i].reshape(-1, 128)[:k].double())[0])
    many = 2_000_000  # 4.6 GB of 4-bit pages, 16 GB of bf16 pages
    src = torch.empty((many, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda)
    dst = torch.empty((many, 1, 1, 2304), dtype=torch.uint8, device=cuda)
    at = torch.tensor([many - 1, many - 2], dtype=torch.int32, device=cuda)
    src[many - 2:] = torch.randn((2, 1, 2, 16, 128), device=cuda).to(torch.bfloat16)
    one, off = torch.tensor([[30]], dtype=torch.int32, device=cuda), torch.tensor([0, 2], device=cuda)
    back = torch.zeros((2, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda)
    z = torch.zeros(1, dtype=torch.int32, device=cuda)
    lib.tg_quant_pages(z, one, 1, 16, 128, off, at, src, many, off, at, dst, many)
    lib.tg_dequant_pages(z, one, 1, 16, 128, off, at, dst, many, off, torch.arange(2, dtype=torch.int32, device=cuda), back, 2)
    for i in (0, 1):
        want = hold(src[[many - 1, many - 2], 0, i].reshape(-1, 128)[:30].double())[0]
        assert torch.equal(back[:, 0, i].reshape(-1, 128)[:30].double(), want)


def test_binding_refusals(lib, cuda):
    order, ntok = torch.zeros(1, dtype=torch.int32, device=cuda), torch.tensor([[16]], dtype=torch.int32, device=cuda)
    off, ids = torch.tensor([0, 1], device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    bf, four = torch.zeros((1, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda), torch.zeros((1, 2304), dtype=torch.uint8, device=cuda)
    args = dict(head_order=order, ntok=ntok, H_p=1, P=16, d=128, src_off=off, src_ids=ids, src=bf, src_pages=1, dst_off=off,
                dst_ids=ids, dst=four, dst_pages=1)
    lib.tg_quant_pages(**args)
    for bad in (dict(ntok=ntok[0]), dict(head_order=order.repeat(2)), dict(src_off=off[:1]), dict(src_pages=2), dict(dst_pages=2)):
        with pytest.raises(ValueError):
            lib.tg_quant_pages(**dict(args, **bad))
    for bad in (dict(src=four.expand(4, 2304).contiguous()), dict(dst=bf), dict(ntok=ntok.long()), dict(off=None), dict(dst_ids=ids.cpu())):
        with pytest.raises((TypeError, ValueError)):
            lib.tg_quant_pages(**dict(args, **bad))
