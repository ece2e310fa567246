"""Host side of pages that grow: lists with a reserve, page sizes, the 64-bit definition of 4-bit values against
spelt-out cases, and what the calls refuse before they launch anything (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from pages4_helpers import E2M1, e4m3_grid, hold, nearest, places

OK, INVALID, SHAPE, NONFINITE, CAPACITY = 0, -1, -2, -3, -4


@pytest.mark.parametrize("reserve", [0, 1, 15, 16, 1000])
@pytest.mark.parametrize("H_p,P,cluster", [(1, 16, False), (2, 32, True), (4, 48, True)])
def test_lists_hold_the_longest_head_and_the_reserve(lib, reserve, H_p, P, cluster):
    w = synth.small(L=3, batch=4, H=4, H_q=8, H_p=H_p, P=P, cluster=cluster)
    N = synth.contexts(w)
    N[1] = 0
    t = lib.tg_build_pages(w.L, w.batch, w.H, w.H_p, w.P, w.alpha, synth.budgets_hat(w), N, cluster)
    off, ids, n = lib.tg_reserve_pages(t["order"], t["ntok"], H_p, P, reserve)
    G, at, next_id = w.H // H_p, 0, 0
    want = {}
    for l in range(w.L):
        for b in range(w.batch):
            for g in range(G):
                most = max(t["ntok"][l, b, h] for h in t["order"][l, g * H_p:(g + 1) * H_p]) + reserve
                i = (l * w.batch + b) * G + g
                assert off[i] == at
                at += -(-most // P)
                assert off[i + 1] == at
    for b in range(w.batch):
        for l in range(w.L):
            for g in range(G):
                i = (l * w.batch + b) * G + g
                want[i] = list(range(next_id, next_id + off[i + 1] - off[i]))
                next_id += off[i + 1] - off[i]
    assert n == next_id == at and all(ids[off[i]:off[i + 1]].tolist() == v for i, v in want.items())
    if reserve == 0:
        assert np.array_equal(off, t["pt_off"]) and np.array_equal(ids, t["pt_ids"])


def test_refused_tables(lib):
    order, ntok = np.arange(4, dtype=np.int32)[None], np.full((1, 2, 4), 20, np.int32)
    for bad in (dict(H_p=3), dict(P=24), dict(reserve=-1), dict(H_p=0)):
        with pytest.raises((lib.TGError, ZeroDivisionError)):
            lib.tg_reserve_pages(**dict(dict(head_order=order, ntok=ntok, H_p=2, P=16, reserve=4), **bad))
    for o, t in ((order + 1, ntok), (order - 1, ntok), (order, ntok - 21), (order, ntok + (2 ** 31 - 30))):
        with pytest.raises(lib.TGError) as e:
            lib.tg_reserve_pages(o, t, 2, 16, 4)
        assert e.value.code == INVALID
    so, n = lib.load(), ctypes.c_int64(0)
    ids = np.zeros(3, np.int32)
    assert so.tg_reserve_pages(1, 2, 4, 2, 16, order.ctypes.data, ntok.ctypes.data, 4, None, ids.ctypes.data, 3,
                               ctypes.addressof(n)) == CAPACITY
    assert n.value == 8 and not ids.any()


def test_owners_refuse_before_they_take_anything(lib):
    from non_uniform_paged_gb300.ragged import GrowingCache, GrowingLists

    class Never:
        def admit(self, counts):
            raise AssertionError("pages were taken")

    for bad in (dict(pages="e4m3"), dict(reserve=-1)):
        with pytest.raises(ValueError):
            GrowingLists(**dict(dict(H_q=4, H_p=1, P=16, d=128, order=[0, 1], ntok=[[5, 5]], reserve=3, n_cta=4, device="cpu"), **bad))
        w = synth.small()
        with pytest.raises(ValueError):
            GrowingCache(w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, synth.budgets_hat(w), synth.contexts(w), n_cta=24,
                         device="cpu", allocator=Never(), **dict(dict(reserve=3), **bad))


def test_page_bytes(lib):
    assert lib.tg_page_bytes(lib.PAGES_BF16, 4, 16, 128) == 4 * 2 * 16 * 128 * 2
    assert lib.tg_page_bytes(lib.PAGES_E2M1, 4, 48, 256) == 4 * 3 * 2 * 2304
    for bad in ((2, 4, 16, 128), (1, 0, 16, 128), (1, 4, 24, 128), (0, 4, 16, 64), (0, 2 ** 30, 2 ** 30, 256)):
        with pytest.raises(lib.TGError):
            lib.tg_page_bytes(*bad)


def test_every_place_of_a_tile_is_used_once():
    for d in (128, 256):
        nibbles, scales = set(), set()
        for V in (False, True):
            for t in range(16):
                for e in range(d):
                    byte, upper, sc = places(t, e, V)
                    nibbles.add((byte, upper))
                    scales.add(sc)
        assert len(nibbles) == 2 * 16 * d and len(scales) == 2 * d
        assert {b for b, _ in nibbles} | scales == set(range(d // 128 * 2304))


def test_the_definition_of_held_values():
    assert torch.equal(e4m3_grid().float(), torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
    x = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)  # ties go to the even code
    assert nearest(x, E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6]
    row = torch.zeros(32, dtype=torch.float64)
    row[:8] = torch.tensor([6.0, -5.0, 5.01, 0.25, 0.26, -0.26, 2.5, -3.5])
    row[16] = 1e9
    row[17] = 1.0
    v, code = hold(row)
    assert v[:8].tolist() == [6.0, -4.0, 6.0, 0.0, 0.5, -0.5, 2.0, -4.0] and code[0] == 56  # scale 1
    assert v[16] == 6 * 448 and v[17] == 0 and code[1] == 126
    tiny, code = hold(torch.full((16,), 1e-4, dtype=torch.float64))
    assert not tiny.any() and code[0] == 1
    v, _ = hold(row, unit=4.0)
    assert v[0] == 6.0 and v[16] == 6 * 448 * 4
    v, _ = hold(torch.tensor([float("inf"), float("nan"), -float("inf"), 1.0] * 4, dtype=torch.float64))
    assert v[:4].tolist() == [2688.0, 2688.0, -2688.0, 0.0]


FAKE = 1 << 20  # aligned, never read: every refusal below comes first


def _append(lib, **change):
    a = dict(stream=None, batch=2, T=2, H_q=4, H=2, H_p=2, P=16, d=128, rot=128, max_pos=64, flags=0, cu_q=FAKE, qkv=FAKE,
             stride=8 * 128, qw=None, kw=None, eps=1e-6, axes=1, positions=None, axis_of=None, origin=FAKE, cos_sin=FAKE,
             head_order=FAKE, ntok=FAKE, added=None, reserve=4, pt_off=FAKE, pt_ids=FAKE, format=0, k_unit=1.0, v_unit=1.0,
             pool=FAKE, pool_pages=8, q=FAKE, K=None, V=None, Nmax=0, start=None, status=None)
    assert set(change) <= set(a)
    a.update(change)
    return lib.load().tg_append_rope(*a.values())


def test_append_refusals(lib):
    axis = np.zeros(64, np.uint8)
    axis[63] = 3
    cases = [(dict(batch=0), INVALID), (dict(T=-1), INVALID), (dict(H_q=0), INVALID), (dict(H=0), INVALID), (dict(H_p=0), INVALID),
             (dict(P=0), INVALID), (dict(reserve=-1), INVALID), (dict(d=64), SHAPE), (dict(H=3, stride=10 * 128), SHAPE),
             (dict(P=24), SHAPE), (dict(rot=136), SHAPE), (dict(rot=8), SHAPE), (dict(rot=-16), SHAPE), (dict(flags=2), INVALID),
             (dict(format=2), INVALID), (dict(format=-1), INVALID), (dict(format=1, k_unit=3.0), INVALID),
             (dict(format=1, v_unit=0.0), INVALID), (dict(format=1, k_unit=-2.0), INVALID),
             (dict(format=1, v_unit=float("nan")), INVALID), (dict(format=1, k_unit=2.0 ** 61), INVALID), (dict(axes=0), SHAPE),
             (dict(axes=5), SHAPE), (dict(stride=8 * 128 - 8), SHAPE), (dict(stride=8 * 128 + 4), SHAPE),
             (dict(eps=float("inf")), NONFINITE), (dict(eps=-1.0), INVALID), (dict(pool_pages=0), CAPACITY),
             (dict(pool_pages=2 ** 31), CAPACITY), (dict(K=FAKE), INVALID), (dict(V=FAKE), INVALID),
             (dict(K=FAKE, V=FAKE, start=FAKE), INVALID), (dict(K=FAKE, V=FAKE, Nmax=4), INVALID), (dict(cos_sin=None), INVALID),
             (dict(max_pos=0), INVALID), (dict(origin=None), INVALID), (dict(axes=3), INVALID),
             (dict(axes=3, positions=FAKE), INVALID), (dict(axes=3, positions=FAKE, axis_of=axis.ctypes.data), INVALID),
             (dict(axes=4, axis_of=axis.ctypes.data), INVALID)]
    cases += [({k: None}, INVALID) for k in ("cu_q", "qkv", "head_order", "ntok", "pt_off", "pt_ids", "pool", "q")]
    cases += [({k: FAKE + 8}, INVALID) for k in ("qkv", "q", "pool", "cos_sin", "qw", "kw")]
    cases += [(dict(K=FAKE + 8, V=FAKE, Nmax=4, start=FAKE), INVALID)]
    for change, code in cases:
        assert _append(lib, **change) == code, change
        assert lib.load().tg_last_error_string()
    assert _append(lib, T=0, cu_q=None) == OK  # nothing to do
    assert _append(lib, T=0, axes=4, positions=FAKE, axis_of=axis.ctypes.data) == OK


def _convert(lib, name, **change):
    a = dict(stream=None, batch=2, H=2, H_p=2, P=16, d=128, head_order=FAKE, ntok=FAKE)
    if name == "tg_dequant_pages":
        a.update(added=None, plus=0, reserve=0)
    a.update(src_off=FAKE, src_ids=FAKE, src=FAKE, src_pages=4, dst_off=FAKE, dst_ids=FAKE, dst=FAKE, dst_pages=4, k_unit=1.0,
             v_unit=1.0, status=None)
    assert set(change) <= set(a)
    a.update(change)
    return getattr(lib.load(), name)(*a.values())


@pytest.mark.parametrize("name", ["tg_quant_pages", "tg_dequant_pages"])
def test_conversion_refusals(lib, name):
    cases = [(dict(batch=0), INVALID), (dict(H=0), INVALID), (dict(H_p=0), INVALID), (dict(P=0), INVALID), (dict(d=96), SHAPE),
             (dict(H_p=3), SHAPE), (dict(P=8), SHAPE), (dict(batch=2 ** 30, H=2), SHAPE), (dict(k_unit=0.3), INVALID),
             (dict(v_unit=float("inf")), INVALID), (dict(src_pages=0), CAPACITY), (dict(dst_pages=2 ** 31), CAPACITY),
             (dict(src=FAKE + 2), INVALID), (dict(dst=FAKE + 8), INVALID)]
    cases += [({k: None}, INVALID) for k in ("head_order", "ntok", "src_off", "src_ids", "src", "dst_off", "dst_ids", "dst")]
    if name == "tg_dequant_pages":
        cases += [(dict(plus=-1), INVALID), (dict(plus=3, reserve=2), INVALID), (dict(reserve=-1), INVALID)]
    for change, code in cases:
        assert _convert(lib, name, **change) == code, change


def _grown(lib, plan, ws, **change):
    a = dict(stream=None, plan_host=plan.ctypes.data, plan_dev=FAKE, layer=0, format=1, q=FAKE, pool=FAKE, pool_pages=8,
             pt_off=FAKE, pt_ids=FAKE, ntok=FAKE, added=None, plus=1, reserve=4, scale=1.0, k_unit=1.0, v_unit=1.0,
             workspace=FAKE, workspace_bytes=ws, out=FAKE, lse=None, status=None, cta_time=None)
    assert set(change) <= set(a)
    a.update(change)
    return lib.load().tg_decode_grown(*a.values())


def test_decode_grown_refusals(lib):
    ntok = np.full((1, 2, 2), 24, np.int32)
    plan, ws = lib.tg_plan_decode(lib.tg_split_map([[96]], 4), np.arange(2, dtype=np.int32)[None], ntok, 4, 2, 16, 128)
    junk = np.zeros_like(plan)
    cases = [(dict(format=2), INVALID), (dict(plus=-1), INVALID), (dict(reserve=-1, plus=0), INVALID), (dict(plus=5), INVALID),
             (dict(layer=1), INVALID), (dict(layer=-1), INVALID), (dict(plan_host=junk.ctypes.data), INVALID),
             (dict(scale=float("nan")), NONFINITE), (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 8), INVALID), (dict(pool=FAKE + 8), INVALID),
             (dict(plan_dev=FAKE + 8), INVALID), (dict(workspace=FAKE + 128), INVALID), (dict(workspace_bytes=ws - 1), CAPACITY),
             (dict(k_unit=1.5), INVALID), (dict(v_unit=2.0 ** -61), INVALID), (dict(pool_pages=0), CAPACITY),
             (dict(pool_pages=2 ** 31), CAPACITY)]
    cases += [({k: None}, INVALID) for k in ("plan_host", "plan_dev", "q", "pool", "pt_off", "pt_ids", "ntok", "workspace", "out")]
    for change, code in cases:
        assert _grown(lib, plan, ws, **change) == code, change
