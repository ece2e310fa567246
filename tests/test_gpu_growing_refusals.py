"""Refusals of the calls on growing and 4-bit pages, each named by an argument that the call has, and their counterparts that pass."""
import inspect

import pytest
import torch

from test_gpu_append import Case
from test_gpu_grown import Lists

pytestmark = pytest.mark.gpu


def _pages(cuda):
    order, ntok = torch.zeros(1, dtype=torch.int32, device=cuda), torch.tensor([[16]], dtype=torch.int32, device=cuda)
    off, ids = torch.tensor([0, 1], device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    bf, four = torch.ones((1, 1, 2, 16, 128), dtype=torch.bfloat16, device=cuda), torch.zeros((1, 2304), dtype=torch.uint8, device=cuda)
    return dict(head_order=order, ntok=ntok, H_p=1, P=16, d=128, src_off=off, src_ids=ids, src=bf, src_pages=1, dst_off=off,
                dst_ids=ids, dst=four, dst_pages=1)


def _refused(call, args, errors, bad):
    assert set(bad) <= set(inspect.signature(call).parameters), bad
    with pytest.raises(errors):
        call(**dict(args, **bad))


def test_conversions(lib, cuda):
    into, names = _pages(cuda), ("head_order", "ntok", "src_off", "src_ids", "src", "dst_off", "dst_ids", "dst")
    out_of = dict(into, src=into["dst"], dst=into["src"])
    lib.tg_quant_pages(**into)
    lib.tg_dequant_pages(**out_of)
    kept = into["src"].clone(), into["dst"].clone()
    for call, args in ((lib.tg_quant_pages, into), (lib.tg_dequant_pages, out_of)):
        for name in names:
            _refused(call, args, (TypeError, ValueError), {name: None})
            _refused(call, args, TypeError, {name: args[name].cpu()})
        for name in ("src_off", "dst_off"):
            _refused(call, args, ValueError, {name: args[name][:1]})
            _refused(call, args, TypeError, {name: args[name].int()})
        for bad in (dict(k_unit=3.0), dict(v_unit=0.0), dict(P=24), dict(d=64), dict(H_p=0), dict(src_pages=0), dict(dst_pages=-1)):
            _refused(call, args, (lib.TGError, ValueError), bad)
    for bad in (dict(plus=1), dict(plus=-1), dict(reserve=-1)):
        _refused(lib.tg_dequant_pages, out_of, lib.TGError, bad)
    _refused(lib.tg_dequant_pages, out_of, ValueError, dict(added=torch.zeros(2, dtype=torch.int32, device=cuda)))
    assert torch.equal(into["src"], kept[0]) and torch.equal(into["dst"], kept[1])


@pytest.mark.parametrize("fmt", [0, 1])
def test_an_append_on_two_axes_passes_and_one_position_past_the_table_is_left_out(lib, cuda, fmt):
    c = Case(cuda, fmt, [4], [[6]], 2, 1, 128, axes=2)
    assert c.call(lib) == 0
    c.verify()
    assert all(bool((c.q[i] != c.mark).any()) for i in range(4))
    c = Case(cuda, fmt, [4], [[6]], 2, 1, 128, axes=2)
    c.positions[2, c.axis_of[0]] = 600
    assert c.call(lib) == lib.STATUS_BAD_INPUT
    assert [bool((c.q[i] != c.mark).any()) for i in range(4)] == [True, True, False, True]


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
def test_decode(lib, cuda, pages):
    x = Lists(cuda, pages, [[20, 3], [30, 1]], 4, 128, H_p=2, reserve=10, n_cta=4, hostile=False)
    out = torch.zeros_like(x.q)
    args = dict(plan=x.lists.plan, layer=0, fmt=x.lists.format, q=x.q, pool=x.pool, pool_pages=x.n, pt_off=x.off, pt_ids=x.ids,
                ntok=x.lists.ntok[0], added=x.lists.added, plus=1, reserve=10, scale=0.1, out=out, workspace=x.lists.workspace)
    for name in ("q", "pool", "pt_off", "pt_ids", "ntok", "out", "workspace"):
        _refused(lib.tg_decode_grown, args, (TypeError, ValueError, lib.TGError), {name: None})
    for bad in (dict(plus=11), dict(plus=-1), dict(reserve=0), dict(scale=float("nan")), dict(layer=1), dict(fmt=2), dict(pool_pages=0),
                dict(workspace=x.lists.workspace[:256])):
        _refused(lib.tg_decode_grown, args, (ValueError, TypeError, lib.TGError), bad)
    if pages == "e2m1":
        _refused(lib.tg_decode_grown, args, lib.TGError, dict(v_unit=3.0))
    _refused(lib.tg_decode_grown, args, ValueError, dict(added=x.lists.added[:1]))
    assert not out.any()
    lib.tg_decode_grown(**args)
    assert bool(out.any()) and int(x.lists.status) == 0
