"""PrefillPass and SharedPrefix on other streams than the one they were made on."""
import math

import numpy as np
import pytest
import torch

from prompt_helpers import attend64, check, seen_keys

pytestmark = pytest.mark.gpu
D, H, G = 128, 2, 4
Q_LEN, KV_LEN = [1, 40], [9000, 4000]  # cut runs: a workspace
NTOK = np.array([[20000, 9000]], np.int32)


def _prompt_case(cuda):
    from non_uniform_paged_gb300.ragged import PrefillPass
    g = torch.Generator(device=cuda).manual_seed(11)
    q = torch.randn((sum(Q_LEN), H * G, D), generator=g, device=cuda).to(torch.bfloat16)
    K, V = (torch.randn((2, H, max(KV_LEN), D), generator=g, device=cuda).to(torch.bfloat16) for _ in range(2))

    def right(out, lse):
        at = 0
        for b, (nq, nk) in enumerate(zip(Q_LEN, KV_LEN)):
            for j in range(H * G):
                ref = attend64(q[at:at + nq, j], K[b, j // G, :nk], V[b, j // G, :nk], 1 / math.sqrt(D), seen_keys(nq, nk, 0, cuda))
                check(out[at:at + nq, j], lse[at:at + nq, j], ref, (b, j))
            at += nq

    return (lambda: PrefillPass(H, H * G, D, Q_LEN, KV_LEN, device=cuda),
            lambda p, out, lse, **kw: p.attend(q, K, V, out, lse, **kw), right, q)


def _prefix_case(cuda):
    from non_uniform_paged_gb300.ragged import SharedPrefix
    g = torch.Generator(device=cuda).manual_seed(12)
    pages = 20000 // 16
    pool = torch.randn((pages, H, 2, 16, D), generator=g, device=cuda).to(torch.bfloat16)
    ids = torch.randperm(pages, generator=g, device=cuda).to(torch.int32)
    off = torch.tensor([0, pages], device=cuda)
    q = torch.randn((7, H * G, D), generator=g, device=cuda).to(torch.bfloat16)

    def right(out, lse):
        for j in range(H * G):
            kv = pool[ids.long(), j // G].transpose(0, 1).reshape(2, -1, D)[:, :NTOK[0, j // G]]
            check(out[:, j], lse[:, j], attend64(q[:, j], kv[0], kv[1], 1 / math.sqrt(D)), j)

    return (lambda: SharedPrefix(H * G, H, 16, D, [0, 7], np.arange(H), NTOK, device=cuda),
            lambda p, out, lse, **kw: p.attend(0, q, pool, pages, off, ids, out, lse, **kw), right, q)


def _ranges(p):
    return [(t.data_ptr(), t.data_ptr() + max(1, t.numel() * t.element_size())) for t in p._buffers]


@pytest.mark.parametrize("case", [_prompt_case, _prefix_case])
@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_dropped_while_its_stream_is_busy(lib, cuda, case, how):
    """Memory of a dropped pass is not handed out while a stream that ran it still has work queued.
    (The pass's own call is complete before it is dropped: nothing here reads memory that is gone.)"""
    make, attend, right, q = case(cuda)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    side = torch.cuda.Stream()
    p = make()
    assert p.workspace is not None
    torch.cuda.synchronize()
    if how == "current":
        with torch.cuda.stream(side):
            attend(p, out, lse)
    else:
        attend(p, out, lse, stream=side if how == "argument" else side.cuda_stream)
    side.synchronize()
    right(out, lse)
    with torch.cuda.stream(side):
        torch.cuda._sleep(600_000_000)
    old = _ranges(p)
    del p
    again = make()
    assert not side.query()
    assert all(b <= lo or hi <= a for lo, hi in old for a, b in _ranges(again))
    torch.cuda.synchronize()


@pytest.mark.parametrize("case", [_prompt_case, _prefix_case])
def test_made_while_busy_and_run_on_another_stream(lib, cuda, case):
    """Made while the current stream still writes memory that the constructor is given, and run on
    another stream at once: results as ever."""
    make, attend, right, q = case(cuda)
    first = make()
    sizes = [t.numel() * t.element_size() for t in first._buffers]
    del first
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.empty(n, dtype=torch.uint8, device=cuda) for n in sizes]
    busy = torch.zeros(1 << 28, dtype=torch.uint8, device=cuda)
    for _ in range(200):
        busy.add_(1)
    for t in held:
        t.fill_(0xff)
    places = {t.data_ptr() for t in held}
    del held, t
    p = make()
    assert places & {a for a, _ in _ranges(p)}
    attend(p, out, lse, stream=side)
    side.synchronize()
    assert int(p.status.item()) == 0
    right(out, lse)


@pytest.mark.parametrize("case", [_prompt_case, _prefix_case])
def test_a_refused_call_uses_no_stream(lib, cuda, case):
    make, attend, _, q = case(cuda)
    p = make()
    before = set(p._streams)
    with pytest.raises(ValueError):
        attend(p, torch.empty_like(q)[:1], None, stream=torch.cuda.Stream())
    assert p._streams == before
