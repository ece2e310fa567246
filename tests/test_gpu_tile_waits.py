"""The bounded waits of the tile kernel: work that takes longer than a wait's limit is no reason to
give up."""
import math

import pytest
import torch

from prompt_helpers import attend64, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,n", [(128, 131040), (256, 92000)])
def test_a_pass_of_seconds_on_one_block(lib, cuda, d, n):
    """A long prompt and a short one on a single thread block, for more than the 2 s after which a
    block gives up that makes no progress.  The clearing warp has work at the end of the contexts
    only (the long one ends with a block), so it waits for nearly the whole pass."""
    from non_uniform_paged_gb300.ragged import PrefillPass
    assert n % 80 == 0
    short, g = 17, 8
    gen = torch.Generator(device=cuda).manual_seed(d)
    q = torch.randn((n + short, g, d), generator=gen, device=cuda).to(torch.bfloat16)
    K, V = (torch.randn((2, 1, n, d), generator=gen, device=cuda).to(torch.bfloat16) for _ in range(2))
    V[1, :, short:] = float("nan")
    p = PrefillPass(1, g, d, [n, short], [n, short], n_cta=1, device=cuda)
    assert p.plan.header["N_CTA"] == 1
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device=cuda)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    p.attend(q, K, V, out, lse)
    end.record()
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    # (a faster device needs a longer prompt)
    assert start.elapsed_time(end) > 2100
    # rows spread over the long prompt -- the first ones are worked on last -- and the short one
    rows = torch.cat([torch.arange(40, device=cuda), torch.linspace(40, n - 1, 88, device=cuda).long()])
    seen = torch.arange(n, device=cuda)[None] <= rows[:, None]
    few = torch.arange(short, device=cuda)
    for j in (0, 3, g - 1):
        ref = attend64(q[rows, j], K[0, 0], V[0, 0], 1 / math.sqrt(d), seen)
        check(out[rows, j], lse[rows, j], ref, f"long, head {j}")
        ref = attend64(q[n:, j], K[1, 0, :short], V[1, 0, :short], 1 / math.sqrt(d), few[None] <= few[:, None])
        check(out[n:, j], lse[n:, j], ref, f"short, head {j}")
    assert bool((out != 9.0).any(-1).all()) and bool((lse != 9.0).all())


def test_waits_that_run_out(lib, cuda, tmp_path):
    """The kernel built with waits that give up at once: a call ends with TG_STATUS_TIMEOUT, whatever
    step each warp was at, and the device goes on working."""
    import ctypes
    import os
    import subprocess
    from non_uniform_paged_gb300 import _build
    from non_uniform_paged_gb300.ragged import PrefillPass
    so = str(tmp_path / "libshort.so")
    src = [os.path.join(_build.CSRC, f) for f in ("prefill_attn.cu", "planner.cpp")]
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-DTG_TILE_SHORT_WAIT", "-shared", *src, "-o", so], check=True)
    call = ctypes.CDLL(so).tg_prefill_attn
    call.argtypes = lib._SIGS["tg_prefill_attn"][1]
    gen = torch.Generator(device=cuda).manual_seed(7)
    stream = torch.cuda.current_stream().cuda_stream
    ran_out = 0
    for d in (128, 256):
        # one block with items of all lengths; cut runs, which a merge joins; many blocks at once
        for q_len, kv_len, window, n_cta in (([600, 17, 40], [600, 17, 2000], 0, 1), ([1, 3], [9000, 5000], 0, 152),
                                             ([700] * 6, [1400] * 6, 300, 152)):
            H, g = 2, 4
            q = torch.randn((sum(q_len), H * g, d), generator=gen, device=cuda).to(torch.bfloat16)
            K, V = (torch.randn((len(q_len), H, max(kv_len), d), generator=gen, device=cuda).to(torch.bfloat16) for _ in range(2))
            p = PrefillPass(H, H * g, d, q_len, kv_len, window=window, n_cta=n_cta, device=cuda)
            ref, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
            p.attend(q, K, V, ref)
            for _ in range(5):
                p.status.zero_()
                ws = p.workspace
                assert call(stream, p.plan.host_ptr, p.plan.dev_ptr, q.data_ptr(), K.data_ptr(), V.data_ptr(), max(kv_len),
                            p.scale, None if ws is None else ws.data_ptr(), p.workspace_bytes, out.data_ptr(), lse.data_ptr(),
                            p.status.data_ptr()) == 0
                status = int(p.status.item())
                assert status in (0, lib.STATUS_TIMEOUT)
                ran_out += status == lib.STATUS_TIMEOUT
                if status == 0:
                    assert torch.equal(out, ref)
            p.status.zero_()
            p.attend(q, K, V, out, lse)
            assert lib.tg_check_status(p.status) == 0 and torch.equal(out, ref)
    assert ran_out > 0
