"""The first call that a host thread makes into CUDA at all is one of the library's: each call gives what it gives elsewhere."""
import threading

import pytest
import torch

import synth
import test_gpu_pass_streams as passes
from test_gpu_grown import Lists

pytestmark = pytest.mark.gpu


def _in_a_thread(call):
    raised = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001 (what the call raised is what is tested)
            raised.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert raised == []


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [128, 256])
def test_grown_decode(lib, cuda, pages, d):
    x = Lists(cuda, pages, [[100, 30]], 4, d, reserve=2, n_cta=4, hostile=False)
    want = x.run([1], 1)[:2]
    out, lse = (torch.zeros_like(t) for t in want)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    _in_a_thread(lambda: x.lists.attend(0, x.q, x.pool, x.n, x.off, x.ids, out, lse=lse, stream=stream))
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("case", [passes._prompt_case, passes._prefix_case])
def test_prompt_and_prefix_attention(lib, cuda, case):
    make, attend, right, q = case(cuda)
    p = make()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=cuda)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    _in_a_thread(lambda: attend(p, out, lse, stream=stream))
    right(out, lse)


def test_static_decode(lib, cuda):
    from non_uniform_paged_gb300.ragged import RaggedCache
    w = synth.small(L=1, batch=2, N=100, H=2, H_q=4, H_p=1)
    c = RaggedCache(w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, synth.budgets_hat(w), synth.contexts(w), n_cta=4, device=cuda)
    c.compact_layer(0, synth.scores(w, 0, cuda), *synth.keys_values(w, 0, cuda))
    q = torch.randn((2, 4, w.d), device=cuda).to(torch.bfloat16)
    want, out = torch.empty_like(q), torch.zeros_like(q)
    c.decode_layer(0, q, want)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    _in_a_thread(lambda: c.decode_layer(0, q, out, stream=stream))
    assert torch.equal(out, want)


def test_fused_sparse_layer(lib, cuda):
    from non_uniform_paged_gb300.ragged import SparseDecoder, build_minmax
    w = synth.workload(4, batch=2, N=400, L=1)
    n = w.N // w.P
    K, V = (t.view(w.batch, w.H, n, w.P, w.d) for t in synth.keys_values(w, 0, cuda))
    pool, mm = torch.stack([K, V], 3).contiguous(), build_minmax(K.reshape(w.batch, w.H, -1, w.d), w.P)
    q = torch.randn((w.batch, w.H_q, w.d), device=cuda).to(torch.bfloat16)
    dec = SparseDecoder(w.batch, w.H, w.H_q, w.d, w.P, n, 10, device=cuda)
    want, out = torch.empty_like(q), torch.zeros_like(q)
    dec.step(q, mm, pool, want)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    _in_a_thread(lambda: dec.step_fused(q, mm, pool, out, stream=stream))
    assert torch.equal(out, want)
    lib.tg_check_status(dec.status)
