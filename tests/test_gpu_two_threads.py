"""Decode calls from two host threads at once, each with its plan, workspace and stream: plans of unlike head counts, whose launches
take unlike amounts of shared memory."""
import threading

import numpy as np
import pytest
import torch

import synth
from test_gpu_grown import Lists

pytestmark = pytest.mark.gpu


def _at_once(jobs, calls):
    """Each job `calls` times in a thread of its own; the exceptions that they raised."""
    failed, go = [], threading.Barrier(len(jobs))

    def work(job):
        try:
            go.wait(30)
            for _ in range(calls):
                job()
        except Exception as e:  # noqa: BLE001 (what a call raised is what is tested)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return failed


@pytest.mark.parametrize("pages", ["bf16", "e2m1"])
@pytest.mark.parametrize("d", [128, 256])
def test_grown_decodes_of_one_and_of_eight_heads(lib, cuda, pages, d):
    xs = [Lists(cuda, pages, [[100, 30]], 2 * g, d, reserve=2, n_cta=4, hostile=False, seed=g) for g in (1, 8)]
    want = [x.run([1], 1)[:2] for x in xs]
    got = [[torch.empty_like(t) for t in w] for w in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()

    def job(i):
        x = xs[i]
        return lambda: x.lists.attend(0, x.q, x.pool, x.n, x.off, x.ids, got[i][0], lse=got[i][1], stream=streams[i])

    assert _at_once([job(0), job(1)], 4000) == []
    for w, y in zip(want, got):
        assert torch.equal(w[0], y[0]) and torch.equal(w[1], y[1])


def test_static_decodes_of_one_and_of_eight_heads(lib, cuda):
    """(The bare calls: what the ctypes binding does around each takes longer than a call, so that two hardly ever meet.)"""
    from non_uniform_paged_gb300.ragged import RaggedCache
    so, jobs, want, got, kept = lib.load(), [], [], [], []
    for g in (1, 8):
        w = synth.small(L=1, batch=2, N=100, H=2, H_q=2 * g, H_p=1)
        c = RaggedCache(w.L, w.batch, w.H, w.H_q, w.d, w.P, w.H_p, w.alpha, synth.budgets_hat(w), synth.contexts(w), n_cta=4,
                        device=cuda)
        c.compact_layer(0, synth.scores(w, 0, cuda), *synth.keys_values(w, 0, cuda))
        q = torch.randn((2, w.H_q, w.d), device=cuda).to(torch.bfloat16)
        ref, out, s = torch.empty_like(q), torch.empty_like(q), torch.cuda.Stream()
        c.decode_layer(0, q, ref)
        want.append(ref), got.append(out), kept.append((c, q, s))
        args = [s.cuda_stream, c.plan.ctypes.data, c.plan_dev.data_ptr(), 0, q.data_ptr(), c.pool.data_ptr(), c.n_pages,
                c.list_offsets(0).data_ptr(), c.pt_ids_dev.data_ptr(), c.scale, c.workspace.data_ptr(), c.workspace_bytes,
                out.data_ptr(), None, c.status.data_ptr(), None]

        def job(args=args, call=so.tg_decode_attn):
            for _ in range(10):
                assert call(*args) == 0

        jobs.append(job)
    torch.cuda.synchronize()
    assert _at_once(jobs, 2000) == []
    assert all(torch.equal(a, b) for a, b in zip(want, got))
