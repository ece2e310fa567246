"""tg_prefill_attn against its 64-bit definition: lengths, masks, windows, heads, cut runs, rows
that hold anything behind the contexts."""
import math

import pytest
import torch

from prompt_helpers import attend64, check, seen_keys

pytestmark = pytest.mark.gpu


def _inputs(cuda, q_len, kv_len, H, H_q, d, Nmax, seed=0, gain=1.0):
    g = torch.Generator(device=cuda).manual_seed(seed)
    q = (gain * torch.randn((sum(q_len), H_q, d), generator=g, device=cuda)).to(torch.bfloat16)
    K = torch.randn((len(q_len), H, Nmax, d), generator=g, device=cuda).to(torch.bfloat16)
    V = torch.randn((len(q_len), H, Nmax, d), generator=g, device=cuda).to(torch.bfloat16)
    for b, n in enumerate(kv_len):  # what lies behind a context is anybody's
        K[b, :, n:] = float("nan")
        V[b, :, n:] = float("inf")
    return q, K, V


def _run(lib, cuda, q_len, kv_len, H, g, d, window=0, n_cta=None, Nmax=None, seed=0, gain=1.0, rows=None):
    from non_uniform_paged_gb300.ragged import PrefillPass
    Nmax = Nmax or max(max(kv_len), 1)
    q, K, V = _inputs(cuda, q_len, kv_len, H, H * g, d, Nmax, seed, gain)
    p = PrefillPass(H, H * g, d, q_len, kv_len, window=window, n_cta=n_cta, device=cuda)
    out = torch.full_like(q, 9.0)
    lse = torch.full(q.shape[:2], 9.0, device=cuda)
    p.attend(q, K, V, out, lse)
    torch.cuda.synchronize()
    assert lib.tg_check_status(p.status) == 0
    at = 0
    for b, (nq, nk) in enumerate(zip(q_len, kv_len)):
        seen = seen_keys(nq, nk, window, cuda)
        for j in range(H * g):
            if nq:
                ref = attend64(q[at:at + nq, j], K[b, j // g, :nk], V[b, j // g, :nk], 1 / math.sqrt(d), seen)
                check(out[at:at + nq, j], lse[at:at + nq, j], ref, f"request {b} head {j}")
        at += nq
    return p, q, K, V, out, lse


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n", [1, 2, 31, 64, 127, 128, 129, 255, 256, 257, 515])
def test_whole_prompts(lib, cuda, d, n):
    _run(lib, cuda, [n], [n], 2, 4, d, seed=n)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 6, 7, 8])
def test_head_groups(lib, cuda, d, g):
    _run(lib, cuda, [70, 1, 130], [70, 90, 400], 2, g, d, seed=g)


@pytest.mark.parametrize("d", [128, 256])
def test_packed_lengths_with_empty_requests(lib, cuda, d):
    _run(lib, cuda, [0, 5, 0, 300, 1, 64, 0], [0, 5, 17, 300, 1, 640, 0], 1, 2, d, Nmax=700)


@pytest.mark.parametrize("d", [128, 256])
def test_rows_ahead_of_the_context_see_nothing(lib, cuda, d):
    """More queries than keys: the first rows get out 0 and lse -inf, also with no key at all."""
    for q_len, kv_len in (([200], [60]), ([40], [0]), ([3, 300, 5], [1, 130, 0])):
        _, _, _, _, out, lse = _run(lib, cuda, q_len, kv_len, 2, 3, d)
        first = q_len[0] - kv_len[0]
        assert bool((out[:first] == 0).all()) and bool(torch.isneginf(lse[:first]).all())


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000])
def test_windows(lib, cuda, d, window):
    _run(lib, cuda, [300, 90, 1], [300, 700, 520], 1, 4, d, window=window)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("n_cta", [1, 2, 5, 152])
def test_results_do_not_hang_on_the_block_count(lib, cuda, d, n_cta):
    """Few blocks: many items one after the other; many: cut runs and the merge."""
    _run(lib, cuda, [150, 40, 700], [1500, 2000, 700], 2, 2, d, n_cta=n_cta)


@pytest.mark.parametrize("d", [128, 256])
def test_single_tokens_on_long_contexts_are_cut(lib, cuda, d):
    p, *_ = _run(lib, cuda, [1, 2, 1], [9000, 4097, 20001], 2, 4, d)
    assert p.plan.header["n_merge"] > 0


@pytest.mark.parametrize("d", [128, 256])
def test_peaked_and_rising_logits(lib, cuda, d):
    """Large logits whose maximum keeps rising along the keys: the reference moves many times."""
    from non_uniform_paged_gb300.ragged import PrefillPass
    g = torch.Generator(device=cuda).manual_seed(1)
    n, H, gq = 700, 1, 4
    q = (3 * torch.randn((n, H * gq, d), generator=g, device=cuda)).to(torch.bfloat16)
    K = torch.randn((1, H, n, d), generator=g, device=cuda)
    K = (K * torch.linspace(0.1, 4, n, device=cuda)[:, None]).to(torch.bfloat16)
    V = torch.randn((1, H, n, d), generator=g, device=cuda).to(torch.bfloat16)
    p = PrefillPass(H, H * gq, d, [n], [n], device=cuda)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    p.attend(q, K, V, out, lse)
    for j in range(gq):
        check(out[:, j], lse[:, j], attend64(q[:, j], K[0, 0], V[0, 0], 1 / math.sqrt(d), seen_keys(n, n, 0, cuda)), j)


def test_scale_and_missing_lse(lib, cuda):
    from non_uniform_paged_gb300.ragged import PrefillPass
    q, K, V = _inputs(cuda, [50], [50], 1, 2, 128, 50)
    p = PrefillPass(1, 2, 128, [50], [50], device=cuda)
    out = torch.empty_like(q)
    p.attend(q, K, V, out, scale=0.5)
    for j in range(2):
        check(out[:, j], None, attend64(q[:, j], K[0, 0], V[0, 0], 0.5, seen_keys(50, 50, 0, cuda)))


def test_same_bits_every_time_and_in_a_graph(lib, cuda):
    p, q, K, V, out, lse = _run(lib, cuda, [64, 3], [5000, 9000], 2, 4, 128)
    again, l2 = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(3):
        p.attend(q, K, V, again, l2)
        assert torch.equal(again, out) and torch.equal(l2, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        p.attend(q, K, V, again, l2)
    for _ in range(2):
        again.zero_(), l2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out) and torch.equal(l2, lse)


def test_two_passes_on_two_streams(lib, cuda):
    a = _run(lib, cuda, [64, 3], [5000, 9000], 2, 4, 128, seed=1)
    b = _run(lib, cuda, [700, 1], [700, 12000], 2, 4, 256, seed=2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    for _ in range(5):
        for (p, q, K, V, out, lse), s in zip((a, b), streams):
            o, l = torch.empty_like(out), torch.empty_like(lse)
            with torch.cuda.stream(s):
                p.attend(q, K, V, o, l)
            got.append((o, l, out, lse))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ro) and torch.equal(l, rl) for o, l, ro, rl in got)


def test_window_as_large_as_it_gets(lib, cuda):
    for w in (130, 2**31 - 1):
        _run(lib, cuda, [40, 200], [130, 60], 1, 4, 128, window=w)


def test_more_blocks_than_the_device_has(lib, cuda):
    """A plan for 1000 blocks on fewer SMs: they follow one another."""
    p, *_ = _run(lib, cuda, [300, 700, 90], [3000, 700, 9000], 4, 4, 128, n_cta=1000)
    assert p.plan.header["N_CTA"] > torch.cuda.get_device_properties(0).multi_processor_count


def test_keys_that_raise_the_reference_in_every_block(lib, cuda):
    """Each block's logits tower over the ones before, by more than the weights may grow: the block
    is done again with its own maximum, in all rows or in some of a warp's."""
    from non_uniform_paged_gb300.ragged import PrefillPass
    for d in (128, 256):
        n = 500
        q = torch.ones((n, 2, d), device=cuda).to(torch.bfloat16)
        q[::3] = 0.01  # these rows' logits stay small
        K = (torch.arange(n, device=cuda) // 40 * (400.0 / d))[None, None, :, None].expand(1, 1, n, d).to(torch.bfloat16).contiguous()
        V = torch.randn((1, 1, n, d), generator=torch.Generator(device=cuda).manual_seed(4), device=cuda).to(torch.bfloat16)
        p = PrefillPass(1, 2, d, [n], [n], device=cuda)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
        p.attend(q, K, V, out, lse, scale=1 / 16)
        for j in range(2):
            check(out[:, j], lse[:, j], attend64(q[:, j], K[0, 0], V[0, 0], 1 / 16, seen_keys(n, n, 0, cuda)), (d, j))


def test_contexts_past_32_bit_offsets(lib, cuda):
    """2^31 and more values ahead of the rows that are read; a window keeps the work small."""
    from non_uniform_paged_gb300.ragged import PrefillPass
    n, d = 17_000_001, 128
    K = torch.zeros((1, 1, n, d), dtype=torch.bfloat16, device=cuda)
    V = torch.zeros_like(K)
    g = torch.Generator(device=cuda).manual_seed(5)
    K[0, 0, -400:] = torch.randn((400, d), generator=g, device=cuda).to(torch.bfloat16)
    V[0, 0, -400:] = torch.randn((400, d), generator=g, device=cuda).to(torch.bfloat16)
    q = torch.randn((5, 2, d), generator=g, device=cuda).to(torch.bfloat16)
    p = PrefillPass(1, 2, d, [5], [n], window=300, device=cuda)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=cuda)
    p.attend(q, K, V, out, lse)
    for j in range(2):
        check(out[:, j], lse[:, j], attend64(q[:, j], K[0, 0, -400:], V[0, 0, -400:], 1 / math.sqrt(d),
                                            seen_keys(5, 400, 300, cuda)))


def test_binding_refusals(lib, cuda):
    p, q, K, V, out, lse = _run(lib, cuda, [5], [9], 1, 2, 128)
    for bad in (dict(q=q[:4]), dict(K=K[:, :, :, :64]), dict(V=V[:, :, :8]), dict(out=out[:, :1]), dict(lse=lse[:4])):
        with pytest.raises(ValueError):
            p.attend(**dict(dict(q=q, K=K, V=V, out=out, lse=lse), **bad))
    with pytest.raises(TypeError):
        p.attend(q.float(), K, V, out)
    with pytest.raises(TypeError):
        p.attend(q.cpu(), K, V, out)
    with pytest.raises(lib.TGError) as e:
        p.attend(q, K[:, :, :8].contiguous(), V[:, :, :8].contiguous(), out)
    assert e.value.code == lib.ERR_SHAPE
    with pytest.raises(lib.TGError):
        p.attend(q, K, V, out, scale=0.0)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("window", [1, 50, 79, 80, 81, 300])
def test_rows_ahead_of_every_window_hold_anything(lib, cuda, d, window):
    """Rows that no token of the pass sees, ahead of its first window as behind its end."""
    from non_uniform_paged_gb300.ragged import PrefillPass
    q_len, kv_len, H, g = [1, 90, 300, 40], [700, 333, 1203, 60], 2, 4
    for n_cta in (1, 152):
        q, K, V = _inputs(cuda, q_len, kv_len, H, H * g, d, max(kv_len), seed=window)
        for b in range(len(q_len)):
            first = max(0, kv_len[b] - q_len[b] - window + 1)
            K[b, :, :first] = float("inf")
            V[b, :, :first] = float("nan")
        p = PrefillPass(H, H * g, d, q_len, kv_len, window=window, n_cta=n_cta, device=cuda)
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device=cuda)
        p.attend(q, K, V, out, lse)
        at = 0
        for b, (nq, nk) in enumerate(zip(q_len, kv_len)):
            first = max(0, nk - nq - window + 1)
            seen = seen_keys(nq, nk, window, cuda)[:, first:]
            for j in range(H * g):
                ref = attend64(q[at:at + nq, j], K[b, j // g, first:nk], V[b, j // g, first:nk], 1 / math.sqrt(d), seen)
                check(out[at:at + nq, j], lse[at:at + nq, j], ref, f"request {b} head {j}")
            at += nq
