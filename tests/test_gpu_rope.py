"""tg_qk_norm_rope against its 64-bit definition, and what it leaves alone."""
import pytest
import torch

from prompt_helpers import rope64

pytestmark = pytest.mark.gpu


def _table(max_pos, rot, cuda, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=cuda) / max(rot, 1))
    a = torch.arange(max_pos, dtype=torch.float64, device=cuda)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _run(lib, cuda, lens, start, Nmax, H_q, H, d, rot, pairs=False, qw=True, kw=True, pad=0, eps=1e-6, extra=0, positions=None,
         max_pos=None, seed=0):
    g = torch.Generator(device=cuda).manual_seed(seed)
    T, batch, heads = sum(lens) + pad, len(lens), H_q + 2 * H
    wide = torch.randn((T, heads * d + extra), generator=g, device=cuda).to(torch.bfloat16)
    qkv = wide[:, :heads * d].view(T, heads, d)
    cu = torch.tensor([sum(lens[:i]) for i in range(batch + 1)], dtype=torch.int32, device=cuda)
    st = torch.tensor(start, dtype=torch.int32, device=cuda)
    w = [torch.randn(d, generator=g, device=cuda) if on else None for on in (qw, kw)]
    tab = _table(max_pos or Nmax, rot, cuda) if rot else None
    mark = 7.0
    q = torch.full((T, H_q, d), mark, dtype=torch.bfloat16, device=cuda)
    K = torch.full((batch, H, Nmax, d), mark, dtype=torch.bfloat16, device=cuda)
    V = torch.full_like(K, mark)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device=cuda)
    lib.tg_qk_norm_rope(qkv, cu, st, tab, q, K, V, q_weight=w[0], k_weight=w[1], eps=eps, pairs=pairs, positions=pos,
                        dev_status=status)
    torch.cuda.synchronize()
    return qkv, w, tab, q, K, V, int(status.item()), mark


def _verify(out, lens, start, H_q, H, rot, pairs, eps=1e-6, positions=None, skip=()):
    qkv, w, tab, q, K, V, _, mark = out
    d = q.shape[-1]
    left_k = torch.ones(K.shape[:3], dtype=torch.bool, device=K.device)
    at = 0
    for b, n in enumerate(lens):
        for_rows = range(n)
        for i in for_rows:
            left_k[b, :, start[b] + i] = False
        if n:
            pos = torch.arange(start[b], start[b] + n, device=q.device)
            if positions is not None:
                pos = torch.tensor(positions[at:at + n], device=q.device)
            ref, tol = rope64(qkv[at:at + n], tab[pos] if rot else None, H_q, H, w[0], w[1], eps, pairs, rot)
            got = torch.cat([q[at:at + n], K[b, :, start[b]:start[b] + n].transpose(0, 1),
                             V[b, :, start[b]:start[b] + n].transpose(0, 1)], 1).double()
            d_ = (got - ref).abs()
            assert bool((d_ <= tol).all()), (b, (d_ / tol.clamp_min(1e-30)).max().item())
            assert torch.equal(got[:, H_q + H:], ref[:, H_q + H:])
        at += n
    # rows that no token owns are as they were
    assert bool((K[left_k] == mark).all()) and bool((V[left_k] == mark).all())
    assert bool((q[at:] == mark).all())


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("H_q,H", [(8, 2), (5, 1), (7, 7), (32, 8)])
@pytest.mark.parametrize("rot_of,pairs", [(1, False), (1, True), (2, False), (2, True), (0, False)])
def test_against_definition(lib, cuda, d, H_q, H, rot_of, pairs):
    lens, start, rot = [1, 0, 37, 200], [299, 12, 0, 41], d // rot_of if rot_of else 0
    out = _run(lib, cuda, lens, start, 300, H_q, H, d, rot, pairs, pad=3)
    assert out[6] == 0
    _verify(out, lens, start, H_q, H, rot, pairs)


@pytest.mark.parametrize("rot", [16, 48, 112])
@pytest.mark.parametrize("pairs", [False, True])
def test_odd_rotations(lib, cuda, rot, pairs):
    out = _run(lib, cuda, [9, 4], [3, 0], 16, 3, 1, 128, rot, pairs)
    _verify(out, [9, 4], [3, 0], 3, 1, rot, pairs)


@pytest.mark.parametrize("qw,kw", [(False, False), (True, False), (False, True)])
def test_norm_of_one_side_only(lib, cuda, qw, kw):
    out = _run(lib, cuda, [19], [0], 19, 6, 2, 128, 128, qw=qw, kw=kw)
    _verify(out, [19], [0], 6, 2, 128, False)


def test_many_requests_one_token_each_strided_rows(lib, cuda):
    """A decode step of 200 requests; the rows are slices of a wider buffer."""
    lens, start = [1] * 200, [(i * 37) % 500 for i in range(200)]
    out = _run(lib, cuda, lens, start, 500, 8, 2, 128, 128, extra=24)
    assert out[6] == 0
    _verify(out, lens, start, 8, 2, 128, False)


def test_positions_apart_from_rows(lib, cuda):
    pos = [5, 99, 0, 63, 64, 7]
    out = _run(lib, cuda, [4, 2], [10, 0], 20, 4, 2, 128, 128, positions=pos, max_pos=100)
    _verify(out, [4, 2], [10, 0], 4, 2, 128, False, positions=pos)


def test_zero_rows_stay_finite(lib, cuda):
    """A head of zeros has norm sqrt(eps): 0 comes out."""
    qkv = torch.zeros((2, 3, 128), dtype=torch.bfloat16, device=cuda)
    q = torch.full((2, 1, 128), 5.0, dtype=torch.bfloat16, device=cuda)
    K = torch.full((1, 1, 2, 128), 5.0, dtype=torch.bfloat16, device=cuda)
    w = torch.ones(128, device=cuda)
    cu = torch.tensor([0, 2], dtype=torch.int32, device=cuda)
    lib.tg_qk_norm_rope(qkv, cu, cu[:1].clone(), _table(2, 128, cuda), q, K, K.clone(), q_weight=w, k_weight=w)
    assert bool((q == 0).all()) and bool((K == 0).all())


def test_rows_and_positions_outside_write_nothing(lib, cuda):
    """Context rows past Nmax and positions past the table set the status; their neighbours are written."""
    out = _run(lib, cuda, [4], [6], 8, 2, 1, 128, 128)  # rows 6..9 of 8
    assert out[6] == lib.STATUS_BAD_INPUT
    q, mark = out[3], out[7]
    assert bool((q[2:] == mark).all()) and not bool((q[:2] == mark).all(-1).any())
    out = _run(lib, cuda, [3], [0], 8, 2, 1, 128, 128, positions=[0, -1, 9], max_pos=8)
    assert out[6] == lib.STATUS_BAD_INPUT
    assert bool((out[3][1:] == mark).all()) and bool((out[4][0, :, 1:] == mark).all())
    out = _run(lib, cuda, [3], [-2], 8, 2, 1, 128, 0)
    assert out[6] == lib.STATUS_BAD_INPUT and bool((out[3][:2] == mark).all())


def test_offsets_past_32_bits(lib, cuda):
    """A context buffer of more than 2^31 values: the last request's rows lie behind them."""
    H, Nmax, d = 1, 8_400_000, 128
    K = torch.empty((2, H, Nmax, d), dtype=torch.bfloat16, device=cuda)
    V = torch.empty_like(K)
    qkv = torch.randn((2, 3, d), device=cuda).to(torch.bfloat16)
    q = torch.empty((2, 1, d), dtype=torch.bfloat16, device=cuda)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda)
    start = torch.tensor([0, Nmax - 1], dtype=torch.int32, device=cuda)
    lib.tg_qk_norm_rope(qkv, cu, start, None, q, K, V)
    assert torch.equal(K[1, 0, Nmax - 1], qkv[1, 1]) and torch.equal(V[1, 0, Nmax - 1], qkv[1, 2])
    assert torch.equal(K[0, 0, 0], qkv[0, 1]) and torch.equal(q, qkv[:, :1])


@pytest.mark.parametrize("T", [16, 3000])
def test_same_bits_in_a_graph_and_on_two_streams(lib, cuda, T):
    ins, ref = [], []
    for seed in (1, 2):
        out = _run(lib, cuda, [T], [0], T, 8, 2, 128, 128, seed=seed)
        qkv, w, tab, q, K, V, status, _ = out
        assert status == 0
        ins.append((qkv, w, tab)), ref.append((q.clone(), K.clone(), V.clone()))
    cu = torch.tensor([0, T], dtype=torch.int32, device=cuda)
    start = torch.zeros(1, dtype=torch.int32, device=cuda)
    bufs = [tuple(torch.empty_like(t) for t in r) for r in ref]

    def call(i):
        (qkv, w, tab), (q, K, V) = ins[i], bufs[i]
        lib.tg_qk_norm_rope(qkv, cu, start, tab, q, K, V, q_weight=w[0], k_weight=w[1])

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(i)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(bufs, ref) for a, b in zip(x, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        call(0), call(1), call(0)
    for x in bufs:
        for t in x:
            t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(bufs, ref) for a, b in zip(x, y))


def test_long_rows_past_the_first_batches(lib, cuda):
    """Head counts that leave batches and warps half filled, with more tokens than one warp each."""
    for H_q, H, d, T in ((33, 3, 128, 2100), (9, 1, 256, 2050), (64, 8, 128, 70), (1, 1, 256, 5)):
        out = _run(lib, cuda, [T], [0], T, H_q, H, d, d, seed=T)
        assert out[6] == 0
        _verify(out, [T], [0], H_q, H, d, False)


def test_binding_refusals(lib, cuda):
    qkv = torch.zeros((2, 3, 128), dtype=torch.bfloat16, device=cuda)
    q, K = torch.zeros((2, 1, 128), dtype=torch.bfloat16, device=cuda), torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16, device=cuda)
    cu, st = torch.tensor([0, 2], dtype=torch.int32, device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
    for bad in (dict(qkv=qkv[:1]), dict(qkv=qkv.transpose(1, 2).contiguous().transpose(1, 2)), dict(K=K[0]), dict(V=K[:, :, :2]),
                dict(cu_q=cu[:1]), dict(q_weight=torch.ones(64, device=cuda))):
        with pytest.raises(ValueError):
            lib.tg_qk_norm_rope(**dict(dict(qkv=qkv, cu_q=cu, start=st, cos_sin=None, q=q, K=K, V=K), **bad))
    for bad in (dict(qkv=qkv.float()), dict(q=q.half()), dict(start=st.long()), dict(cu_q=cu.cpu())):
        with pytest.raises(TypeError):
            lib.tg_qk_norm_rope(**dict(dict(qkv=qkv, cu_q=cu, start=st, cos_sin=None, q=q, K=K, V=K), **bad))


def test_more_heads_than_a_product_of_batches_holds(lib, cuda):
    """A token's batches squared pass 2^31."""
    out = _run(lib, cuda, [1], [2], 4, 400_000, 1, 128, 128, seed=5)
    assert out[6] == 0
    _verify(out, [1], [2], 400_000, 1, 128, False)
