"""Cases that measure the operators of a cache that grows and of pages held in 4 bits.

Five operators work on the ragged pages beside retention and the static decode step:

  append   the packed projections of new tokens -> normalised and rotated queries, and their K and V
           rows behind the retained ones in the pages, which hold bf16 or 4 bits; positions of one or
           several axes (tg_append_rope);
  quant    retained bf16 pages into 4-bit pages (tg_quant_pages; read back by tg_dequant_pages, so
           that what the pages stand for is compared);
  dequant  4-bit pages into bf16 pages, for the operators that read those (tg_dequant_pages);
  decode   decode attention over retained and appended tokens, of bf16 pages and of 4-bit pages
           (tg_decode_grown).

With ``own`` false, ``run`` computes each in elementary torch operations; with ``own`` true it makes
the library's calls.  ``exact`` is a separate 64-bit computation from the definitions.

4-bit pages: blocks of 16 consecutive values of a row share a scale s, the e4m3 number nearest to
max|x| / (6 unit), at least 2^-9; a value is held as the e2m1 number nearest to x / (unit s), both with
ties to the even code, both saturating.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: 16 requests, one new token each, bf16 pages
        dict(name="append-step-16", op="append", fmt="bf16", H_q=32, H=8, d=128, P=16, H_p=4, batch=16, q_lo=1, q_hi=1,
             kept_lo=400, kept_hi=4096, grown=37, axes=1, rot=128, pairs=False, norm=True, dense=False, pad=0),
        # prompts of text and images (time, height, width) behind nothing retained yet
        dict(name="append-image-8", op="append", fmt="bf16", H_q=32, H=8, d=128, P=16, H_p=4, batch=8, q_lo=700,
             q_hi=4096, kept_lo=1, kept_hi=1, grown=0, axes=3, rot=128, pairs=False, norm=True, dense=False, pad=13),
        # follow-up turns onto 4-bit pages, whose tokens the pass itself attends to as the pages hold them
        dict(name="append4-turns-12", op="append", fmt="e2m1", H_q=16, H=8, d=256, P=16, H_p=4, batch=12, q_lo=60,
             q_hi=1500, kept_lo=2000, kept_hi=9000, grown=11, axes=1, rot=256, pairs=False, norm=True, dense=True, pad=0),
        # a short prompt's layer into 4 bits: latency counts
        dict(name="quant-short-1", op="quant", H=8, d=128, P=16, H_p=4, batch=1, N=700, b_lo=0.1, b_hi=1.0),
        # a layer of a batch of long prompts into 4 bits
        dict(name="quant-long-16", op="quant", H=8, d=128, P=16, H_p=4, batch=16, N=32768, b_lo=0.1, b_hi=0.5),
        # one conversation's layer out of 4 bits, before a turn attends to it
        dict(name="dequant-turn-1", op="dequant", H=8, d=128, P=16, H_p=4, batch=1, N=4096, b_lo=0.1, b_hi=1.0),
        # a layer with 256-wide heads of a batch out of 4 bits, single-head lists
        dict(name="dequant-wide-16", op="dequant", H=8, d=256, P=32, H_p=1, batch=16, N=16384, b_lo=0.2, b_hi=1.0),
        # one request's decode step over bf16 pages: latency counts
        dict(name="decode-short-1", op="decode", fmt="bf16", H_q=32, H=8, d=128, P=16, H_p=4, batch=1, N=4096, b_lo=0.1,
             b_hi=1.0, reserve=256, grown=99),
        # a batch of long contexts with head-wise budgets, bf16 pages
        dict(name="decode-long-16", op="decode", fmt="bf16", H_q=32, H=8, d=128, P=16, H_p=4, batch=16, N=32768, b_lo=0.1,
             b_hi=0.5, reserve=1024, grown=700),
        # one request's decode step over 4-bit pages: latency counts
        dict(name="decode4-short-1", op="decode", fmt="e2m1", H_q=32, H=8, d=128, P=16, H_p=4, batch=1, N=4096, b_lo=0.1,
             b_hi=1.0, reserve=256, grown=99),
        # a batch of long contexts, 4-bit pages
        dict(name="decode4-long-32", op="decode", fmt="e2m1", H_q=32, H=8, d=128, P=16, H_p=4, batch=32, N=32768,
             b_lo=0.1, b_hi=0.5, reserve=1024, grown=700),
        # 256-wide heads, two query heads to a KV head
        dict(name="decode4-wide-16", op="decode", fmt="e2m1", H_q=16, H=8, d=256, P=16, H_p=4, batch=16, N=65536,
             b_lo=0.05, b_hi=0.4, reserve=512, grown=17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "quant", "dequant", "decode", "decode", "decode"])
    d = rng.choice([128, 128, 256])
    H = rng.choice([1, 2, 3, 4, 8])
    H_q = H * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    P = rng.choice([16, 16, 32, 48, 64])
    H_p = rng.choice([p for p in (1, 2, 3, 4) if H % p == 0])
    fmt = rng.choice(["bf16", "e2m1"])
    if op == "append":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, min(8192, 60000000 // ((H_q + 2 * H) * d)) // batch))
        kept = _log(rng, 1, 4096 if batch < 9 else 1024)
        return dict(op=op, fmt=fmt, H_q=H_q, H=H, d=d, P=P, H_p=H_p, batch=batch, q_lo=max(1, hi // rng.choice([1, 4, 16])),
                    q_hi=hi, kept_lo=max(1, kept // rng.choice([1, 8])), kept_hi=kept, grown=rng.choice([0, 1, _log(rng, 1, 200)]),
                    axes=rng.choice([1, 1, 2, 3, 4]), rot=rng.choice([d, d, d // 2, d - 16, 48]), pairs=rng.random() < 0.3,
                    norm=rng.random() < 0.8, dense=fmt == "e2m1" or rng.random() < 0.3, pad=rng.choice([0, 0, 5, 100]))
    batch = _log(rng, 1, 32)
    N = _log(rng, 16, min(65536, 1200000 // (batch * H) * 128 // d))  # rows of 1.2M x 128 at most
    b_lo = rng.choice([0.03, 0.3, 1.0])
    if op != "decode":
        return dict(op=op, H=H, d=d, P=P, H_p=H_p, batch=batch, N=N, b_lo=b_lo, b_hi=max(b_lo, 0.6))
    reserve = _log(rng, 1, 2000)
    return dict(op=op, fmt=fmt, H_q=H_q, H=H, d=d, P=P, H_p=H_p, batch=batch, N=N, b_lo=b_lo, b_hi=max(b_lo, 0.6),
                reserve=reserve, grown=rng.choice([0, reserve - 1, rng.randrange(reserve)]))


def _lengths(case):
    """Tokens that each request brings: log-uniform in [q_lo, q_hi]; they follow from the case, not from the
    seed, so that every seed is the same amount of work."""
    lo, hi = case["q_lo"], case["q_hi"]
    g = torch.Generator().manual_seed(case["batch"] * 7919 + hi * 31 + lo * 17)
    u = torch.rand(case["batch"], generator=g, dtype=torch.float64)
    return [min(hi, max(lo, int(round(math.exp(math.log(lo) + float(x) * (math.log(hi) - math.log(lo))))))) for x in u]


def _kept(case):
    """Retained tokens of each (request, head), evenly spread and shuffled: ceil(B N), or kept_lo to kept_hi."""
    n = case["batch"] * case["H"]
    if case["op"] == "append":
        lo, hi, N = float(case["kept_lo"]), float(case["kept_hi"]), 1 << 30
    else:
        N = case["N"]
        lo, hi = case["b_lo"] * N, case["b_hi"] * N
    g = torch.Generator().manual_seed(n * 13 + case["P"])
    at = torch.randperm(n, generator=g).tolist()
    kept = [max(1, min(N, math.ceil(lo + (hi - lo) * i / max(1, n - 1)))) for i in at]
    return [kept[b * case["H"]:(b + 1) * case["H"]] for b in range(case["batch"])]


def _reserve(case):
    return case["grown"] + case["q_hi"] if case["op"] == "append" else case.get("reserve", 0)


def _page_counts(case):
    """Pages of each list (request, group): its longest head and the reserve."""
    H_p, P = case["H_p"], case["P"]
    return [-(-(max(k[i:i + H_p]) + _reserve(case)) // P) for k in _kept(case) for i in range(0, case["H"], H_p)]


# ------------------------------------------------------------------ inputs

def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * scale


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def _pool4(pages, case, g):
    """4-bit pages [pages][H_p][P/16][d/128][2304] with any codes, and scales from 2^-3 to 2."""
    pool = torch.randint(0, 256, (pages, case["H_p"], case["P"] // 16, case["d"] // 128, 2304), generator=g, device=DEV,
                         dtype=torch.uint8)
    pool[..., 2048:] = pool[..., 2048:] % 0x20 + 0x20
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    H, d, P, H_p, batch = case["H"], case["d"], case["P"], case["H_p"], case["batch"]
    kept = _kept(case)
    off = _offsets(_page_counts(case))
    s["pages"] = off[-1]
    s["ntok"] = _ints(kept)
    s["most"] = max(map(max, kept)) + case.get("grown", 0) + 1  # of a decode step
    s["pt_off"] = _ints(off, torch.int64)
    s["pt_ids"] = torch.randperm(off[-1], generator=g, device=DEV).to(torch.int32)  # pages lie anywhere
    if own:
        import numpy as np
        from non_uniform_paged_gb300.ragged import GrowingLists
        s["lists"] = GrowingLists(case.get("H_q", H), H_p, P, d, np.arange(H, dtype=np.int32), np.asarray(kept, np.int32),
                                  _reserve(case), pages=case.get("fmt", "e2m1"), device=DEV)
        s["lists"].added.fill_(case.get("grown", 0))
    if case["op"] == "append":
        return _prepare_append(s, case, g)
    bf16 = (off[-1], H_p, 2, P, d)
    if case["op"] == "quant":
        s["src"] = _randn(bf16, g, 1.3)
        s["pool"] = torch.zeros((off[-1], H_p, P // 16, d // 128, 2304), dtype=torch.uint8, device=DEV)
        s["back"] = torch.zeros(bf16, dtype=torch.bfloat16, device=DEV)
    elif case["op"] == "dequant":
        s["pool"] = _pool4(off[-1], case, g)
        s["back"] = torch.zeros(bf16, dtype=torch.bfloat16, device=DEV)
    else:
        s["pool"] = _randn(bf16, g) if case["fmt"] == "bf16" else _pool4(off[-1], case, g)
        s["q"] = _randn((batch, case["H_q"], d), g, 1.5)
        s["out"] = torch.zeros((batch, case["H_q"], d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((batch, case["H_q"]), dtype=torch.float32, device=DEV)
    return s


def _prepare_append(s, case, g):
    H, H_q, d, P, batch, rot, axes = (case[k] for k in ("H", "H_q", "d", "P", "batch", "rot", "axes"))
    lens = _lengths(case)
    off = _offsets(lens)
    rows, far = off[-1] + case["pad"], 8192
    s["tokens"] = off[-1]
    s["cu_q"] = _ints(off)
    s["qkv"] = _randn((rows, H_q + 2 * H, d), g, 1.7)
    s["q_weight"] = torch.rand(d, generator=g, device=DEV) + 0.5 if case["norm"] else None
    s["k_weight"] = torch.rand(d, generator=g, device=DEV) + 0.5 if case["norm"] else None
    # the rotation's table, made in 64 bits once and kept: cos and sin of position * base^(-2i/rot)
    freq = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * freq
    s["table"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
    # one axis: token i of request b stands at origin[b] + grown + i; several: a position for each, pairs dealt out in turn
    s["origin"] = torch.randint(0, far - s["grown"] - case["q_hi"], (batch,), generator=g, device=DEV).to(torch.int32)
    s["positions"] = torch.randint(0, far, (rows, axes), generator=g, device=DEV).to(torch.int32) if axes > 1 else None
    s["axis_of"] = [i % axes for i in range(rot // 2)] if axes > 1 else None
    s["q"] = torch.zeros((rows, H_q, d), dtype=torch.bfloat16, device=DEV)
    s["pool"] = torch.zeros((s["pages"], case["H_p"], 2, P, d), dtype=torch.bfloat16, device=DEV) if case["fmt"] == "bf16" \
        else torch.zeros((s["pages"], case["H_p"], P // 16, d // 128, 2304), dtype=torch.uint8, device=DEV)
    s["K"] = torch.zeros((batch, H, max(lens), d), dtype=torch.bfloat16, device=DEV) if case["dense"] else None
    s["V"] = torch.zeros_like(s["K"]) if case["dense"] else None
    s["start"] = torch.zeros(batch, dtype=torch.int32, device=DEV) if case["dense"] else None
    return s


# ------------------------------------------------------------------ one pass, plain

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _held(x):
    """What 4-bit pages hold of x [...][d]: blocks of 16 with a scale of their own."""
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1, keepdim=True) / 6).clamp(max=448).to(torch.float8_e4m3fn).to(x.dtype).clamp_min(2.0 ** -9)
    r = b.abs() / s
    code = (r > 0.25).int() + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5)
    v = torch.tensor(E2M1, dtype=x.dtype, device=x.device)[code] * s
    return torch.where(b < 0, -v, v).flatten(-2)


def _values(tiles, V):
    """What 4-bit tiles [...][d/128][2304] stand for: K (or V) rows [...][16][d] in 32 bits."""
    at, sc = (1024, 2176) if V else (0, 2048)
    byte = tiles[..., at:at + 1024]
    s = tiles[..., sc:sc + 128].contiguous().view(torch.float8_e4m3fn).float()
    if V:  # [half of 8 tokens][block of 16 values][token][8 bytes], scales [block][token]
        byte = byte.unflatten(-1, (2, 8, 8, 8)).transpose(-2, -3).flatten(-2).flatten(-3, -2).flatten(-2).unflatten(-1, (16, 64))
        s = s.unflatten(-1, (8, 16)).transpose(-1, -2)
    else:  # [token][64 bytes], scales [token][block]
        byte, s = byte.unflatten(-1, (16, 64)), s.unflatten(-1, (16, 8))
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=tiles.device)
    v = table[torch.stack([byte & 15, byte >> 4], -1).int()].flatten(-2)  # the low four bits first
    v = (v.unflatten(-1, (8, 16)) * s[..., None]).flatten(-2)             # [...][d/128][16][128]
    return v.transpose(-2, -3).flatten(-2)


def _append_plain(s):
    H_q, H, d, rot, n, P, H_p = (s[k] for k in ("H_q", "H", "d", "rot", "tokens", "P", "H_p"))
    # in 64 bits where a value goes to 4: next to the border of two of them 32 say the wrong one
    kind = torch.float32 if s["fmt"] == "bf16" else torch.float64
    x = s["qkv"][:n].to(kind)
    t = torch.arange(n, device=DEV, dtype=torch.int32)
    req = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    i = t - s["cu_q"][req]
    if s["positions"] is None:
        cs = s["table"][(s["origin"][req] + s["grown"] + i).long()]
    else:
        axis = torch.tensor(s["axis_of"], device=DEV)
        cs = s["table"][s["positions"][:n].long()[:, axis], torch.arange(rot // 2, device=DEV)]
    c, sn = cs.to(kind)[:, None].unbind(-1)
    parts = []
    for y, w in ((x[:, :H_q], s["q_weight"]), (x[:, H_q:H_q + H], s["k_weight"])):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.to(kind)
        if s["pairs"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        parts.append(torch.cat([z, y[..., rot:]], -1))
    s["q"][:n] = parts[0].to(torch.bfloat16)
    k, v = parts[1], x[:, H_q + H:]
    if s["fmt"] == "e2m1":
        k, v = _held(k), _held(v)
    else:
        head = torch.arange(H, device=DEV)
        slot = s["ntok"][req] + s["grown"] + i[:, None]
        first = s["pt_off"][req[:, None] * (H // H_p) + head // H_p]
        page = s["pt_ids"][first + slot // P].long()
        s["pool"][page, head % H_p, 0, slot % P] = k.to(torch.bfloat16)
        s["pool"][page, head % H_p, 1, slot % P] = v.to(torch.bfloat16)
    if s["K"] is not None:
        s["K"][req, :, i] = k.to(torch.bfloat16)
        s["V"][req, :, i] = v.to(torch.bfloat16)
    return _append_out(s)


def _append_out(s):
    out = {"q": s["q"]}
    if s["fmt"] == "bf16":
        out["pool"] = s["pool"]
    if s["K"] is not None:
        out["K"], out["V"] = s["K"], s["V"]  # of 4-bit pages: what they hold of the new tokens
    return out


def _rows_of_pages(s):
    """For each page of the lists: [pages][H_p][P] bool, whether the row is a token, and whether it is a row
    behind the last one in its page."""
    H_p, P, G = s["H_p"], s["P"], s["H"] // s["H_p"]
    counts = s["pt_off"].diff()
    lst = torch.repeat_interleave(torch.arange(counts.numel(), device=DEV), counts, output_size=s["pages"])
    k = torch.arange(s["pages"], device=DEV) - s["pt_off"][lst]
    n = s["ntok"].view(-1, G, H_p).flatten(0, 1)[lst][:, :, None]
    row = (k[:, None] * P + torch.arange(P, device=DEV))[:, None]
    return row < n, (row >= n) & (row < (n + P - 1) // P * P)


def _pages_plain(s):
    live, tail = _rows_of_pages(s)
    ids = s["pt_ids"].long()
    if s["op"] == "quant":
        v = _held(s["src"][ids].float()).to(torch.bfloat16)
    else:
        tiles = s["pool"][ids]  # [pages][H_p][P/16][d/128][2304]
        v = torch.stack([_values(tiles, False).flatten(2, 3), _values(tiles, True).flatten(2, 3)], 2).to(torch.bfloat16)
    v = torch.where(live[:, :, None, :, None], v, torch.zeros((), dtype=v.dtype, device=DEV))
    old = s["back"][ids]
    s["back"][ids] = torch.where((live | tail)[:, :, None, :, None], v, old)
    return {"back": s["back"]}


def _decode_plain(s):
    H, H_q, d, P, H_p, batch = (s[k] for k in ("H", "H_q", "d", "P", "H_p", "batch"))
    g, scale = H_q // H, 1.0 / math.sqrt(d)
    n = (s["ntok"] + s["grown"] + 1).long()
    most = s["most"]
    head = torch.arange(H, device=DEV)[:, None]
    tile = torch.arange(-(-most // 16), device=DEV)
    tile = torch.minimum(tile, (n[..., None] - 1) // 16)  # [batch][H][tiles], the last one again behind it
    lst = torch.arange(batch, device=DEV)[:, None, None] * (H // H_p) + head // H_p
    page = s["pt_ids"][s["pt_off"][lst] + tile // (P // 16)].long()
    if s["fmt"] == "bf16":
        view = s["pool"].unflatten(3, (P // 16, 16))
        K, V = (view[page, head % H_p, i, tile % (P // 16)].float().flatten(2, 3) for i in (0, 1))
    else:
        tiles = s["pool"][page, head % H_p, tile % (P // 16)]
        K, V = _values(tiles, False).flatten(2, 3), _values(tiles, True).flatten(2, 3)
    hide = torch.arange(K.shape[2], device=DEV) >= n[..., None]
    q = s["q"].float().view(batch, H, g, d)
    x = torch.matmul(q, K.transpose(-1, -2)).mul_(scale).masked_fill_(hide[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    s["out"].copy_((torch.matmul(x, V) / total).view(batch, H_q, d))
    s["lse"].copy_((total.log() + m).view(batch, H_q))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if not own:
        return {"append": _append_plain, "quant": _pages_plain, "dequant": _pages_plain, "decode": _decode_plain}[s["op"]](s)
    lists, pages, off, ids = s["lists"], s["pages"], s["pt_off"], s["pt_ids"]
    if s["op"] == "append":
        lists.append(0, s["qkv"], s["table"], s["q"], s["pool"], pages, off, ids, cu_q=s["cu_q"], origin=s["origin"],
                     positions=s["positions"], axis_of=s["axis_of"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                     pairs=s["pairs"], K=s["K"], V=s["V"], start=s["start"])
        return _append_out(s)
    if s["op"] == "decode":
        lists.attend(0, s["q"], s["pool"], pages, off, ids, s["out"], lse=s["lse"], plus=1)
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "quant":
        lists.quantize(0, s["src"], pages, off, ids, s["pool"], pages, off, ids)
    lists.dequantize(0, s["pool"], pages, off, ids, s["back"], pages, off, ids)
    return {"back": s["back"]}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    H, d = case["H"], case["d"]
    kept = _kept(case)
    bits4 = 9 / 16  # bytes of a value: four bits, and a scale for sixteen
    if case["op"] == "append":
        n, H_q = sum(_lengths(case)), case["H_q"]
        held = 2 if case["fmt"] == "bf16" else bits4
        rows = n * case["axes"] if case["axes"] > 1 else min(n, 8192)
        byts = 2 * n * (2 * H_q + 2 * H) * d + 2 * n * H * d * (held + (2 if case["dense"] else 0))
        return {"bytes": byts + min(rows, 8192) * case["rot"] * 4, "flops": 7 * n * (H_q + H) * d}
    tokens = sum(map(sum, kept))
    if case["op"] == "quant":
        return {"bytes": 2 * tokens * d * (2 + bits4 + bits4 + 2), "flops": 6 * tokens * d}
    if case["op"] == "dequant":
        return {"bytes": 2 * tokens * d * (2 + bits4), "flops": 2 * tokens * d}
    tokens += (case["grown"] + 1) * H * case["batch"]
    g, io = case["H_q"] // H, case["batch"] * case["H_q"] * (4 * d + 4)
    held = 2 if case["fmt"] == "bf16" else bits4
    return {"bytes": 2 * tokens * d * held + 4 * tokens // case["P"] // case["H_p"] + io, "flops": 4 * tokens * g * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _nearest(x, grid):
    """The place of the number in grid (ascending) nearest to x, ties to the even place."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.bucketize(x, mid), torch.bucketize(x, mid, right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _exact_held(x):
    scales = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    codes = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    blocks = x.double().reshape(*x.shape[:-1], -1, 16)
    top = blocks.abs().max(-1, keepdim=True).values
    s = scales[_nearest(top / 6, scales).clamp_min(1)]
    return (codes[_nearest(blocks.abs() / s, codes)] * s * blocks.sign()).reshape(x.shape)


def _exact_rows(s, b, h, n):
    """K and V rows of n tokens of request b, head h, in 64 bits: out of the bytes one by one."""
    H_p, P, d = s["H_p"], s["P"], s["d"]
    lst = b * (s["H"] // H_p) + h // H_p
    t = torch.arange(n, device=DEV)
    page = s["pt_ids"].long()[s["pt_off"][lst] + t // P]
    if s["pool"].dtype == torch.bfloat16:
        rows = s["pool"][page, h % H_p, :, t % P].double()
        return rows[:, 0], rows[:, 1]
    flat = s["pool"].reshape(-1)
    tile = ((page * H_p + h % H_p) * (P // 16) + t % P // 16) * (d // 128)
    e = torch.arange(d, device=DEV)
    base = (tile[:, None] + e // 128) * 2304
    r, i, j = (t % 16)[:, None], e % 128, e % 128 // 16
    magnitude = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    out = []
    for code_at, scale_at in ((64 * r + i // 2, 2048 + 8 * r + j),
                              (1024 + 512 * (r // 8) + 64 * j + 8 * (r % 8) + i % 16 // 2, 2176 + 16 * j + r)):
        code = (flat[base + code_at] >> (4 * (i % 2)).to(torch.uint8)) & 15
        v = magnitude[(code & 7).long()] * flat[base + scale_at].view(torch.float8_e4m3fn).double()
        out.append(torch.where(code >= 8, -v, v))
    return out


def _exact_append(s):
    H_q, H, rot = s["H_q"], s["H"], s["rot"]
    q, cu = s["q"].double(), s["cu_q"].tolist()
    dense = [torch.zeros(s["K"].shape, dtype=torch.float64, device=DEV) for _ in range(2)] if s["K"] is not None else None
    pool = s["pool"].double() if s["fmt"] == "bf16" else None
    pair = torch.arange(rot // 2, device=DEV)
    first, second = (2 * pair, 2 * pair + 1) if s["pairs"] else (pair, pair + rot // 2)
    for b in range(s["batch"]):
        x = s["qkv"][cu[b]:cu[b + 1]].double()
        n = x.shape[0]
        if s["positions"] is None:
            at = (int(s["origin"][b]) + s["grown"] + torch.arange(n, device=DEV))[:, None].expand(n, rot // 2)
        else:
            at = s["positions"][cu[b]:cu[b + 1], pair % s["axes"]].long()
        cs = s["table"][at, pair].double()
        y = x[:, :H_q + H]
        if s["q_weight"] is not None:
            w = torch.cat([s["q_weight"].double().expand(H_q, -1), s["k_weight"].double().expand(H, -1)])
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w
        z = y.clone()
        z[..., first] = y[..., first] * cs[:, None, :, 0] - y[..., second] * cs[:, None, :, 1]
        z[..., second] = y[..., first] * cs[:, None, :, 1] + y[..., second] * cs[:, None, :, 0]
        q[cu[b]:cu[b + 1]] = z[:, :H_q]
        kv = [z[:, H_q:], x[:, H_q + H:]]
        if s["fmt"] == "e2m1":
            kv = [_exact_held(v) for v in kv]
        for h in range(H):
            slot = int(s["ntok"][b, h]) + s["grown"] + torch.arange(n, device=DEV)
            page = s["pt_ids"].long()[s["pt_off"][b * (H // s["H_p"]) + h // s["H_p"]] + slot // s["P"]]
            for i, v in enumerate(kv):
                if pool is not None:
                    pool[page, h % s["H_p"], i, slot % s["P"]] = v[:, h]
                if dense is not None:
                    dense[i][b, h, :n] = v[:, h]
    out = {"q": q}
    if pool is not None:
        out["pool"] = pool
    if dense is not None:
        out["K"], out["V"] = dense
    return out


def exact(case, seed):
    s = prepare(case, seed)
    H, H_p, P, d = case["H"], case["H_p"], case["P"], case["d"]
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "decode":
        g = case["H_q"] // H
        out, lse = s["out"].double(), s["lse"].double()
        for b in range(case["batch"]):
            for h in range(H):
                K, V = _exact_rows(s, b, h, int(s["ntok"][b, h]) + case["grown"] + 1)
                a = d ** -0.5 * (s["q"][b, h * g:(h + 1) * g].double() @ K.T)
                lse[b, h * g:(h + 1) * g] = torch.logsumexp(a, -1)
                out[b, h * g:(h + 1) * g] = torch.softmax(a, -1) @ V
        return {"out": out, "lse": lse}
    back = s["back"].double()
    for b in range(case["batch"]):
        for h in range(H):
            n = int(s["ntok"][b, h])
            t = torch.arange(n, device=DEV)
            page = s["pt_ids"].long()[s["pt_off"][b * (H // H_p) + h // H_p] + t // P]
            if case["op"] == "quant":
                rows = s["src"][page, h % H_p, :, t % P]
                back[page, h % H_p, :, t % P] = _exact_held(rows)
            else:
                back[page, h % H_p, :, t % P] = torch.stack(_exact_rows(s, b, h, n), 1)
    return {"back": back}
