"""Cases that measure the prompt-side and shared-prefix operators.

Three operators work around the ragged cache:

  rope    the packed projections of a forward pass -> normalised and rotated queries, and
          the K and V rows of the contexts they belong to (tg_qk_norm_rope);
  prompt  causal attention of those queries over the contexts (tg_prefill_attn);
  prefix  decode attention of a batch over retained tokens that all its requests share,
          merged with what each request attended to on its own (tg_prefix_attn).

With ``own`` false, ``run`` computes each in elementary torch operations in 32 bits, rounded
once at the end; with ``own`` true it makes the library's calls.  ``exact`` is a separate
64-bit computation from the definitions.
"""
import math

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: 16 requests, one new token each, far into their contexts
        dict(name="rope-decode-16", op="rope", H_q=32, H=8, d=128, batch=16, q_lo=1, q_hi=1, ctx=4096, rot=128,
             pairs=False, norm=True, pad=0),
        # a packed prefill pass over 16 whole prompts of different lengths
        dict(name="rope-prefill-16", op="rope", H_q=32, H=8, d=128, batch=16, q_lo=200, q_hi=4096, ctx=4096, rot=128,
             pairs=False, norm=True, pad=0),
        # long mixed prompts of a model with 256-wide heads, in a buffer padded behind the last one
        dict(name="rope-wide-6", op="rope", H_q=16, H=8, d=256, batch=6, q_lo=4096, q_hi=16384, ctx=16384, rot=256,
             pairs=False, norm=True, pad=37),
        # one short question: latency counts
        dict(name="prompt-short-17", op="prompt", H_q=32, H=8, d=128, batch=1, q_lo=17, q_hi=17, old_lo=0, old_hi=0,
             window=0),
        # follow-up turns of a conversation: a few new tokens on long contexts
        dict(name="prompt-turn-8", op="prompt", H_q=32, H=8, d=128, batch=8, q_lo=1, q_hi=64, old_lo=4096,
             old_hi=32768, window=0),
        # a packed prefill pass over 16 whole prompts of different lengths
        dict(name="prompt-ragged-16", op="prompt", H_q=32, H=8, d=128, batch=16, q_lo=64, q_hi=4096, old_lo=0,
             old_hi=0, window=0),
        # long mixed prompts of a model with 256-wide heads
        dict(name="prompt-wide-4", op="prompt", H_q=16, H=8, d=256, batch=4, q_lo=4096, q_hi=9000, old_lo=0, old_hi=0,
             window=0),
        # the last chunk of a chunked prefill of 100000 tokens
        dict(name="prompt-chunk-100k", op="prompt", H_q=32, H=8, d=128, batch=1, q_lo=4096, q_hi=4096, old_lo=95904,
             old_hi=95904, window=0),
        # a few requests behind a short system prompt: latency counts
        dict(name="prefix-small-4", op="prefix", H_q=32, H=8, d=128, P=16, H_p=4, groups=1, batch=4, N=500, b_lo=1.0,
             b_hi=1.0, suffix=True),
        # a decode batch behind one shared document, every token kept
        dict(name="prefix-doc-40", op="prefix", H_q=32, H=8, d=128, P=16, H_p=1, groups=1, batch=40, N=10000, b_lo=1.0,
             b_hi=1.0, suffix=True),
        # a long shared document with head-wise budgets
        dict(name="prefix-ragged-64", op="prefix", H_q=32, H=8, d=128, P=16, H_p=4, groups=1, batch=64, N=100000,
             b_lo=0.03, b_hi=0.6, suffix=True),
        # 256-wide heads, two documents shared by half of the batch each
        dict(name="prefix-wide-32", op="prefix", H_q=16, H=8, d=256, P=16, H_p=4, groups=2, batch=32, N=65536,
             b_lo=0.2, b_hi=1.0, suffix=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "prefix"])
    d = rng.choice([128, 128, 256])
    H = rng.choice([1, 2, 4, 8])
    H_q = H * rng.choice([1, 2, 3, 4, 5, 6, 7, 8] if d == 128 else [1, 2, 3, 4])
    if op == "rope":
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, 49152 // batch)
        ctx = max(hi, min(_log(rng, 64, 16384), 65536 // batch))
        return dict(op=op, H_q=H_q, H=H, d=d, batch=batch, q_lo=max(1, hi // rng.choice([1, 4, 16])), q_hi=hi, ctx=ctx,
                    rot=d if rng.random() < 0.7 else d // 2, pairs=rng.random() < 0.3, norm=rng.random() < 0.8,
                    pad=rng.choice([0, 0, 5, 100]))
    if op == "prompt":
        batch = _log(rng, 1, 32)
        hi = _log(rng, 1, 16384 // batch)
        old = rng.choice([0, 0, _log(rng, 1, 32768)])
        return dict(op=op, H_q=H_q, H=H, d=d, batch=batch, q_lo=max(1, hi // rng.choice([1, 4, 64])), q_hi=hi,
                    old_lo=old // rng.choice([1, 8]), old_hi=old, window=rng.choice([0, 0, _log(rng, 64, 4096)]))
    groups = rng.choice([1, 1, 2, 3])
    return dict(op=op, H_q=H_q, H=H, d=d, P=rng.choice([16, 16, 32, 64, 48]), H_p=rng.choice([p for p in (1, 2, 4) if H % p == 0]),
                groups=groups, batch=groups * _log(rng, 1, 64), N=_log(rng, 100, 100000 // groups),
                b_lo=rng.choice([0.03, 0.3, 1.0]), b_hi=1.0, suffix=rng.random() < 0.7)


def _lengths(case, seed, lo, hi, salt):
    """Lengths log-uniform in [lo, hi]; they follow from the case, not from the seed, so that every
    seed is the same amount of work."""
    if hi <= lo:
        return [int(lo)] * case["batch"]
    g = torch.Generator().manual_seed(case["batch"] * 7919 + hi * 31 + lo * 17 + salt)
    u = torch.rand(case["batch"], generator=g, dtype=torch.float64)
    a = math.log(max(lo, 1))
    return [min(hi, max(lo, int(round(math.exp(a + float(x) * (math.log(hi) - a)))))) for x in u]


def _kept(case):
    """Retained tokens of each (group, head): ceil(B * N), budgets evenly spread and shuffled."""
    n = case["groups"] * case["H"]
    g = torch.Generator().manual_seed(case["N"] * 13 + n)
    at = torch.randperm(n, generator=g).tolist()
    kept = [max(1, min(case["N"], math.ceil(case["N"] * (case["b_lo"] + (case["b_hi"] - case["b_lo"]) * i / max(1, n - 1)))))
            for i in at]
    return [kept[r * case["H"]:(r + 1) * case["H"]] for r in range(case["groups"])]


def _prompt_lengths(case):
    q_len = _lengths(case, 0, case["q_lo"], case["q_hi"], 1)
    old = _lengths(case, 0, case["old_lo"], case["old_hi"], 2)
    return q_len, [a + b for a, b in zip(q_len, old)]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) * scale


def _offsets(lens):
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    return off


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    H, H_q, d, batch = case["H"], case["H_q"], case["d"], case["batch"]
    if case["op"] == "rope":
        lens = _lengths(case, 0, case["q_lo"], case["q_hi"], 1)
        off = _offsets(lens)
        rows = off[-1] + case["pad"]
        s["tokens"] = off[-1]
        s["cu_q"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        s["start"] = torch.tensor([case["ctx"] - n for n in lens] if case["q_hi"] < case["ctx"] else [0] * batch,
                                  dtype=torch.int32, device=DEV)
        s["qkv"] = _randn((rows, H_q + 2 * H, d), g, 1.7)
        s["q_weight"] = torch.rand(d, generator=g, device=DEV) + 0.5 if case["norm"] else None
        s["k_weight"] = torch.rand(d, generator=g, device=DEV) + 0.5 if case["norm"] else None
        # the rotation's table, made in 64 bits once and kept: cos and sin of position * base^(-2i/rot)
        freq = 500000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
        angle = torch.arange(case["ctx"], dtype=torch.float64, device=DEV)[:, None] * freq
        s["table"] = torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()
        s["q"] = torch.zeros((rows, H_q, d), dtype=torch.bfloat16, device=DEV)
        s["K"] = torch.zeros((batch, H, case["ctx"], d), dtype=torch.bfloat16, device=DEV)
        s["V"] = torch.zeros_like(s["K"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "prompt":
        s["q_len"], s["kv_len"] = _prompt_lengths(case)
        s["off"] = _offsets(s["q_len"])
        T, Nmax = s["off"][-1], max(s["kv_len"])
        s["q"] = _randn((T, H_q, d), g, 1.5)
        s["K"] = _randn((batch, H, Nmax, d), g)
        s["V"] = _randn((batch, H, Nmax, d), g)
        s["out"] = torch.zeros((T, H_q, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, H_q), dtype=torch.float32, device=DEV)
        if own:
            from non_uniform_paged_gb300.ragged import PrefillPass
            s["pass"] = PrefillPass(H, H_q, d, s["q_len"], s["kv_len"], window=case["window"], device=DEV)
        return s
    P, H_p, groups = case["P"], case["H_p"], case["groups"]
    G = H // H_p
    s["kept"] = _kept(case)
    s["req_off"] = [r * (batch // groups) for r in range(groups)] + [batch]
    counts = [-(-max(s["kept"][r][i * H_p:(i + 1) * H_p]) // P) for r in range(groups) for i in range(G)]
    off = _offsets(counts)
    s["pages"] = off[-1]
    s["pt_off"] = torch.tensor(off, dtype=torch.int64, device=DEV)
    s["pt_ids"] = torch.randperm(off[-1], generator=g, device=DEV).to(torch.int32)  # pages lie anywhere
    s["off"] = off
    s["pool"] = _randn((off[-1], H_p, 2, P, d), g)
    s["q"] = _randn((batch, H_q, d), g, 1.5)
    s["own_out"] = _randn((batch, H_q, d), g, 0.3) if case["suffix"] else None
    s["own_lse"] = torch.randn((batch, H_q), generator=g, device=DEV) + math.log(case["N"]) if case["suffix"] else None
    s["out"] = torch.zeros((batch, H_q, d), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((batch, H_q), dtype=torch.float32, device=DEV)
    if own:
        import numpy as np
        from non_uniform_paged_gb300.ragged import SharedPrefix
        s["prefix"] = SharedPrefix(H_q, H_p, P, d, s["req_off"], np.arange(H, dtype=np.int32),
                                   np.asarray(s["kept"], np.int32), device=DEV)
    return s


# ------------------------------------------------------------------ one pass

def _rope_plain(s):
    H_q, H, d, rot, n = s["H_q"], s["H"], s["d"], s["rot"], s["tokens"]
    x = s["qkv"][:n].float()
    t = torch.arange(n, device=DEV, dtype=torch.int32)
    req = torch.searchsorted(s["cu_q"][1:].contiguous(), t, right=True)
    row = s["start"][req].long() + t - s["cu_q"][req]
    c, sn = s["table"][row][:, None].unbind(-1)
    parts = []
    for y, w in ((x[:, :H_q], s["q_weight"]), (x[:, H_q:H_q + H], s["k_weight"])):
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        if s["pairs"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        parts.append(torch.cat([z, y[..., rot:]], -1).to(torch.bfloat16))
    s["q"][:n] = parts[0]
    s["K"][req, :, row] = parts[1]
    s["V"][req, :, row] = s["qkv"][:n, H_q + H:]
    return {"q": s["q"], "K": s["K"], "V": s["V"]}


def _softmax_v(q, K, V, scale, hide=None):
    """softmax(scale q K^T) V and the log of its sum, in 32 bits; hide: True where a key is not seen."""
    x = torch.matmul(q, K.transpose(-1, -2)).mul_(scale)
    if hide is not None:
        x.masked_fill_(hide, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, V) / total.clamp_min(1e-30)
    return o, (total.log() + m).squeeze(-1)


def _prompt_plain(s):
    H, H_q, d = s["H"], s["H_q"], s["d"]
    scale, gq = 1.0 / math.sqrt(d), H_q // H
    for b, (nq, nk) in enumerate(zip(s["q_len"], s["kv_len"])):
        K, V = s["K"][b, :, :nk].float(), s["V"][b, :, :nk].float()
        step = max(1, (1 << 30) // (H_q * nk))  # queries at a time: 4 GB of scores
        for i in range(0, nq, step):
            n = min(step, nq - i)
            at = slice(s["off"][b] + i, s["off"][b] + i + n)
            q = s["q"][at].float().view(n, H, gq, d).permute(1, 2, 0, 3).reshape(H, gq * n, d)
            pos = torch.arange(nk - nq + i, nk - nq + i + n, device=DEV)[:, None]
            key = torch.arange(nk, device=DEV)[None]
            hide = key > pos
            if s["window"]:
                hide = hide | (key <= pos - s["window"])
            o, lse = _softmax_v(q, K, V, scale, hide.repeat(gq, 1))
            s["out"][at] = o.view(H, gq, n, d).permute(2, 0, 1, 3).reshape(n, H_q, d).to(torch.bfloat16)
            s["lse"][at] = lse.view(H, gq, n).permute(2, 0, 1).reshape(n, H_q)
    return {"out": s["out"], "lse": s["lse"]}


def _prefix_rows(s, r):
    """The retained K and V rows of every head of group r, out of its pages: [H][most][d] in 32 bits, with
    zeros where a head keeps fewer tokens, and a mask of those places."""
    H, H_p, P = s["H"], s["H_p"], s["P"]
    kept = torch.tensor(s["kept"][r], device=DEV)[:, None]
    head = torch.arange(H, device=DEV)[:, None]
    token = torch.arange(max(s["kept"][r]), device=DEV)[None]
    hide = token >= kept
    token = torch.minimum(token, kept - 1)
    first = s["pt_off"][r * (H // H_p) + head // H_p]
    page = s["pt_ids"][first + token // P].long()
    kv = s["pool"][page, head % H_p, :, token % P].float().masked_fill_(hide[..., None, None], 0.0)
    return kv[:, :, 0], kv[:, :, 1], hide


def _prefix_plain(s):
    H, H_q, d = s["H"], s["H_q"], s["d"]
    scale, gq = 1.0 / math.sqrt(d), H_q // H
    for r in range(s["groups"]):
        at = slice(s["req_off"][r], s["req_off"][r + 1])
        n = at.stop - at.start
        K, V, hide = _prefix_rows(s, r)
        q = s["q"][at].float().view(n, H, gq, d).transpose(0, 1).reshape(H, n * gq, d)
        o, lse = _softmax_v(q, K, V, scale, hide[:, None])
        o = o.view(H, n, gq, d).transpose(0, 1).reshape(n, H_q, d)
        lse = lse.view(H, n, gq).transpose(0, 1).reshape(n, H_q)
        if s["own_lse"] is not None:
            own_lse = s["own_lse"][at]
            both = torch.logaddexp(lse, own_lse)
            o = o * (lse - both).exp()[..., None] + s["own_out"][at].float() * (own_lse - both).exp()[..., None]
            lse = both
        s["out"][at] = o.to(torch.bfloat16)
        s["lse"][at] = lse
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    s = state
    if s["op"] == "rope":
        if not own:
            return _rope_plain(s)
        from non_uniform_paged_gb300 import tg_qk_norm_rope
        tg_qk_norm_rope(s["qkv"], s["cu_q"], s["start"], s["table"], s["q"], s["K"], s["V"], q_weight=s["q_weight"],
                        k_weight=s["k_weight"], eps=1e-6, pairs=s["pairs"], dev_status=s["status"])
        return {"q": s["q"], "K": s["K"], "V": s["V"]}
    if s["op"] == "prompt":
        if not own:
            return _prompt_plain(s)
        s["pass"].attend(s["q"], s["K"], s["V"], s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if not own:
        return _prefix_plain(s)
    s["prefix"].attend(0, s["q"], s["pool"], s["pages"], s["pt_off"], s["pt_ids"], s["out"], lse=s["lse"],
                       own_out=s["own_out"], own_lse=s["own_lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs_seen(nq, nk, window):
    """Number of (query, key) pairs that the causal mask and the window leave."""
    first = nk - nq  # position of the first query
    if window <= 0 or window >= nk:
        return nq * first + nq * (nq + 1) // 2
    full = max(0, nk - max(first, window - 1))  # queries that see a whole window
    rest = nq - full
    return full * window + rest * first + rest * (rest + 1) // 2


def work(case):
    H, H_q, d, batch = case["H"], case["H_q"], case["d"], case["batch"]
    if case["op"] == "rope":
        lens = _lengths(case, 0, case["q_lo"], case["q_hi"], 1)
        n = sum(lens)
        # every projection read once and written once, and the table rows of the positions met
        rows = max(lens)
        return {"bytes": 4 * n * (H_q + 2 * H) * d + 4 * rows * case["rot"], "flops": 7 * n * (H_q + H) * d}
    if case["op"] == "prompt":
        q_len, kv_len = _prompt_lengths(case)
        seen = sum(_pairs_seen(a, b, case["window"]) for a, b in zip(q_len, kv_len))
        keys = sum(min(b, case["window"] + a - 1) if case["window"] else b for a, b in zip(q_len, kv_len))
        return {"bytes": 4 * sum(q_len) * H_q * d + 4 * sum(q_len) * H_q + 4 * keys * H * d, "flops": 4 * seen * H_q * d}
    kept = _kept(case)
    rows = batch // case["groups"] * (H_q // H)
    tokens = sum(map(sum, kept))
    io = batch * H_q * (4 * d + 4) + (batch * H_q * (2 * d + 4) if case["suffix"] else 0)
    pages = sum(-(-max(k[i:i + case["H_p"]]) // case["P"]) for k in kept for i in range(0, H, case["H_p"]))
    return {"bytes": 4 * tokens * d + 4 * pages + io, "flops": 4 * tokens * rows * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows(q, K, V, scale, first=None, last=None):
    """Rows of q (float64 [n][d]) over K, V: weights exp(scale q.k) / sum; row i sees keys first[i]..last[i]."""
    a = (q * scale) @ K.T
    if last is not None:
        key = torch.arange(K.shape[0], device=K.device)
        seen = (key[None] <= last[:, None]) & (key[None] >= first[:, None])
        a = torch.where(seen, a, torch.full((), -math.inf, dtype=torch.float64, device=K.device))
    lse = torch.logsumexp(a, -1)
    top = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    return torch.exp(a - top[:, None]) @ V, lse


def exact(case, seed):
    s = prepare(case, seed)
    H, H_q, d = case["H"], case["H_q"], case["d"]
    gq, scale = H_q // H, d ** -0.5
    if case["op"] == "rope":
        rot = case["rot"]
        q, K, V = s["q"].double(), s["K"].double(), s["V"].double()
        cu, start = s["cu_q"].tolist(), s["start"].tolist()
        i0 = torch.arange(rot // 2, device=DEV)
        first = 2 * i0 if case["pairs"] else i0
        second = 2 * i0 + 1 if case["pairs"] else i0 + rot // 2
        for b in range(case["batch"]):
            x = s["qkv"][cu[b]:cu[b + 1]].double()
            n = x.shape[0]
            cs = s["table"][start[b]:start[b] + n].double()
            x[:, :H_q + H] = _exact_norm_turn(x[:, :H_q + H], s, H_q, cs, first, second)
            q[cu[b]:cu[b + 1]] = x[:, :H_q]
            K[b, :, start[b]:start[b] + n] = x[:, H_q:H_q + H].transpose(0, 1)
            V[b, :, start[b]:start[b] + n] = x[:, H_q + H:].transpose(0, 1)
        return {"q": q, "K": K, "V": V}
    out, lse = s["out"].double(), s["lse"].double()
    if case["op"] == "prompt":
        if work(case)["flops"] > 8e12:
            return None
        for b, (nq, nk) in enumerate(zip(s["q_len"], s["kv_len"])):
            for h in range(H):
                K, V = s["K"][b, h, :nk].double(), s["V"][b, h, :nk].double()
                for j in range(h * gq, (h + 1) * gq):
                    for i in range(0, nq, 4096):
                        rows = slice(s["off"][b] + i, s["off"][b] + min(nq, i + 4096))
                        last = torch.arange(i, min(nq, i + 4096), device=DEV) + (nk - nq)
                        first = last - case["window"] + 1 if case["window"] else torch.zeros_like(last)
                        out[rows, j], lse[rows, j] = _exact_rows(s["q"][rows, j].double(), K, V, scale, first, last)
        return {"out": out, "lse": lse}
    for r in range(case["groups"]):
        for h in range(H):
            n, P, lst = s["kept"][r][h], case["P"], r * (H // case["H_p"]) + h // case["H_p"]
            token = torch.arange(n, device=DEV)
            page = s["pt_ids"].long()[s["off"][lst] + token // P]
            K = s["pool"][page, h % case["H_p"], 0, token % P].double()
            V = s["pool"][page, h % case["H_p"], 1, token % P].double()
            for b in range(s["req_off"][r], s["req_off"][r + 1]):
                at = slice(h * gq, (h + 1) * gq)
                o, le = _exact_rows(s["q"][b, at].double(), K, V, scale)
                if case["suffix"]:
                    w = s["own_lse"][b, at].double()
                    e1, e2 = torch.exp(le - torch.maximum(le, w)), torch.exp(w - torch.maximum(le, w))
                    o = (o * e1[:, None] + s["own_out"][b, at].double() * e2[:, None]) / (e1 + e2)[:, None]
                    le = torch.maximum(le, w) + torch.log(e1 + e2)
                out[b, at], lse[b, at] = o, le
    return {"out": out, "lse": lse}


def _exact_norm_turn(x, s, H_q, cs, first, second):
    """RMS norm of each head, then the plane rotation of each pair (first, second), in 64 bits."""
    if s["q_weight"] is not None:
        w = torch.cat([s["q_weight"].double().expand(H_q, -1), s["k_weight"].double().expand(x.shape[1] - H_q, -1)])
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w
    y = x.clone()
    c, t = cs[:, None, :, 0], cs[:, None, :, 1]
    y[..., first] = x[..., first] * c - x[..., second] * t
    y[..., second] = x[..., first] * t + x[..., second] * c
    return y
