"""The operators of serving and training with a bounded key/value memory, as cases to measure.

Six operators, all on [batch, heads, tokens, head dimension] tensors in bfloat16 or float16:

``window_sink``       attention in which query i, at key position p = i + Nkv - Nq, sees the keys j <= p with
                      j >= p - left (a sliding window; left < 0: no bound) or j < sinks (the first tokens, which stay
                      visible); H query heads share Hkv key/value heads.  Returns O and the row log-sum-exp.
``window_sink_grad``  its gradients dQ, dK, dV from O, LSE and dO.
``cache_append``      tokens written into a 4-bit cache: per token and head one scale and one minimum for the D values,
                      codes 0..15 (the cache's own format, below); returns the values that the written rows stand for.
``cache_attention``   the last Nq tokens of each sequence against that cache (lengths differ per sequence), with the
                      same mask.  Returns O and LSE.
``cache_weights``     what each cached token weighs in it: sum over the query rows of exp(scale q.k - LSE).
``cache_evict``       keep the first `sinks`, the last `recent` and, between them, the heaviest tokens up to `keep` in
                      all, per head, in order; returns the kept rows, their weights, positions and the new lengths.

4-bit format of a row x of D values (in the input type t): min = min(x), scale = t((max(x) - min) / 15),
code = clamp(round_half_even((x - min) / scale), 0, 15) (0 where scale is 0), value = min + code * scale.  Codes are
packed two to a byte, the even channel in the low four bits; (scale, min) follow one another in a tensor of type t.

With ``own`` false ``run`` computes the operators in plain torch operations, with it the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short ragged prompt of a small model: latency of a single call
        {"name": "window_sink small", "op": "window_sink", "B": 1, "H": 4, "Hkv": 2, "Nq": 300, "Nkv": 300, "D": 64,
         "left": 127, "sinks": 4, "dtype": "fp16"},
        # prefill of a long prompt, grouped heads, a window of 1024 tokens and four sinks
        {"name": "window_sink long", "op": "window_sink", "B": 1, "H": 32, "Hkv": 8, "Nq": 8192, "Nkv": 8192, "D": 128,
         "left": 1023, "sinks": 4, "dtype": "bf16"},
        # a training step's attention layer at the D = 64 workload's batch and length
        {"name": "window_sink_grad D64", "op": "window_sink_grad", "B": 4, "H": 16, "Hkv": 16, "Nq": 1024, "Nkv": 1024,
         "D": 64, "left": 255, "sinks": 4, "dtype": "bf16"},
        # a long training sequence with grouped heads, odd length
        {"name": "window_sink_grad D128", "op": "window_sink_grad", "B": 1, "H": 16, "Hkv": 4, "Nq": 8001, "Nkv": 8001,
         "D": 128, "left": 1023, "sinks": 16, "dtype": "bf16"},
        # one decoded token of each of 64 sequences goes into the cache
        {"name": "cache_append token", "op": "cache_append", "B": 64, "Hkv": 8, "N": 1, "C": 4096, "D": 128,
         "dtype": "bf16"},
        # padded prompts of different lengths go into the cache
        {"name": "cache_append prompts", "op": "cache_append", "B": 8, "Hkv": 8, "N": 8192, "C": 8200, "D": 128,
         "dtype": "bf16"},
        # one sequence of one short chat: latency
        {"name": "cache_attention small", "op": "cache_attention", "B": 1, "H": 8, "Hkv": 8, "Nq": 1, "C": 1024,
         "len_min": 777, "len_max": 777, "D": 64, "left": -1, "sinks": 0, "dtype": "fp16"},
        # a decode batch over long contexts of different lengths, eight query heads to a key head
        {"name": "cache_attention long", "op": "cache_attention", "B": 16, "H": 64, "Hkv": 8, "Nq": 1, "C": 32768,
         "len_min": 16001, "len_max": 32768, "D": 128, "left": -1, "sinks": 0, "dtype": "bf16"},
        # weights of a decoded token, a middle-sized batch
        {"name": "cache_weights token", "op": "cache_weights", "B": 8, "H": 32, "Hkv": 8, "Nq": 1, "C": 16384,
         "len_min": 9001, "len_max": 16384, "D": 128, "left": -1, "sinks": 0, "dtype": "bf16"},
        # weights of a prompt's last 16 tokens, the observation window before an eviction
        {"name": "cache_weights prompt", "op": "cache_weights", "B": 2, "H": 32, "Hkv": 8, "Nq": 16, "C": 32768,
         "len_min": 20000, "len_max": 32768, "D": 128, "left": -1, "sinks": 0, "dtype": "bf16"},
        # a batch brought down to its budget
        {"name": "cache_evict batch", "op": "cache_evict", "B": 16, "Hkv": 8, "C": 8192, "len_min": 3000,
         "len_max": 8192, "D": 128, "keep": 2048, "sinks": 4, "recent": 512, "dtype": "bf16"},
        # one very long context brought down to its budget
        {"name": "cache_evict long", "op": "cache_evict", "B": 1, "Hkv": 8, "C": 131072, "len_min": 130001,
         "len_max": 130001, "D": 128, "keep": 8192, "sinks": 4, "recent": 1024, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["window_sink", "window_sink_grad", "cache_append", "cache_attention", "cache_weights",
                     "cache_evict"])
    c = {"op": op, "D": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "fp16"])}
    if op in ("window_sink", "window_sink_grad"):
        c["B"] = rng.choice([1, 1, 2, 3])
        c["Hkv"] = rng.choice([1, 2, 4, 8])
        c["H"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4])
        top = int(min(8192, math.sqrt(2.0e9 / (c["B"] * c["H"])) if op == "window_sink" else
                      math.sqrt(1.0e9 / (c["B"] * c["H"]))))
        c["Nkv"] = _log(rng, 64, top)
        c["Nq"] = c["Nkv"] if rng.random() < 0.7 else _log(rng, 1, c["Nkv"])
        c["left"] = rng.choice([-1, _log(rng, 1, 2048), _log(rng, 1, 2048), _log(rng, 1, 2048)])
        c["sinks"] = rng.choice([0, 1, 4, 4, 16, _log(rng, 1, 300)])
        return c
    c["B"] = _log(rng, 1, 32)
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    if op == "cache_append":
        c["N"] = rng.choice([1, _log(rng, 1, 4096)])
        c["C"] = c["N"] + _log(rng, 1, 2000)
        return c
    c["C"] = _log(rng, 128, 32768)
    c["len_max"] = rng.randint(max(1, c["C"] // 2), c["C"])
    c["len_min"] = rng.randint(1, c["len_max"])
    if op == "cache_evict":
        c["keep"] = _log(rng, 32, c["C"])
        c["sinks"] = rng.randint(0, min(16, c["keep"]))
        c["recent"] = rng.randint(0, c["keep"] - c["sinks"])
        return c
    c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
    c["Nq"] = rng.choice([1, 1, 1, 2, 3, 5])
    c["left"] = rng.choice([-1, -1, _log(rng, 1, c["C"])])
    c["sinks"] = rng.choice([0, 4, _log(rng, 1, 200)])
    return c


# ------------------------------------------------------------------ inputs

def _lens(c, seed=None):
    lens = np.rint(np.linspace(c["len_min"], c["len_max"], c["B"])).astype(np.int64)
    return lens if seed is None else np.random.RandomState(seed % (1 << 31)).permutation(lens)


def _keys(shape, g, dev):
    # keys have channels with an offset and channels that are larger than the rest
    D = shape[-1]
    gain = torch.where(torch.rand(D, generator=g, device=dev) < 0.06, 4.0, 1.0)
    off = torch.randn(D, generator=g, device=dev) * 0.5
    return torch.randn(shape, generator=g, device=dev) * gain + off


def _pack(x):
    """Codes [..., D / 2] and (scale, min) [..., 2] of x [..., D], in the format above."""
    t, d = x.dtype, x.double()
    mn, mx = d.amin(-1, keepdim=True), d.amax(-1, keepdim=True)
    sc = ((mx - mn) / 15).to(t).double()
    code = torch.where(sc > 0, torch.round((d - mn) / torch.where(sc > 0, sc, 1.0)), 0.0).clamp(0, 15).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([sc, mn], -1).to(t)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    t, D, B, Hkv = _T[c["dtype"]], c["D"], c["B"], c["Hkv"]
    s = {"case": c, "scale": 1.0 / math.sqrt(D)}
    if c["op"] in ("window_sink", "window_sink_grad"):
        s["q"] = torch.randn((B, c["H"], c["Nq"], D), generator=g, device=dev).to(t)
        s["k"] = torch.randn((B, Hkv, c["Nkv"], D), generator=g, device=dev).to(t)
        s["v"] = torch.randn((B, Hkv, c["Nkv"], D), generator=g, device=dev).to(t)
        if c["op"] == "window_sink_grad":
            s["do"] = torch.randn((B, c["H"], c["Nq"], D), generator=g, device=dev).to(t)
            s["o"], s["lse"] = _plain_forward(s)
        return s
    if c["op"] == "cache_append":
        N, C = c["N"], c["C"]
        s["k"] = _keys((B, Hkv, N, D), g, dev).to(t)
        s["v"] = torch.randn((B, Hkv, N, D), generator=g, device=dev).to(t)
        s["start"] = torch.randint(0, C - N + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s["count"] = torch.randint((N + 1) // 2, N + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s["cache"] = [torch.zeros((B, Hkv, C, D // 2), dtype=torch.uint8, device=dev),
                      torch.zeros((B, Hkv, C, 2), dtype=t, device=dev),
                      torch.zeros((B, Hkv, C, D // 2), dtype=torch.uint8, device=dev),
                      torch.zeros((B, Hkv, C, 2), dtype=t, device=dev)]
        return s
    C = c["C"]
    cache = []
    for x in ("k", "v"):   # head by head: the unpacked tensors never exist whole
        codes = torch.empty((B, Hkv, C, D // 2), dtype=torch.uint8, device=dev)
        par = torch.empty((B, Hkv, C, 2), dtype=t, device=dev)
        for b in range(B):
            y = _keys((Hkv, C, D), g, dev) if x == "k" else torch.randn((Hkv, C, D), generator=g, device=dev)
            codes[b], par[b] = _pack(y.to(t))
        cache += [codes, par]
    s["cache"] = cache
    s["lens"] = torch.tensor(_lens(c, seed), dtype=torch.int32, device=dev)
    if c["op"] == "cache_evict":
        # accumulated weights: a few heavy tokens, many light ones, some never seen (ties at zero)
        u = torch.rand((B, Hkv, C), generator=g, device=dev)
        acc = torch.exp(4 * torch.randn((B, Hkv, C), generator=g, device=dev) - 8)
        s["acc"] = torch.where(u < 0.2, torch.zeros_like(acc), acc)
        return s
    s["q"] = torch.randn((B, c["H"], c["Nq"], D), generator=g, device=dev).to(t)
    if c["op"] == "cache_weights":
        s["lse"] = _plain_cache_scores(s)[1]
    return s


# ------------------------------------------------------------------ plain forms

def _visible(pos, Nkv, left, sinks, dev):
    """[..., Nkv]: which keys a query at position pos [..., 1] sees."""
    j = torch.arange(Nkv, device=dev)
    vis = j <= pos
    if left >= 0:
        vis = vis & ((j >= pos - left) | (j < sinks))
    return vis


def _soft(s, vis):
    """Masked scores -> (exp(s - max), sum, LSE), rows that see nothing all zero."""
    s = torch.where(vis, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    return p, l, (m + torch.log(l)).squeeze(-1)


def _plain_scores(s):
    c, q, k = s["case"], s["q"].float(), s["k"].float()
    B, H, Nq, D = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    pos = torch.arange(Nq, device=q.device)[:, None] + (Nkv - Nq)
    vis = _visible(pos, Nkv, c["left"], c["sinks"], q.device)
    return torch.matmul(q.view(B, Hkv, H // Hkv, Nq, D), k[:, :, None].transpose(-1, -2)) * s["scale"], vis


def _plain_forward(s):
    x, vis = _plain_scores(s)
    p, l, lse = _soft(x, vis)
    o = torch.matmul(p, s["v"].float()[:, :, None]) / torch.where(l > 0, l, 1.0)
    return o.view(s["q"].shape).to(s["q"].dtype), lse.reshape(s["q"].shape[:3])


def _plain_backward(s):
    x, vis = _plain_scores(s)
    shape, (Hkv, D) = x.shape, (s["k"].shape[1], s["q"].shape[3])
    lse = s["lse"].view(shape[:4] + (1,))
    p = torch.where(vis, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)), 0.0)
    q, do, o = (s[n].float().view(shape[:4] + (D,)) for n in ("q", "do", "o"))
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * s["scale"]
    t = s["q"].dtype
    return dq.view(s["q"].shape).to(t), dk.to(t), dv.to(t)


def _plain_unpack(codes, par):
    lo, hi = (codes & 15).float(), (codes >> 4).float()
    return torch.stack([lo, hi], -1).flatten(-2) * par[..., 0:1].float() + par[..., 1:2].float()


def _plain_append(s):
    c, (kc, kp, vc, vp) = s["case"], s["cache"]
    B, Hkv, N, D = s["k"].shape
    i = torch.arange(N, device=kc.device)
    row = (s["start"].long()[:, None] + i).clamp(max=c["C"] - 1)           # [B, N]
    real = (i < s["count"][:, None])[:, None, :, None]                      # [B, 1, N, 1]
    out = []
    for x, codes, par in ((s["k"], kc, kp), (s["v"], vc, vp)):
        at = row[:, None, :, None].expand(B, Hkv, N, 1)
        for new, held in zip(_pack(x), (codes, par)):
            a = at.expand(B, Hkv, N, held.shape[-1])
            held.scatter_(2, a, torch.where(real, new, held.gather(2, a)))
        got = _plain_unpack(codes.gather(2, at.expand(B, Hkv, N, D // 2)), par.gather(2, at.expand(B, Hkv, N, 2)))
        out.append(torch.where(real, got, 0.0).to(x.dtype))
    return tuple(out)


def _plain_cache_scores(s):
    """(exp(s - max), LSE, sum), [B, Hkv, G, Nq, C], of the queries against the cache."""
    c, q = s["case"], s["q"].float()
    B, H, Nq, D = q.shape
    k = _plain_unpack(s["cache"][0], s["cache"][1])
    pos = s["lens"].view(B, 1, 1, 1, 1) - Nq + torch.arange(Nq, device=q.device)[:, None]
    vis = _visible(pos, c["C"], c["left"], c["sinks"], q.device)
    x = torch.matmul(q.view(B, c["Hkv"], (H // c["Hkv"]) * Nq, D), k.transpose(-1, -2)) * s["scale"]
    p, l, lse = _soft(x.view(B, c["Hkv"], H // c["Hkv"], Nq, c["C"]), vis)
    return p, lse.reshape(B, H, Nq), l


def _plain_cache_attention(s):
    p, lse, l = _plain_cache_scores(s)
    v = _plain_unpack(s["cache"][2], s["cache"][3])
    o = torch.matmul((p / torch.where(l > 0, l, 1.0)).flatten(2, 3), v)
    return o.view(s["q"].shape).to(s["q"].dtype), lse


def _plain_cache_weights(s):
    c, q = s["case"], s["q"].float()
    B, H, Nq, D = q.shape
    k = _plain_unpack(s["cache"][0], s["cache"][1])
    pos = s["lens"].view(B, 1, 1, 1, 1) - Nq + torch.arange(Nq, device=q.device)[:, None]
    vis = _visible(pos, c["C"], c["left"], c["sinks"], q.device)
    x = torch.matmul(q.view(B, c["Hkv"], (H // c["Hkv"]) * Nq, D), k.transpose(-1, -2)) * s["scale"]
    lse = s["lse"].view(B, c["Hkv"], H // c["Hkv"], Nq, 1)
    x = x.view(B, c["Hkv"], H // c["Hkv"], Nq, c["C"])
    return torch.where(vis, torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)), 0.0).sum((2, 3))


def _plain_evict(s):
    c, lens, acc = s["case"], s["lens"].long(), s["acc"]
    B, Hkv, C, keep = c["B"], c["Hkv"], c["C"], c["keep"]
    j = torch.arange(C, device=acc.device)
    n = lens.view(B, 1, 1)
    fixed = (j < c["sinks"]) | (j >= n - c["recent"])
    # rank: tokens that always stay, then the others by weight (ties: the lowest position first), then none at all
    order = torch.sort(torch.where(j >= n, -math.inf, torch.where(fixed, math.inf, acc)), dim=-1, descending=True,
                       stable=True).indices
    at = torch.where(j[:keep] < n, order[..., :keep], C).sort(-1).values    # positions in order, C where there is none
    real = at < C
    at = torch.where(real, at, 0)
    out = []
    for codes, par in (s["cache"][0:2], s["cache"][2:4]):
        codes = codes.gather(2, at[..., None].expand(B, Hkv, keep, codes.shape[-1]))
        x = _plain_unpack(codes, par.gather(2, at[..., None].expand(B, Hkv, keep, 2)))
        out.append(torch.where(real[..., None], x, 0.0).to(par.dtype))
    return {"k": out[0], "v": out[1], "acc": torch.where(real, acc.gather(2, at), 0.0),
            "index": torch.where(real, at, -1).int(), "lens": lens.clamp(max=keep).int()}


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"window_sink": _plain_forward, "window_sink_grad": _plain_backward, "cache_append": _plain_append,
                "cache_attention": lambda s: _plain_cache_attention(s), "cache_weights": _plain_cache_weights,
                "cache_evict": _plain_evict}[op](state)
    return _own(state, c, op)


# ------------------------------------------------------------------ the framework's operators

def _own(s, c, op):
    from exact_attention_10_gb300 import fa
    if op == "window_sink":
        return fa.forward(s["q"], s["k"], s["v"], scale=s["scale"], window=(c["left"], 0), sinks=c["sinks"])
    if op == "window_sink_grad":
        return fa.backward(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], scale=s["scale"], window=(c["left"], 0),
                           sinks=c["sinks"])
    cache = fa.PackedCache(*s["cache"])
    if op == "cache_append":
        fa.cache_append(cache, s["k"], s["v"], s["start"], count=s["count"])
        return fa.cache_read(cache, s["start"], c["N"], count=s["count"])
    if op == "cache_attention":
        return fa.cache_forward(s["q"], cache, s["lens"], scale=s["scale"], window=(c["left"], 0), sinks=c["sinks"])
    if op == "cache_weights":
        return fa.cache_weights(s["q"], cache, s["lse"], s["lens"], scale=s["scale"], window=(c["left"], 0),
                                sinks=c["sinks"])
    kept, acc, lens, index = fa.cache_evict(cache, s["acc"], s["lens"], c["keep"], sinks=c["sinks"],
                                            recent=c["recent"])
    k, v = fa.cache_read(kept, torch.zeros_like(lens), c["keep"], count=lens)
    return {"k": k, "v": v, "acc": acc, "index": index, "lens": lens}


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(Nq, length, left, sinks):
    """Visible (query, key) pairs of one head, and the keys that some query sees."""
    pos = np.arange(length - Nq, length)
    pos = pos[pos >= 0]
    if not len(pos):
        return 0, 0
    if left < 0:
        return int((pos + 1).sum()), length
    lo = np.maximum(pos - left, 0)
    pairs = (pos + 1 - lo) + np.minimum(sinks, lo)
    return int(pairs.sum()), int(length - lo[0] + min(sinks, lo[0]))


def work(case):
    c, D = case, case["D"]
    row = D // 2 + 4      # a packed row: codes, scale and minimum
    if c["op"] in ("window_sink", "window_sink_grad"):
        pairs, keys = _pairs(c["Nq"], c["Nkv"], c["left"], c["sinks"])
        q, kv = c["B"] * c["H"] * c["Nq"] * D * 2, c["B"] * c["Hkv"] * c["Nkv"] * D * 2
        lse = c["B"] * c["H"] * c["Nq"] * 4
        if c["op"] == "window_sink":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4.0 * c["B"] * c["H"] * pairs * D}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10.0 * c["B"] * c["H"] * pairs * D}
    heads = c["B"] * c["Hkv"]
    if c["op"] == "cache_append":   # the new rows read, packed rows written and read, values written
        rows = 2 * heads * c["N"]
        return {"bytes": rows * (2 * D + 2 * row + 2 * D), "flops": rows * D * 6.0}
    lens = _lens(c)
    if c["op"] == "cache_evict":
        kept = int(np.minimum(lens, c["keep"]).sum()) * c["Hkv"]
        return {"bytes": int(lens.sum()) * c["Hkv"] * 4 + kept * (2 * row * 3 + 4 + 4) + heads * c["keep"] * 4 * D,
                "flops": 2.0 * kept * 2 * D}
    got = [_pairs(c["Nq"], int(n), c["left"], c["sinks"]) for n in lens]
    pairs, keys = sum(x for x, _ in got) * c["H"], sum(x for _, x in got) * c["Hkv"]
    q = c["B"] * c["H"] * c["Nq"] * D * 2
    if c["op"] == "cache_attention":
        return {"bytes": 2 * keys * row + 2 * q + q // (D // 2), "flops": 4.0 * pairs * D}
    return {"bytes": keys * row + q + q // (D // 2) + heads * c["C"] * 4, "flops": 2.0 * pairs * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def _values64(codes, par):
    """[C, D] float64 of one head's packed rows."""
    n = codes.to(torch.int64)
    x = torch.empty(n.shape[0], n.shape[1] * 2, dtype=torch.float64, device=n.device)
    x[:, 0::2] = torch.remainder(n, 16)
    x[:, 1::2] = torch.div(n, 16, rounding_mode="floor")
    return par[:, 1:].double() + x * par[:, :1].double()


def _hidden64(first, count, keys, left, sinks, dev):
    """[count, keys] true where the query at position first + i must not see key j."""
    d = (first + torch.arange(count, device=dev)).view(-1, 1) - torch.arange(keys, device=dev).view(1, -1)
    hid = d < 0
    if left >= 0:
        hid |= (d > left) & (torch.arange(keys, device=dev).view(1, -1) >= sinks)
    return hid


def _rows64(q, k, first, left, sinks, scale):
    x = (q @ k.t()) * scale
    x.masked_fill_(_hidden64(first, q.shape[0], k.shape[0], left, sinks, q.device), -math.inf)
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]), lse


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, scale = c["op"], s["scale"]
    if op in ("window_sink", "window_sink_grad"):
        G, block = c["H"] // c["Hkv"], 1024
        o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), []
        dq = torch.zeros_like(o)
        dk = torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
        dv = torch.zeros_like(dk)
        for b in range(c["B"]):
            for h in range(c["H"]):
                k, v = s["k"][b, h // G].double(), s["v"][b, h // G].double()
                for i in range(0, c["Nq"], block):
                    q = s["q"][b, h, i:i + block].double()
                    first = c["Nkv"] - c["Nq"] + i
                    if op == "window_sink":
                        p, l = _rows64(q, k, first, c["left"], c["sinks"], scale)
                        o[b, h, i:i + block] = p @ v
                        lse.append(l)
                        continue
                    x = (q @ k.t()) * scale - s["lse"][b, h, i:i + block, None].double()
                    p = torch.exp(x).masked_fill_(_hidden64(first, q.shape[0], c["Nkv"], c["left"], c["sinks"], "cuda"), 0)
                    do, got = s["do"][b, h, i:i + block].double(), s["o"][b, h, i:i + block].double()
                    ds = p * (do @ v.t() - torch.einsum("id,id->i", do, got)[:, None])
                    dq[b, h, i:i + block] = scale * (ds @ k)
                    dk[b, h // G] += scale * (ds.t() @ q)
                    dv[b, h // G] += p.t() @ do
        if op == "window_sink":
            return o, torch.cat(lse).view(s["q"].shape[:3])
        return dq, dk, dv
    if op == "cache_append":
        got = []
        for x in (s["k"], s["v"]):
            d = x.double()
            mn = d.min(-1, keepdim=True).values
            sc = ((d.max(-1, keepdim=True).values - mn) / 15).to(x.dtype).double()
            code = torch.round((d - mn) / sc).nan_to_num(0.0).clamp(0, 15)
            real = torch.arange(c["N"], device="cuda") < s["count"][:, None]
            got.append((code * sc + mn) * real[:, None, :, None])
        return tuple(got)
    if op == "cache_evict":
        B, Hkv, keep = c["B"], c["Hkv"], c["keep"]
        k = torch.zeros((B, Hkv, keep, c["D"]), dtype=torch.float64, device="cuda")
        v, w = torch.zeros_like(k), torch.zeros((B, Hkv, keep), dtype=torch.float64, device="cuda")
        index = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            for h in range(Hkv):
                a = s["acc"][b, h, :n].cpu().numpy()
                if n <= keep:
                    pick = np.arange(n)
                else:
                    first, last = np.arange(c["sinks"]), np.arange(max(c["sinks"], n - c["recent"]), n)
                    mid = np.arange(c["sinks"], max(c["sinks"], n - c["recent"]))
                    heavy = mid[np.lexsort((mid, -a[mid]))][:keep - len(first) - len(last)]
                    pick = np.sort(np.concatenate([first, heavy, last]))
                pick = torch.from_numpy(pick).cuda()
                m = len(pick)
                index[b, h, :m] = pick.int()
                w[b, h, :m] = s["acc"][b, h].double()[pick]
                k[b, h, :m] = _values64(s["cache"][0][b, h][pick], s["cache"][1][b, h][pick])
                v[b, h, :m] = _values64(s["cache"][2][b, h][pick], s["cache"][3][b, h][pick])
        return {"k": k, "v": v, "acc": w, "index": index, "lens": torch.clamp(s["lens"], max=keep)}
    G, Nq = c["H"] // c["Hkv"], c["Nq"]
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    w = torch.zeros((c["B"], c["Hkv"], c["C"]), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        for h in range(c["Hkv"]):
            k = _values64(s["cache"][0][b, h, :n], s["cache"][1][b, h, :n])
            if op == "cache_attention":
                v = _values64(s["cache"][2][b, h, :n], s["cache"][3][b, h, :n])
            for hq in range(h * G, h * G + G):
                q = s["q"][b, hq].double()
                if op == "cache_attention":
                    p, lse[b, hq] = _rows64(q, k, n - Nq, c["left"], c["sinks"], scale)
                    o[b, hq] = p @ v
                else:
                    x = (q @ k.t()) * scale - s["lse"][b, hq, :, None].double()
                    w[b, h, :n] += torch.exp(x).masked_fill_(_hidden64(n - Nq, Nq, n, c["left"], c["sinks"], "cuda"), 0).sum(0)
    return (o, lse) if op == "cache_attention" else w
