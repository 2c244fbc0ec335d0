"""The operators of batches of different lengths, as cases to measure: packed sequences and a paged key/value cache.

Packed sequences: the tokens of S sequences stand behind one another, q [T, H, D], k and v [T, Hkv, D] in bfloat16 or
float16, sequence s in rows cu[s] .. cu[s + 1] - 1 (`cu` int32 [S + 1]); H query heads share Hkv key heads.

``packed``        attention inside each sequence, causal (query i sees the keys j <= i + Lk - Lq of its sequence) or full;
                  queries and keys may have sequences of their own lengths.  Returns O [T, H, D] and the row
                  log-sum-exp [H, T].
``packed_grad``   its gradients dQ, dK, dV from O, LSE and dO.

Paged cache: pages [P, Hkv, page, D] for K and for V; token t of sequence b is row t % page of page table[b, t // page].
With `bits` 16 the pages are of the model's type; with 8 they hold e4m3 codes with one float32 scale per token and key
head [P, Hkv, page]: scale = max |x| / 448, code = e4m3(x / scale) (0 where scale is 0), value = code * scale.

``paged_append``  packed tokens k, v written behind what each sequence holds; returns the values that the new rows stand
                  for, read back.
``paged_attention``  the last Nq tokens of each sequence, q [B, H, Nq, D], against its cached tokens.  Returns O and LSE
                  [B, H, Nq].

With `own` false ``run`` computes the operators in plain torch operations, with it the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # three short prompts of a small model, slices of a fused projection: latency of a single call
        {"name": "packed small", "op": "packed", "S": 3, "len_min": 1, "len_max": 300, "prefix": 0, "H": 4, "Hkv": 2,
         "D": 64, "causal": True, "fused": True, "dtype": "fp16"},
        # a prefill batch of many prompts of different lengths, grouped heads
        {"name": "packed batch", "op": "packed", "S": 64, "len_min": 64, "len_max": 2048, "prefix": 0, "H": 32,
         "Hkv": 8, "D": 128, "causal": True, "fused": True, "dtype": "bf16"},
        # a few long documents
        {"name": "packed long", "op": "packed", "S": 4, "len_min": 4001, "len_max": 16384, "prefix": 0, "H": 32,
         "Hkv": 8, "D": 128, "causal": True, "fused": False, "dtype": "bf16"},
        # a training step's attention layer on packed short documents
        {"name": "packed_grad D64", "op": "packed_grad", "S": 16, "len_min": 100, "len_max": 1024, "prefix": 0, "H": 16,
         "Hkv": 16, "D": 64, "causal": True, "fused": False, "dtype": "bf16"},
        # a training step's attention layer on packed documents up to long ones, grouped heads
        {"name": "packed_grad D128", "op": "packed_grad", "S": 6, "len_min": 500, "len_max": 8001, "prefix": 0, "H": 16,
         "Hkv": 4, "D": 128, "causal": True, "fused": True, "dtype": "bf16"},
        # one decoded token of each of 64 sequences goes into the cache
        {"name": "paged_append token", "op": "paged_append", "S": 64, "len_min": 1, "len_max": 1, "held": 4000,
         "Hkv": 8, "D": 128, "page": 16, "bits": 16, "dtype": "bf16"},
        # prompts of different lengths go into a cache of 8 bits
        {"name": "paged_append prompts", "op": "paged_append", "S": 8, "len_min": 1000, "len_max": 8192, "held": 100,
         "Hkv": 8, "D": 128, "page": 64, "bits": 8, "dtype": "bf16"},
        # one sequence of one short chat: latency
        {"name": "paged_attention small", "op": "paged_attention", "S": 1, "len_min": 777, "len_max": 777, "Nq": 1,
         "H": 8, "Hkv": 8, "D": 64, "page": 16, "bits": 16, "dtype": "fp16"},
        # a decode batch of chats of different lengths, four query heads to a key head
        {"name": "paged_attention batch", "op": "paged_attention", "S": 64, "len_min": 1001, "len_max": 8192, "Nq": 1,
         "H": 32, "Hkv": 8, "D": 128, "page": 16, "bits": 16, "dtype": "bf16"},
        # two very long contexts, eight query heads to a key head: the cache's length is what there is to split
        {"name": "paged_attention long", "op": "paged_attention", "S": 2, "len_min": 100001, "len_max": 131072, "Nq": 1,
         "H": 64, "Hkv": 8, "D": 128, "page": 64, "bits": 16, "dtype": "bf16"},
        # a decode batch over long contexts in 8 bits
        {"name": "paged_attention e4m3", "op": "paged_attention", "S": 32, "len_min": 4001, "len_max": 32768, "Nq": 1,
         "H": 32, "Hkv": 8, "D": 128, "page": 32, "bits": 8, "dtype": "bf16"},
        # four drafted tokens of each sequence checked at once
        {"name": "paged_attention drafts", "op": "paged_attention", "S": 16, "len_min": 2000, "len_max": 16384, "Nq": 4,
         "H": 32, "Hkv": 8, "D": 128, "page": 16, "bits": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["packed", "packed_grad", "paged_append", "paged_attention", "paged_attention"])
    c = {"op": op, "D": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "fp16"])}
    c["Hkv"] = rng.choice([1, 2, 4, 8])
    if op in ("packed", "packed_grad"):
        c["H"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4])
        c["S"] = _log(rng, 1, 64)
        top = int(min(8192, math.sqrt((2.0e9 if op == "packed" else 5.0e8) / (c["S"] * c["H"]))))
        c["len_max"] = _log(rng, min(64, top), top)
        c["len_min"] = _log(rng, 1, c["len_max"])
        c["prefix"] = rng.choice([0, 0, 0, _log(rng, 1, 500)])
        c["causal"] = rng.random() < 0.8
        c["fused"] = c["prefix"] == 0 and rng.random() < 0.5
        return c
    c["page"] = rng.choice([16, 16, 32, 64, 128])
    c["bits"] = rng.choice([16, 16, 8])
    c["S"] = _log(rng, 1, 64)
    if op == "paged_append":
        c["len_max"] = rng.choice([1, _log(rng, 1, 2048)])
        c["len_min"] = _log(rng, 1, c["len_max"])
        c["held"] = _log(rng, 1, 2000)
        return c
    c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 8])
    c["len_max"] = _log(rng, 64, int(min(131072, 1.6e6 / (c["S"] * c["Hkv"]))))
    c["len_min"] = _log(rng, 1, c["len_max"])
    c["Nq"] = rng.choice([1, 1, 1, 2, 3, 5])
    return c


# ------------------------------------------------------------------ inputs

def _lens(c, seed=None):
    """Lengths spread evenly over their logarithm, in an order of the seed's."""
    lens = np.rint(np.geomspace(c["len_min"], c["len_max"], c["S"])).astype(np.int64)
    return lens if seed is None else np.random.RandomState(seed % (1 << 31)).permutation(lens)


def _keys(shape, g, dev):
    # keys have channels with an offset and channels that are larger than the rest
    D = shape[-1]
    gain = torch.where(torch.rand(D, generator=g, device=dev) < 0.06, 4.0, 1.0)
    off = torch.randn(D, generator=g, device=dev) * 0.5
    return torch.randn(shape, generator=g, device=dev) * gain + off


def _cu(lens, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev)


def _quantise(x):
    """Codes and scales of rows x [..., D] in the 8-bit format."""
    x = x.float()
    top = x.abs().amax(-1)
    scale = top / torch.full_like(top, 448.0)   # (by a tensor: the quotient rounded once, not a product with 1/448)
    code = torch.where(scale[..., None] > 0, x / torch.where(scale > 0, scale, 1.0)[..., None], 0.0)
    return code.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _table(lens, page, g, dev):
    """Pages of each sequence in a pool in which they are scattered; -1 behind a sequence's last."""
    need = [-(-int(n) // page) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device=dev).int()
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    t, D, Hkv = _T[c["dtype"]], c["D"], c["Hkv"]
    lens = _lens(c, seed)
    s = {"case": c, "scale": 1.0 / math.sqrt(D), "lens_list": [int(n) for n in lens]}
    if c["op"] in ("packed", "packed_grad"):
        H, Tq = c["H"], int(lens.sum())
        klens = lens + c["prefix"]
        Tk = int(klens.sum())
        if c["fused"]:
            qkv = torch.randn((Tq, H + 2 * Hkv, D), generator=g, device=dev).to(t)
            s["q"], s["k"], s["v"] = qkv.split([H, Hkv, Hkv], 1)
        else:
            s["q"] = torch.randn((Tq, H, D), generator=g, device=dev).to(t)
            s["k"] = torch.randn((Tk, Hkv, D), generator=g, device=dev).to(t)
            s["v"] = torch.randn((Tk, Hkv, D), generator=g, device=dev).to(t)
        s["klens_list"] = [int(n) for n in klens]
        s["cu"] = _cu(lens, dev)
        s["cu_k"] = _cu(klens, dev) if c["prefix"] else s["cu"]
        if c["op"] == "packed_grad":
            s["do"] = torch.randn((Tq, H, D), generator=g, device=dev).to(t)
            s["o"], s["lse"] = _plain_packed(s)
        if own:   # the batch's plan: the same for every layer
            from exact_attention_10_gb300 import fa
            s["plan"] = fa.packed_plan(s["cu"], Tq, H, Hkv, cu_k=s["cu_k"], tokens_k=Tk, causal=c["causal"],
                                       grad=c["op"] == "packed_grad")
        return s
    page = c["page"]
    if c["op"] == "paged_append":
        T = int(lens.sum())
        start = torch.randint(0, c["held"] + 1, (c["S"],), generator=g, device=dev, dtype=torch.int32)
        s["k"], s["v"] = _keys((T, Hkv, D), g, dev).to(t), torch.randn((T, Hkv, D), generator=g, device=dev).to(t)
        s["start"], s["cu"] = start, _cu(lens, dev)
        s["table"], pool = _table(start.cpu().numpy() + lens, page, g, dev)
    else:
        s["table"], pool = _table(lens, page, g, dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = torch.randn((c["S"], c["H"], c["Nq"], D), generator=g, device=dev).to(t)
    pages, scales = [], []
    for make in (_keys, lambda shape, g, dev: torch.randn(shape, generator=g, device=dev)):
        if c["op"] == "paged_append":
            x = torch.zeros((pool, Hkv, page, D), dtype=t, device=dev)
        else:
            x = make((pool, Hkv, page, D), g, dev).to(t)
        if c["bits"] == 8:
            x, sc = _quantise(x)
            scales.append(sc)
        pages.append(x)
    s["cache"] = pages + scales
    if own:   # the cache that such a program keeps
        from exact_attention_10_gb300 import fa
        s["cache"] = fa.PagedCache(*s["cache"])
    return s


# ------------------------------------------------------------------ plain forms

def _plain_scores(s, b, q0, k0, h):
    """Scores [G, Lq, Lk] of key head h of sequence b, hidden ones -inf, in 32 bits."""
    c, Lq, Lk = s["case"], s["lens_list"][b], s["klens_list"][b]
    G = c["H"] // c["Hkv"]
    q = s["q"][q0:q0 + Lq, h * G:h * G + G].float().transpose(0, 1)
    k = s["k"][k0:k0 + Lk, h].float()
    x = torch.matmul(q, k.t()) * s["scale"]
    if c["causal"]:
        i = torch.arange(Lq, device=q.device)[:, None] + (Lk - Lq)
        x = torch.where(torch.arange(Lk, device=q.device) <= i, x, -math.inf)
    return x, q, k


def _plain_packed(s):
    c = s["case"]
    H, G = c["H"], c["H"] // c["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
    lse = torch.full((H, s["q"].shape[0]), -math.inf, dtype=torch.float32, device=o.device)
    q0 = k0 = 0
    for b, (Lq, Lk) in enumerate(zip(s["lens_list"], s["klens_list"])):
        for h in range(c["Hkv"]):
            x, _, _ = _plain_scores(s, b, q0, k0, h)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
            l = p.sum(-1, keepdim=True)
            y = torch.matmul(p, s["v"][k0:k0 + Lk, h].float()) / torch.where(l > 0, l, 1.0)
            o[q0:q0 + Lq, h * G:h * G + G] = y.transpose(0, 1).to(o.dtype)
            lse[h * G:h * G + G, q0:q0 + Lq] = (m + torch.log(l)).squeeze(-1)
        q0, k0 = q0 + Lq, k0 + Lk
    return o, lse


def _plain_packed_grad(s):
    c, t = s["case"], s["q"].dtype
    G = c["H"] // c["Hkv"]
    dq = torch.zeros(s["q"].shape, dtype=t, device=s["q"].device)
    dk = torch.zeros(s["k"].shape, dtype=t, device=s["q"].device)
    dv = torch.zeros_like(dk)
    q0 = k0 = 0
    for b, (Lq, Lk) in enumerate(zip(s["lens_list"], s["klens_list"])):
        for h in range(c["Hkv"]):
            rows, heads = slice(q0, q0 + Lq), slice(h * G, h * G + G)
            x, q, k = _plain_scores(s, b, q0, k0, h)
            lse = s["lse"][heads, rows, None]
            p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse))
            do = s["do"][rows, heads].float().transpose(0, 1)
            o = s["o"][rows, heads].float().transpose(0, 1)
            v = s["v"][k0:k0 + Lk, h].float()
            dv[k0:k0 + Lk, h] = torch.matmul(p.transpose(-1, -2), do).sum(0).to(t)
            ds = p * (torch.matmul(do, v.t()) - (do * o).sum(-1, keepdim=True))
            dq[rows, heads] = (torch.matmul(ds, k) * s["scale"]).transpose(0, 1).to(t)
            dk[k0:k0 + Lk, h] = (torch.matmul(ds.transpose(-1, -2), q).sum(0) * s["scale"]).to(t)
        q0, k0 = q0 + Lq, k0 + Lk
    return dq, dk, dv


def _plain_append(s):
    c, cache, table = s["case"], s["cache"], s["table"].long()
    T, Hkv, D = s["k"].shape
    i = torch.arange(T, device=table.device)
    b = torch.searchsorted(s["cu"][1:].long(), i, right=True)
    tok = s["start"].long()[b] + i - s["cu"].long()[b]
    pid, row = table[b, tok // c["page"]], tok % c["page"]
    out = []
    for n, x in enumerate((s["k"], s["v"])):
        if c["bits"] == 16:
            cache[n][pid, :, row] = x
            out.append(cache[n][pid, :, row])
        else:
            code, sc = _quantise(x)
            cache[n].view(torch.uint8)[pid, :, row] = code.view(torch.uint8)
            cache[2 + n][pid, :, row] = sc
            got = cache[n].view(torch.uint8)[pid, :, row].view(torch.float8_e4m3fn).float()
            out.append((got * cache[2 + n][pid, :, row][..., None]).to(x.dtype))
    return tuple(out)


def _plain_attention(s):
    c, q = s["case"], s["q"].float()
    B, H, Nq, D = q.shape
    Hkv, G = c["Hkv"], H // c["Hkv"]
    o, lse = torch.empty_like(s["q"]), torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    for b, n in enumerate(s["lens_list"]):
        at = s["table"][b, :-(-n // c["page"])].long()
        kv = []
        for i in (0, 1):
            x = s["cache"][i].view(torch.uint8)[at].view(s["cache"][i].dtype).float() if c["bits"] == 8 else s["cache"][i][at].float()
            if c["bits"] == 8:
                x = x * s["cache"][2 + i][at][..., None]
            kv.append(x.transpose(0, 1).reshape(Hkv, -1, D)[:, :n])
        x = torch.matmul(q[b].view(Hkv, G * Nq, D), kv[0].transpose(-1, -2)) * s["scale"]
        pos = torch.arange(Nq, device=q.device).repeat(G)[:, None] + (n - Nq)
        x = torch.where(torch.arange(n, device=q.device) <= pos, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        o[b] = (torch.matmul(p, kv[1]) / torch.where(l > 0, l, 1.0)).view(H, Nq, D).to(o.dtype)
        lse[b] = (m + torch.log(l)).view(H, Nq)
    return o, lse


def run(state):
    c = state["case"]
    if not own:
        return {"packed": _plain_packed, "packed_grad": _plain_packed_grad, "paged_append": _plain_append,
                "paged_attention": _plain_attention}[c["op"]](state)
    return _own(state, c)


# ------------------------------------------------------------------ the framework's operators

def _own(s, c):
    from exact_attention_10_gb300 import fa
    if c["op"] == "packed":
        return fa.packed_forward(s["q"], s["k"], s["v"], s["plan"], scale=s["scale"])
    if c["op"] == "packed_grad":
        return fa.packed_backward(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["plan"], scale=s["scale"])
    if c["op"] == "paged_append":
        fa.paged_append(s["cache"], s["table"], s["k"], s["v"], s["start"], cu=s["cu"])
        return fa.paged_read(s["cache"], s["table"], s["start"], s["k"].shape[0], cu=s["cu"], dtype=s["k"].dtype)
    return fa.paged_forward(s["q"], s["cache"], s["table"], s["lens"], scale=s["scale"])


# ------------------------------------------------------------------ what a pass cannot do without

def _pairs(Lq, Lk, causal):
    """Visible (query, key) pairs of one head of a sequence."""
    if not causal:
        return Lq * Lk
    n = np.arange(Lk - Lq + 1, Lk + 1, dtype=np.int64)
    return int(n[n > 0].sum())


def work(case):
    c, D, lens = case, case["D"], _lens(case)
    if c["op"] in ("packed", "packed_grad"):
        Tq, Tk = int(lens.sum()), int((lens + c["prefix"]).sum())
        pairs = sum(_pairs(int(n), int(n) + c["prefix"], c["causal"]) for n in lens) * c["H"]
        q, kv, lse = Tq * c["H"] * D * 2, Tk * c["Hkv"] * D * 2, Tq * c["H"] * 4
        if c["op"] == "packed":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4.0 * pairs * D}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10.0 * pairs * D}
    row = 2 * D if c["bits"] == 16 else D + 4
    if c["op"] == "paged_append":   # the new rows read, held rows written and read, values written
        rows = 2 * int(lens.sum()) * c["Hkv"]
        return {"bytes": rows * (2 * D + 2 * row + 2 * D), "flops": rows * D * (1.0 if c["bits"] == 16 else 4.0)}
    keys = int(lens.sum()) * c["Hkv"]
    q = c["S"] * c["H"] * c["Nq"] * D * 2
    pairs = sum(_pairs(c["Nq"], int(n), True) for n in lens) * c["H"]
    table = sum(-(-int(n) // c["page"]) for n in lens) * 4
    return {"bytes": 2 * keys * row + 2 * q + q // (D // 2) + table, "flops": 4.0 * pairs * D}


# ------------------------------------------------------------------ the definitions in 64 bits

def _softmax64(q, k, first, causal, scale):
    """(weights, LSE) of queries at positions first + i against keys 0 .. len(k) - 1."""
    x = (q @ k.t()) * scale
    if causal:
        ahead = torch.arange(k.shape[0], device=q.device)[None] - (first + torch.arange(q.shape[0], device=q.device))[:, None]
        x.masked_fill_(ahead > 0, -math.inf)
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]), lse


def _held64(s, n, pid):
    """[tokens, Hkv, D] float64: what the rows of pages `pid` stand for."""
    x = s["cache"][n][pid.long()] if s["case"]["bits"] == 16 else \
        s["cache"][n].view(torch.uint8)[pid.long()].view(torch.float8_e4m3fn)
    x = x.double()
    if s["case"]["bits"] == 8:
        x = x * s["cache"][2 + n][pid.long()].double().unsqueeze(-1)
    return x.permute(0, 2, 1, 3).flatten(0, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op, scale, block = c["op"], s["scale"], 1024
    if op == "paged_append":
        out = []
        for x in (s["k"], s["v"]):
            d = x.double()
            if c["bits"] == 8:
                sc = (d.abs().max(-1, keepdim=True).values / torch.full((1,), 448.0, dtype=d.dtype, device=d.device)).float().double()
                code = (x.float() / torch.where(sc > 0, sc, torch.ones_like(sc)).float()).clamp(-448, 448)
                d = code.to(torch.float8_e4m3fn).double() * sc
            out.append(d)
        return tuple(out)
    G = c["H"] // c["Hkv"]
    if op == "paged_attention":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens_list"]):
            pid = s["table"][b, :(n + c["page"] - 1) // c["page"]]
            k, v = _held64(s, 0, pid)[:n], _held64(s, 1, pid)[:n]
            for hq in range(c["H"]):
                p, lse[b, hq] = _softmax64(s["q"][b, hq].double(), k[:, hq // G], n - c["Nq"], True, scale)
                o[b, hq] = p @ v[:, hq // G]
        return o, lse
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["H"], o.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk = torch.zeros_like(o), torch.zeros(s["k"].shape, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    cq, ck = s["cu"].tolist(), s["cu_k"].tolist()
    for q0, q1, k0, k1 in zip(cq, cq[1:], ck, ck[1:]):
        for hq in range(c["H"]):
            k, v = s["k"][k0:k1, hq // G].double(), s["v"][k0:k1, hq // G].double()
            for i in range(q0, q1, block):
                e = min(i + block, q1)
                first = (k1 - k0) - (q1 - q0) + i - q0
                last = min(k1 - k0, max(1, first + e - i)) if c["causal"] else k1 - k0   # (keys that some row sees)
                p, l = _softmax64(s["q"][i:e, hq].double(), k[:last], first, c["causal"], scale)
                if op == "packed":
                    lse[hq, i:e] = l
                    o[i:e, hq] = p @ v[:last]
                    continue
                p = p * torch.exp(l - s["lse"][hq, i:e].double()).nan_to_num(0.0)[:, None]
                do, got = s["do"][i:e, hq].double(), s["o"][i:e, hq].double()
                ds = p * (do @ v[:last].t() - torch.einsum("id,id->i", do, got)[:, None])
                dq[i:e, hq] = scale * (ds @ k[:last])
                dk[k0:k0 + last, hq // G] += scale * (ds.t() @ s["q"][i:e, hq].double())
                dv[k0:k0 + last, hq // G] += p.t() @ do
    return (o, lse) if op == "packed" else (dq, dk, dv)
