"""The paged key/value cache (fa_paged_append, fa_paged_read, fa_paged_fwd) on the
GPU, in full against plain float64 arithmetic.

Attention, from the arithmetic: scores are fp32 sums of products that are exact
(16-bit operands; at 8 bits codes against q, which keeps its bits but for 2^-40 of
a row's largest element) times one or two fp32 factors, off by at most delta =
(2 D + 8) 2^-24 scale max_j sum_d |q_d k_jd|; weights are rounded to 16 bits for the
product (eps/2 of the type of the product: bf16 rows bf16, else fp16, which also
rounds weights below 2^-14 of its range, here 2^-21 of a row's largest, by up to
2^-25 each, i.e. 2^-32 of that largest) and the result once more; fp32 sums and the
exponential add 2^-15.  So per element, with w the weights' eps/2 and n the tokens,
  |O - ref| <= eps/2 |ref| + (w + 2^-15 + 2 delta) sum_j p_j |v_j| + 2^-32 p_max sum_j |v_j|
  |LSE - ref| <= delta + 2^-18 (1 + |ref|)
Append and read are exact: codes and scales as float32 quotients give them.
"""
from __future__ import annotations

import copy
import math
import os

import pytest
import torch

from exact_attention_10_gb300 import fa

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()


def _ok():
    rc = fa.sync_status(torch.cuda.current_stream().cuda_stream)
    assert rc == 0, fa.status_string(rc)


def quantise(x):
    """Codes (as float) and scales of rows, quotients rounded once to float32."""
    f = x.float()
    top = f.abs().amax(-1)
    sc = top / torch.full_like(top, 448.0)
    q = torch.where(sc[..., None] > 0, f / sc[..., None], 0.0)
    return q.to(torch.float8_e4m3fn), sc


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(lens, Hkv, D, page, bits, dtype, seed, spare=2):
    """A cache that holds sequences of `lens` tokens in scattered pages, garbage everywhere else."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cache = fa.paged_empty(P, Hkv, page, D, T[dtype], bits)
    for t in cache[:2]:   # infinities and NaN, in either format
        t.view(torch.uint8).fill_(0xFF)
    for t in cache[2:]:
        t.fill_(math.nan)
    n = sum(lens)
    gain = torch.where(torch.rand(D, generator=g, device="cuda") < 0.06, 4.0, 1.0)
    k = (torch.randn((max(n, 1), Hkv, D), generator=g, device="cuda") * gain + 0.3).to(T[dtype])
    v = torch.randn((max(n, 1), Hkv, D), generator=g, device="cuda").to(T[dtype])
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    if n:
        fa.paged_append(cache, table, k, v, ints([0] * len(lens)), cu=ints(cu))
    return cache, table, k, v, cu, g


def held(x, bits):
    if bits == 16:
        return x.double()
    c, s = quantise(x)
    return c.double() * s[..., None].double()


def check(q, o, lse, k, v, cu, lens, scale, bits, dtype, hidden=()):
    """Every element against float64; `hidden`: (b, first, last) tokens that do not exist."""
    B, H, Nq, D = q.shape
    G = H // k.shape[1]
    eps = torch.finfo(T[dtype]).eps / 2
    we = 2.0 ** -8 if (dtype == "bf16" and bits == 16) else 2.0 ** -11
    for b in range(B):
        n = lens[b]
        kk, vv = held(k[cu[b]:cu[b] + n], bits), held(v[cu[b]:cu[b] + n], bits)
        for h in range(H):
            x, y, z = q[b, h].double(), kk[:, h // G], vv[:, h // G]
            s = scale * x @ y.T
            vis = torch.arange(n, device="cuda")[None] <= torch.arange(Nq, device="cuda")[:, None] + (n - Nq)
            for bb, t0, t1 in hidden:
                if bb == b:
                    vis[:, t0:t1] = False
            s = torch.where(vis, s, -math.inf)
            l = torch.logsumexp(s, 1) if n else torch.full((Nq,), -math.inf, dtype=torch.float64, device="cuda")
            p = torch.exp(s - torch.where(l == -math.inf, 0.0, l)[:, None])
            r, none = p @ z, l == -math.inf
            if n:
                delta = (2 * D + 8) * 2.0 ** -24 * scale * (x.abs() @ y.abs().T).amax(1)
                bound = (eps * r.abs() + (we + 2.0 ** -15 + 2 * delta[:, None]) * (p @ z.abs())
                         + 2.0 ** -32 * p.amax(1, keepdim=True) * (vis.double() @ z.abs()))
                assert bool(((o[b, h].double() - r).abs() <= bound).all()), (b, h)
                err = (lse[b, h].double() - l).abs()[~none]
                assert bool((err <= (delta + 2.0 ** -18 * (1 + l.abs()))[~none]).all()), (b, h)
            assert bool((o[b, h][none] == 0).all()) and bool((lse[b, h][none] == -math.inf).all()), (b, h)


CASES = [
    # lens, H, Hkv, Nq, page
    ([1], 1, 1, 1, 16),
    ([16, 17, 0, 300], 4, 2, 1, 16),
    ([777], 8, 8, 1, 16),
    ([5, 1, 64, 200], 8, 2, 4, 32),           # more queries than tokens in one
    ([1000, 63, 2049], 5, 1, 3, 64),          # 15 rows
    ([129, 700], 16, 2, 5, 128),              # 40 rows: three blocks in a CTA of four
    ([90, 40, 33], 8, 1, 4, 16),              # 32 rows
    ([256], 64, 1, 5, 256),                   # 320 rows: five CTA blocks
    ([4000, 9000, 1, 2500, 6], 8, 2, 1, 16),  # shares and a join
    ([40000], 4, 2, 2, 1024),
    ([2000] * 70, 4, 4, 1, 64),
    ([30] * 700, 2, 1, 1, 16),
]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, dtype, D, bits):
    lens, H, Hkv, Nq, page = CASES[case]
    cache, table, k, v, cu, g = make(lens, Hkv, D, page, bits, dtype, seed=case)
    q = torch.randn((len(lens), H, Nq, D), generator=g, device="cuda").to(T[dtype])
    o, lse = fa.paged_forward(q, cache, table, ints(lens))
    _ok()
    if len(lens) > 100:   # a few of the many are enough
        keep = list(range(0, len(lens), 97))
        check(q[keep], o[keep], lse[keep], k, v, [cu[b] for b in keep], [lens[b] for b in keep], D ** -0.5, bits, dtype)
    else:
        check(q, o, lse, k, v, cu, lens, D ** -0.5, bits, dtype)


@pytest.mark.parametrize("bits", [16, 8])
def test_lengths_follow_the_device_and_are_clamped(bits):
    """Shorter lens, negative ones and ones past the table."""
    lens = [300, 200, 100]
    cache, table, k, v, cu, g = make(lens, 2, 64, 16, bits, "bf16", seed=3)
    q = torch.randn((3, 4, 2, 64), generator=g, device="cuda").bfloat16()
    for now in ([300, 7, 0], [-5, 200, 99], [33, 16, 100]):
        o, lse = fa.paged_forward(q, cache, table, ints(now))
        _ok()
        check(q, o, lse, k, v, cu, [max(0, n) for n in now], 0.125, bits, "bf16")
    o, lse = fa.paged_forward(q[:1], cache, table[:1, :10].contiguous(), ints([1 << 30]))
    _ok()
    check(q[:1], o, lse, k, v, cu, [160], 0.125, bits, "bf16")


@pytest.mark.parametrize("bits", [16, 8])
def test_pages_outside_the_pool(bits):
    """Tokens of a page that does not exist are not written, read as zeros and seen by no query."""
    lens = [100, 90]
    cache, table, k, v, cu, g = make(lens, 2, 64, 16, bits, "bf16", seed=5)
    P = cache.k.shape[0]
    table[0, 1], table[1, 5], table[1, 0] = P, -1, -(1 << 31)
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").bfloat16()
    o, lse = fa.paged_forward(q, cache, table, ints(lens))
    _ok()
    check(q, o, lse, k, v, cu, lens, 0.125, bits, "bf16", hidden=[(0, 16, 32), (1, 0, 16), (1, 80, 96)])
    before = [t.clone() for t in cache]
    fa.paged_append(cache, table, k + 1, v + 1, ints([16, 0]), cu=ints([0, 16, 32]))
    rk, rv = fa.paged_read(cache, table, ints([16, 0]), 32, cu=ints([0, 16, 32]), dtype=torch.bfloat16)
    _ok()
    assert not rk.any() and not rv.any()
    for a, b in zip(cache, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_and_read_exactly(dtype, D, bits):
    """Packed tokens of several sequences, strided inputs, rows of no sequence, appends that start inside a page."""
    g = torch.Generator(device="cuda").manual_seed(7)
    Hkv, page = 3, 32
    start, cu = [0, 5, 31, 64, 2], [3, 4, 50, 50, 115, 120]
    n = 130
    qkv = torch.randn((n, 3 * Hkv, D), generator=g, device="cuda")
    qkv[10] *= 300.0
    qkv[20] *= 1e-4
    qkv[21] = 0.0
    qkv[22, :, ::2] = 0.0
    qkv = qkv.to(T[dtype])
    _, k, v = qkv.split(Hkv, 1)
    table = torch.randperm(20, generator=g, device="cuda").int().view(5, 4)
    cache = fa.paged_empty(20, Hkv, page, D, T[dtype], bits)
    fa.paged_append(cache, table, k, v, ints(start), cu=ints(cu))
    rk, rv = fa.paged_read(cache, table, ints(start), n, cu=ints(cu), dtype=T[dtype])
    _ok()
    want = [torch.zeros_like(t) for t in cache]
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    for b in range(5):
        for i in range(cu[b], cu[b + 1]):
            t = start[b] + i - cu[b]
            if t >= 4 * page:   # past the table (sequence 3's last): not written, read as zeros
                continue
            pid = int(table[b, t // page])
            inside[i] = True
            for m, x in enumerate((k, v)):
                if bits == 16:
                    want[m][pid, :, t % page] = x[i]
                else:
                    c, s = quantise(x[i])
                    want[m].view(torch.uint8)[pid, :, t % page] = c.view(torch.uint8)
                    want[2 + m][pid, :, t % page] = s
    for a, b in zip(cache, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for r, x in ((rk, k), (rv, v)):
        val = x if bits == 16 else held(x, 8).float().to(T[dtype])
        assert torch.equal(r[inside], val[inside]) and not r[~inside].any()


def test_append_one_token_each_and_into_a_graph():
    """A captured decoding step: append, attention; replays follow lens, tables and tokens."""
    B, H, Hkv, D, page, steps = 3, 4, 2, 64, 16, 40
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = fa.paged_empty(30, Hkv, page, D, torch.float16, 8)
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(30, generator=g, device="cuda").int().tolist()
    lens = ints([0, 3, 30])
    k = torch.randn((steps, B, Hkv, D), generator=g, device="cuda").half()
    v = torch.randn((steps, B, Hkv, D), generator=g, device="cuda").half()
    old = [torch.randn((33, Hkv, D), generator=g, device="cuda").half() for _ in range(2)]
    for b in range(B):
        for j in range(2 if b == 2 else 1):
            table[b, j] = free.pop()
    fa.paged_append(cache, table, old[0], old[1], ints([0, 0, 0]), cu=ints([0, 0, 3, 33]))
    q, kn, vn = torch.zeros((B, H, 1, D), dtype=torch.float16, device="cuda"), k[0].clone(), v[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fa.paged_forward(q, cache, table, lens)   # (loads the kernels outside the capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_append(cache, table, kn, vn, lens)
        lens.add_(1)
        o, lse = fa.paged_forward(q, cache, table, lens)
    lens.copy_(ints([0, 3, 30]))
    hist_k = [[], [x for x in old[0][:3]], [x for x in old[0][3:]]]
    hist_v = [[], [x for x in old[1][:3]], [x for x in old[1][3:]]]
    for s in range(steps):
        now = lens.tolist()
        for b in range(B):
            if now[b] % page == 0 and int(table[b, now[b] // page]) < 0:
                table[b, now[b] // page] = free.pop()
            hist_k[b].append(k[s, b])
            hist_v[b].append(v[s, b])
        kn.copy_(k[s])
        vn.copy_(v[s])
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        graph.replay()
        if s % 8 == 0 or s == steps - 1:
            _ok()
            n = [len(x) for x in hist_k]
            cu = [0, n[0], n[0] + n[1]]
            check(q, o, lse, torch.stack(sum(hist_k, [])), torch.stack(sum(hist_v, [])), cu, n, 0.125, 8, "fp16")


def test_many_graphs_streams_and_strided_queries():
    """Two captured calls replayed at once keep their workspaces apart; q is a slice of a projection's output."""
    lens = [5000, 3000, 7000]
    cache, table, k, v, cu, g = make(lens, 2, 128, 16, 16, "bf16", seed=13)
    base = torch.randn((2, 3, 2, 12, 128), generator=g, device="cuda").bfloat16()   # [call, B, Nq, heads, D]
    n = ints(lens)
    res, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        q = base[i].transpose(1, 2)[:, 2:10]
        fa.paged_forward(q, cache, table, n)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res.append((q, *fa.paged_forward(q, cache, table, n)))
        graphs.append(gr)
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                gr.replay()
        for st in streams:
            torch.cuda.current_stream().wait_stream(st)
    _ok()
    for q, o, lse in res:
        check(q, o, lse, k, v, cu, lens, 128 ** -0.5, 16, "bf16")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o, lse = fa.paged_forward(res[0][0], cache, table, n, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(o, res[0][1]) and torch.equal(lse, res[0][2])


def test_same_bits_every_time_and_shared_pages():
    """The join's order is fixed; two sequences with the same first pages see the same tokens."""
    lens = [9000, 9000, 4000]
    cache, table, k, v, cu, g = make(lens, 2, 128, 64, 8, "bf16", seed=17)
    table[1] = table[0]
    q = torch.randn((1, 8, 1, 128), generator=g, device="cuda").bfloat16().expand(3, 8, 1, 128).contiguous()
    o, lse = fa.paged_forward(q, cache, table, ints(lens))
    for _ in range(3):
        o2, lse2 = fa.paged_forward(q, cache, table, ints(lens))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _ok()
    check(q[:1], o[1:2], lse[1:2], k, v, cu, [9000], 128 ** -0.5, 8, "bf16")


@pytest.mark.parametrize("bits", [16, 8])
def test_values_that_are_not_finite(bits):
    """A NaN or infinity in a sequence stays in it, and in the key heads that hold it."""
    lens = [50, 70, 4000]
    cache, table, k, v, cu, g = make(lens, 2, 64, 16, bits, "bf16", seed=19)
    q = torch.randn((3, 4, 1, 64), generator=g, device="cuda").bfloat16()
    bad = k[cu[1]:cu[1] + 1].clone()
    bad[0, 1, 3] = math.nan
    fa.paged_append(cache, table[1:2].contiguous(), bad, v[cu[1]:cu[1] + 1], ints([20]))
    o, lse = fa.paged_forward(q, cache, table, ints(lens))
    _ok()
    assert bool(o[1, 2:].isnan().all()) and bool(lse[1, 2:].isnan().all())
    assert bool(o[1, :2].isfinite().all())
    check(q[[0, 2]], o[[0, 2]], lse[[0, 2]], k, v, [cu[0], cu[2]], [50, 4000], 0.125, bits, "bf16")


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_of_queries_keys_and_values(dtype, bits):
    """Large and small queries and values, rows whose scales differ by powers of ten, one heavy token among many."""
    lens = [3000]
    for gain, vgain, scale in ((8.0, 1.0, 0.125), (1e-3, 100.0, 0.125), (30.0, 1e-2, 1e-2)):
        g = torch.Generator(device="cuda").manual_seed(23)
        cache, table, k, v, cu, _ = make(lens, 1, 64, 16, bits, dtype, seed=23)
        mag = 10.0 ** (3 * torch.rand((3000, 1, 1), generator=g, device="cuda") - 2)
        v = (v.float() * vgain * mag).to(T[dtype])
        k = k.clone()
        k[1234] *= 3
        fa.paged_append(cache, table, k, v, ints([0]), cu=ints([0, 3000]))
        q = (torch.randn((1, 4, 1, 64), generator=g, device="cuda") * gain).to(T[dtype])
        o, lse = fa.paged_forward(q, cache, table, ints(lens), scale=scale)
        _ok()
        check(q, o, lse, k, v, cu, lens, scale, bits, dtype)


def test_prompts_then_decoding():
    """The serving path together: a packed prefill, its keys into the cache, decoding, drafted tokens."""
    H, Hkv, D, page, lens = 8, 2, 128, 16, [40, 1, 333]
    g = torch.Generator(device="cuda").manual_seed(29)
    n, total = sum(lens), [x + 6 for x in lens]
    cache = fa.paged_empty(64, Hkv, page, D)
    table = torch.randperm(64, generator=g, device="cuda").int()[:63].view(3, 21).contiguous()
    table = torch.cat([table, torch.full((3, 3), -1, dtype=torch.int32, device="cuda")], 1)
    qkv = torch.randn((sum(total), H + 2 * Hkv, D), generator=g, device="cuda").bfloat16()   # all tokens of all sequences
    first = [0, total[0], total[0] + total[1]]
    rows = torch.cat([torch.arange(f, f + m, device="cuda") for f, m in zip(first, lens)])
    q, k, v = qkv[rows].split([H, Hkv, Hkv], 1)
    cu = ints([0, 40, 41, 374])
    plan = fa.packed_plan(cu, n, H, Hkv, causal=True)
    o, lse = fa.packed_forward(q, k, v, plan)
    fa.paged_append(cache, table, k, v, ints([0, 0, 0]), cu=cu)
    got = {i: o[j] for j, i in enumerate(rows.tolist())}
    at = ints(lens)
    for new in (1, 1, 4):   # two decoded tokens, then four drafted ones
        idx = torch.cat([torch.arange(f + m, f + m + new, device="cuda") for f, m in zip(first, at.tolist())])
        q, k, v = qkv[idx].split([H, Hkv, Hkv], 1)
        fa.paged_append(cache, table, k, v, at, cu=ints([0, new, 2 * new, 3 * new]))
        at = at + new
        o, _ = fa.paged_forward(q.reshape(3, new, H, D).transpose(1, 2), cache, table, at)
        for b in range(3):
            for i in range(new):
                got[int(idx[b * new + i])] = o[b, :, i]
    _ok()
    qq, kk, vv = qkv.split([H, Hkv, Hkv], 1)
    full = fa.packed_plan(ints(first + [sum(total)]), sum(total), H, Hkv, causal=True)
    want, _ = fa.packed_forward(qq, kk, vv, full)
    _ok()
    for b in range(3):   # against float64, every token
        for h in range(H):
            x, y, z = (t[first[b]:first[b] + total[b], i].double() for t, i in ((qq, h), (kk, h // 4), (vv, h // 4)))
            s = D ** -0.5 * x @ y.T
            s.masked_fill_(torch.ones_like(s).triu(1).bool(), -math.inf)
            delta = (2 * D + 8) * 2.0 ** -24 * D ** -0.5 * (x.abs() @ y.abs().T).amax(1, keepdim=True)
            r = torch.stack([got[first[b] + i][h] for i in range(total[b])]).double()
            for res in (want[first[b]:first[b] + total[b], h].double(), r):
                if res is r:   # the last sequence's 21 pages end before its last three tokens, which the cache does not hold
                    s[:, 21 * page:] = -math.inf
                p = torch.softmax(s, 1)
                bound = 2.0 ** -8 * (p @ z).abs() + (2.0 ** -8 + 2.0 ** -15 + 2 * delta) * (p @ z.abs())
                assert bool(((res - p @ z).abs() <= bound).all())


def test_streams_of_their_own():
    """Append, read and attention on a stream given by the call."""
    lens = [70, 33]
    g = torch.Generator(device="cuda").manual_seed(37)
    k, v = (torch.randn((103, 2, 64), generator=g, device="cuda").half() for _ in range(2))
    q = torch.randn((2, 4, 1, 64), generator=g, device="cuda").half()
    cache, table = fa.paged_empty(8, 2, 32, 64, torch.float16, 8), ints([[5, 0, 7], [2, 1, -1]])
    zero, cu, n = ints([0, 0]), ints([0, 70, 103]), ints(lens)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    fa.paged_append(cache, table, k, v, zero, cu=cu, stream=st)
    rk, _ = fa.paged_read(cache, table, zero, 103, cu=cu, dtype=torch.float16, stream=st)
    o, lse = fa.paged_forward(q, cache, table, n, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    _ok()
    assert torch.equal(rk, held(k, 8).float().half())
    check(q, o, lse, k, v, [0, 70], lens, 0.125, 8, "fp16")


def test_the_readme_block():
    """The README's python block on packed sequences and the paged cache, run as it stands with small sizes."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        blocks = [b.split("```")[0] for b in f.read().split("```python\n")[1:]]
    text, = (b for b in blocks if b.startswith("# packed sequences"))
    g = torch.Generator(device="cuda").manual_seed(41)
    H, Hkv, D, lens, T = 4, 2, 64, ints([50, 3]), 53
    q, do = (torch.randn((T, H, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    k, v = (torch.randn((T, Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))
    tokens = [(torch.randn((2, H, 1, D), generator=g, device="cuda").bfloat16(),
               *(torch.randn((2, Hkv, D), generator=g, device="cuda").bfloat16() for _ in range(2))) for _ in range(20)]
    names = dict(fa=fa, torch=torch, q=q, k=k, v=v, do=do, H=H, Hkv=Hkv, D=D, T=T, cu=ints([0, 50, 53]), start=ints([0, 0]),
                 lens=lens, pages=12, table=torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6), tokens=tokens)
    exec(compile(text, "README.md", "exec"), names)
    _ok()
    assert lens.tolist() == [70, 23]
    hk = [torch.cat([x[a:b], *(t[1 + i][s:s + 1] for t in tokens)]) for i, x in ((0, k), (1, v)) for s, a, b in ((0, 0, 50), (1, 50, 53))]
    check(tokens[-1][0], names["o"], names["lse"], torch.cat(hk[:2]), torch.cat(hk[2:]), [0, 70], [70, 23], D ** -0.5, 16, "bf16")


def test_copies_of_a_cache():
    cache = fa.paged_empty(4, 2, 16, 64, bits=8)
    twin = copy.deepcopy(cache)
    assert isinstance(twin, fa.PagedCache) and twin.k.data_ptr() != cache.k.data_ptr()
    assert twin.args(torch.bfloat16).k == twin.k.data_ptr()
