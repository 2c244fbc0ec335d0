"""The 4-bit key/value cache on the GPU (fa_cache_append, _read, _fwd,
_weights, _evict) against plain float64 implementations of their definitions.

The packed format is compared bit for bit.  Attention and weights are compared
with tolerances that follow the arithmetic:

* scores.  x = scale (ks dot + kmin sum q), where dot = sum code q is formed in
  fp32 from exact products (q scaled by a power of two) in chains of at most D
  + 8 additions, and sum q likewise: |dx| <= (D + 8) 2^-24 A with A = scale (ks
  sum code |q| + |kmin| sum |q|), the sum of all magnitudes; twice that covers
  the products and the final additions.  `delta` below is its largest value
  over a row's visible tokens.
* weights: p has the relative error delta + 2^-21 (the exponential); w = p vs
  is rounded to fp16, 2^-11 relative, as it enters the product with the codes:
  2^-11 of sum p vs code (2^-22 for fp16 results), part of B = sum p (vs code +
  |vmin|), the sum of all magnitudes in O's numerator.
* sums over n tokens in fp32: each chain has at most n / 8 + 64 additions
  (eight warps, then the joins): (n / 8 + 64) 2^-24 of the magnitudes.
* the result: half a unit of its type, finfo(t).eps / 2.
"""
from __future__ import annotations

import math

import numpy as np
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
    assert fa.sync_status(torch.cuda.current_stream().cuda_stream) == 0


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def pack64(x):
    """(codes, params) of x [..., D] by the definition, in float64."""
    t, d = x.dtype, x.double()
    mn, mx = d.amin(-1, keepdim=True), d.amax(-1, keepdim=True)
    sc = ((mx - mn) / 15).to(t)
    s = sc.double()
    code = torch.where(s > 0, torch.round((d - mn) / torch.where(s > 0, s, 1.0)), torch.zeros_like(d)).clamp(0, 15)
    code = code.to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.cat([sc, mn.to(t)], -1)


def unpack64(codes, params):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    return c * params[..., 0:1].double() + params[..., 1:2].double()


def random_cache(B, Hkv, C, D, dtype, seed):
    """A cache of plausible rows (keys with a few large channels)."""
    g = _gen(seed)
    k = torch.randn((B, Hkv, C, D), generator=g, device="cuda")
    k = k * torch.where(torch.rand(D, generator=g, device="cuda") < 0.05, 4.0, 1.0) + torch.randn(D, generator=g, device="cuda") / 2
    v = torch.randn((B, Hkv, C, D), generator=g, device="cuda")
    kc, kp = pack64(k.to(T[dtype]))
    vc, vp = pack64(v.to(T[dtype]))
    return fa.PackedCache(kc.contiguous(), kp.contiguous(), vc.contiguous(), vp.contiguous())


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hkv,N,C", [(1, 1, 1, 1), (3, 2, 1, 40), (2, 3, 77, 100), (5, 1, 33, 64), (2, 8, 300, 301)])
def test_append_and_read(B, Hkv, N, C, D, dtype):
    g = _gen(N + C + D)
    k = (torch.randn((B, Hkv, N, D), generator=g, device="cuda") * 3).to(T[dtype])
    v = torch.randn((B, Hkv, N, D), generator=g, device="cuda").to(T[dtype])
    start = torch.randint(0, C - N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    count = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    count[0] = N
    for cnt in (None, count):
        cache = fa.cache_empty(B, Hkv, C, D, T[dtype])
        for x in cache:   # a pattern in the rows that stay untouched
            x.view(torch.uint8).fill_(0x5A)
        want = [x.clone() for x in cache]
        fa.cache_append(cache, k, v, start, count=cnt)
        _ok()
        for x, at in ((k, 0), (v, 2)):
            codes, params = pack64(x)
            for b in range(B):
                s, n = int(start[b]), N if cnt is None else int(cnt[b])
                want[at][b, :, s:s + n] = codes[b, :, :n]
                want[at + 1][b, :, s:s + n] = params[b, :, :n]
        for got, ref in zip(cache, want):
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8))
        rk, rv = fa.cache_read(cache, start, N, count=cnt)
        u = torch.finfo(T[dtype]).eps / 2
        for got, x in ((rk, k), (rv, v)):
            ref = unpack64(*pack64(x))
            real = torch.ones((B, N), dtype=torch.bool, device="cuda") if cnt is None else (
                torch.arange(N, device="cuda") < cnt[:, None])
            ref = ref * real[:, None, :, None]
            # half a unit of the type, and fp32's rounding before it
            tol = ref.abs() * (u + 2.0 ** -23) + torch.finfo(T[dtype]).smallest_normal * u
            assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_places_outside_the_cache(dtype):
    """Tokens before 0 and from C on are not written; reads of them are zeros."""
    B, Hkv, N, C, D = 4, 2, 10, 16, 64
    k = torch.randn((B, Hkv, N, D), device="cuda").to(T[dtype])
    start = torch.tensor([-3, 12, 2 ** 31 - 4, -2 ** 31], dtype=torch.int32, device="cuda")
    cache = fa.cache_empty(B, Hkv, C, D, T[dtype])
    fa.cache_append(cache, k, k, start)
    got = fa.cache_read(cache, start, N)[0]
    _ok()
    codes, params = pack64(k)
    want = [torch.zeros_like(x) for x in cache[:2]]
    want[0][0, :, :7], want[1][0, :, :7] = codes[0, :, 3:], params[0, :, 3:]
    want[0][1, :, 12:], want[1][1, :, 12:] = codes[1, :, :4], params[1, :, :4]
    assert torch.equal(cache.k_codes, want[0]) and torch.equal(cache.k_params, want[1])
    assert torch.equal(cache.v_codes, want[0]) and torch.equal(cache.v_params, want[1])
    assert bool((got[0, :, :3] == 0).all()) and bool((got[1, :, 4:] == 0).all()) and bool((got[2:] == 0).all())
    assert bool((got[0, :, 3:] != 0).any())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_borders_and_extremes(D, dtype):
    """Rows whose values lie exactly on and next to borders between codes,
    constant rows, single steps, the type's largest and smallest values."""
    t = T[dtype]
    fi = torch.finfo(t)
    rows = []
    for s in (1.0, 0.5, 3.0, 2.0 ** -10, 48.0):           # scale s (max - min = 15 s): halves are borders
        for lo in (0.0, -7.5 * s, 64 * s, -15 * s):
            x = lo + torch.arange(D, dtype=torch.float64) % 31 * 0.5 * s
            x[0], x[1] = lo, lo + 15 * s
            rows.append(x)
            rows.append(torch.nextafter(x.to(t).float(), torch.tensor(1e30)).double())
    rows += [torch.zeros(D), torch.full((D,), 3.25), torch.full((D,), -float(fi.max))]
    rows.append(torch.linspace(-1, 1, D).double() * fi.max)                      # the range overflows fp32 in bf16
    rows.append(torch.linspace(0, 1, D).double() * fi.smallest_normal * 40)
    one = torch.zeros(D)
    one[D // 2] = fi.smallest_normal * 2
    rows.append(one)
    rows.append(torch.where(torch.arange(D) == 5, fi.max, 1.0))
    mixed = torch.randn(D, generator=torch.Generator().manual_seed(1)) * 1e-4
    mixed[3] = 7.0
    rows.append(mixed)
    x = torch.stack([r.double() for r in rows]).to(t).cuda()[None, None].contiguous()
    N = x.shape[2]
    cache = fa.cache_empty(1, 1, N, D, t)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, x, x, start)
    got = fa.cache_read(cache, start, N)[0]
    _ok()
    codes, params = pack64(x)
    bad = (cache.k_codes != codes).any(-1)[0, 0].nonzero().flatten().tolist()
    assert not bad, bad
    assert torch.equal(cache.k_params, params) and torch.equal(cache.v_codes, codes)
    ref = unpack64(codes, params)
    tol = ref.abs() * (fi.eps / 2 + 2.0 ** -23) + fi.smallest_normal * fi.eps
    assert bool(torch.isfinite(got[ref.abs() <= fi.max]).all())
    inside = ref.abs() < fi.max * (1 - fi.eps)
    assert bool(((got.double() - ref).abs() <= tol)[inside].all())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rows_that_are_not_finite_stand_for_nan(dtype):
    x = torch.randn((1, 1, 5, 64), device="cuda").to(T[dtype])
    x[0, 0, 1, 7], x[0, 0, 2, 63], x[0, 0, 3, 0] = math.nan, math.inf, -math.inf
    cache = fa.cache_empty(1, 1, 5, 64, T[dtype])
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, x, x, start)
    for got in fa.cache_read(cache, start, 5):
        assert bool(torch.isnan(got[0, 0, 1:4]).all()) and bool(torch.isfinite(got[0, 0, [0, 4]]).all())


# ------------------------------------------------------------------ attention and weights

def reference(q, cache, lens, left, sinks, scale):
    """Per sequence and head, float64: O, LSE, token weights and the bounds of
    the module's docstring, (O tolerance without the final rounding, delta per row)."""
    B, H, Nq, D = q.shape
    Hkv, C = cache.k_codes.shape[1:3]
    G = H // Hkv
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    w = torch.zeros((B, Hkv, C), dtype=torch.float64, device="cuda")
    w_tol = torch.zeros_like(w)
    o_tol = torch.zeros_like(o)
    delta = torch.zeros_like(lse)
    for b in range(B):
        n = max(0, min(int(lens[b]), C))
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        for h in range(Hkv):
            k, v = (unpack64(cache[i][b, h, :n], cache[i + 1][b, h, :n]) for i in (0, 2))
            ks, kmin = cache.k_params[b, h, :n].double().unbind(-1)
            vs, vmin = cache.v_params[b, h, :n].double().unbind(-1)
            codes = (k - kmin[:, None]) / torch.where(ks > 0, ks, 1.0)[:, None]
            for g in range(G):
                for i in range(Nq):
                    pos = n - Nq + i
                    vis = j <= pos
                    if left >= 0:
                        vis &= (j >= pos - left) | (j < sinks)
                    at = vis.nonzero().flatten()
                    if not len(at):
                        continue
                    x = q[b, h * G + g, i].double()
                    s = (k[at] @ x) * scale
                    mag = scale * (ks[at] * (codes[at] @ x.abs()) + kmin[at].abs() * x.abs().sum())
                    d = 2 * (D + 8) * 2.0 ** -24 * float(mag.max())
                    L = torch.logsumexp(s, 0)
                    p = torch.exp(s - L)
                    o[b, h * G + g, i] = p @ v[at]
                    lse[b, h * G + g, i] = L
                    delta[b, h * G + g, i] = d
                    part = p @ (v - vmin[:, None])[at]
                    o_tol[b, h * G + g, i] = part * 2.0 ** -11 + (part + p @ vmin[at].abs()) * (n / 8 + 64) * 2.0 ** -24 + (
                        2 * (d + 2.0 ** -21) * (p @ v[at].abs()))
                    w[b, h, at] += p
                    w_tol[b, h, at] += p * (d + 2.0 ** -20 + abs(float(L)) * 2.0 ** -22)
    return o, lse, w, o_tol, w_tol, delta


def check_attention(q, cache, lens, left, sinks, scale, o, lse, ref):
    o_ref, lse_ref, _, o_tol, _, delta = ref
    t = q.dtype
    empty = torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse), empty)
    assert bool((o[empty] == 0).all())
    C = cache.k_codes.shape[2]
    tol = o_ref.abs() * torch.finfo(t).eps / 2 * (1 + 2.0 ** -10) + o_tol + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    err = (o.double() - o_ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    fine = ~empty
    ltol = delta + (C / 8 + 64) * 2.0 ** -24 + (1 + lse_ref.abs().where(fine, torch.zeros_like(lse_ref))) * 2.0 ** -21
    lerr = (lse.double() - lse_ref).abs()[fine]
    assert bool((lerr <= ltol[fine]).all()), float((lerr / ltol[fine]).max())


ATTENTION = [  # (B, H, Hkv, Nq, C, lens, left, sinks)
    (1, 1, 1, 1, 1, [1], -1, 0),
    (1, 2, 1, 1, 64, [64], -1, 0),
    (3, 4, 2, 1, 100, [1, 33, 100], -1, 0),
    (2, 8, 1, 1, 777, [777, 500], -1, 0),               # eight rows per key head
    (2, 5, 1, 1, 300, [300, 257], -1, 0),
    (2, 9, 1, 1, 300, [300, 257], -1, 0),               # more than eight: 16-row tiles
    (1, 16, 1, 3, 700, [700], -1, 0),                   # 48 rows: three row blocks
    (2, 4, 2, 4, 90, [3, 90], -1, 0),                   # the first queries see nothing
    (4, 2, 2, 1, 50, [0, 50, 60, -5], -1, 0),           # no tokens; lengths outside [0, C]
    (1, 8, 8, 1, 2000, [1999], 255, 4),                 # a window and sinks: units left out between them
    (2, 8, 2, 2, 2000, [1500, 130], 64, 70),            # sinks past a unit
    (2, 4, 4, 1, 1000, [1000, 999], 0, 0),              # the query's own token alone
    (1, 4, 1, 5, 1000, [640], 100, 1000),               # sinks that cover everything
    (2, 3, 3, 1, 5000, [5000, 4097], 4096, 1),
    (40, 4, 2, 1, 200, None, -1, 0),                    # many short sequences
    (300, 1, 1, 1, 70, None, 20, 3),                    # more sequences than threads in a block
]


def _attention_case(case, D, dtype, seed=0, gain=1.0):
    B, H, Hkv, Nq, C, lens, left, sinks = case
    cache = random_cache(B, Hkv, C, D, dtype, seed + C)
    g = _gen(seed + 1)
    q = (torch.randn((B, H, Nq, D), generator=g, device="cuda") * gain).to(T[dtype])
    if lens is None:
        lens = torch.randint(0, C + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    else:
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return q, cache, lens, left, sinks


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "-".join(map(str, c[:5])) + f"-w{c[6]}s{c[7]}")
def test_attention_and_weights(case, D, dtype):
    q, cache, lens, left, sinks = _attention_case(case, D, dtype)
    scale = D ** -0.5
    o, lse = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks)
    _ok()
    ref = reference(q, cache, lens, left, sinks, scale)
    check_attention(q, cache, lens, left, sinks, scale, o, lse, ref)
    w = fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks)
    acc = torch.full_like(w, 3.0)
    got = fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks, acc=acc)
    _ok()
    assert got is acc
    w_ref, w_tol = ref[2], ref[4]
    # (an LSE that is off by its own tolerance scales every weight)
    rows = q.shape[1] // cache.k_codes.shape[1] * q.shape[2]
    tol = 2 * w_tol + w_ref * (rows + 8) * 2.0 ** -23 + w_ref * (cache.k_codes.shape[2] / 8 + 64) * 2.0 ** -23
    err = (w.double() - w_ref).abs()
    assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())
    C = cache.k_codes.shape[2]
    n = lens.clamp(0, C)
    behind = torch.arange(C, device="cuda")[None, None] >= n[:, None, None]
    assert bool((w[behind.expand_as(w)] == 0).all()) and bool((acc[behind.expand_as(w)] == 3.0).all())
    assert bool(((acc - 3.0).double() - w_ref).abs().le(tol + 2.0 ** -21).all())


ROWS = [  # as above, with more than 16 query rows per key head
    (1, 17, 1, 1, 1, [1], -1, 0),
    (1, 4, 1, 5, 64, [64], -1, 0),
    (2, 8, 2, 8, 200, [65, 200], -1, 0),                # 32 rows; an odd number of units
    (1, 3, 1, 11, 500, [500], -1, 0),                   # 33
    (1, 8, 1, 8, 1000, [937], -1, 0),                   # 64, one whole block
    (2, 5, 1, 13, 700, [700, 129], -1, 0),              # 65: a second block of one row
    (2, 8, 1, 20, 600, [600, 10], 64, 5),               # 160; some queries see nothing
    (3, 20, 1, 1, 300, [0, 400, -5], 20, 3),            # no tokens; lengths outside [0, C]
    (1, 8, 2, 5, 3001, [2999], 255, 4),                 # units left out between sinks and window: tiles of two places
    (2, 16, 4, 6, 2000, [1500, 130], 64, 70),
    (1, 24, 1, 1, 4000, [3999], 1000, 65),
    (1, 6, 1, 3, 40000, [39990], -1, 0),                # shared out over many CTAs
    (40, 18, 1, 1, 200, None, -1, 0),
    (300, 20, 1, 1, 70, None, 20, 3),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(map(str, c[:5])) + f"-w{c[6]}s{c[7]}")
def test_attention_and_weights_of_many_rows(case, D, dtype):
    test_attention_and_weights(case, D, dtype)


@pytest.mark.parametrize("B", [31, 32, 33, 256, 257])
@pytest.mark.parametrize("H", [2, 20])
def test_batches_around_what_a_warp_or_a_block_holds(B, H):
    """The search for a CTA's share of the tokens takes a sequence to a lane, or
    several to a thread; empty sequences among them, at either end."""
    for lens in (None, [0] * (B - 1) + [900], [900] + [0] * (B - 1)):
        test_attention_and_weights((B, H, 1, 1, 1500, lens, -1, 0), 64, "bf16")


@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_many_rows_run_to_run_and_hidden(D):
    """The same bits on every call and beside another stream's calls; rows that a
    query does not see, and those behind the sequence, may hold anything."""
    q, cache, lens, left, sinks = _attention_case((3, 12, 2, 9, 3000, [2900, 64, 1501], 700, 9), D, "bf16", seed=21)
    _, lse = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks)
    want = fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks)
    dirty = fa.PackedCache(*(x.clone() for x in cache))
    for b, n in enumerate(lens.tolist()):
        dirty[0][b, :, n:] = 255
        dirty[1][b, :, n:] = math.nan
        first = max(0, n - 9 - left)   # the first query's window
        if first > sinks:
            dirty[1][b, :, sinks:first] = math.inf
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(20):
        got = fa.cache_weights(q, dirty, lse, lens, window=(left, 0), sinks=sinks)
        with torch.cuda.stream(side):
            other = fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(other, want)
    _ok()


@pytest.mark.parametrize("D", [64, 128])
def test_large_scores(D):
    """Queries four times larger: the maximum moves often, single tokens dominate."""
    for dtype in ("bf16", "fp16"):
        q, cache, lens, left, sinks = _attention_case((2, 8, 2, 1, 3000, [3000, 2047], -1, 0), D, dtype, seed=5, gain=6.0)
        o, lse = fa.cache_forward(q, cache, lens)
        _ok()
        check_attention(q, cache, lens, left, sinks, D ** -0.5, o, lse, reference(q, cache, lens, left, sinks, D ** -0.5))


@pytest.mark.parametrize("Nq,G", [(1, 4), (3, 4)])
def test_hidden_rows_may_hold_anything(Nq, G):
    """Rows behind the last token, and rows that no query sees between the
    sinks and the window, hold NaN and infinities: the results are those of a
    cache whose rows there are zeros, bit for bit."""
    B, Hkv, C, D, left, sinks = 2, 2, 500, 128, 90, 5
    q, cache, lens, _, _ = _attention_case((B, G * Hkv, Hkv, Nq, C, [433, 300], left, sinks), D, "bf16", seed=3)
    clean = fa.PackedCache(*(x.clone() for x in cache))
    dirty = fa.PackedCache(*(x.clone() for x in cache))
    for b in range(B):
        n = int(lens[b])
        hidden = list(range(sinks, n - Nq - left)) + list(range(n, C))
        for i, x in enumerate(dirty):
            x[b, :, hidden] = 0xFF if i in (0, 2) else (math.nan if i == 1 else math.inf)
            clean[i][b, :, hidden] = 0
    res = []
    for c in (clean, dirty):
        o, lse = fa.cache_forward(q, c, lens, window=(left, 0), sinks=sinks)
        w = fa.cache_weights(q, c, lse, lens, window=(left, 0), sinks=sinks)
        res.append((o, lse, w))
    _ok()
    for a, b in zip(*res):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_a_visible_nan_row_reaches_only_its_queries():
    q, cache, lens, _, _ = _attention_case((2, 4, 2, 2, 300, [300, 300], 40, 2), 64, "bf16", seed=9)
    cache.v_params[0, 1, 258] = math.nan    # seen by query 0 (position 298: 258 ..) alone of key head 1
    o, lse = fa.cache_forward(q, cache, lens, window=(40, 0), sinks=2)
    _ok()
    bad = torch.isnan(o).any(-1)
    want = torch.zeros_like(bad)
    want[0, 2:4, 0] = True
    assert torch.equal(bad, want) and bool(torch.isfinite(lse).all())


def test_long_context_split_over_all_ctas():
    """One sequence of two key heads over every CTA (parts joined by the merge),
    and a ragged batch whose shares cut tiles: rows sampled against float64."""
    for case in ((1, 16, 2, 1, 60001, [60001], -1, 0), (3, 8, 2, 1, 30000, [30000, 17, 12345], -1, 0),
                 (1, 24, 2, 1, 20000, [20000], 9999, 64)):
        for D, dtype in ((128, "bf16"), (64, "fp16")):
            q, cache, lens, left, sinks = _attention_case(case, D, dtype, seed=11)
            o, lse = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks)
            _ok()
            ref = reference(q, cache, lens, left, sinks, D ** -0.5)
            check_attention(q, cache, lens, left, sinks, D ** -0.5, o, lse, ref)
            again = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks)
            assert torch.equal(o, again[0]) and torch.equal(lse, again[1])   # the same bits on every call


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes of codes: the last sequence's rows."""
    B, Hkv, C, D = 5, 4, 3400000, 128    # 68 M rows, 4.4 GB of codes for K
    row = random_cache(1, Hkv, 700, D, "bf16", 3)
    parts = []
    for x in row:
        y = torch.zeros((B, Hkv, C, x.shape[3]), dtype=x.dtype, device="cuda")
        y[-1, :, :700] = x[0]
        parts.append(y)
    cache = fa.PackedCache(*parts)
    q = torch.randn((B, 8, 1, D), generator=_gen(4), device="cuda").to(torch.bfloat16)
    lens = torch.tensor([0, 1, 0, 2, 700], dtype=torch.int32, device="cuda")
    o, lse = fa.cache_forward(q, cache, lens)
    want = fa.cache_forward(q[-1:].contiguous(), row, lens[-1:].contiguous())
    _ok()
    assert torch.allclose(o[-1:].float(), want[0].float(), rtol=2 ** -7, atol=1e-3)   # split differently: one rounding apart
    assert torch.allclose(lse[-1:], want[1], rtol=1e-5, atol=1e-5)
    k = torch.randn((B, Hkv, 3, D), generator=_gen(5), device="cuda").to(torch.bfloat16)
    start = torch.full((B,), C - 3, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, k, k, start)
    codes, params = pack64(k)
    _ok()
    assert torch.equal(cache.k_codes[:, :, -3:], codes) and torch.equal(cache.v_params[:, :, -3:], params)
    assert torch.equal(cache.k_codes[-1, :, :700], row.k_codes[0])


def test_graph_replay_follows_lens_and_two_graphs_overlap():
    """A decode step captured once (append, attention, weights) and replayed
    while lens grow; two captured graphs replayed on two streams at a time."""
    B, H, Hkv, C, D = 3, 8, 2, 4000, 128
    q, cache, lens, _, _ = _attention_case((B, H, Hkv, 1, C, [700, 3000, 1], -1, 0), D, "bf16", seed=21)
    k = torch.randn((B, Hkv, 1, D), generator=_gen(6), device="cuda").to(torch.bfloat16)
    acc = torch.zeros((B, Hkv, C), device="cuda")

    def step():
        fa.cache_append(cache, k, k, lens)
        lens.add_(1)
        o, lse = fa.cache_forward(q, cache, lens)
        fa.cache_weights(q, cache, lse, lens, acc=acc)
        return o, lse

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    lens.copy_(torch.tensor([710, 3100, 50], dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [713, 3103, 53]
    want = fa.cache_forward(q, cache, lens)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])

    caches = [random_cache(B, Hkv, C, D, "bf16", 30 + i) for i in range(2)]
    ln = torch.tensor([4000, 2000, 3999], dtype=torch.int32, device="cuda")
    wants = [fa.cache_forward(q, c, ln) for c in caches]
    graphs, outs = [], []
    for c in caches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.cache_forward(q, c, ln))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_on_another_stream():
    q, cache, lens, _, _ = _attention_case((4, 8, 2, 1, 3000, [3000, 5, 700, 2999], -1, 0), 64, "bf16", seed=8)
    want = fa.cache_forward(q, cache, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs = [fa.cache_forward(q, cache, lens) for _ in range(8)]
    given = fa.cache_forward(q, cache, lens, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    for got in outs + [given]:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ eviction

def evict_reference(acc, lens, keep, sinks, recent):
    """Kept positions [B, Hkv, keep] (-1 behind them) by sorting, in numpy."""
    B, Hkv, C = acc.shape
    out = np.full((B, Hkv, keep), -1, dtype=np.int64)
    for b in range(B):
        n = max(0, min(int(lens[b]), C))
        for h in range(Hkv):
            if n <= keep:
                out[b, h, :n] = np.arange(n)
                continue
            mid = np.arange(sinks, n - recent)
            a = acc[b, h, mid].astype(np.float64) + 0.0
            low = np.isnan(a)
            order = np.lexsort((mid, np.where(low, 0.0, -np.where(low, 0.0, a)), low))
            pick = np.concatenate([np.arange(sinks), mid[order[:keep - sinks - recent]], np.arange(n - recent, n)])
            out[b, h] = np.sort(pick)
    return out


EVICT = [  # (B, Hkv, C, lens, keep, sinks, recent)
    (1, 1, 1, [1], 1, 0, 0),
    (2, 2, 50, [50, 20], 30, 4, 8),
    (3, 1, 100, [100, 0, 31], 30, 0, 0),
    (1, 3, 777, [777], 776, 0, 0),            # one token goes
    (2, 2, 777, [700, 650], 64, 0, 64),       # the recent ones alone
    (2, 2, 777, [700, 650], 64, 60, 4),       # nothing to choose
    (1, 2, 5000, [4999], 1, 0, 0),
    (1, 1, 40000, [39999], 20001, 3, 100),    # a cluster per row
    (2, 4, 20000, [20000, 15000], 2048, 4, 512),
    (1, 2, 400000, [399999], 3000, 4, 100),   # slices longer than shared memory holds
    (70, 8, 300, None, 100, 1, 20),           # more rows than SMs
    (2, 1, 64, [70, -3], 32, 1, 1),           # lengths outside [0, C]
    (2, 1, 20, [20, 7], 33, 1, 1),            # a budget that no sequence can reach
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(map(str, (c[0], c[1], c[2], c[4], c[5], c[6]))))
def test_evict(case, kind, D):
    B, Hkv, C, lens, keep, sinks, recent = case
    g = _gen(C + keep)
    acc = torch.exp(4 * torch.randn((B, Hkv, C), generator=g, device="cuda") - 6)
    if kind == "ties":      # few distinct weights, many zeros of both signs
        acc = torch.floor(acc * 4).clamp(max=3)
        acc = torch.where((torch.arange(C, device="cuda") % 3 == 0) & (acc == 0), -torch.zeros_like(acc), acc)
    if kind == "special":   # negative weights, infinities, NaN, subnormals
        acc = acc - 0.01
        r = torch.rand(acc.shape, generator=g, device="cuda")
        for lo, x in ((0.0, math.nan), (0.05, math.inf), (0.1, -math.inf), (0.15, 1e-42), (0.2, -1e-42)):
            acc = torch.where((r >= lo) & (r < lo + 0.05), x, acc)
    lens = (torch.randint(0, C + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if lens is None
            else torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cache = fa.PackedCache(torch.randint(0, 256, (B, Hkv, C, D // 2), generator=g, device="cuda", dtype=torch.uint8),
                           torch.randn((B, Hkv, C, 2), generator=g, device="cuda").bfloat16(),
                           torch.randint(0, 256, (B, Hkv, C, D // 2), generator=g, device="cuda", dtype=torch.uint8),
                           torch.randn((B, Hkv, C, 2), generator=g, device="cuda").bfloat16())
    cap = keep + 5
    out = fa.cache_empty(B, Hkv, cap, D)
    for x in out:
        x.view(torch.uint8).fill_(0x77)
    got, acc2, lens2, index = fa.cache_evict(cache, acc, lens, keep, sinks=sinks, recent=recent, out=out)
    _ok()
    assert got is out
    n = lens.clamp(0, C)
    assert torch.equal(lens2, n.clamp(max=keep).int())
    want = torch.from_numpy(evict_reference(acc.cpu().numpy(), n.cpu().numpy(), keep, sinks, recent)).cuda()
    assert torch.equal(index.long(), want)
    real = want >= 0
    at = want.clamp(min=0)
    a = torch.where(real, acc.gather(2, at), torch.zeros((), device="cuda"))
    assert torch.equal(acc2[:, :, :keep].view(torch.int32), a.view(torch.int32)) and bool((acc2[:, :, keep:] == 0).all())
    for x, y in zip(cache, out):
        moved = x.gather(2, at[..., None].expand(B, Hkv, keep, x.shape[3]))
        old = torch.full_like(y[:, :, :keep].view(torch.uint8), 0x77).view(y.dtype)
        ref = torch.where(real[..., None], moved.view(torch.int16) if x.dtype != torch.uint8 else moved,
                          old.view(torch.int16) if x.dtype != torch.uint8 else old)
        mine = y[:, :, :keep]
        assert torch.equal(mine.view(torch.int16) if x.dtype != torch.uint8 else mine, ref)
        assert bool((y[:, :, keep:].reshape(-1).view(torch.uint8) == 0x77).all())


def test_evict_into_a_new_cache():
    q, cache, lens, _, _ = _attention_case((2, 4, 2, 1, 500, [500, 40], -1, 0), 64, "bf16", seed=2)
    lse = fa.cache_forward(q, cache, lens)[1]
    acc = fa.cache_weights(q, cache, lse, lens)
    kept, acc2, lens2, index = fa.cache_evict(cache, acc, lens, 64, sinks=4, recent=16)
    _ok()
    assert kept.k_codes.shape == (2, 2, 64, 32) and acc2.shape == (2, 2, 64) and lens2.tolist() == [64, 40]
    # what remains attends like the kept tokens alone
    o, _ = fa.cache_forward(q, kept, lens2)
    at = index.clamp(min=0).long()
    picked = fa.PackedCache(*(x.gather(2, at[..., None].expand(2, 2, 64, x.shape[3])).contiguous() for x in cache))
    assert torch.equal(o, fa.cache_forward(q, picked, lens2)[0])


def test_serving_step_with_eviction_captured():
    """Append, attention, weights, eviction and read-out in one captured graph,
    replayed on other lengths and contents: what the eager calls give."""
    B, H, Hkv, C, D = 2, 8, 2, 3000, 64
    q, cache, lens, _, _ = _attention_case((B, H, Hkv, 1, C, [2900, 50], -1, 0), D, "fp16", seed=31)
    k = torch.randn((B, Hkv, 1, D), generator=_gen(6), device="cuda").half()
    zero = torch.zeros_like(lens)

    def step():
        fa.cache_append(cache, k, k, lens)
        n = lens + 1
        o, lse = fa.cache_forward(q, cache, n, window=(2000, 0), sinks=4)
        acc = fa.cache_weights(q, cache, lse, n, window=(2000, 0), sinks=4)
        kept, acc2, n2, index = fa.cache_evict(cache, acc, n, 700, sinks=4, recent=200)
        return (o, lse, acc, acc2, n2, index, *fa.cache_read(kept, zero, 700, count=n2))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for new in ([1500, 2999], [0, 699]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        k.copy_(torch.randn((B, Hkv, 1, D), generator=_gen(new[0]), device="cuda").half())
        graph.replay()
        got = [x.clone() for x in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    _ok()


def test_many_query_rows():
    """A prompt's last 100 tokens: 400 query rows per key head, in row blocks."""
    case = (1, 4, 1, 100, 600, [555], 300, 7)
    for D, dtype in ((64, "fp16"), (128, "bf16")):
        q, cache, lens, left, sinks = _attention_case(case, D, dtype, seed=13)
        o, lse = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks)
        ref = reference(q, cache, lens, left, sinks, D ** -0.5)
        check_attention(q, cache, lens, left, sinks, D ** -0.5, o, lse, ref)
        w = fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks)
        _ok()
        assert abs(float(w.sum()) - 400) <= 400 * 2.0 ** -14   # every query's weights sum to 1
        assert bool(((w.double() - ref[2]).abs() <= 4 * ref[4] + ref[2] * 2.0 ** -14).all())


def test_same_tensor_for_keys_and_values_and_queries_that_are_not_finite():
    q, cache, lens, _, _ = _attention_case((2, 4, 2, 1, 300, [300, 100], -1, 0), 128, "bf16", seed=17)
    want = fa.cache_forward(q, cache, lens)
    bad = q.clone()
    bad[0, 1, 0, 3], bad[1, 2, 0, 0] = math.nan, math.inf
    o, lse = fa.cache_forward(bad, cache, lens)
    _ok()
    hit = torch.zeros((2, 4, 1), dtype=torch.bool, device="cuda")
    hit[0, 1], hit[1, 2] = True, True
    assert bool(torch.isnan(o[hit]).all()) and torch.equal(o[~hit], want[0][~hit]) and torch.equal(lse[~hit], want[1][~hit])
    x = torch.randn((2, 2, 5, 128), device="cuda").bfloat16()
    fa.cache_append(cache, x, x, lens - 5)
    got = fa.cache_read(cache, lens - 5, 5)
    _ok()
    assert torch.equal(got[0], got[1])


# ------------------------------------------------------------------ refusals that need device memory

def test_refusals():
    q, cache, lens, _, _ = _attention_case((2, 4, 2, 1, 100, [100, 50], -1, 0), 64, "bf16", seed=2)
    with pytest.raises(fa.FAError):   # the output over the codes
        fa.cache_forward(q, cache, lens, out=cache.k_codes.view(-1)[:q.numel() * 2].view(torch.bfloat16).view(q.shape))
    with pytest.raises(fa.FAError):   # in place
        fa.cache_evict(cache, torch.zeros((2, 2, 100), device="cuda"), lens, 50, out=cache)
    with pytest.raises(fa.FAError):   # host memory
        fa.cache_forward(q, cache, lens.cpu())
    for bad in (lens.long(), lens.float()):
        with pytest.raises(TypeError):
            fa.cache_forward(q, cache, bad)
    with pytest.raises(ValueError):
        fa.cache_forward(q, cache, lens, window=(5, 1))
    with pytest.raises(ValueError):
        fa.cache_forward(q, cache, lens, sinks=-1)
    with pytest.raises(ValueError):
        fa.cache_forward(q[:, :3].contiguous(), cache, lens)   # three query heads for two key heads
    with pytest.raises(ValueError):
        fa.cache_forward(q.transpose(1, 2).contiguous().transpose(1, 2), cache, lens) if q.shape[2] > 1 else \
            fa.cache_forward(q.expand(2, 4, 2, 64), cache, lens)   # not contiguous
    with pytest.raises(TypeError):
        fa.cache_forward(q.half(), cache, lens)
    with pytest.raises(ValueError):
        fa.cache_evict(cache, torch.zeros((2, 2, 100), device="cuda"), lens, 50, sinks=30, recent=30)
