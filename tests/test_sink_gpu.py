"""Causal windows with sinks and shared key heads (fa_fwd_sink, fa_bwd_sink)
on the GPU, in full against plain float64 attention.

Forward tolerance, from the arithmetic: the scores are fp32 sums of exact
products, off by at most delta = 2 D 2^-24 scale max_j sum_d |q_d k_jd|; the
probabilities are rounded to the input type for the product with V and the
result once more (finfo(t).eps / 2 each); sums over n keys in fp32 and the
exponential add 2^-15.  So per element
  |O - ref| <= eps/2 |ref| + (eps/2 + 2^-15 + 2 delta) sum_j p_j |v_j|
and |LSE - ref| <= delta + 2^-18 (1 + |ref|).
The backward's bounds are those of tests/test_bwd_gpu.py: normwise 1.5 u and
per row 12 u of (its largest element + the gradient's RMS), u = 2^-8 (bf16) or
2^-11 (fp16); shared heads sum exact fp32 products and add no rounding.
"""
from __future__ import annotations

import math

import pytest
import torch

from exact_attention_10_gb300 import fa
from exact_attention_10_gb300.inputs import make_custom

pytestmark = pytest.mark.gpu
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()


def _ok():
    rc = fa.sync_status(torch.cuda.current_stream().cuda_stream)
    assert rc == 0, fa.status_string(rc)


def _inputs(B, H, Hkv, Nq, Nkv, D, dtype, seed, gain=1.0):
    q, do, _ = make_custom(B, H, Nq, D, dtype, seed=seed, qk_gain=gain)
    _, k, v = make_custom(B, Hkv, Nkv, D, dtype, seed=seed + 1)
    return q.cuda(), k.cuda(), v.cuda(), (do / gain).cuda()


def visible(Nq, Nkv, left, sinks):
    pos = torch.arange(Nq, device="cuda")[:, None] + (Nkv - Nq)
    j = torch.arange(Nkv, device="cuda")[None]
    vis = j <= pos
    if left >= 0:
        vis &= (j >= pos - left) | (j < sinks)
    return vis


def reference(q, k, v, left, sinks, scale, do=None):
    """float64: O, LSE, sum p |v|, delta and, with do, (dQ, dK, dV) of this O."""
    B, H, Nq, D = q.shape
    G = H // k.shape[1]
    vis = visible(Nq, k.shape[2], left, sinks)
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    pv = torch.zeros_like(o)
    lse = torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    delta = torch.zeros_like(lse)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(k.shape, dtype=torch.float64, device="cuda"), None
    dv = torch.zeros_like(dk)
    for b in range(B):
        for h in range(H):
            x, y, z = q[b, h].double(), k[b, h // G].double(), v[b, h // G].double()
            s = torch.where(vis, (x @ y.T) * scale, -math.inf)
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(torch.isinf(lse[b, h]), 0.0, lse[b, h])[:, None])
            o[b, h] = p @ z
            pv[b, h] = p @ z.abs()
            mag = torch.where(vis, (x.abs() @ y.abs().T) * scale, torch.zeros((), dtype=torch.float64, device="cuda"))
            delta[b, h] = 2 * D * 2.0 ** -24 * mag.amax(-1)
            if do is not None:
                g = do[b, h].double()
                ds = p * (g @ z.T - (g * o[b, h]).sum(-1, keepdim=True))
                dq[b, h] = scale * (ds @ y)
                dk[b, h // G] += scale * (ds.T @ x)
                dv[b, h // G] += p.T @ g
    return o, lse, pv, delta, (dq, dk, dv)


def check_forward(o, lse, ref, dtype, label):
    o_ref, lse_ref, pv, delta, _ = ref
    eps2 = torch.finfo(o.dtype).eps / 2
    empty = torch.isneginf(lse_ref)
    assert torch.equal(torch.isneginf(lse), empty), label
    assert bool((o[empty] == 0).all()), label
    tol = eps2 * o_ref.abs() + (eps2 + 2.0 ** -15 + 2 * delta[..., None]) * pv + 1e-7
    err = (o.double() - o_ref).abs()
    assert bool((err <= tol).all()), (label, float((err / tol).max()))
    ltol = delta + 2.0 ** -18 * (1 + lse_ref.abs())
    lerr = (lse.double() - lse_ref).abs()
    assert bool((lerr[~empty] <= ltol[~empty]).all()), (label, float((lerr / ltol)[~empty].max()))


def check_grads(grads, refs, dtype, label):
    u = U[dtype]
    rms_all = math.sqrt(float(torch.cat([r.flatten() for r in refs]).square().mean()))
    for name, g, ref in zip(("dQ", "dK", "dV"), grads, refs):
        g = g.double()
        assert bool(torch.isfinite(g).all()), (label, name)
        rms = math.sqrt(float(ref.square().mean())) or rms_all
        norm = float((g - ref).norm()) / (float(ref.norm()) or rms * math.sqrt(ref.numel()))
        row = ((g - ref).abs().amax(-1) / (ref.abs().amax(-1) + rms)).max()
        print(f"{label} {name}: normwise {norm / u:.2f}u worst row {float(row) / u:.2f}u")
        assert norm <= 1.5 * u and float(row) <= 12 * u, (label, name, norm / u, float(row) / u)


CASES = [  # (B, H, Hkv, Nq, Nkv, left, sinks)
    (1, 1, 1, 1, 1, 0, 1),
    (1, 2, 1, 2, 2, 0, 0),
    (2, 4, 2, 300, 300, 127, 4),          # shared heads, ragged
    (1, 3, 3, 1000, 1000, 200, 1),
    (1, 4, 1, 777, 777, 0, 5),            # the diagonal and the sinks alone
    (1, 2, 2, 1000, 1000, 255, 128),      # sinks fill a key tile
    (1, 2, 1, 1000, 1000, 100, 300),      # sinks over three key tiles
    (1, 2, 1, 900, 900, 64, 5000),        # every key is a sink: plain causal
    (1, 4, 2, 900, 900, -1, 7),           # no window: plain causal
    (1, 2, 1, 600, 600, 5000, 7),         # a window that cannot bind
    (2, 6, 2, 64, 1500, 300, 10),         # the last queries of a longer sequence
    (1, 4, 2, 300, 120, 30, 3),           # more queries than keys: the first see nothing
    (1, 8, 8, 1, 3001, 500, 4),           # one query
    (1, 4, 4, 129, 129, 1, 130),
]


@pytest.mark.parametrize("schedule", ["auto", "whole_tiles", "balanced"])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (64, "fp16"), (128, "fp16")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward(case, D, dtype, schedule):
    B, H, Hkv, Nq, Nkv, left, sinks = case
    q, k, v, _ = _inputs(B, H, Hkv, Nq, Nkv, D, dtype, seed=Nq + Nkv + left)
    o, lse = fa.forward(q, k, v, window=(left, 0), sinks=sinks, schedule=schedule)
    _ok()
    check_forward(o, lse, reference(q, k, v, left, sinks, D ** -0.5), dtype, f"{case} {D} {dtype} {schedule}")


@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "bf16"), (64, "fp16"), (128, "fp16")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward(case, D, dtype, deterministic):
    B, H, Hkv, Nq, Nkv, left, sinks = case
    q, k, v, do = _inputs(B, H, Hkv, Nq, Nkv, D, dtype, seed=Nq + Nkv + left)
    o, lse = fa.forward(q, k, v, window=(left, 0), sinks=sinks)
    grads = fa.backward(q, k, v, o, do, lse, window=(left, 0), sinks=sinks, deterministic=deterministic)
    _ok()
    ref = reference(q, k, v, left, sinks, D ** -0.5, do)
    check_grads(grads, ref[4], dtype, f"{case} {D} {dtype}")
    again = fa.backward(q, k, v, o, do, lse, window=(left, 0), sinks=sinks, deterministic=deterministic)
    _ok()
    for i, (a, b) in enumerate(zip(grads, again)):
        if i or deterministic or D == 128:
            assert torch.equal(a, b)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("B,H,Hkv,N,left,sinks", [(1, 4, 1, 5000, 255, 4), (2, 8, 4, 2500, 511, 20), (1, 2, 2, 9000, 63, 200),
                                                  (3, 24, 8, 1300, 300, 2)])
def test_long(B, H, Hkv, N, left, sinks, D, dtype):
    """Sink tiles cut into many parts, several tiles per CTA, split forward tiles."""
    q, k, v, do = _inputs(B, H, Hkv, N, N, D, dtype, seed=N)
    o, lse = fa.forward(q, k, v, window=(left, 0), sinks=sinks)
    grads = fa.backward(q, k, v, o, do, lse, window=(left, 0), sinks=sinks)
    _ok()
    ref = reference(q, k, v, left, sinks, D ** -0.5, do)
    check_forward(o, lse, ref, dtype, f"N={N} D={D}")
    check_grads(grads, ref[4], dtype, f"N={N} D={D}")


@pytest.mark.parametrize("D", [64, 128])
def test_large_scores(D):
    q, k, v, _ = _inputs(1, 4, 2, 700, 700, D, "fp16", seed=3, gain=4.0)
    o, lse = fa.forward(q, k, v, window=(150, 0), sinks=9)
    _ok()
    check_forward(o, lse, reference(q, k, v, 150, 9, D ** -0.5), "fp16", "gain 4")


@pytest.mark.parametrize("D", [64, 128])
def test_agrees_with_the_band(D):
    """No sinks and a head of its own for each query head: fa_fwd_band's mask
    and, tile for tile, its arithmetic."""
    q, k, v, do = _inputs(1, 4, 4, 1500, 1500, D, "bf16", seed=D)
    want = fa.forward(q, k, v, window=(300, 0), schedule="whole_tiles")
    got = fa.forward(q, k, v, window=(300, 0), sinks=0, schedule="whole_tiles")
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    a = fa.backward(q, k, v, *want[:1], do, want[1], window=(300, 0), deterministic=True)
    b = fa.backward(q, k, v, *want[:1], do, want[1], window=(300, 0), sinks=0, deterministic=True)
    _ok()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_gradient_against_differences():
    """dQ, dK, dV along a direction, against the change of sum(O dO) computed
    in float64 (the definition) around the same point."""
    for D, Hkv in ((64, 1), (128, 2)):
        q, k, v, do = _inputs(1, 4, Hkv, 200, 200, D, "bf16", seed=7)
        o, lse = fa.forward(q, k, v, window=(40, 0), sinks=3)
        grads = fa.backward(q, k, v, o, do, lse, window=(40, 0), sinks=3)
        _ok()
        for i, x in enumerate((q, k, v)):
            d = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                            dtype=torch.float64)
            h = 1e-4

            def f(e):
                y = [t.double() for t in (q, k, v)]
                y[i] = y[i] + e * d
                return float((reference(*y, 40, 3, D ** -0.5)[0] * do.double()).sum())
            diff = (f(h) - f(-h)) / (2 * h)
            got = float((grads[i].double() * d).sum())
            # the gradient's own error, u per element at most 1.5 normwise, along d
            tol = 1.5 * U["bf16"] * float(grads[i].double().norm()) * 6 + 1e-4 * abs(diff)
            assert abs(got - diff) <= tol, (i, got, diff, tol)


@pytest.mark.parametrize("D", [64, 128])
def test_hidden_keys_may_hold_anything(D):
    """NaN and infinities in keys and values that lie in no visited tile leave
    every result as it was."""
    N, left, sinks = 1200, 63, 4
    q, k, v, do = _inputs(1, 2, 1, 100, N, D, "bf16", seed=5)
    dirty_k, dirty_v = k.clone(), v.clone()
    dirty_k[:, :, 128:896] = math.nan    # tiles between the sinks' and the windows' (queries sit at 1100 ..)
    dirty_v[:, :, 128:896] = math.inf
    want = fa.forward(q, k, v, window=(left, 0), sinks=sinks)
    got = fa.forward(q, dirty_k, dirty_v, window=(left, 0), sinks=sinks)
    a = fa.backward(q, k, v, want[0], do, want[1], window=(left, 0), sinks=sinks, deterministic=True)
    b = fa.backward(q, dirty_k, dirty_v, want[0], do, want[1], window=(left, 0), sinks=sinks, deterministic=True)
    _ok()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and torch.equal(a[0], b[0])
    assert torch.equal(a[1][:, :, :128], b[1][:, :, :128]) and torch.equal(a[1][:, :, 1024:], b[1][:, :, 1024:])


@pytest.mark.parametrize("schedule", ["whole_tiles", "balanced"])
@pytest.mark.parametrize("D", [64, 128])
def test_keys_that_are_not_finite_reach_only_their_queries(D, schedule):
    """Keys of visited tiles -- one next to the sinks, two in the windows -- that
    hold NaN or infinities: the rows that do not see them keep every bit."""
    N, left, sinks = 1200, 200, 4
    q, k, v, _ = _inputs(1, 4, 2, N, N, D, "bf16", seed=6)
    dirty = k.clone()
    rows = torch.arange(N, device="cuda")
    blind = torch.ones(N, dtype=torch.bool, device="cuda")
    for j, x in ((10, math.nan), (500, math.inf), (900, -math.inf)):
        dirty[:, :, j] = x
        blind &= ~((rows >= j) & (rows - left <= j))
    want = fa.forward(q, k, v, window=(left, 0), sinks=sinks, schedule=schedule)
    got = fa.forward(q, dirty, v, window=(left, 0), sinks=sinks, schedule=schedule)
    _ok()
    assert int(blind.sum()) == N - 3 * (left + 1)
    assert torch.equal(want[0][:, :, blind], got[0][:, :, blind])
    assert torch.equal(want[1][:, :, blind], got[1][:, :, blind])


def test_graphs_and_streams():
    """Captured forward and backward, two graphs replayed at once on two
    streams while eager calls run on a third: the same bits."""
    sets = [_inputs(1, 4, 2, 16, 6000, 128, "bf16", seed=i) for i in range(3)]

    def run(q, k, v, do):
        o, lse = fa.forward(q, k, v, window=(2000, 0), sinks=4, schedule="balanced")
        return (o, lse, *fa.backward(q, k, v, o, do, lse, window=(2000, 0), sinks=4, deterministic=True))

    wants = [run(*s) for s in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    eager = []
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager.append(run(*sets[2]))
    torch.cuda.synchronize()
    _ok()
    for got, want in zip(outs + eager, wants[:2] + [wants[2]] * 10):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_prompt_to_cache_to_eviction():
    """The operators as a serving loop uses them: a prompt through the window
    with sinks, its tokens packed, decoded tokens appended and attended with
    the same mask, weights gathered, the cache cut to its budget, decoding on."""
    B, H, Hkv, N, D, left, sinks, C = 2, 8, 2, 700, 64, 255, 4, 1024
    q, k, v, _ = _inputs(B, H, Hkv, N + 8, N + 8, D, "bf16", seed=1)
    prompt = [x[:, :, :N].contiguous() for x in (q, k, v)]
    fa.forward(*prompt, window=(left, 0), sinks=sinks)
    cache = fa.cache_empty(B, Hkv, C, D)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, prompt[1], prompt[2], lens)
    lens += N
    acc = torch.zeros((B, Hkv, C), device="cuda")
    start = torch.zeros_like(lens)
    for i in range(N, N + 8):
        one = [x[:, :, i:i + 1].contiguous() for x in (q, k, v)]
        fa.cache_append(cache, one[1], one[2], lens)
        lens += 1
        o, lse = fa.cache_forward(one[0], cache, lens, window=(left, 0), sinks=sinks)
        fa.cache_weights(one[0], cache, lse, lens, window=(left, 0), sinks=sinks, acc=acc)
        # the same step in float64 on the values that the cache stands for
        kk, vv = fa.cache_read(cache, start, i + 1)
        ref = reference(one[0], kk, vv, left, sinks, D ** -0.5)
        # (the read-out rounds each value once more: u relative to it, on top of the result's own)
        scores = 2.0 ** -8 * (one[0].double().abs() @ kk.double().abs().repeat_interleave(H // Hkv, 1).transpose(-1, -2)).amax(-1) * D ** -0.5
        tol = 2.0 ** -8 * ref[0].abs() + (2.0 ** -8 + 2.0 ** -14 + 2 * scores[..., None]) * ref[2]
        assert bool(((o.double() - ref[0]).abs() <= tol).all())
    _ok()
    rows = H // Hkv * 8
    total = acc.sum(-1)
    assert bool(((total - rows).abs() <= rows * 2.0 ** -14).all())   # each query's weights sum to 1
    seen = acc > 0
    assert bool(seen[:, :, :sinks].all()) and not bool(seen[:, :, sinks:N - left].any())
    kept, acc, lens, index = fa.cache_evict(cache, acc, lens, 200, sinks=sinks, recent=64)
    assert lens.tolist() == [200, 200] and bool((index[:, :, 1:] > index[:, :, :-1]).all())
    o, lse = fa.cache_forward(one[0], kept, lens)
    _ok()
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())


def test_refusals():
    q, k, v, do = _inputs(1, 4, 2, 100, 100, 64, "bf16", seed=2)
    o, lse = fa.forward(q, k, v, window=(10, 0), sinks=1)
    for bad in (dict(window=(10, 1), sinks=1), dict(window=(10, 0), sinks=-1), dict(window=(10, 0), sinks=1, schedule="x")):
        with pytest.raises(ValueError):
            fa.forward(q, k, v, **bad)
    with pytest.raises(ValueError):
        fa.forward(q[:, :3].contiguous(), k, v, window=(10, 0), sinks=1)
    with pytest.raises(ValueError):
        fa.forward(q.transpose(1, 2), k, v, window=(10, 0), sinks=1)
    with pytest.raises(TypeError):
        fa.forward(q, k.half(), v.half(), window=(10, 0), sinks=1)
    with pytest.raises(fa.FAError):
        fa.forward(q, k, v, window=(10, 0), sinks=1, out=q)
    with pytest.raises(fa.FAError):
        fa.backward(q, k, v, o, do, lse, window=(10, 0), sinks=1, dk=v)
    with pytest.raises(fa.FAError):
        fa.forward(q, k, v, window=(10, 0), sinks=1, scale=-1.0)
    lib = fa.load()
    ws = torch.empty(64, dtype=torch.uint8, device="cuda")   # too small a workspace
    rc = lib.fa_bwd_sink(*(x.data_ptr() for x in (q, k, v, o, do, lse)), *(torch.empty_like(x).data_ptr() for x in (q, k, v)),
                         1, 4, 2, 100, 100, 64, 10, 1, 0.125, 0, 0, ws.data_ptr(), 64, None)
    assert rc == 1
