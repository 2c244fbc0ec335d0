"""Attention over packed sequences (fa_packed_plan, fa_packed_fwd, fa_packed_bwd)
on the GPU, in full against plain float64 attention sequence by sequence.

Tolerances as in tests/test_sink_gpu.py, whose kernels' arithmetic this shares:
scores are fp32 sums of exact products, off by at most delta = 2 D 2^-24 scale
max_j sum_d |q_d k_jd|; P is rounded to the input type for its product and the
result once more (finfo(t).eps / 2 each); fp32 sums and the exponential add 2^-15:
  |O - ref| <= eps/2 |ref| + (eps/2 + 2^-15 + 2 delta) sum_j p_j |v_j|
  |LSE - ref| <= delta + 2^-18 (1 + |ref|)
The backward's gradients: normwise 1.5 u per tensor and per row 12 u of (its
largest element + the gradient's RMS), u = 2^-8 (bf16) or 2^-11 (fp16).  Where a
query sees one key its gradients dQ and dK are exactly 0, the difference of two
fp32 sums of D products that are the same but for their order and the roundings
of their partial sums: |dP - delta| <= e = 2 D 2^-24 sum_d (|dO v| + |dO O|), to
which the bounds add its way into them, scale sum_j p e |k| and scale sum_i p e |q|.
Where a query sees a few keys and one has nearly all the weight, its gradients are
small against what delta = rowsum(dO O) makes of O's own rounding to the type, off by
up to d = eps/2 sum_d |dO O|: dS is off by p d, and a row of dQ by scale sum_j p d |k|, of
dK by scale sum_i p d |q|, which the bounds of single rows add.
"""
from __future__ import annotations

import math

import pytest
import torch

from exact_attention_10_gb300 import fa

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()


def _ok():
    rc = fa.sync_status(torch.cuda.current_stream().cuda_stream)
    assert rc == 0, fa.status_string(rc)


def _cu(lens, front=0):
    cu = [front]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu, torch.tensor(cu, dtype=torch.int32, device="cuda")


def _randn(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def reference(q, k, v, cq, ck, causal, scale, do=None):
    """float64 [T, H, D]: O, LSE [H, T], sum p |v|, delta [H, T] (and dQ, dK, dV and what their bounds add); rows of no
    sequence stay 0."""
    Tq, H, D = q.shape
    G = H // k.shape[1]
    o = torch.zeros((Tq, H, D), dtype=torch.float64, device="cuda")
    pv, dq = torch.zeros_like(o), torch.zeros_like(o)
    lse = torch.zeros((H, Tq), dtype=torch.float64, device="cuda")
    delta = torch.zeros_like(lse)
    dk, dv, fk = (torch.zeros(k.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    fq, gq, gk = torch.zeros_like(o), torch.zeros_like(o), torch.zeros_like(fk)
    half = torch.finfo(q.dtype).eps / 2 if q.dtype != torch.float64 else 0.0
    for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
        if a == b:
            continue
        for h in range(H):
            x, y, z = q[a:b, h].double(), k[c:d, h // G].double(), v[c:d, h // G].double()
            s = scale * x @ y.T
            if causal:
                i = torch.arange(b - a, device="cuda")[:, None] + (d - c) - (b - a)
                s.masked_fill_(torch.arange(d - c, device="cuda")[None] > i, -math.inf)
            l = torch.logsumexp(s, 1) if d > c else torch.full((b - a,), -math.inf, dtype=torch.float64, device="cuda")
            p = torch.exp(s - torch.where(l == -math.inf, 0.0, l)[:, None])
            o[a:b, h], pv[a:b, h], lse[h, a:b] = p @ z, p @ z.abs(), l
            if d > c:
                delta[h, a:b] = 2 * D * 2.0 ** -24 * scale * (x.abs() @ y.abs().T).amax(1)
            if do is not None:
                w = do[a:b, h].double()
                ds = p * (w @ z.T - (w * o[a:b, h]).sum(1, keepdim=True))
                dq[a:b, h] = scale * ds @ y
                dk[c:d, h // G] += scale * ds.T @ x
                dv[c:d, h // G] += p.T @ w
                e = p * (2 * D * 2.0 ** -24) * (w.abs() @ z.abs().T + (w * o[a:b, h]).abs().sum(1, keepdim=True))
                fq[a:b, h] = scale * e @ y.abs()
                fk[c:d, h // G] += scale * e.T @ x.abs()
                e = p * (half * (w * o[a:b, h]).abs().sum(1, keepdim=True))
                gq[a:b, h] = scale * e @ y.abs()
                gk[c:d, h // G] += scale * e.T @ x.abs()
    none = torch.zeros_like(fk)
    return o, lse, pv, delta, dq, dk, dv, fq, fk, none, gq, gk, none


def check_forward(o, lse, ref, dtype):
    r, rl, pv, delta = ref[:4]
    eps = torch.finfo(T[dtype]).eps / 2
    bound = eps * r.abs() + (eps + 2.0 ** -15 + 2 * delta.T[..., None]) * pv
    assert bool(((o.double() - r).abs() <= bound).all())
    hidden = rl == -math.inf
    assert bool((lse[hidden] == -math.inf).all())
    err = (lse.double() - rl).abs()[~hidden]
    assert bool((err <= (delta + 2.0 ** -18 * (1 + rl.abs()))[~hidden]).all())


def check_grads(got, ref, dtype):
    u = U[dtype]
    for name, g, r, f, gr in zip(("dQ", "dK", "dV"), got, ref, ref[3:], ref[6:]):
        g = g.double()
        assert bool(g.isfinite().all()), name
        rms = r.square().mean().sqrt()
        assert float((g - r).norm()) <= 1.5 * u * float(r.norm()) + float(f.norm()), name
        row = 12 * u * (r.abs().amax(-1) + rms) + (f + gr).amax(-1)
        assert bool(((g - r).abs().amax(-1) <= row).all()), name


def batch(lens, klens, H, Hkv, D, dtype, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Tq, Tk = sum(lens), sum(klens)
    t = T[dtype]
    q = (_randn(g, Tq, H, D, dtype=torch.float32) * gain).to(t)
    k, v = _randn(g, Tk, Hkv, D, dtype=t), _randn(g, Tk, Hkv, D, dtype=t)
    return q, k, v, (_randn(g, Tq, H, D, dtype=torch.float32) / gain).to(t)


SHAPES = [
    # lens, klens (None: the same), H, Hkv
    ([1], None, 1, 1),
    ([7, 0, 130], None, 2, 1),
    ([128, 256, 1, 127, 129], None, 4, 2),
    ([300, 1, 511], [300, 40, 700], 2, 2),
    ([5, 200, 3, 0], [0, 77, 3, 50], 3, 1),       # no keys, fewer keys than queries, no queries
    ([700, 2, 385, 64], None, 6, 2),
    ([1] * 40 + [260] + [0] * 3 + [33] * 9, None, 2, 1),
    ([60, 68], [500, 1000], 4, 1),                # at most 128 query tokens in all
    ([1030], [2100], 2, 1),
    # enough tiles for those of 256 rows (the others are of 128)
    ([300] * 20 + [513, 1, 0], None, 12, 4),
    ([200, 290, 129] * 7, [0, 350, 100] * 7, 12, 12),
    # ... and pairs of heads
    ([300] * 20 + [513, 1, 0], None, 16, 4),
    ([200, 290, 129] * 7, [0, 350, 100] * 7, 12, 6),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_forward_and_gradients(shape, causal, dtype, D):
    lens, klens, H, Hkv = SHAPES[shape]
    klens = lens if klens is None else klens
    q, k, v, do = batch(lens, klens, H, Hkv, D, dtype, seed=shape)
    cq, cu = _cu(lens)
    ck, cu_k = _cu(klens)
    plan = fa.packed_plan(cu, q.shape[0], H, Hkv, cu_k=cu_k, tokens_k=k.shape[0], causal=causal, grad=True)
    o, lse = fa.packed_forward(q, k, v, plan)
    _ok()
    ref = reference(q, k, v, cq, ck, causal, D ** -0.5, do)
    check_forward(o, lse, ref, dtype)
    for det in (False, True):
        grads = fa.packed_backward(q, k, v, o, do, lse, plan, deterministic=det)
        _ok()
        check_grads(grads, ref[4:], dtype)


def test_strided_slices_in_and_out():
    """q, k, v as slices of one buffer, the gradients into slices of another; and heads outermost."""
    H, Hkv, D, lens = 4, 2, 128, [100, 270, 31]
    g = torch.Generator(device="cuda").manual_seed(5)
    n = sum(lens)
    qkv = _randn(g, n, H + 2 * Hkv, D, dtype=torch.bfloat16)
    q, k, v = qkv.split([H, Hkv, Hkv], 1)
    cq, cu = _cu(lens)
    plan = fa.packed_plan(cu, n, H, Hkv, causal=True, grad=True)
    out = torch.full((n, H + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.packed_forward(q, k, v, plan, out=out[:, :H])
    do = _randn(g, H, n, D, dtype=torch.bfloat16).transpose(0, 1)
    d = torch.full_like(qkv, 7.0)
    dq, dk, dv = d.split([H, Hkv, Hkv], 1)
    fa.packed_backward(q, k, v, o, do, lse, plan, dq=dq, dk=dk, dv=dv)
    _ok()
    ref = reference(q, k, v, cq, cq, True, D ** -0.5, do)
    check_forward(o, lse, ref, "bf16")
    check_grads((dq, dk, dv), ref[4:], "bf16")
    assert bool((out[:, H] == 7.0).all())
    o2, lse2 = fa.packed_forward(*(x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)), plan)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_outside_and_neighbours_that_are_not_finite(D):
    """Rows of no sequence are neither read nor written, and a sequence of NaN and infinities spoils no other."""
    H, Hkv, lens = 2, 1, [130, 200, 70, 90]
    q, k, v, do = batch([10] + lens + [40], [10] + lens + [40], H, Hkv, D, "bf16", seed=9)
    n = q.shape[0]
    cq, cu = _cu(lens, front=10)
    plan = fa.packed_plan(cu, n, H, Hkv, causal=False, grad=True)
    want = fa.packed_forward(q, k, v, plan)
    wgrad = fa.packed_backward(q, k, v, want[0], do, want[1], plan, deterministic=True)
    _ok()
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[:10] = bad[cq[-1]:] = bad[cq[1]:cq[2]] = True
    for x in (q, k, v, do):
        x[bad] = torch.tensor([math.nan, math.inf, -math.inf, math.nan] * (D // 4), dtype=x.dtype, device="cuda")
    out, lse = torch.full_like(q, 3.0), torch.full((H, n), 3.0, device="cuda")
    fa.packed_forward(q, k, v, plan, out=out, lse=lse)
    got = [torch.full_like(x, 3.0) for x in (q, k, v)]
    fa.packed_backward(q, k, v, out, do, lse, plan, dq=got[0], dk=got[1], dv=got[2], deterministic=True)
    _ok()
    good = ~bad
    assert torch.equal(out[good], want[0][good]) and torch.equal(lse[:, good], want[1][:, good])
    for x, y in zip(got, wgrad):
        assert torch.equal(x[good], y[good])
    outside = bad.clone()
    outside[cq[1]:cq[2]] = False
    for x in (out, lse.T, *got):
        assert bool((x[outside] == 3.0).all())
    if D == 64:   # the single pass, whose order of adds varies
        fused = fa.packed_backward(q, k, v, out, do, lse, plan)
        _ok()
        ref = reference(*(torch.where(bad[:, None, None], torch.zeros_like(x), x) for x in (q, k, v)), cq, cq, False,
                        D ** -0.5, torch.where(bad[:, None, None], torch.zeros_like(do), do))
        check_grads([x[good] for x in fused], [x[good] for x in ref[4:]], "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_key_tiles_in_parts(causal, D):
    """Few key tiles, many query rows to each: their query tiles are cut into parts, whose sums are the same bits every
    time; sequences without queries or keys among them, and gradients into slices."""
    lens, klens, H, Hkv = [2000, 130, 0, 700, 5], [2000, 300, 90, 650, 0], 8, 1
    q, k, v, do = batch(lens, klens, H, Hkv, D, "bf16", seed=31)
    cq, cu = _cu(lens)
    ck, cu_k = _cu(klens)
    plan = fa.packed_plan(cu, q.shape[0], H, Hkv, cu_k=cu_k, tokens_k=k.shape[0], causal=causal, grad=True)
    o, lse = fa.packed_forward(q, k, v, plan)
    kv = torch.full((k.shape[0], 3, D), 5.0, dtype=q.dtype, device="cuda")
    dq, dk, dv = fa.packed_backward(q, k, v, o, do, lse, plan, dk=kv[:, 0:1], dv=kv[:, 2:3])
    _ok()
    check_grads((dq, dk, dv), reference(q, k, v, cq, ck, causal, D ** -0.5, do)[4:], "bf16")
    assert bool((kv[:, 1] == 5.0).all())
    for _ in range(3):
        again = fa.packed_backward(q, k, v, o, do, lse, plan, deterministic=D == 64)
        assert torch.equal(again[1], dk) and torch.equal(again[2], dv)
    _ok()


def test_low_scores_in_a_ragged_tile():
    """All scores of a sequence far below zero: exp(-LSE) overflows, and must not reach dQ from the rows behind its end."""
    D = 64
    for dtype in ("fp16", "bf16"):
        q, k, v, do = batch([70, 90], [70, 90], 1, 1, D, dtype, seed=3)
        q, k = q.abs() + 1, -(k.abs() + 1)
        cq, cu = _cu([70, 90])
        plan = fa.packed_plan(cu, 160, 1, causal=False, grad=True)
        o, lse = fa.packed_forward(q, k, v, plan, scale=0.25)
        grads = fa.packed_backward(q, k, v, o, do, lse, plan, scale=0.25)
        _ok()
        ref = reference(q, k, v, cq, cq, False, 0.25, do)
        assert float(ref[1].max()) < -20
        check_forward(o, lse, ref, dtype)
        # Keys with a common part, which cancels in dQ = scale sum_j dS_j k_j but for the
        # errors of dS: element by element, dS is off by its rounding to the type, eps/2
        # |dS|, by p (eps/2 sum_d |dO O|) through the rounded O in delta, by the 2^-15 + 2
        # delta of p and by the fp32 sums' p e; P by its rounding and 2^-15 + 2 delta; the
        # result by eps/2 once more; each of the three roundings to the type also by half a
        # step of its subnormals (weights reach down to exp(-40) here).
        eps = torch.finfo(T[dtype]).eps / 2
        sub = torch.finfo(T[dtype]).smallest_normal * eps
        want = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v)]
        for a, b in zip(cq, cq[1:]):
            x, y, z, w = (t[a:b, 0].double() for t in (q, k, v, do))
            p = torch.exp(0.25 * x @ y.T - ref[1][0, a:b, None])
            dp, wo = w @ z.T, w * ref[0][a:b, 0]
            ds = p * (dp - wo.sum(1, keepdim=True))
            rel = 2.0 ** -15 + 2 * ref[3][0, a:b, None]
            e = (eps + rel) * ds.abs() + p * (eps * wo.abs().sum(1, keepdim=True) + 2 * D * 2.0 ** -24 * (
                w.abs() @ z.abs().T + wo.abs().sum(1, keepdim=True)))
            want[0][a:b, 0] = 0.25 * (e + sub) @ y.abs()
            want[1][a:b, 0] = 0.25 * (e + sub).T @ x.abs()
            want[2][a:b, 0] = (p * (eps + rel) + sub).T @ w.abs()
        for g, r, bound in zip(grads, ref[4:], want):
            assert bool(((g.double() - r).abs() <= (1 + eps) * bound + eps * r.abs() + sub).all())


def test_bounds_that_are_no_sequences():
    """Boundaries outside the tensors or falling are clamped: the sequences stay apart and inside."""
    H, D, n = 2, 64, 300
    q, k, v, _ = batch([n], [n], H, H, D, "bf16", seed=4)
    for cu, same in (([-5, 100, 50, 1000], [0, 100, 100, 300]), ([200, 100, 300, 300], [200, 200, 300, 300])):
        a = fa.packed_plan(torch.tensor(cu, dtype=torch.int32, device="cuda"), n, H, causal=True)
        b = fa.packed_plan(torch.tensor(same, dtype=torch.int32, device="cuda"), n, H, causal=True)
        out = [torch.zeros_like(q) for _ in range(2)]
        fa.packed_forward(q, k, v, a, out=out[0])
        fa.packed_forward(q, k, v, b, out=out[1])
        _ok()
        assert torch.equal(*out)


def test_one_sequence_is_the_unpacked_call():
    """One sequence, heads outermost: the tensors of forward, near the same sums."""
    H, N, D = 2, 700, 128
    q, k, v, do = batch([N], [N], H, H, D, "bf16", seed=8)
    plan = fa.packed_plan(torch.tensor([0, N], dtype=torch.int32, device="cuda"), N, H, causal=True, grad=True)
    o, lse = fa.packed_forward(q, k, v, plan)
    a, b = (x.transpose(0, 1).unsqueeze(0).contiguous() for x in (o, do))
    qq, kk, vv = (x.transpose(0, 1).unsqueeze(0).contiguous() for x in (q, k, v))
    oo, ll = fa.forward(qq, kk, vv, causal=True)
    _ok()
    assert torch.equal(a, oo) and torch.equal(lse[None], ll)
    for x, y in zip(fa.packed_backward(q, k, v, o, do, lse, plan), fa.backward(qq, kk, vv, oo, b, ll, causal=True)):
        assert torch.equal(x.transpose(0, 1)[None], y)


def test_another_stream_and_a_captured_graph():
    """Plan, forward and backward captured; replays follow the lengths and tensors."""
    H, Hkv, D, n = 4, 2, 128, 600
    q, k, v, do = batch([n], [n], H, Hkv, D, "bf16", seed=11)
    _, cu = _cu([100, 400, 100])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan = fa.packed_plan(cu, n, H, Hkv, causal=True, grad=True)
        fa.packed_backward(q, k, v, *fa.packed_forward(q, k, v, plan)[:1], do, fa.packed_forward(q, k, v, plan)[1], plan)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = fa.packed_plan(cu, n, H, Hkv, causal=True, grad=True)
        o, lse = fa.packed_forward(q, k, v, plan)
        grads = fa.packed_backward(q, k, v, o, do, lse, plan)
    for lens in ([100, 400, 100], [1, 2, 597], [0, 600, 0]):
        cq, new = _cu(lens)
        cu.copy_(new)
        q.mul_(0.75)
        graph.replay()
        _ok()
        ref = reference(q, k, v, cq, cq, True, D ** -0.5, do)
        check_forward(o, lse, ref, "bf16")
        check_grads(grads, ref[4:], "bf16")


def test_a_stream_of_its_own():
    """Plan, forward and backward on a stream given by the call, while the current one does something else."""
    lens, H, Hkv, D = [300, 41], 4, 2, 64
    q, k, v, do = batch(lens, lens, H, Hkv, D, "fp16", seed=15)
    cq, cu = _cu(lens)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    plan = fa.packed_plan(cu, sum(lens), H, Hkv, causal=True, grad=True, stream=st)
    o, lse = fa.packed_forward(q, k, v, plan, stream=st)
    junk = [torch.full((1 << 20,), 9.0, device="cuda") for _ in range(4)]   # (must not get the results' memory)
    grads = fa.packed_backward(q, k, v, o, do, lse, plan, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    _ok()
    ref = reference(q, k, v, cq, cq, True, D ** -0.5, do)
    check_forward(o, lse, ref, "fp16")
    check_grads(grads, ref[4:], "fp16")
    assert all(bool((x == 9.0).all()) for x in junk)


def test_gradient_against_differences():
    """The directional derivative of sum(O dO) in float64 arithmetic, against the kernel's gradients."""
    H, Hkv, D, lens = 2, 1, 64, [40, 150]
    q, k, v, do = batch(lens, lens, H, Hkv, D, "fp16", seed=21)
    cq, cu = _cu(lens)
    plan = fa.packed_plan(cu, sum(lens), H, Hkv, causal=True, grad=True)
    o, lse = fa.packed_forward(q, k, v, plan)
    grads = fa.packed_backward(q, k, v, o, do, lse, plan)
    _ok()
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(3):
        x = [q.double(), k.double(), v.double()]
        dx = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h, f = 1e-4, []
        for sgn in (1, -1):
            y = list(x)
            y[i] = x[i] + sgn * h * dx
            f.append(float((reference(*y, cq, cq, True, D ** -0.5)[0] * do.double()).sum()))
        want = (f[0] - f[1]) / (2 * h)
        got = float((grads[i].double() * dx).sum())
        # each element of the gradient is off by at most 12 u (row maximum + RMS) (as above), along dx at random
        r = grads[i].double()
        row = 12 * U["fp16"] * (r.abs().amax(-1, keepdim=True) + r.square().mean().sqrt())
        assert abs(got - want) <= float((row * dx.abs()).sum())
