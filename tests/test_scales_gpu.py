"""The operators on windows with sinks and on the 4-bit cache at softmax scales
other than D**-0.5, and the weights' accuracy by itself.

Tolerances: those of tests/test_sink_gpu.py and tests/test_cache_gpu.py, whose
score bounds grow with the scale; the gradients' and the weights' own below.
"""
from __future__ import annotations

import math

import pytest
import torch

from exact_attention_10_gb300 import fa
from test_cache_gpu import T, _attention_case, _gen, _ok, check_attention, unpack64
from test_cache_gpu import reference as cache_reference
from test_sink_gpu import U, _inputs, check_forward, visible
from test_sink_gpu import reference as sink_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()


# a sink tile in one part (few sinks, as long as the share of a CTA) and in several, tiles of one and of two Q tiles
WINDOWS = [(2, 4, 2, 300, 300, 127, 4), (1, 4, 1, 2500, 2500, 200, 20), (1, 8, 4, 64, 1500, 300, 10)]


@pytest.mark.parametrize("scale", [0.07, 0.3])
@pytest.mark.parametrize("schedule", ["whole_tiles", "balanced"])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_window_forward(case, D, dtype, schedule, scale):
    B, H, Hkv, Nq, Nkv, left, sinks = case
    q, k, v, _ = _inputs(B, H, Hkv, Nq, Nkv, D, dtype, seed=Nq)
    o, lse = fa.forward(q, k, v, window=(left, 0), sinks=sinks, scale=scale, schedule=schedule)
    _ok()
    check_forward(o, lse, sink_reference(q, k, v, left, sinks, scale), dtype, f"{case} {D} {scale}")


def _gradient_bounds(q, k, v, do, left, sinks, scale, u):
    """Bounds on the errors of (dQ, dK, dV), element by element, from the arithmetic:

    * P_ij = exp(x_ij - LSE_i) is off by E_i relatively: delta_i from the scores
      (tests/test_sink_gpu.py), as much and 2^-18 (1 + |LSE_i|) from the LSE,
      2^-15 from the exponential; in dV's product it is rounded besides: u.
    * dS_ij = P_ij (dP_ij - Delta_i): dP is an fp32 sum of D exact products, off
      by 2 D 2^-24 sum |do v|; Delta_i = sum do o takes the O that was rounded
      to the input type, u of each term, and is an fp32 sum too.  So
        |d dS| <= P (E |dP - Delta| + 2 D 2^-24 sum |do v| + (u + 2 D 2^-24) sum |do o|),
      and its own rounding u (|dS| + that).  (Where one key has nearly all of a
      row's weight, dP and Delta nearly cancel and the term of O's rounding is
      all that is left of dS: the larger the scale, the more such rows.)
    * the sums over keys or queries run in fp32: 2^-15 of their magnitudes; the
      result is rounded: u.
    * Roundings to 16 bits below the type's normal range are half of its least
      step instead (`least`), of P, of dS and of the result.
    """
    least = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2
    B, H, Nq, D = q.shape
    G = H // k.shape[1]
    o, lse, _, delta, grads = sink_reference(q, k, v, left, sinks, scale, do)
    vis = visible(Nq, k.shape[2], left, sinks)
    bq, bk, bv = (torch.zeros_like(g) for g in grads)
    for b in range(B):
        for h in range(H):
            x, y, z, g = (t.double() for t in (q[b, h], k[b, h // G], v[b, h // G], do[b, h]))
            seen = torch.where(torch.isinf(lse[b, h]), 0.0, lse[b, h])
            p = torch.exp(torch.where(vis, (x @ y.T) * scale, -math.inf) - seen[:, None])
            e = (2 * delta[b, h] + 2.0 ** -18 * (1 + seen.abs()) + 2.0 ** -15)[:, None]
            mag = (g * o[b, h]).abs().sum(-1, keepdim=True)
            diff = g @ z.T - (g * o[b, h]).sum(-1, keepdim=True)
            ds = p * (e * diff.abs() + 2 * D * 2.0 ** -24 * (g.abs() @ z.abs().T) + (u + 2 * D * 2.0 ** -24) * mag)
            ds = ds * (1 + u) + (u + 2.0 ** -15) * (p * diff).abs() + least * vis
            bq[b, h] = scale * (ds @ y.abs())
            bk[b, h // G] += scale * (ds.T @ x.abs())
            bv[b, h // G] += (p * (e + u + 2.0 ** -15) + least * vis).T @ g.abs()
    return grads, [bound * (1 + u) + u * g.abs() + least for bound, g in zip((bq, bk, bv), grads)]


@pytest.mark.parametrize("scale", [0.07, 0.3])
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (64, "bf16"), (128, "bf16")])
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_window_backward(case, D, dtype, deterministic, scale):
    B, H, Hkv, Nq, Nkv, left, sinks = case
    q, k, v, do = _inputs(B, H, Hkv, Nq, Nkv, D, dtype, seed=Nq)
    o, lse = fa.forward(q, k, v, window=(left, 0), sinks=sinks, scale=scale)
    got = fa.backward(q, k, v, o, do, lse, window=(left, 0), sinks=sinks, scale=scale, deterministic=deterministic)
    _ok()
    refs, bounds = _gradient_bounds(q, k, v, do, left, sinks, scale, U[dtype])
    for name, g, ref, bound in zip(("dQ", "dK", "dV"), got, refs, bounds):
        err = (g.double() - ref).abs()
        norm = float(err.norm() / ref.norm())
        print(f"{name}: normwise {norm / U[dtype]:.2f}u, of the bound {float((err / bound).max()):.2f}")
        assert bool((err <= bound).all()), name
        assert norm <= 1.5 * U[dtype], name


CACHES = [(2, 8, 2, 1, 2000, [1500, 130], 64, 70), (2, 9, 1, 1, 300, [300, 257], -1, 0), (1, 8, 1, 5, 1000, [937], -1, 0),
          (2, 4, 2, 1, 5000, [5000, 17], -1, 0)]   # up to 8, 16 and 64 rows per key head; tiles cut between CTAs


@pytest.mark.parametrize("scale", [0.07, 0.3])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("case", CACHES, ids=lambda c: "-".join(map(str, c[:5])))
def test_cache_attention_and_weights(case, D, dtype, scale):
    q, cache, lens, left, sinks = _attention_case(case, D, dtype, seed=4)
    o, lse = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks, scale=scale)
    ref = cache_reference(q, cache, lens, left, sinks, scale)
    check_attention(q, cache, lens, left, sinks, scale, o, lse, ref)
    w = fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks, scale=scale)
    _ok()
    rows = q.shape[1] // cache.k_codes.shape[1] * q.shape[2]
    C = cache.k_codes.shape[2]
    tol = 2 * ref[4] + ref[2] * (rows + 8) * 2.0 ** -23 + ref[2] * (C / 8 + 64) * 2.0 ** -23
    assert bool(((w.double() - ref[2]).abs() <= tol).all())


@pytest.mark.parametrize("schedule", ["whole_tiles", "balanced"])
@pytest.mark.parametrize("D", [64, 128])
def test_window_output_that_is_only_16_byte_aligned(D, schedule):
    """An O that starts in the middle of a 32-byte sector is stored 16 bytes at
    a time: the same bits, and nothing beside it touched."""
    q, k, v, _ = _inputs(2, 4, 2, 333, 333, D, "bf16", seed=8)
    want = fa.forward(q, k, v, window=(100, 0), sinks=4, schedule=schedule)
    room = torch.full((q.numel() + 32,), 7.0, dtype=q.dtype, device="cuda")
    assert room.data_ptr() % 32 == 0
    out = room[8:8 + q.numel()].view(q.shape)
    assert out.data_ptr() % 32 == 16 and out.is_contiguous()
    got = fa.forward(q, k, v, window=(100, 0), sinks=4, schedule=schedule, out=out)
    _ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((room[:8] == 7).all()) and bool((room[8 + q.numel():] == 7).all())


# ------------------------------------------------------------------ the weights' accuracy

def _weights64(q, cache, lse, lens, scale):
    """sum exp(scale q.k - lse) in float64 for exactly this lse, and the scores'
    largest magnitude over the rows that weigh at a token."""
    B, H, Nq, D = q.shape
    Hkv, C = cache.k_codes.shape[1:3]
    w = torch.zeros((B, Hkv, C), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            k = unpack64(cache.k_codes[b, h, :n], cache.k_params[b, h, :n])
            x = q.view(B, Hkv, -1, Nq, D)[b, h].double() @ k.T * scale
            pos = n - Nq + torch.arange(Nq, device="cuda")
            x = x.masked_fill(torch.arange(n, device="cuda") > pos[:, None], -math.inf)
            w[b, h, :n] = torch.exp(x - lse.view(B, Hkv, -1, Nq)[b, h, ..., None].double()).sum((0, 1))
    return w


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (64, "bf16"), (128, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("H,Nq", [(8, 1), (4, 4), (8, 8)])   # 8 and 16 rows (mma.sync), 64 (tcgen05)
def test_weights_against_their_own_lse(H, Nq, D, dtype):
    """The relative error over all tokens (2-norm), with float64 fed the very
    LSE that the kernel gets, so that nothing but the weights' own arithmetic is
    in it.

    A weight is exp(x - LSE) with x of a few units here.  Its relative error is
    that of the exponent.  The product of D centred codes ((code - 7.5) 2^-9,
    against a row of q scaled to 2^14) is summed in fp32 with partial sums no
    larger than the scores, up to about 8, in a dozen roundings of 2^-24 of
    them, and the constants, the last sums and 2^x add 2^-23 or so: independent
    of one another, sqrt(12) 8 2^-24 / sqrt(3) + 2^-23 = 1.1e-6 at the very
    most, 3e-7 where the partial sums are of one or two units.  The bound is
    6e-7, twice the latter; codes from 0 on, whose partial sums are several
    times the scores, gave 1.1e-6."""
    B, Hkv, C = 2, 1, 6000
    q, cache, _, _, _ = _attention_case((B, H, Hkv, Nq, C, [C, C - 777], -1, 0), D, dtype, seed=40)
    lens = torch.tensor([C, C - 777], dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    _, lse = fa.cache_forward(q, cache, lens, scale=scale)
    w = fa.cache_weights(q, cache, lse, lens, scale=scale).double()
    _ok()
    ref = _weights64(q, cache, lse, lens, scale)
    err = float((w - ref).norm() / ref.norm())
    print(f"H={H} Nq={Nq} D={D} {dtype}: {err:.2e}, LSE up to {float(lse.abs().max()):.1f}")
    assert err <= 6e-7, err


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H", [1, 20])   # mma.sync; tcgen05, with one row of the twenty that weighs anything
def test_weights_of_a_row_add_up(H, dtype):
    """What the LSE's rounding to log2 units leaves out scales all weights of a
    row alike; it must not.  Over a row's tokens the roundings of single weights
    average out, so the row's sum shows it.

    The LSEs fed are the true ones + 6, about 16: in log2 units between 16 and
    32, where fp32 holds them to 2^-20 (relative to a weight ln 2 / 2^20 = 6.6e-7
    at most, 3.8e-7 rms).  What remains beside it: log2(e) in fp32, 1.3e-8 of a
    score of up to 8 units, 1e-7; and 2^x, 2^-22 / sqrt(tokens that count).  Bound:
    2e-7 rms over 96 rows; an oracle that leaves the LSE's rounding in must be
    told apart by it."""
    B, C, D = 96, 2000, 64
    q, cache, _, _, _ = _attention_case((B, H, 1, 1, C, [C] * B, -1, 0), D, dtype, seed=50)
    lens = torch.full((B,), C, dtype=torch.int32, device="cuda")
    _, lse = fa.cache_forward(q, cache, lens)
    lse = lse + 6
    heavy = torch.arange(H, device="cuda")[None, :, None] == (torch.arange(B, device="cuda") % H)[:, None, None]
    lse = torch.where(heavy, lse, 1000.0).contiguous()   # exp(x - 1000): 0
    w = fa.cache_weights(q, cache, lse, lens).double()
    _ok()
    ref = _weights64(q, cache, lse, lens, D ** -0.5)
    one = lse[heavy]
    assert 16 < float(one.min()) * 1.4427 and float(one.max()) * 1.4427 < 32
    left_out = one.double() / math.log(2) - (one * torch.tensor(1.4426950408889634, device="cuda")).double()
    biased = ref.sum((1, 2)) * torch.exp2(left_out)   # 2^-(the rounded one) instead of 2^-(the exact one)

    def rms(x):
        return float((w.sum((1, 2)) / x - 1).square().mean().sqrt())

    print(f"H={H} {dtype}: {rms(ref.sum((1, 2))):.2e}, against the biased oracle {rms(biased):.2e}")
    assert rms(ref.sum((1, 2))) <= 2e-7 < rms(biased)
