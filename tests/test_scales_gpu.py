"""The operators on windows with sinks and on the 4-bit cache at softmax scales
other than D**-0.5, and the weights' accuracy by itself.

Tolerances: those of tests/test_sink_gpu.py and tests/test_cache_gpu.py, whose
score bounds grow with the scale; the weights' own below.
"""
from __future__ import annotations

import math

import pytest
import torch

from exact_attention_10_gb300 import fa
from test_cache_gpu import T, _attention_case, _gen, _ok, check_attention, unpack64
from test_cache_gpu import reference as cache_reference
from test_sink_gpu import _inputs, check_forward, check_grads
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


@pytest.mark.parametrize("scale", [0.07, 0.3])
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (64, "bf16"), (128, "bf16")])
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_window_backward(case, D, dtype, deterministic, scale):
    B, H, Hkv, Nq, Nkv, left, sinks = case
    q, k, v, do = _inputs(B, H, Hkv, Nq, Nkv, D, dtype, seed=Nq)
    o, lse = fa.forward(q, k, v, window=(left, 0), sinks=sinks, scale=scale)
    grads = fa.backward(q, k, v, o, do, lse, window=(left, 0), sinks=sinks, scale=scale, deterministic=deterministic)
    _ok()
    check_grads(grads, sink_reference(q, k, v, left, sinks, scale, do)[4], dtype, f"{case} {D} {scale}")


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
    that of the exponent: the product of D centred codes (|code - 7.5| 2^-9 with
    a row of q scaled to 2^14) is summed in fp32 with partial sums no larger
    than sum |code - 7.5| |q| scale ks -- about 4 sqrt(D) standard deviations of
    a term, x itself a few units, so roundings of 2^-24 of values up to about 8
    at a dozen places, and the final ones (mul, sum, ref, and 2^x to 2^-22):
    independent, they add up to sqrt(12) 8 2^-24 / sqrt(3) + 2^-23 = 1.1e-6 at
    the very most and 3e-7 where the sums are as small as the scores.  The bound
    is 6e-7, twice the latter: codes from 0 on (partial sums several times the
    scores) measured 1.1e-6, and an LSE whose rounding to log2 units is left in
    scales whole rows by up to LSE 2^-24 log2(e), 1.2e-6 at the LSE of 14 that
    the scale below gives."""
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
