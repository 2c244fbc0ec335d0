"""CPU-only checks of the entry points for windows with sinks and for the 4-bit
cache: bad arguments are refused before any device is touched, sound ones reach
the device check.  (Fake addresses, never dereferenced.)"""
from __future__ import annotations

import ctypes
import os

import pytest

from exact_attention_10_gb300 import build as fa_build
from exact_attention_10_gb300 import fa

OK, INVALID, MISALIGNED, UNSUPPORTED = 0, 1, 2, 3
A = 0x10000000
STEP = 0x1000000
P = [A + i * STEP for i in range(16)]
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fa_build.LIB_PATH):
        fa_build.build()
    return fa.load()


def _no_gpu():
    torch = pytest.importorskip("torch")
    return not torch.cuda.is_available()


def _call(fn, base, names, over):
    a = dict(base, **over)
    return fn(*(a[n] for n in names))


FWD = dict(q=P[0], k=P[1], v=P[2], o=P[3], lse=P[4], B=1, H=4, Hkv=2, Nq=256, Nkv=256, D=64, left=31, sinks=4,
           scale=F(0.125), dtype=0, schedule=0, ws=P[5], nws=1 << 20, stream=None)
BWD = dict(q=P[0], k=P[1], v=P[2], o=P[3], do=P[4], lse=P[5], dq=P[6], dk=P[7], dv=P[8], B=1, H=4, Hkv=2, Nq=256,
           Nkv=256, D=64, left=31, sinks=4, scale=F(0.125), dtype=0, flags=0, ws=P[9], nws=1 << 22, stream=None)
BAD_SIZES = [dict(D=32), dict(D=256), dict(B=0), dict(H=0), dict(Hkv=0), dict(H=5), dict(Nq=0), dict(Nkv=-1),
             dict(sinks=-1), dict(scale=F(0.0)), dict(scale=F(float("nan"))), dict(scale=F(-1.0)), dict(dtype=2),
             dict(B=1 << 20, H=1 << 10, Hkv=1 << 10, Nq=4),           # B*H*Nq >= 2^31
             dict(B=1 << 15, H=1, Hkv=1, Nkv=1 << 16)]                 # B*Hkv*Nkv >= 2^31


@pytest.mark.parametrize("over", BAD_SIZES + [dict(q=0), dict(lse=0), dict(schedule=3), dict(o=P[0]), dict(o=P[1] + 64),
                                              dict(lse=P[3] + 128), dict(ws=P[2])], ids=str)
def test_forward_refusals(lib, over):
    assert _call(lib.fa_fwd_sink, FWD, FWD, over) == INVALID


@pytest.mark.parametrize("over", BAD_SIZES + [dict(flags=2), dict(do=0), dict(dv=0), dict(ws=0), dict(dq=P[1]),
                                              dict(dk=P[6] + 64), dict(dv=P[5]), dict(ws=P[7])], ids=str)
def test_backward_refusals(lib, over):
    assert _call(lib.fa_bwd_sink, BWD, BWD, over) == INVALID


def test_alignment_and_device(lib):
    for name, base, fn in (("o", FWD, lib.fa_fwd_sink), ("lse", FWD, lib.fa_fwd_sink), ("ws", FWD, lib.fa_fwd_sink),
                           ("dk", BWD, lib.fa_bwd_sink), ("ws", BWD, lib.fa_bwd_sink)):
        assert _call(fn, base, base, {name: base[name] + 8}) == MISALIGNED
    if _no_gpu():
        for left, sinks in ((31, 4), (-1, 0), (-5, 9), (0, 0), (2 ** 31 - 1, 2 ** 31 - 1)):
            assert _call(lib.fa_fwd_sink, FWD, FWD, dict(left=left, sinks=sinks)) == UNSUPPORTED
            assert _call(lib.fa_bwd_sink, BWD, BWD, dict(left=left, sinks=sinks)) == UNSUPPORTED
        n = ctypes.c_size_t()
        assert lib.fa_fwd_sink_workspace(1, 4, 2, 256, 256, 64, 31, 4, 0, ctypes.byref(n)) == UNSUPPORTED
        assert lib.fa_bwd_sink_workspace(1, 4, 2, 256, 256, 64, 31, 4, 0, ctypes.byref(n)) == UNSUPPORTED
        assert lib.fa_cache_workspace(1, 4, 2, 1, 100, 64, ctypes.byref(n)) == UNSUPPORTED
    assert lib.fa_fwd_sink_workspace(1, 5, 2, 256, 256, 64, 31, 4, 0, None) == INVALID
    assert lib.fa_cache_workspace(1, 5, 2, 1, 100, 64, ctypes.byref(ctypes.c_size_t())) == INVALID


APPEND = dict(kc=P[0], kp=P[1], vc=P[2], vp=P[3], k=P[4], v=P[5], start=P[6], count=None, B=2, Hkv=2, N=8, C=64, D=64,
              dtype=0, stream=None)
CACHE = dict(q=P[0], kc=P[1], kp=P[2], vc=P[3], vp=P[4], lens=P[5], o=P[6], lse=P[7], B=2, H=4, Hkv=2, Nq=1, C=5000, D=64,
             left=-1, sinks=0, scale=F(0.125), dtype=0, ws=P[8], nws=1 << 24, stream=None)
WEIGHTS = dict(q=P[0], kc=P[1], kp=P[2], lse=P[3], lens=P[4], acc=P[5], add=0, B=2, H=4, Hkv=2, Nq=1, C=64, D=64, left=-1,
               sinks=0, scale=F(0.125), dtype=0, stream=None)
EVICT = dict(kc=P[0], kp=P[1], vc=P[2], vp=P[3], acc=P[4], lens=P[5], kc2=P[6], kp2=P[7], vc2=P[8], vp2=P[9], acc2=P[10],
             lens2=P[11], index=P[12], B=2, Hkv=2, C=64, C2=32, D=64, keep=32, sinks=4, recent=8, stream=None)


@pytest.mark.parametrize("fn,base,bad", [
    ("fa_cache_append", APPEND, [dict(D=48), dict(B=0), dict(Hkv=0), dict(N=0), dict(C=0), dict(dtype=7), dict(kc=0),
                                 dict(start=0), dict(vc=P[0]), dict(kp=P[4] + 8), dict(C=1 << 30, B=2),
                                 dict(N=1 << 30, B=2)]),
    ("fa_cache_read", APPEND, [dict(D=48), dict(N=0), dict(k=0), dict(v=P[4] + 64), dict(k=P[0])]),
    ("fa_cache_fwd", CACHE, [dict(D=96), dict(H=3), dict(Nq=0), dict(sinks=-1), dict(scale=F(0.0)), dict(lens=0), dict(o=0),
                             dict(o=P[0]), dict(lse=P[6]), dict(ws=P[1]), dict(C=1 << 30)]),
    ("fa_cache_weights", WEIGHTS, [dict(D=96), dict(H=3), dict(add=2), dict(scale=F(float("inf"))), dict(acc=0),
                                   dict(acc=P[3]), dict(sinks=-2)]),
    ("fa_cache_evict", EVICT, [dict(D=96), dict(keep=0), dict(keep=33), dict(sinks=-1), dict(recent=-1), dict(sinks=25),
                               dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(index=0), dict(kc2=P[0]), dict(acc2=P[4]),
                               dict(lens2=P[5]), dict(vc2=P[6]), dict(B=1 << 29, Hkv=1)]),
])
def test_cache_refusals(lib, fn, base, bad):
    f = getattr(lib, fn)
    for over in bad:
        assert _call(f, base, base, over) == INVALID, over
    if _no_gpu():
        assert _call(f, base, base, {}) == UNSUPPORTED
        if "count" in base:
            assert _call(f, base, base, dict(count=P[7])) == UNSUPPORTED
    first = "q" if "q" in base else "kc"
    assert _call(f, base, base, {first: base[first] + 8}) == MISALIGNED
    for name in ("start", "lens", "acc", "index", "kp"):
        if name in base:
            assert _call(f, base, base, {name: base[name] + 2}) == MISALIGNED, name
            if _no_gpu():
                assert _call(f, base, base, {name: base[name] + 4}) == UNSUPPORTED, name


@pytest.mark.parametrize("fn,base,sizes", [
    ("fa_cache_append", APPEND, ("C", "N")), ("fa_cache_read", APPEND, ("C", "N")), ("fa_cache_fwd", CACHE, ("C",)),
    ("fa_cache_weights", WEIGHTS, ("C",)), ("fa_cache_evict", EVICT, ("C", "C2")),
    ("fa_fwd_sink", FWD, ("Nkv", "Nq")), ("fa_bwd_sink", BWD, ("Nkv", "Nq"))])
def test_sizes_next_to_the_32_bit_limit(lib, fn, base, sizes):
    """Lengths whose last block's or cluster's indices would pass 2^31 are
    refused, the ones below them are not (pointers 2^40 bytes apart, so that no
    tensor overlaps another)."""
    f = getattr(lib, fn)
    far = {name: (i + 1) << 40 for i, name in enumerate(n for n in base if base[n] in P)}
    one = dict(B=1, Hkv=1) | ({"H": 1} if "H" in base else {})
    small = {n: 64 for n in ("N", "C", "C2", "Nq", "Nkv", "keep") if n in base}
    for name in sizes:
        for n in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 65535):
            assert _call(f, base, base, far | one | small | {name: n}) == INVALID, (name, n)
        if _no_gpu() and name != "Nq":   # (its rows are not the largest tensor of every call)
            assert _call(f, base, base, far | one | small | {name: 2 ** 31 - 65536}) == UNSUPPORTED, name


def test_python_refusals_before_the_library():
    torch = pytest.importorskip("torch")
    c = fa.cache_empty(2, 2, 16, 64, torch.bfloat16, device="cpu")
    assert c.sizes == (2, 2, 16, 64, 0) and c.k_codes.shape == (2, 2, 16, 32) and c.v_params.shape == (2, 2, 16, 2)
    with pytest.raises(ValueError):
        fa.cache_empty(1, 1, 4, 80, device="cpu")
    with pytest.raises(TypeError):
        fa.cache_empty(1, 1, 4, 64, torch.float32, device="cpu")
    with pytest.raises(ValueError):
        fa.PackedCache(c[0], c[1][:, :, :8], c[2], c[3])
    with pytest.raises(TypeError):
        fa.PackedCache(c[0], c[1], c[2], c[3].half())
    with pytest.raises(ValueError):
        fa.PackedCache(c[0].transpose(0, 1), *c[1:])
    k = torch.zeros((2, 2, 3, 64), dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.cache_append(c, k[:, :1], k[:, :1], ints)
    with pytest.raises(TypeError):
        fa.cache_append(c, k.half(), k.half(), ints)
    with pytest.raises(TypeError):
        fa.cache_append(c, k, k, ints.long())
    with pytest.raises(ValueError):
        fa.cache_append(c, k, k, ints[:1])
    with pytest.raises(ValueError):
        fa.cache_read(c, ints, 0)
    q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16)
    for bad in (dict(window=(3, 1)), dict(sinks=-1), dict(sinks=2 ** 32)):
        with pytest.raises(ValueError):
            fa.cache_forward(q, c, ints, **bad)
        with pytest.raises(ValueError):
            fa.forward(q, k, k, sinks=bad.get("sinks", 0), window=bad.get("window", (3, 0)))
    with pytest.raises(ValueError):
        fa.cache_evict(c, torch.zeros(2, 2, 16), ints, 4, sinks=3, recent=2)


@pytest.mark.parametrize("sizes", [(0, 2, 16), (2, 0, 16), (2, 2, 0)], ids=str)
def test_empty_caches_are_refused(sizes):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        fa.cache_empty(*sizes, 64, torch.bfloat16, device="cpu")
