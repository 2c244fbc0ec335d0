"""Packed sequences without a GPU: refusals of the entry points and of the Python
calls, and the plan's room (no address here is ever read)."""
from __future__ import annotations

import ctypes
import os

import pytest
import torch

from exact_attention_10_gb300 import build as fa_build
from exact_attention_10_gb300 import fa

INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
A = 0x10000000


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fa_build.LIB_PATH):
        fa_build.build()
    return fa.load()


def _sizes(**over):
    z = dict(seqs=3, tokens_q=100, tokens_k=100, heads=4, key_heads=2, causal=1)
    z.update(over)
    return fa.PackedSizes(*z.values())


BAD_SIZES = [dict(seqs=0), dict(tokens_q=0), dict(tokens_k=-1), dict(heads=0), dict(key_heads=0), dict(heads=5),
             dict(causal=2), dict(heads=65536), dict(tokens_q=1 << 30), dict(tokens_k=(1 << 31) - 1), dict(seqs=1 << 24),
             dict(seqs=(1 << 31) - 1)]


@pytest.mark.parametrize("over", BAD_SIZES, ids=str)
def test_bad_sizes(lib, over):
    n = ctypes.c_size_t()
    assert lib.fa_packed_plan_bytes(_sizes(**over), 1, n) == INVALID
    assert lib.fa_packed_bwd_workspace(_sizes(**over), 64, 0, n) == INVALID
    assert lib.fa_packed_plan(A, A, _sizes(**over), 1, A + 4096, 1 << 30, None) == INVALID
    assert _fwd(lib, sizes=_sizes(**over)) == INVALID
    assert _bwd(lib, sizes=_sizes(**over)) == INVALID


def _tensor(i, row=1024, head=128):
    return fa.Rows(A + i * 0x1000000, row, head)


def _fwd(lib, sizes=None, D=128, scale=0.1, dtype=0, plan=A - 0x100000, plan_bytes=1 << 18, lse=A - 0x400000, **over):
    t = dict(q=_tensor(0), k=_tensor(1), v=_tensor(2), o=_tensor(3))
    t.update(over)
    return lib.fa_packed_fwd(t["q"], t["k"], t["v"], t["o"], lse, sizes or _sizes(), D, scale, dtype, plan, plan_bytes, None)


def _bwd(lib, sizes=None, D=128, scale=0.1, dtype=0, flags=0, plan=A - 0x100000, plan_bytes=1 << 18, ws=A - 0x4000000,
         ws_bytes=1 << 24, lse=A - 0x400000, **over):
    t = {n: _tensor(i) for i, n in enumerate(("q", "k", "v", "o", "do", "dq", "dk", "dv"))}
    t.update(over)
    return lib.fa_packed_bwd(t["q"], t["k"], t["v"], t["o"], t["do"], lse, t["dq"], t["dk"], t["dv"], sizes or _sizes(), D,
                             scale, dtype, flags, plan, plan_bytes, ws, ws_bytes, None)


BAD_CALLS = [dict(D=96), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(dtype=2), dict(lse=None),
             dict(plan=None), dict(plan_bytes=64), dict(q=fa.Rows(None, 1024, 128)), dict(k=_tensor(1, row=64)),
             dict(k=_tensor(1, row=1028)), dict(v=_tensor(2, head=100)), dict(v=_tensor(2, row=0)), dict(q=_tensor(0, row=1 << 40)),
             dict(lse=A + 0x3000000)]
FWD_CALLS = [dict(o=_tensor(0)), dict(o=fa.Rows(A + 0x1000000 + 128, 1024, 128)), dict(o=_tensor(3, row=256))]
BWD_CALLS = [dict(flags=2), dict(ws=None), dict(ws_bytes=100), dict(dq=_tensor(0)), dict(dk=_tensor(7)),
             dict(dk=fa.Rows(A + 0x7000000 + 256, 1024, 128)), dict(ws=A + 0x6000000 - 64), dict(dv=_tensor(7, row=128))]


@pytest.mark.parametrize("over", BAD_CALLS + FWD_CALLS, ids=lambda o: ",".join(o))
def test_bad_forward(lib, over):
    assert _fwd(lib, **over) == INVALID


@pytest.mark.parametrize("over", [o for o in BAD_CALLS if o != dict(lse=A + 0x3000000)] + BWD_CALLS, ids=lambda o: ",".join(o))
def test_bad_backward(lib, over):
    assert _bwd(lib, **over) == INVALID


def test_misaligned(lib):
    assert _fwd(lib, q=fa.Rows(A + 8, 1024, 128)) == MISALIGNED
    assert _bwd(lib, dv=fa.Rows(A + 0x7000002, 1024, 128)) == MISALIGNED
    assert _fwd(lib, lse=A - 0x400002) == MISALIGNED


def test_sound_calls_need_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    assert _fwd(lib) == UNSUPPORTED and _bwd(lib) == UNSUPPORTED
    # slices of one buffer lie in one another's ranges and are apart
    part = [fa.Rows(A + 0x5000000 + 256 * h, 8 * 128, 128) for h in (0, 4, 6)]
    assert _bwd(lib, dq=part[0], dk=part[1], dv=part[2]) == UNSUPPORTED
    assert _bwd(lib, dq=part[0], dk=part[1], dv=fa.Rows(A + 0x5000000 + 256 * 5, 8 * 128, 128)) == INVALID
    assert lib.fa_packed_plan(A, A, _sizes(), 1, A + 4096, 1 << 18, None) == UNSUPPORTED


def test_plan_room(lib):
    """A plan's bytes: header, per list two words a slot (a tile, and 160 more), an entry and a sequence and two, the tables."""
    n = ctypes.c_size_t()
    for S, tq, tk in ((1, 1, 1), (3, 100, 700), (64, 36000, 36001)):
        keys = tk // 128 + S
        parts = min(16, -(-640 // (2 * keys)), -(-(tq // 128 + 1) * 2 // 8))
        few = (tq // 256 + S) * 4 <= 213
        caps = [tq // 128 + S, tq // 128 + S, keys * parts]   # (pairs of heads, or few: tiles of 128 rows)
        h0 = 4 if few else 2
        words = [1 + 2 * (caps[0] * h0 + 160 + caps[0] + S + 1)]
        words.append(1 + sum(2 * (c * h + 160 + c + S + 1) for c, h in zip(caps, (h0, 4, 2))) + caps[1] + 1 + keys)
        for grad in (0, 1):
            assert lib.fa_packed_plan_bytes(_sizes(seqs=S, tokens_q=tq, tokens_k=tk), grad, n) == 0
            assert n.value == 16 * words[grad]


def test_python_refusals():
    q, k = torch.zeros(10, 4, 64, dtype=torch.bfloat16), torch.zeros(10, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.packed_plan(cu.long(), 10, 4)
    with pytest.raises(ValueError):
        fa.packed_plan(cu[:1], 10, 4)
    with pytest.raises(ValueError):
        fa.packed_plan(cu, 10, 4, cu_k=cu)
    with pytest.raises(ValueError):
        fa.packed_plan(cu, 10, 4, cu_k=cu[:1], tokens_k=10)
    with pytest.raises(ValueError):
        fa.packed_plan(cu, 1 << 32, 4)
    with pytest.raises(fa.FAError):
        fa.packed_plan(cu, 10, 4, 3)
    plan = fa.PackedPlan(torch.zeros(16, dtype=torch.uint8), fa.PackedSizes(1, 10, 10, 4, 2, 1), False)
    lse = torch.zeros(4, 10)
    for bad in (dict(q=q[:9]), dict(k=k[:, :1]), dict(q=q.float()), dict(k=k.half()), dict(out=q[:, :2]),
                dict(lse=lse.double()), dict(lse=lse.T), dict(plan=None), dict(q=q[0]),
                dict(v=torch.zeros(10, 64, 2, dtype=torch.bfloat16).transpose(1, 2))):
        a = dict(dict(q=q, k=k, v=k, plan=plan), **bad)
        with pytest.raises((TypeError, ValueError)):
            fa.packed_forward(**a)
    with pytest.raises(ValueError):
        fa.packed_backward(q, k, k, q, q, lse, plan)   # made without grad
