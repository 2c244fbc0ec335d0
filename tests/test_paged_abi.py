"""The paged cache without a GPU: refusals of the entry points and of the Python
calls (no address here is ever read)."""
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


def _pages(bits=16, **over):
    c = dict(k=A, v=A + 0x1000000, k_scale=A + 0x2000000, v_scale=A + 0x3000000, pages=20, key_heads=2, page=16, D=64,
             bits=bits, dtype=0)
    c.update(over)
    return fa.Pages(*c.values())


def _move(lib, name, cache=None, table=A + 0x4000000, width=5, B=3, k=None, v=None, tokens=10, start=A + 0x5000000,
          cu=A + 0x6000000):
    return getattr(lib, name)(cache or _pages(), table, width, B, k or fa.Rows(A + 0x7000000, 128, 64),
                              v or fa.Rows(A + 0x8000000, 128, 64), tokens, start, cu, None)


def _fwd(lib, q=A + 0x7000000, strides=(256, 64, 64), cache=None, table=A + 0x4000000, width=5, lens=A + 0x5000000,
         o=A + 0x8000000, lse=A + 0x9000000, B=3, H=4, Nq=1, scale=0.1, ws=A + 0xA000000, ws_bytes=1 << 24):
    return lib.fa_paged_fwd(q, *strides, cache or _pages(), table, width, lens, o, lse, B, H, Nq, scale, ws, ws_bytes, None)


BAD_PAGES = [dict(pages=0), dict(key_heads=0), dict(key_heads=65536), dict(page=8), dict(page=24), dict(page=2048),
             dict(D=96), dict(bits=4), dict(dtype=2), dict(k=None), dict(v=None), dict(bits=8, k_scale=None),
             dict(bits=8, v_scale=None)]


@pytest.mark.parametrize("over", BAD_PAGES, ids=str)
def test_bad_caches(lib, over):
    n = ctypes.c_size_t()
    c = _pages(**over)
    assert _move(lib, "fa_paged_append", cache=c) == INVALID
    assert _move(lib, "fa_paged_read", cache=c) == INVALID
    assert _fwd(lib, cache=c) == INVALID
    if not any(x in over for x in ("k", "v", "k_scale", "v_scale")):   # (the workspace query looks at sizes alone)
        assert lib.fa_paged_workspace(c, 5, 3, 4, 1, n) == INVALID


@pytest.mark.parametrize("over", [
    dict(table=None), dict(width=0), dict(B=0), dict(tokens=0), dict(start=None), dict(cu=None), dict(width=1 << 28),
    dict(B=1 << 30), dict(tokens=(1 << 31) - 1), dict(k=fa.Rows(None, 128, 64)), dict(k=fa.Rows(A + 0x7000000, 60, 64)),
    dict(v=fa.Rows(A + 0x8000000, 132, 64)), dict(v=fa.Rows(A + 0x8000000, 128, 0))], ids=str)
def test_bad_moves(lib, over):
    for name in ("fa_paged_append", "fa_paged_read"):
        assert _move(lib, name, **over) == INVALID


def test_overlaps_and_alignment(lib):
    inside = fa.Rows(A + 256, 128, 64)
    assert _move(lib, "fa_paged_append", k=inside) == INVALID   # tokens in the pages
    assert _move(lib, "fa_paged_read", k=inside) == INVALID
    assert _move(lib, "fa_paged_read", k=fa.Rows(A + 0x8000000, 128, 64)) == INVALID   # k and v the same
    assert _move(lib, "fa_paged_read", k=fa.Rows(A + 0x7000000, 64, 64)) == INVALID    # rows in one another
    assert _move(lib, "fa_paged_append", table=A + 64) == INVALID
    assert _fwd(lib, o=A) == INVALID
    assert _fwd(lib, lse=A + 0x8000000) == INVALID
    assert _fwd(lib, ws=A + 0x9000000) == INVALID
    assert _move(lib, "fa_paged_append", k=fa.Rows(A + 0x7000008, 128, 64)) == MISALIGNED
    assert _move(lib, "fa_paged_read", start=A + 0x5000002) == MISALIGNED
    assert _fwd(lib, q=A + 0x7000002) == MISALIGNED
    assert _fwd(lib, cache=_pages(8, k_scale=A + 0x2000004)) == MISALIGNED


@pytest.mark.parametrize("over", [
    dict(q=None), dict(lens=None), dict(o=None), dict(lse=None), dict(table=None), dict(H=3), dict(H=0), dict(Nq=0),
    dict(B=0), dict(scale=0.0), dict(scale=float("inf")), dict(strides=(256, 60, 64)), dict(strides=(-256, 64, 64)),
    dict(strides=(256, 32, 64)), dict(strides=(256, 64, 1), Nq=2), dict(H=1 << 30), dict(Nq=1 << 29)], ids=str)
def test_bad_attention(lib, over):
    assert _fwd(lib, **over) == INVALID


def test_sound_calls_need_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    n = ctypes.c_size_t()
    for c in (_pages(), _pages(8)):
        assert _move(lib, "fa_paged_append", cache=c) == UNSUPPORTED
        assert _move(lib, "fa_paged_read", cache=c) == UNSUPPORTED
        assert _move(lib, "fa_paged_append", cache=c, cu=None, tokens=3) == UNSUPPORTED
        assert _fwd(lib, cache=c) == UNSUPPORTED
        assert lib.fa_paged_workspace(c, 5, 3, 4, 1, n) == UNSUPPORTED
    assert _fwd(lib, strides=(256, 64, 7)) == UNSUPPORTED   # (the stride of a dimension of one does not count)


def test_python_refusals():
    z = torch.zeros
    k16, k8, sc = z(4, 2, 16, 64, dtype=torch.bfloat16), z(4, 2, 16, 64).to(torch.float8_e4m3fn), z(4, 2, 16)
    for bad in ((k16, k16[:3]), (k16, k16.half()), (k16[0], k16[0]), (z(4, 2, 8, 64).half(), z(4, 2, 8, 64).half()),
                (z(4, 2, 16, 32).half(), z(4, 2, 16, 32).half()), (k8, k8), (k8, k8, sc), (k8, k8, sc, sc[:3]),
                (k8, k8, sc, sc.double()), (k16, k16, sc, sc), (k16.float(), k16.float()),
                (k16.transpose(0, 1), k16.transpose(0, 1)), (k16[:0], k16[:0])):
        with pytest.raises((TypeError, ValueError)):
            fa.PagedCache(*bad)
    with pytest.raises(ValueError):
        fa.paged_empty(4, 2, 16, 64, bits=4, device="cpu")
    with pytest.raises(TypeError):
        fa.paged_empty(4, 2, 16, 64, torch.float32, device="cpu")
    cache, c8 = fa.PagedCache(k16, k16.clone()), fa.PagedCache(k8, k8.clone(), sc, sc.clone())
    table, lens = z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32)
    new, q = z(3, 2, 64, dtype=torch.bfloat16), z(3, 4, 1, 64, dtype=torch.bfloat16)
    for bad in (dict(table=table.long()), dict(table=table[0]), dict(table=table.T), dict(k=new.half()), dict(k=new[:2]),
                dict(k=new[0]), dict(v=new[:, :1]), dict(start=lens[:2]), dict(start=lens.long()), dict(cu=lens),
                dict(cache=tuple(cache)), dict(k=new.transpose(1, 2).contiguous().transpose(1, 2)), dict(table=table[:, :0])):
        with pytest.raises((TypeError, ValueError)):
            fa.paged_append(**dict(dict(cache=cache, table=table, k=new, v=new, start=lens), **bad))
    with pytest.raises(TypeError):
        fa.paged_read(cache, table, lens, 3, dtype=torch.float16)
    with pytest.raises(TypeError):
        fa.paged_read(c8, table, lens, 3, dtype=torch.float32)
    with pytest.raises(ValueError):
        fa.paged_read(cache, table, lens, 0)
    for bad in (dict(q=q[:2]), dict(q=q[:, :3]), dict(q=q.half()), dict(q=q[0]), dict(q=q[..., :32]), dict(lens=lens[:2]),
                dict(table=table.T), dict(out=q[:, :2]), dict(lse=z(3, 4, 1).double()), dict(lse=z(3, 4)),
                dict(q=z(3, 4, 64, 2, dtype=torch.bfloat16).transpose(2, 3))):
        with pytest.raises((TypeError, ValueError)):
            fa.paged_forward(**dict(dict(q=q, cache=cache, table=table, lens=lens), **bad))
    assert c8.args(torch.bfloat16).bits == 8 and c8.args(torch.float16).dtype == 1
