"""Serving on from an evicted cache: append, attention, weights and eviction
over several turns, against float64 on a mirror of the kept rows that is kept
apart from the library's cache; and the README's loop, as it stands there.

Tolerances as in tests/test_cache_gpu.py.
"""
from __future__ import annotations

import os

import pytest
import torch

from exact_attention_10_gb300 import fa
from test_cache_gpu import T, _gen, _ok, check_attention, evict_reference, pack64, reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load()


def _tokens(B, H, Hkv, n, D, dtype, seed):
    g = _gen(seed)
    return [(torch.randn((B, h, 1, D), generator=g, device="cuda")).to(T[dtype]) for _ in range(n) for h in (H, Hkv, Hkv)]


@pytest.mark.parametrize("left,sinks", [(-1, 0), (25, 4)])
@pytest.mark.parametrize("D,dtype,G", [(64, "bf16", 4), (128, "fp16", 20)])
def test_turns_of_appends_and_evictions(D, dtype, G, left, sinks):
    """Two caches in turn: each eviction goes into the other one.  After it the
    positions count the kept tokens alone, for lens, the window and the sinks."""
    B, Hkv, N, keep, room = 3, 2, 90, 64, 40
    H, C = Hkv * G, keep + room
    start = torch.tensor([90, 50, 3], dtype=torch.int32, device="cuda")
    g = _gen(D)
    prompt = [torch.randn((B, Hkv, N, D), generator=g, device="cuda").to(T[dtype]) for _ in range(2)]
    cache, spare = (fa.cache_empty(B, Hkv, C, D, T[dtype]) for _ in range(2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, *prompt, lens, count=start)
    lens += start
    weights = torch.zeros((B, Hkv, C), device="cuda")
    # the mirror: packed rows by the definition, in tensors of another capacity
    mirror = fa.PackedCache(*(torch.zeros((B, Hkv, 200, x.shape[3]), dtype=x.dtype, device="cuda") for x in cache))
    for i, x in enumerate(prompt):
        for b in range(B):
            n = int(start[b])
            mirror[2 * i][b, :, :n], mirror[2 * i + 1][b, :, :n] = (y[b, :, :n] for y in pack64(x))
    n = start.tolist()
    tokens = iter(_tokens(B, H, Hkv, 60, D, dtype, 5))
    cuts = 0
    for turn in range(60):
        q, k, v = (next(tokens) for _ in range(3))
        fa.cache_append(cache, k, v, lens)
        lens += 1
        for i, x in enumerate((k, v)):
            codes, params = pack64(x)
            for b in range(B):
                mirror[2 * i][b, :, n[b]], mirror[2 * i + 1][b, :, n[b]] = codes[b, :, 0], params[b, :, 0]
        n = [m + 1 for m in n]
        o, lse = fa.cache_forward(q, cache, lens, window=(left, 0), sinks=sinks)
        fa.cache_weights(q, cache, lse, lens, window=(left, 0), sinks=sinks, acc=weights)
        assert lens.tolist() == n and max(n) <= C
        if turn % 7 == 6 or max(n) == C:   # (the float64 reference is slow)
            ref = reference(q, mirror, lens, left, sinks, D ** -0.5)
            check_attention(q, mirror, lens, left, sinks, D ** -0.5, o, lse, ref)
        if max(n) == C:
            cuts += 1
            before = weights
            kept, weights, lens, index = fa.cache_evict(cache, weights, lens, keep, sinks=4, recent=16, out=spare)
            assert kept is spare and weights.shape == (B, Hkv, C)
            spare, cache = cache, kept
            want = torch.from_numpy(evict_reference(before.cpu().numpy(), n, keep, 4, 16)).cuda()
            assert torch.equal(index.long(), want)
            at = want.clamp(min=0)
            for x in mirror:
                x[:, :, :keep] = x.gather(2, at[..., None].expand(B, Hkv, keep, x.shape[3]))
            n = [min(m, keep) for m in n]
    _ok()
    assert cuts >= 2 and lens.tolist() == n


def test_a_cache_without_room_drops_what_is_appended():
    """What the documentation says of a cache of capacity `keep`: it takes no
    more tokens, and nothing else changes."""
    B, Hkv, D = 2, 1, 64
    k = torch.randn((B, Hkv, 9, D), generator=_gen(1), device="cuda").bfloat16()
    cache = fa.cache_empty(B, Hkv, 9, D)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.cache_append(cache, k, k, lens)
    kept, _, lens, _ = fa.cache_evict(cache, torch.zeros((B, Hkv, 9), device="cuda"), lens + 9, 5, recent=5)
    assert kept.sizes[2] == 5 and lens.tolist() == [5, 5]
    was = [x.clone() for x in kept]
    fa.cache_append(kept, k[:, :, :1].contiguous(), k[:, :, :1].contiguous(), lens)
    _ok()
    for a, b in zip(kept, was):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_the_readme_serving_loop():
    """The README's python block on the cache, run as it stands with small
    sizes: every token it decodes is attended with its own key in place, over
    several evictions."""
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = [b.split("```")[0] for b in f.read().split("```python\n")[1:]]
    text = "\n".join(blocks)
    text = text[text.index("# a key/value cache in 4 bits"):]
    B, H, Hkv, D, N, keep, capacity = 2, 8, 2, 64, 100, 64, 128
    tokens = [x for x in zip(*[iter(_tokens(B, H, Hkv, 150, D, "bf16", 9))] * 3)]
    k_prompt, v_prompt = (torch.randn((B, Hkv, N, D), generator=_gen(i), device="cuda").bfloat16() for i in (1, 2))
    q_new, k_new, v_new = tokens[0]
    seen, cuts = [], []

    class Watched:   # the library, with an eye on what the loop attends and evicts
        def __getattr__(self, name):
            return getattr(fa, name)

        def cache_forward(self, q, cache, lens, **kw):
            o, lse = fa.cache_forward(q, cache, lens, **kw)
            k, v = tokens[len(seen)][1:]
            at = (lens.long() - 1)[:, None, None, None]
            assert int(lens.max()) <= cache.sizes[2], "tokens past the capacity"
            for i, x in ((0, k), (2, v)):
                for held, row in zip(cache[i:i + 2], pack64(x)):
                    assert torch.equal(held.gather(2, at.expand(B, Hkv, 1, held.shape[3])), row), "the token's own row"
            if len(seen) % 40 == 0:
                check_attention(q, cache, lens, -1, 0, D ** -0.5, o, lse, reference(q, cache, lens, -1, 0, D ** -0.5))
            seen.append(lens.clone())
            return o, lse

        def cache_evict(self, *a, **kw):
            cuts.append(1)
            return fa.cache_evict(*a, **kw)

    exec(compile(text, "README.md", "exec"), dict(
        fa=Watched(), torch=torch, B=B, H=H, Hkv=Hkv, D=D, keep=keep, capacity=capacity, tokens=tokens, k_prompt=k_prompt,
        v_prompt=v_prompt, q_new=q_new, k_new=k_new, v_new=v_new, lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
        weights=torch.zeros((B, Hkv, capacity), device="cuda")))
    _ok()
    assert len(seen) == len(tokens) and len(cuts) >= 2
