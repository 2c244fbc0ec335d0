"""Results and workspaces of a call with a ``stream`` of its own come from
torch's allocator on that stream.

Memory of the current stream may still be used there by work that is under way
(torch hands a dropped tensor's memory on without waiting), so a result taken
from it and written on another stream would be written too early.  Shown here
on the CPU, with the library and torch's stream context stubbed out; on the GPU
with a fill that is delayed on the current stream.
"""
from __future__ import annotations

import pytest

from exact_attention_10_gb300 import fa

torch = pytest.importorskip("torch")


def _calls(dev, dtype, B=2, H=4, Hkv=2, N=40, D=64, C=48):
    """name -> call(stream) of every entry point that makes results, on inputs
    that do not change."""
    g = torch.Generator().manual_seed(3)

    def rand(*shape):
        return torch.randn(shape, generator=g).to(dtype).to(dev)

    q, do, k, v = rand(B, H, N, D), rand(B, H, N, D), rand(B, Hkv, N, D), rand(B, Hkv, N, D)
    kh, vh = rand(B, H, N, D), rand(B, H, N, D)
    cache = fa.PackedCache(*(torch.randint(0, 256, (B, Hkv, C, D // 2), generator=g, dtype=torch.uint8).to(dev) if i % 2 == 0
                             else rand(B, Hkv, C, 2).abs() for i in range(4)))
    lens = torch.tensor([C, C - 9], dtype=torch.int32, device=dev)
    start = torch.zeros(B, dtype=torch.int32, device=dev)
    one = rand(B, H, 1, D)
    acc = torch.rand((B, Hkv, C), generator=g).to(dev)
    win = dict(window=(20, 0), sinks=3)
    o, lse = torch.zeros_like(q), torch.zeros((B, H, N), device=dev)
    lse1 = torch.zeros((B, H, 1), device=dev)
    return {
        "forward": lambda s: fa.forward(q, kh, vh, causal=True, stream=s),
        "forward band": lambda s: fa.forward(q, kh, vh, window=(20, 3), stream=s),
        "forward sinks": lambda s: fa.forward(q, k, v, schedule="balanced", stream=s, **win),
        "backward": lambda s: fa.backward(q, kh, vh, o, do, lse, causal=True, deterministic=True, stream=s),
        "backward sinks": lambda s: fa.backward(q, k, v, o, do, lse, deterministic=True, stream=s, **win),
        "cache_read": lambda s: fa.cache_read(cache, start, C, stream=s),
        "cache_forward": lambda s: fa.cache_forward(one, cache, lens, stream=s, **win),
        "cache_weights": lambda s: (fa.cache_weights(one, cache, lse1, lens, stream=s, **win),),
        "cache_evict": lambda s: (lambda r: (*r[0], *r[1:]))(fa.cache_evict(cache, acc, lens, C - 9, sinks=2, recent=3, stream=s)),
    }


NAMES = list(_calls("cpu", torch.bfloat16))


class _Foreign:
    """Another library's stream: nothing but a handle."""

    def __init__(self, handle=77):
        self.cuda_stream = handle


class _Lib:
    """Every entry point succeeds; workspace queries ask for 4096 bytes."""

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_workspace"):
                a[-1]._obj.value = 4096
            return 0
        return call


@pytest.mark.parametrize("stream", [_Foreign(), 77], ids=["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_allocations_are_on_the_given_stream(name, stream, monkeypatch):
    call = _calls("cpu", torch.bfloat16)[name]
    on, made = [], []

    class Context:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            on.append(self.stream)

        def __exit__(self, *a):
            on.pop()

    def recorded(make):
        def f(*a, **kw):
            made.append(on[-1] if on else None)
            return make(*a, **kw)
        return f

    queries = (fa._sink_workspace, fa._sink_bwd_workspace, fa._cache_workspace)
    for x in queries:
        x.cache_clear()
    try:
        with monkeypatch.context() as m:
            lib = _Lib()
            m.setattr(fa, "load", lambda *a: lib)
            m.setattr(torch.cuda, "stream", Context)
            m.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
            m.setattr(torch, "empty", recorded(torch.empty))
            m.setattr(torch, "empty_like", recorded(torch.empty_like))
            call(stream)
            assert made and all(x == ("external", 77) for x in made), made
    finally:
        for x in queries:
            x.cache_clear()


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_results_do_not_take_memory_that_is_still_written(name):
    """Tensors of the results' sizes are dropped on the current stream while a
    delayed fill of them is still to run there; the call on another stream does
    not get that memory."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    call = _calls("cuda", torch.bfloat16)[name]
    side = torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)   # about a tenth of a second
    pending = [torch.empty_like(x) for x in want for _ in range(2)]
    for x in pending:
        x.fill_(1)
    held = {x.untyped_storage().data_ptr() for x in pending}
    del pending, x
    got = call(side)
    assert not held & {x.untyped_storage().data_ptr() for x in got}
    side.synchronize()
    torch.cuda.synchronize()
    assert fa.sync_status(side.cuda_stream) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_streams_of_every_kind(name):
    """torch's streams, plain handles (the legacy default stream's 0 among them)
    and objects with nothing but a handle."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    call = _calls("cuda", torch.bfloat16)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, _Foreign(side.cuda_stream), 0):
        got = call(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
