"""CPU models of what packed sequences change in the mbarrier protocols, on the
models of tests/test_pipeline_protocol.py, tests/test_sink_protocol.py and
tests/test_bwd_protocol.py.

Forward at D = 128 (exact_attention_10_gb300/csrc/fa_fwd_kernel.cuh, kSplitQ): the
two halves of the one Q buffer are filled and given back apart.  Per tile the
producer loads Q tile 0, the first step's K and V, Q tile 1 (if the tile has
one), then the other steps; the MMA warp gives half 0 back after Q tile 0's last S
and half 1 after Q tile 1's, and waits for half 1 before its first.  The model
tracks which tile's rows each half holds, and every S must read its own.

Backward (fa_bwd_kernel.cuh, bwd_load): the passes that stream pairs of tiles
load a tile's first step before its resident tiles, which wait for the previous
tile's last products.

Every interleaving tried must finish; planted mistakes must not.
"""
from __future__ import annotations

import random

import pytest
import test_bwd_protocol as bwd
from test_pipeline_protocol import CTA, ORDERS, Barrier, Issuer, epilogue, softmax, wait
from test_sink_protocol import Hazard, interleave


class SplitCTA(CTA):
    def __init__(self, o):
        super().__init__(o)
        self.q1_full, self.q1_empty = Barrier("q1_full"), Barrier("q1_empty")
        self.half = [None, None]


def load_role(c, o, parts, q1_at=0):
    """q1_at: the step behind whose K and V (0) or before whose (1) Q tile 1 is loaded."""
    step = it1 = 0

    def load_q1(t):
        nonlocal it1
        yield wait(c.q1_empty, it1 - 1)
        c.half[1] = t
        c.q1_full.arrive()
        it1 += 1

    for t, (n, _, n1) in enumerate(parts):
        yield wait(c.q_empty[0], t - 1)
        c.half[0] = t
        c.q_full[0].arrive()
        for j in range(n):
            if q1_at == j == 1 and n1:
                yield from load_q1(t)
            st = step % o.stages
            yield wait(c.empty[st], step // o.stages - 1)
            c.full[st].arrive()
            if q1_at == j == 0 and n1:
                yield from load_q1(t)
            step += 1


def mma_parts(c, o, parts, early=False, count_all=False):
    """early: half 0 given back a step too soon; count_all: half 1's phase counted for tiles without a Q tile 1 too."""
    m, m1 = Issuer(c, o, 0), Issuer(c, o, 1)
    step = it1 = 0
    prev, pv, acc = None, False, False

    def reads(half, t):
        if c.half[half] != t:
            raise Hazard

    def finish():
        if pv:
            yield from m1.issue_pv(acc)
        c.empty[prev].arrive()

    for t, (n, n0, n1) in enumerate(parts):
        yield wait(c.q_full[0], t)
        for j in range(n):
            st = step % o.stages
            yield wait(c.full[st], step // o.stages)
            if j < n0:
                yield from m.issue_s()
                reads(0, t)
            if j == max(n0 - (2 if early else 1), 0):
                c.q_empty[0].arrive()
                yield None
            if prev is not None:
                yield from finish()
            if j == 0 and (n1 or count_all):
                if n1:
                    yield wait(c.q1_full, it1)
                it1 += 1
            if j < n1:
                yield from m1.issue_s()
                reads(1, t)
            if j == n1 - 1:
                c.q1_empty.arrive()
                yield None
            if j < n0:
                yield from m.issue_pv(j > 0)
            pv, prev, acc = j < n1, st, j > 0
            step += 1
    if prev is not None:
        yield from finish()


def run(parts, seed, q1_at=0, **mistake):
    o = ORDERS["d128"]
    c = SplitCTA(o)
    roles = [load_role(c, o, parts, q1_at), mma_parts(c, o, parts, **mistake)]
    roles += [softmax(c, o, parts, w, True) for w in range(2)]
    return interleave(roles + [epilogue(c, o, parts)], seed)


def packed_parts(rng):
    """Tiles of one sequence or several: (steps, Q tile 0's, Q tile 1's)."""
    parts = []
    for _ in range(rng.randint(1, 7)):
        n = rng.choice([1, 1, 1, 2, 2, 3, 5, 8])
        parts.append(rng.choice([(n, max(n - 1, 1), n), (n, n, n), (n, n, 0)]))
    return parts


def test_split_q_completes():
    rng = random.Random(1)
    for _ in range(300):
        parts = packed_parts(rng)
        for seed in range(15):
            assert run(parts, seed) == "done", (parts, seed)


@pytest.mark.parametrize("parts", [[(1, 1, 1)], [(2, 1, 2), (1, 1, 1), (2, 2, 2)]])
def test_q_tile_1_before_the_second_step_is_never_loaded_for_one(parts):
    assert all(run(parts, seed, q1_at=1) != "done" for seed in range(50))


def test_a_half_given_back_too_soon_is_found():
    parts = [(3, 3, 3)] * 4
    assert "hazard" in {run(parts, seed, early=True) for seed in range(200)}


def test_a_phase_counted_for_a_tile_without_q_tile_1_is_found():
    parts = [(2, 1, 2), (1, 1, 0), (2, 1, 2), (2, 2, 2)]
    assert all(run(parts, seed, count_all=True) != "done" for seed in range(50))


# ------------------------------------------------------------------ the backward's producer

def early_loader(c, q, tiles):
    """bwd.loader for rings of pairs, the first step before the resident tiles."""
    step = 0

    def load():
        nonlocal step
        yield wait(c.empty[step % q.ring0], step // q.ring0 - 1)
        c.full[step % q.ring0].arrive()
        step += 1

    for t, n in enumerate(tiles):
        yield from load()
        if t > 0:
            yield wait(c.res_empty, t - 1)
        c.res_full.arrive()
        for _ in range(n - 1):
            yield from load()


def early_loader_fused(c, q, tiles, wait_res=True):
    step = 0

    def set_res(v):
        c.res = v

    def set_stage(i):
        return lambda v: c.stage.__setitem__(i, v)

    def load():
        nonlocal step
        yield wait(c.empty[step % q.ring0], step // q.ring0 - 1)
        bwd.copy(c, c.full[step % q.ring0], set_stage(step % q.ring0), step)
        step += 1

    for t, n in enumerate(tiles):
        yield from load()
        if t > 0 and wait_res:
            yield wait(c.res_empty, t - 1)
        bwd.copy(c, c.res_full, set_res, t)
        for _ in range(n - 1):
            yield from load()


@pytest.mark.parametrize("name", ["d64_kv", "d64_dq", "d64_fused", "d128_kv"])
def test_first_step_before_the_resident_tiles_completes(name, monkeypatch):
    monkeypatch.setattr(bwd, "loader", early_loader)
    monkeypatch.setattr(bwd, "loader_fused", early_loader_fused)
    rng = random.Random(len(name))
    for _ in range(120):
        tiles = [rng.choice([1, 1, 2, 3, 4, 7]) for _ in range(rng.randint(1, 6))]
        for seed in range(15):
            assert bwd.run(name, tiles, seed) == "done", (name, tiles, seed)


def test_resident_tiles_that_do_not_wait_are_found(monkeypatch):
    monkeypatch.setattr(bwd, "loader_fused", lambda c, q, tiles: early_loader_fused(c, q, tiles, wait_res=False))
    assert {bwd.run("d64_fused", [3, 2, 4], seed) for seed in range(100)} & {"race", "aliased", "deadlock"}
