"""CPU models of two more mbarrier protocols, with the barriers, waits and
checks of tests/test_pipeline_protocol.py.

mma_parts (exact_attention_10_gb300/csrc/fa_fwd_kernel.cuh), the MMA warps'
order for causal windows with sinks, in its three forms: D = 64 (a warp per Q
tile), D = 128 with two Q tiles (interleaved) and with one (K and V of a stage
on separate barriers).  It carries the steps of a CTA's parts on as one
sequence: the next part's first S is issued before this part's last P.V, the Q
buffer is given back after the part's last S, and the stage of the step whose
P.V is still to come is held across the parts.  The other roles are those of
the other masks.  (A first step of a few sinks waits and arrives like any other.)

weights_rows_kernel (fa_cache_rows.cu): eight warps of sums in two groups that
take every other tile, four that unpack K, the first of which also issues the
MMAs; the tiles are numbered on through the row blocks and segments of a CTA
("passes").  The tensor core is a role of its own that runs each product some
time after its issue, and the model checks what it and the sums read: the tile
that was unpacked, the pass's rows and constants, the tile's scores.

Every interleaving tried must finish; orders with a planted mistake must not.
"""
from __future__ import annotations

import os
import random
import re

import pytest

from test_pipeline_protocol import CTA, ORDERS, Aliased, Barrier, Issuer, epilogue, loader, random_parts, softmax, wait

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_10_gb300", "csrc")


class Hazard(Exception):
    pass


def interleave(roles, seed: int) -> str:
    """'done', 'deadlock', 'aliased' or 'hazard' for one random interleaving.  A
    role yields a wait, or None where others may come in between."""
    blocked = [None] * len(roles)
    live = set(range(len(roles)))
    rng = random.Random(seed)

    def ready(i):
        if blocked[i] is None:
            return True
        _, bar, k = blocked[i]
        if bar.phase > k + 1:
            raise Aliased(f"{bar.name}: phase {bar.phase} while waiting for {k}")
        return bar.phase >= k + 1

    try:
        while live:
            runnable = [i for i in live if ready(i)]
            if not runnable:
                return "deadlock"
            i = rng.choice(runnable)
            try:
                blocked[i] = next(roles[i])
            except StopIteration:
                live.discard(i)
                blocked[i] = None
    except Aliased:
        return "aliased"
    except Hazard:
        return "hazard"
    return "done"


# ------------------------------------------------------------------ mma_parts

def mma_parts(c: CTA, o, parts, w: int, q_after_pv=False, keep_last=False):
    """q_after_pv: the Q buffer given back after the part's last P.V, as the
    other masks' order does; keep_last: the last stage of a part not released
    at the part's end but forgotten."""
    m, m1 = Issuer(c, o, w), Issuer(c, o, 1)
    step = it = 0
    prev, pv, acc = None, False, False
    owed = []   # q_after_pv: buffers still to give back

    def finish(last):
        if o.sep:
            if o.split_kv:
                yield wait(c.v_full[last % o.stages], last // o.stages)
            if pv:
                yield from m.issue_pv(acc)
            (c.v_empty if o.split_kv else c.empty)[prev].arrive()
        else:
            if pv:
                yield from m1.issue_pv(acc)
            c.empty[prev].arrive()
        while owed:
            c.q_empty[owed.pop()].arrive()

    for n, n0, n1 in parts:
        qb = it % o.q_bufs
        yield wait(c.q_full[qb], it // o.q_bufs)
        for j in range(n):
            st = step % o.stages
            yield wait(c.full[st], step // o.stages)
            if o.sep:
                nw = n1 if w else n0
                if j < nw:
                    yield from m.issue_s()
                if o.split_kv:
                    c.empty[st].arrive()
                if j == n - 1 and not q_after_pv:
                    c.q_empty[qb].arrive()
                if prev is not None and not (keep_last and j == 0):
                    yield from finish(step - 1)
                pv = j < nw
            else:
                if j < n0:
                    yield from m.issue_s()
                if prev is not None and not (keep_last and j == 0):
                    yield from finish(step - 1)
                if j < n1:
                    yield from m1.issue_s()
                if j == n - 1 and not q_after_pv:
                    c.q_empty[qb].arrive()
                if j < n0:
                    yield from m.issue_pv(j > 0)
                pv = j < n1
            if j == n - 1 and q_after_pv:
                owed.append(qb)
            prev, acc = st, j > 0
            step += 1
        it += 1
    if prev is not None:
        yield from finish(step - 1)


def run_parts(order: str, parts, seed: int, last_pv_wait=True, flush_before_q=True, **mistake) -> str:
    o = ORDERS[order]
    c = CTA(o)
    roles = [loader(c, o, parts, flush_before_q)]
    roles += [mma_parts(c, o, parts, w, **mistake) for w in range(o.mma_warps)]
    roles += [softmax(c, o, parts, w, last_pv_wait) for w in range(o.tiles)]
    roles.append(epilogue(c, o, parts))
    return interleave(roles, seed)


def sink_parts(rng: random.Random, tiles: int):
    """A CTA's parts under a window: 1 to 6 tiles of 1 to 12 steps, whose Q tile
    0 ends a step before its neighbour or with it, whose Q tile 1 may have no
    rows, and (balanced) later parts that may hold steps of one of them alone."""
    parts = []
    for _ in range(rng.randint(1, 6)):
        n = rng.choice([1, 1, 2, 3, 3, 4, 9, 12])
        if tiles == 1:
            parts.append((n, n, 0))
        else:
            parts.append(rng.choice([(n, max(n - 1, 0), n), (n, n, n), (n, n, 0), (n, 0, n)]))
    return parts


@pytest.mark.parametrize("order", ["d64", "d128", "d128_one_tile"])
def test_mma_parts_completes(order):
    rng = random.Random(len(order))
    for i in range(200):
        parts = (sink_parts if i % 2 else random_parts)(rng, ORDERS[order].tiles)
        for seed in range(15):
            assert run_parts(order, parts, seed) == "done", (order, parts, seed)


@pytest.mark.parametrize("parts", [[(1, 1, 1)] * 5, [(1, 1, 0)] * 4, [(2, 1, 2), (1, 0, 1), (3, 3, 0), (1, 1, 1)]])
def test_mma_parts_of_one_step(parts):
    for order in ("d64", "d128"):
        for seed in range(200):
            assert run_parts(order, parts, seed) == "done", (order, parts, seed)


@pytest.mark.parametrize("order,parts", [("d128", [(3, 2, 3), (3, 3, 3)]), ("d128_one_tile", [(3, 3, 0), (1, 1, 0)])])
def test_a_q_buffer_held_until_the_last_pv_deadlocks(order, parts):
    """With one Q buffer: the next part's first S comes before that P.V and
    needs the buffer."""
    assert all(run_parts(order, parts, seed, q_after_pv=True) == "deadlock" for seed in range(50))


@pytest.mark.parametrize("order", ["d64", "d128", "d128_one_tile"])
def test_a_last_step_forgotten_between_parts_is_found(order):
    parts = [(3, 3, 3), (3, 3, 3), (3, 3, 3)] if ORDERS[order].tiles == 2 else [(3, 3, 0)] * 3
    assert all(run_parts(order, parts, seed, keep_last=True) != "done" for seed in range(50))


@pytest.mark.parametrize("order", ["d64", "d128_one_tile"])
def test_a_lost_phase_is_reported(order):
    """As for the other orders: a softmax that skips the wait for its part's
    last P.V falls behind by a phase."""
    parts = [(3, 3, 3), (2, 2, 2), (4, 4, 4)] if ORDERS[order].tiles == 2 else [(3, 3, 0), (2, 2, 0), (4, 4, 0)]
    assert "aliased" in {run_parts(order, parts, seed, last_pv_wait=False) for seed in range(300)}


def test_the_first_loader_order_is_no_deadlock_here():
    """The Q buffer is free once the part's last S has run, so a producer that
    held the last V past the next Q load would not wait for itself (the other
    masks' order needs its flush, tests/test_pipeline_protocol.py)."""
    for seed in range(100):
        assert run_parts("d128_one_tile", [(4, 4, 0), (1, 1, 0), (3, 3, 0)], seed, flush_before_q=False) == "done"


# ------------------------------------------------------------------ weights_rows_kernel

SUM_WARPS, UNPACK_WARPS = 8, 4


class Rows:
    def __init__(self):
        b = Barrier
        self.full = [b(f"full{s}", UNPACK_WARPS) for s in range(2)]
        self.done = [b(f"done{s}") for s in range(2)]
        self.free = [b(f"free{s}", 4) for s in range(2)]
        self.rows = b("rows", SUM_WARPS)
        self.drain = b("drain")
        self.bar1 = b("bar1", SUM_WARPS)                      # the sums' named barrier
        self.sync = b("sync", SUM_WARPS + UNPACK_WARPS)       # __syncthreads
        # what the memories hold: the tile each unpacking warp last stored to a stage, the pass whose rows and constants
        # each warp brought, the tile whose scores a stage holds
        self.k = [[None] * UNPACK_WARPS for _ in range(2)]
        self.brought = [None] * SUM_WARPS
        self.scores = [None, None]
        self.issued = []   # products under way, in order


def sums(r: Rows, passes, warp: int, restart: bool):
    g, it = warp // 4, 0
    for p, nt in enumerate(passes):
        r.brought[warp] = p
        r.rows.arrive()
        r.bar1.arrive()
        yield wait(r.bar1, p)
        for i in range((g ^ (0 if restart else it)) & 1, nt, 2):
            n = it + i
            yield wait(r.done[g], n >> 1)
            yield None
            if r.scores[g] != n or any(x != p for x in r.brought):
                raise Hazard
            yield None
            r.free[g].arrive()
        it += nt
        r.sync.arrive()
        yield wait(r.sync, p)
    r.sync.arrive()   # before the TMEM is given back
    yield wait(r.sync, len(passes))


def unpack(r: Rows, passes, warp: int, reuse_wait: bool, free_wait: bool, rows_wait: bool):
    it = 0
    for p, nt in enumerate(passes):
        for i in range(nt):
            n = it + i
            s = n & 1
            if n >= 2 and reuse_wait:
                yield wait(r.done[s], (n >> 1) - 1)
            yield None
            r.k[s][warp] = n
            r.full[s].arrive()
            if warp > 0:
                continue
            if i == 0 and rows_wait:
                yield wait(r.rows, p)
            yield wait(r.full[s], n >> 1)
            if n >= 2 and free_wait:
                yield wait(r.free[s], (n >> 1) - 1)
            r.issued.append((n, p))
        it += nt
        r.sync.arrive()
        yield wait(r.sync, p)
    if warp == 0:
        r.issued.append(None)
        yield wait(r.drain, 0)
    r.sync.arrive()
    yield wait(r.sync, len(passes))


def tensor_core(r: Rows):
    while True:
        idle = 0
        while not r.issued:   # (polled: given up where nobody else can go on, which leaves a deadlock to be seen)
            idle += 1
            if idle > 4000:
                return
            yield None
        job = r.issued.pop(0)
        if job is None:
            r.drain.arrive()
            return
        n, p = job
        if any(x != n for x in r.k[n & 1]) or any(x != p for x in r.brought):
            raise Hazard
        yield None
        if any(x != n for x in r.k[n & 1]) or any(x != p for x in r.brought):
            raise Hazard
        r.scores[n & 1] = n
        yield None
        r.done[n & 1].arrive()


def run_rows(passes, seed: int, restart=False, reuse_wait=True, free_wait=True, rows_wait=True) -> str:
    """passes: the tiles of each pass of a CTA."""
    r = Rows()
    roles = [sums(r, passes, w, restart) for w in range(SUM_WARPS)]
    roles += [unpack(r, passes, w, reuse_wait, free_wait, rows_wait) for w in range(UNPACK_WARPS)]
    return interleave(roles + [tensor_core(r)], seed)


PASSES = [[1], [2], [3], [7], [1, 1], [1, 1, 1], [3, 3], [2, 5, 1], [5, 5, 4, 4], [1, 2, 1, 2], [9, 9, 2]]


@pytest.mark.parametrize("passes", PASSES, ids=str)
def test_weights_of_many_rows_complete(passes):
    for seed in range(60):
        assert run_rows(passes, seed) == "done", (passes, seed)


@pytest.mark.parametrize("mistake,passes", [
    (dict(restart=True), [3, 3]),          # the groups take stages from 0 on in each pass
    (dict(reuse_wait=False), [7]),         # K's stage written again before its product has run
    (dict(free_wait=False), [7]),          # scores written over before they are read
    (dict(rows_wait=False), [2, 2]),       # a product before the pass's rows are there
], ids=lambda x: str(x))
def test_planted_mistakes_in_the_weights_are_found(mistake, passes):
    outcomes = [run_rows(passes, seed, **mistake) for seed in range(60)]
    assert any(x != "done" for x in outcomes), outcomes


def test_barrier_counts_are_the_kernels():
    with open(os.path.join(CSRC, "fa_cache_rows.cu")) as f:
        src = f.read()
    counts = dict(re.findall(r"ptx::mbar_init\(b\.(\w+)\((?:s)?\), (\w+)\);", src))
    assert counts == {"full": str(UNPACK_WARPS), "done": "1", "free_": "4", "rows": "kWarps", "drain": "1"}
    assert "kRowsThreads = %d;" % (32 * (SUM_WARPS + UNPACK_WARPS)) in src and "kUnpackWarp = %d;" % SUM_WARPS in src
    with open(os.path.join(CSRC, "fa_cache_kernel.cuh")) as f:
        head = f.read()
    assert "constexpr int kThreads = %d;" % (32 * SUM_WARPS) in head and "kWarps = kThreads / 32;" in head
