"""The tile sequence that the whole-tile kernel runs for causal windows with
sinks (exact_attention_10_gb300/csrc/fa_schedule.h, sched_next_whole), compiled
with g++ and checked on the CPU (tests/sink_tiles_check.cpp) against the
sequence that tests/test_sink_schedule.py checks; planted mistakes in a copy of
the header must be caught."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_10_gb300", "csrc")

CASES = [(N, Nkv, BH, sms, left, sinks)
         for N, Nkv in ((1, 1), (1, 700), (129, 129), (300, 300), (1000, 1000), (2048, 2048), (2900, 2900), (64, 5000),
                        (513, 200), (200, 70), (300, 2000), (1, 65536), (130, 4096))
         for left in (-1, 0, 1, 63, 127, 128, 129, 255, 600, 5000)
         for sinks in (0, 1, 4, 15, 16, 17, 128, 300, 1 << 30)
         for BH in (1, 3, 7, 32, 1000)
         for sms in (7, 152)]
# tiles times heads next to 2^40, where the multiplication gives way to a division
CASES += [(N, 300, BH, 152, 100, 4) for N, BH in ((1, (1 << 20) - 1), (1, 1 << 20), (300, 741455), (300, 741456),
                                                 (300, 3_000_000))]


def _run(tmp, csrc, cases):
    exe = os.path.join(tmp, "sink_tiles_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, os.path.join(ROOT, "tests", "sink_tiles_check.cpp"), "-o",
                    exe], check=True, capture_output=True)
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    return subprocess.run([exe], input=text, capture_output=True, text=True)


def test_sink_tiles(tmp_path):
    r = _run(str(tmp_path), CSRC, CASES)
    assert r.returncode == 0 and r.stdout.strip() == f"ok {len(CASES)}", r.stdout


@pytest.mark.parametrize("old,new", [
    ("s.inv = ((1ull << 40) + (unsigned long long)BH - 1) /", "s.inv = (1ull << 40) /"),           # rounded down
    ("if ((double)s.T * BH < 1099511627776.0)", "if (true)"),                                    # past its range
    ("ct = s.rev ? q : s.C - 1 - q;\n}\n\n// PartIter's", "ct = q;\n}\n\n// PartIter's"),           # rows in the other order
    ("    it.t = it.u * s.G + ((it.u & 1) ? s.G - 1 - it.c : it.c);", "    it.t = it.u * s.G + it.c;"),   # no serpentine
    ("s.sinks <= kSchedFewSinks && a >= 1;", "s.sinks <= kSchedFewSinks && a1 >= 1;"),              # a row's window reaches in
    ("r.few = r.ssz == 1 && s.sinks <= kSchedFewSinks", "r.few = r.ssz == 1 && s.sinks <= kSchedBN"),
    ("r.few = r.ssz == 1 && s.sinks", "r.few = s.sinks"),                                           # tiles without sinks
])
def test_planted_mistakes_are_caught(tmp_path, old, new):
    csrc = os.path.join(str(tmp_path), "csrc")
    shutil.copytree(CSRC, csrc)
    path = os.path.join(csrc, "fa_schedule.h")
    with open(path) as f:
        src = f.read()
    assert src.count(old) == 1, old
    with open(path, "w") as f:
        f.write(src.replace(old, new))
    r = _run(str(tmp_path), csrc, CASES)
    assert r.returncode != 0, r.stdout
