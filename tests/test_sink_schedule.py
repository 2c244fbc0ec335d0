"""The forward's work decomposition for causal windows with sinks
(exact_attention_10_gb300/csrc/fa_schedule.h, SinkSchedule), compiled with g++
and checked exhaustively on the CPU (tests/sink_schedule_check.cpp); a planted
mistake in a copy of the header must be caught."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_10_gb300", "csrc")

CASES = []
for N, Nkv in ((1, 1), (1, 700), (129, 129), (300, 300), (1000, 1000), (2048, 2048), (3000, 3000), (64, 5000),
               (513, 200), (200, 70), (300, 2000), (1, 65536), (130, 4096)):
    for left in (-1, 0, 1, 63, 127, 128, 255, 600, 1023, 5000):
        for sinks in (0, 1, 4, 127, 128, 129, 300, 1 << 30):
            for BH in (1, 7):
                for sms in (7, 152):
                    for mode in (0, 1, 2):
                        CASES.append((N, Nkv, BH, sms, mode, left, sinks))
CASES += [(N, N, 32, 152, mode, left, 4) for N in (4096, 8192) for left in (255, 1023, 4095) for mode in (0, 1, 2)]


def _run(tmp, csrc, cases):
    exe = os.path.join(tmp, "sink_schedule_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, os.path.join(ROOT, "tests", "sink_schedule_check.cpp"), "-o",
                    exe], check=True, capture_output=True)
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    return subprocess.run([exe], input=text, capture_output=True, text=True)


def test_sink_schedules(tmp_path):
    r = _run(str(tmp_path), CSRC, CASES)
    assert r.returncode == 0 and r.stdout.strip() == f"ok {len(CASES)}", r.stdout


@pytest.mark.parametrize("old,new", [
    ("r.ks = a < r.ssz ? r.ssz : a;", "r.ks = a;"),                               # the sinks' steps run twice
    ("s.ss = (s.sinks + kSchedBN - 1) / kSchedBN;", "s.ss = s.sinks / kSchedBN;"),   # the last sinks' tile left out
    ("(j < ssz ? j : j - ssz + ks)", "(j < ssz ? j : j + ks)"),                   # steps left out after the sinks
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
