"""The tiles, parts and plan regions of packed sequences
(exact_attention_10_gb300/csrc/fa_packed.h), compiled with g++ and checked on the
CPU (tests/packed_tiles_check.cpp) against their definition; planted mistakes in a
copy of the header must be caught."""
from __future__ import annotations

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_10_gb300", "csrc")

LENGTHS = (0, 1, 2, 15, 16, 17, 63, 127, 128, 129, 255, 256, 257, 300, 384, 500, 700)
CASES = [f"{q} {k} {c}" for q in LENGTHS for k in LENGTHS for c in (0, 1)]
_rng = random.Random(5)
for _ in range(400):
    _hkv = _rng.choice([1, 1, 2, 8])
    _n = _rng.choice([1, 1, 2, 5, 40, 300])
    _top = _rng.choice([1, 100, 129, 1000, 20000])
    _lens = [_rng.choice([0, 1, 128, 129, _rng.randint(0, _top)]) for _ in range(2 * _n)]
    CASES.append(f"batch {_hkv * _rng.choice([1, 2, 5, 8])} {_hkv} {_n} " + " ".join(map(str, _lens)))


def _run(tmp, csrc):
    exe = os.path.join(tmp, "packed_tiles_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, os.path.join(ROOT, "tests", "packed_tiles_check.cpp"), "-o", exe],
                   check=True, capture_output=True)
    return subprocess.run([exe], input="\n".join(CASES), capture_output=True, text=True)


def test_packed_tiles(tmp_path):
    r = _run(str(tmp_path), CSRC)
    assert r.returncode == 0 and r.stdout.strip() == f"ok {len(CASES)}", r.stdout


@pytest.mark.parametrize("old,new", [
    ("(at >= Lk ? Lk : at + 1)", "(at >= Lk ? Lk : at)"),                                          # the diagonal itself
    ("return n < 1 ? 1 : n;\n}\nFA_HD int key_steps", "return n;\n}\nFA_HD int key_steps"),          # rows without keys take no step
    ("const int last = first + kTile - 1 < rows - 1 ? first + kTile - 1 : rows - 1;", "const int last = first;"),
    ("(long long)kt * kTile - (Lk - (long long)Lq)", "(long long)kt * kTile"),                     # no offset
    ("return (int)((long long)n * i / parts);", "return n / parts * i;"),                          # a remainder lost
    ("(unsigned)(parts - 1) << 28", "(unsigned)parts << 28"),
    ("z.Tk / kTile + (long long)z.S", "(z.Tk + kTile - 1ll) / kTile"),                             # room for one sequence
    ("(z.Tq / kTile + 1ll) * (z.H / z.Hkv)", "(z.Tq / kTile + 1ll)"),                              # the group's steps
    ("capacity(z, l) * heads_of(z, l) + kOrderGrid", "capacity(z, l) * heads_of(z, l)"),            # a last, partial round
    ("n >= kTile ? kTile / 16 : (n + 15) / 16", "n >= kTile ? kTile / 16 : n / 16 + 1"),
    ("table_word(z) + capacity(z, 1) + 1", "table_word(z) + capacity(z, 1) - 1"),
])
def test_planted_mistakes_are_caught(tmp_path, old, new):
    csrc = os.path.join(str(tmp_path), "csrc")
    shutil.copytree(CSRC, csrc)
    path = os.path.join(csrc, "fa_packed.h")
    with open(path) as f:
        src = f.read()
    assert src.count(old) == 1, old
    with open(path, "w") as f:
        f.write(src.replace(old, new))
    r = _run(str(tmp_path), csrc)
    assert r.returncode != 0, r.stdout
