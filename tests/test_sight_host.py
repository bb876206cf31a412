"""The order in which the windowed attention's tiles hold what is seen: the kernels' own struct (csrc/sight.cuh), compiled for
the host, against the oracle's masks."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import kv as okv
from tests.kv_cases import random_tree

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_verification_38_gb300", "csrc")
NOWHERE = 2**31 - 1

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    """places([(T, L, window, sinks, box_log)]): a list of whole numbers for each."""
    exe = str(tmp_path_factory.mktemp("sight") / "sight")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC, "-x", "c++",
                    os.path.join(HERE, "sight_places.cpp"), "-o", exe], check=True)

    def run(cases):
        text = "".join("%d %d %d %d %d\n" % c for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        out = [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
        assert len(out) == len(cases)
        return out

    return run


@pytest.mark.parametrize("as_tree", [False, True])
@pytest.mark.parametrize("box_log", [0, 3, 4])
def test_places_hold_what_is_seen_once(places, box_log, as_tree):
    r = np.random.default_rng(box_log)
    cases, parents = [], []
    for i in range(1500):
        T = int(r.integers(1, 129)) if r.random() < 0.5 else int(r.integers(1, 12))
        window = int(r.integers(1, 700)) if r.random() < 0.6 else int(r.integers(1, 10))
        cases.append((T, T + int(r.integers(0, 600)), window, int(r.choice([0, 0, 1, 4, 16, 17, 100, 900])), box_log))
        parents.append(random_tree(T, i) if as_tree else None)
    box = 1 << box_log
    for (T, L, window, sinks, _), parent, x in zip(cases, parents, places(cases)):
        (s1, i1, end, lo, tail), past = x[:5], x[-2:]
        pos, said = np.array(x[5:-2:2]), np.array(x[6:-2:2])
        assert past == [NOWHERE, NOWHERE] and len(pos) == end and 0 <= s1 <= i1 <= end
        assert (pos >= 0).all() and len(set(pos.tolist())) == end
        assert (pos[::box] % box == 0).all() and end % box == 0
        assert (pos.reshape(-1, box) == pos[::box, None] + np.arange(box)).all()  # whole boxes, as they lie
        see = okv.sight(T, L, parent, window, sinks)
        seen = np.zeros(max(L, pos.max() + 1), dtype=bool)
        seen[:L] = see.any(0)
        assert seen.sum() == seen[pos].sum()  # nothing seen is left out
        assert seen[pos].reshape(-1, box).any(1).all()  # and no box is loaded for nothing
        assert np.array_equal(said, seen[pos])
        inner = pos[s1:i1]
        assert seen[inner[inner < L]].all()  # (a whole tile of these is not looked at position by position)
        early = pos[:tail][pos[:tail] < L]  # before `tail`, a position is seen by every row or by none
        assert (see[:, early].all(0) | ~see[:, early].any(0)).all()


def test_largest_sizes_stay_in_range(places):
    """Lengths, windows and sinks up to the limits of a cache and of a call: no sum passes 32 bits (the sanitizer's word), and
    the list is as long as it must be."""
    top = 2**30
    cases = [(T, L, window, sinks, box_log) for T in (1, 128) for L in (128, top - 1, top) for window in (1, 4096, top - 1, top)
             for sinks in (0, 5, top) for box_log in (0, 4)]
    for (T, L, window, sinks, box_log), x in zip(cases, places(cases)):
        s1, i1, end, lo, tail = x[:5]
        first = max(0, L - T + 1 - window)
        exact = L - first + min(sinks, first)
        assert lo == first and exact <= end < exact + 3 * (1 << box_log) and 0 <= s1 <= i1 <= end and tail <= end
