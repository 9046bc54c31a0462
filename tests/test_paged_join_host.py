"""The join of paged attention reads a pair's partials by a record in the workspace. Where
a bounded wait ran out, its CTA leaves further pairs without one, and the workspace's
former contents stand there: the rule that tells them apart, compiled for the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp4_kv_cache_step_b200", "csrc")

SOURCE = """
#include "paged_join.h"
extern "C" int holds(int first, int last, int slot, int pieces) {
  return csa2::join_record_holds(first, last, slot, pieces);
}
extern "C" int slot_of(int i, int first, int slot) { return csa2::join_slot(i, first, slot); }
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("join")
    (d / "rule.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "rule.cpp"), "-o",
                    str(d / "rule.so")], check=True)
    return ctypes.CDLL(str(d / "rule.so"))


@pytest.mark.parametrize("pieces", [1, 2, 3, 7, 148])
def test_records_of_a_line_hold(rule, pieces):
    """Pairs of any lengths, cut into equal pieces: what the planner writes is accepted,
    and the partials of different pairs never share a slot."""
    r = np.random.RandomState(pieces)
    for _ in range(50):
        units = 5 + r.randint(0, 60, r.randint(1, 40))
        total = int(units.sum())
        n = min(pieces, total)
        begin = [i * total // n for i in range(n + 1)]
        at, taken, seen = 0, set(), [0] * n                  # seen: segments of a piece so far
        for u in units:
            held = [i for i in range(n) if max(begin[i], at) < min(begin[i + 1], at + int(u))]
            first, last = held[0], held[-1]
            slot = 2 * first + (1 if seen[first] else 0)
            for i in held:
                seen[i] += 1
            at += int(u)
            assert rule.holds(first, last, slot, pieces)
            if first == last:
                continue
            slots = {rule.slot_of(i, first, slot) for i in range(first, last + 1)}
            assert len(slots) == last - first + 1 and not slots & taken
            assert min(slots) >= 0 and max(slots) < 2 * pieces
            taken |= slots


@pytest.mark.parametrize("pieces", [1, 5, 148])
def test_former_contents_never_lead_outside(rule, pieces):
    """Bytes of other calls: what is accepted stays inside the 2 * pieces slots."""
    r = np.random.RandomState(3 + pieces)
    edges = [-2 ** 31, -2, -1, 0, 1, pieces - 1, pieces, 2 * pieces - 1, 2 * pieces, 2 ** 30,
             2 ** 31 - 1, 0x7f7f7f7f, 0x3f800000]
    words = np.concatenate([r.randint(-2 ** 31, 2 ** 31, (2000, 3)),
                            r.randint(-2, 2 * pieces + 2, (4000, 3)), r.choice(edges, (4000, 3))])
    for first, last, slot in words.tolist():
        if not rule.holds(first, last, slot, pieces):
            continue
        assert 0 <= first <= last < pieces
        for i in (first, min(first + 1, last), last):
            assert 0 <= rule.slot_of(i, first, slot) < 2 * pieces
    for bad in ((0, pieces, 0), (-1, 0, -2), (1, 0, 2), (0, 0, 2), (0, 0, -1),
                (0x7f7f7f7f, 0x7f7f7f7f, 0x7f7f7f7f)):
        assert not rule.holds(*bad, pieces)
