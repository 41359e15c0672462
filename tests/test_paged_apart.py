"""Host-side answers that tests of ranges leave open, from the library's own code: exactly which pools of one tensor share
bytes, also at distances of part of a row; and that what the calls over pages read of a plan before its header has shown
whose it is lies in every plan, one of packed sequences included."""
import itertools
import random

import pytest

from . import test_packed_layout as L
from .test_packed_layout import program  # noqa: F401  (a fixture)
from .test_paged_layout import run  # noqa: F401  (a fixture)

HALF = 64  # elements of half a row


def half_rows(n, strides, at):
    """The half rows of a pool: n heads, tokens and pages; strides and place in half rows."""
    return {at + h * strides[0] + t * strides[1] + p * strides[2] + half for h in range(n[0]) for t in range(n[1])
            for p in range(n[2]) for half in (0, 1)}


# heads 4, tokens 16, pages 10; page, token and head strides in elements, distance of the values from the keys
H, T, N = 4, 16, 10
ROW = 128 * H
LAYOUTS = [("pages", (2 * T * ROW, ROW, 128), T * ROW), ("tokens", (2 * T * ROW, 2 * ROW, 128), ROW),
           ("heads", (2 * T * ROW, 2 * ROW, 256), 128), ("apart", (T * ROW, ROW, 128), N * T * ROW)]


@pytest.mark.parametrize("name,strides,d", LAYOUTS, ids=[x[0] for x in LAYOUTS])
def test_keys_and_values_of_one_tensor(run, name, strides, d):  # noqa: F811
    """Half a row further on they share bytes, but where the pools lie one behind the other."""
    places = [d, -d, d + HALF, d - HALF, -d + HALF, -d - HALF]
    keys = half_rows((H, T, N), [s // HALF for s in strides[::-1]], 0)
    want = [int(bool(keys & half_rows((H, T, N), [s // HALF for s in strides[::-1]], x // HALF))) for x in places]
    assert want == ([0, 0, 0, 1, 1, 0] if name == "apart" else [0, 0, 1, 1, 1, 1])
    line = " ".join(map(str, (H, T, N, *strides, *strides)))
    assert run([f"pools {line} {x}" for x in places]) == [[0, 0, x] for x in want]


def test_distances_of_part_of_a_row(run):  # noqa: F811
    """Pools of any order and gaps, an odd number of half rows apart: an overlap is never missed."""
    rng = random.Random(4)
    lines, want = [], []
    for _ in range(3000):
        n = [rng.randint(1, 3) for _ in range(3)]
        w, strides = 2, [0, 0, 0]
        for i in rng.sample(range(3), 3):
            strides[i] = w * rng.choice([1, 1, 2, 3]) + rng.choice([0, 0, 1])
            w = strides[i] * n[i]
        d = 2 * rng.randint(-w, w) + 1 if rng.random() < 0.8 else rng.choice(strides) // 2
        want.append(bool(half_rows(n, strides, 0) & half_rows(n, strides, d)))
        s = [HALF * x for x in strides[::-1]]
        lines.append("pools " + " ".join(map(str, (*n, *s, *s, HALF * d))))
    seen = {True: 0, False: 0}
    for line, overlap, (sx, sy, shared) in zip(lines, want, run(lines)):
        assert (sx, sy) == (0, 0), line
        assert shared or not overlap, line
        seen[overlap] += 1
        seen[bool(shared), overlap] = seen.get((bool(shared), overlap), 0) + 1
    assert min(seen[True], seen[False]) > 300
    assert seen[False, False] > 100  # and not everything counts as one


def test_every_plan_has_room_for_what_a_call_over_pages_reads_first(program, run):  # noqa: F811
    """Header, counts, and each CTA's first item and join: a plan of packed sequences passed by mistake is read no further
    than it reaches."""
    for c, got in zip(L.CASES, L.sizes(program, L.CASES)):
        sms = c[-1]
        read = 256 + (4 * sms + 15) // 16 * 16 + sms * (32 + 48)
        assert got[0] >= read, c
    cases = [(1, 1, 1, 0, 16, 1, 0, sms) for sms in (152, 7, 512)]
    for c, got in zip(cases, run(["geom " + " ".join(map(str, c)) for c in cases])):
        assert got[18] == 48 and got[0] >= got[3] + 48 * c[-1] == 256 + (4 * c[-1] + 15) // 16 * 16 + c[-1] * (32 + 48)
