"""Where a new token lies among its stream's keys, from the library's own code: lengths and offsets come from the device
and may be any int, and none of them may lead behind the table."""
import os
import subprocess

import pytest

from video_dit_long_gb300 import build as B

SOURCE = r"""
#include <cstdio>
#include "k6_paged.cuh"
// lines of: Tk t end Lk
int main() {
    k6::PagedGeom g = {};
    int t, end, Lk;
    while (scanf("%d %d %d %d", &g.g.Tk, &t, &end, &Lk) == 4) printf("%d\n", k6::paged_position(g, t, end, Lk));
}
"""


@pytest.fixture(scope="module")
def positions(tmp_path_factory):
    d = tmp_path_factory.mktemp("lengths")
    (d / "lengths.cu").write_text(SOURCE)
    cmd = [B.NVCC, *B.ARCH, "-std=c++17", "-Xcompiler", "-fsanitize=signed-integer-overflow,-fno-sanitize-recover", "-I",
           B.INCLUDE, "-I", B.CSRC, str(d / "lengths.cu"), "-o", str(d / "lengths"), "-Xlinker", "-lubsan"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode and "ubsan" in r.stderr:  # a compiler without the check of overflows
        cmd = [x for x in cmd if "sanitize" not in x and "ubsan" not in x and x not in ("-Xcompiler", "-Xlinker")]
        r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        r = subprocess.run([str(d / "lengths")], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True,
                           text=True)
        assert r.returncode == 0, r.stderr
        return list(map(int, r.stdout.split()))

    return run


def test_a_position_is_in_the_table_or_none(positions):
    """A length below zero is no length, however far: the least int less one token is the largest int."""
    top = 2 ** 31 - 1
    ints = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 15, -2 ** 30, -1, 0, 1, 15, 16, 17, 47, 48, 49, 2 ** 29, top - 1, top]
    cases = [(Tk, t, end, Lk) for Tk in (16, 48, 2 ** 29 - 16) for t in (0, 1, 15, 500) for end in ints if t < end for Lk in ints]
    assert len(cases) > 1000
    for (Tk, t, end, Lk), got in zip(cases, positions(cases)):
        want = Lk - (end - t)
        assert got == (want if 0 <= Lk <= Tk and want >= 0 else -1), (Tk, t, end, Lk)
        assert got < Tk
