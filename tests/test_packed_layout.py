"""Host-side sizes of the packed calls, from the library's own code.

Where a plan's parts lie in its buffer: what a kernel reads of a plan before its
header has shown whose it is must lie in every plan, also in one of a smaller
batch.  And the blocks of the backward pass's pre-pass, and the sizes
that the queries answer."""
import itertools
import os
import subprocess

import pytest

from video_dit_long_gb300 import build as B

SOURCE = r"""
#include <cstdio>
#include "k6_packed.cuh"
// lines of: H kv_heads n_seq q_tokens k_tokens sms
int main() {
    int H, kv, n, sms;
    long q, k;
    while (scanf("%d %d %d %ld %ld %d", &H, &kv, &n, &q, &k, &sms) == 6) {
        k6::Geom g = {};
        g.H = H, g.d = 128;
        const k6attn_packed b = {n, kv, 1, q, k};
        const k6::PackedGeom p = k6::packed_geom(g, b, sms);
        const k6::PackedPlan at = k6::packed_plan_at(nullptr, p);
        k6attn_handle h;
        h.g = g, h.g.dtype = K6ATTN_BF16, h.sms = sms, h.device = 5;  // never the current one
        printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %d %u %u %zu %zu %zu %zu %zu %zu\n", k6::packed_plan_bytes(p), k6::packed_plan_common_bytes(sms),
               (size_t)at.count, (size_t)at.merge, (size_t)at.fwd, (size_t)at.sched, (size_t)at.q, (size_t)at.k,
               sizeof(k6::PackedMerge), p.cap_merge, k6::packed_bwd_rows_blocks(p, true),
               k6::packed_bwd_rows_blocks(p, false), k6attn_packed_plan_bytes(&h, &b),
               k6attn_packed_workspace_bytes(&h, &b), k6::packed_fwd_workspace(p),
               k6attn_packed_backward_workspace_bytes(&h, &b), k6::packed_bwd_workspace(p),
               k6attn_packed_norm_rope_backward_workspace_bytes(&h, q, kv));
    }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    lib = B.build()
    d = tmp_path_factory.mktemp("layout")
    (d / "layout.cu").write_text(SOURCE)
    cmd = [B.NVCC, *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "layout.cu"), "-o", str(d / "layout"), lib,
           "-Xlinker", "-rpath," + os.path.dirname(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "layout")


CASES = [(H, kv, n, q, k, sms)
         for (H, kv), (n, q, k), sms in itertools.product(
             [(1, 1), (4, 2), (24, 1), (24, 8), (24, 24), (128, 1)],
             [(1, 0, 1), (1, 1, 1), (3, 208, 208), (12, 12, 150000), (2, 864, 13824), (1, 25920, 25920), (2000, 9000, 9000)],
             [152, 7, 512])]


def sizes(program, cases):
    text = "\n".join(" ".join(map(str, c)) for c in cases)
    out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(cases)
    return [list(map(int, line.split())) for line in out]


def test_every_plan_holds_what_is_read_before_its_header_is_checked(program):
    common = {}
    for c, got in zip(CASES, sizes(program, CASES)):
        size, shared, count, merge, fwd, sched, q, k, each, cap = got[:10]
        sms = c[-1]
        # the same places in every plan of a GPU: header, counts, the first `sms` split tiles
        assert common.setdefault(sms, (shared, count, merge)) == (shared, count, merge)
        assert count == 256 and merge >= count + 4 * sms and merge % 16 == 0
        assert merge + sms * each == shared <= size, c
        # and room for all of this batch's split tiles, in front of the lists whose places depend on the batch
        assert merge + max(cap, sms) * each <= fwd <= sched <= q <= k <= size, c


def test_the_pre_pass_of_few_queries_over_long_caches_fills_the_gpu(program):
    """With fp16 q and k it takes the norms of every row of v, whatever the number of queries."""
    for H, kv, k in ((24, 4, 134000), (8, 1, 52360), (24, 24, 9000)):
        (got,) = sizes(program, [(H, kv, 3, 12, k, 152)])
        assert got[10] >= 2 * 152, (H, kv, k, got[10])
        assert 1 <= got[11] <= got[10]


def test_sizes_are_host_arithmetic_whichever_device_is_current(program):
    """The queries need no device: they answer for a handle whose device is not the current one, or without any."""
    cases = [c for c in CASES if c[3] > 0]
    for c, got in zip(cases, sizes(program, cases)):
        plan, fwd, fwd_want, bwd, bwd_want, norm = got[12:]
        assert (plan, fwd, bwd) == (got[0], fwd_want, bwd_want), c
        assert plan > 0 and bwd > 0 and norm > 0, c
