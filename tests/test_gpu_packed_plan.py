"""The lists that the plan kernel wrote, read back: every query tile of every key
head is covered once over the keys it sees, whether the batch is cut into one
stretch per SM or dealt out; the backward pass's tiles once; and a plan whose
lists were too short is reported."""
import collections
import os
import subprocess

import pytest

from video_dit_long_gb300 import build as B

from .test_packed_plan import limit

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SOURCE = r"""
#include <cstdio>
#include <vector>
#include "k6_packed.cuh"
// argv-free: H kv_heads block q_tokens k_tokens sms rows n_seq, then n_seq + 1 offsets of q and of k.  rows > 0: forward
// lists cut to that many items per CTA.  Prints the error word, the geometry and places, then the plan's words.
int main() {
    int H, kv, block, sms, rows, n;
    long q, k;
    if (scanf("%d %d %d %ld %ld %d %d %d", &H, &kv, &block, &q, &k, &sms, &rows, &n) != 8) return 1;
    std::vector<int> cu(2 * (n + 1));
    for (int &x : cu)
        if (scanf("%d", &x) != 1) return 1;
    k6::Geom g = {};
    g.H = H, g.d = 128;
    const k6attn_packed b = {n, kv, block, q, k};
    k6::PackedGeom p = k6::packed_geom(g, b, sms);
    if (rows > 0 && rows < p.cap_rows) p.cap_rows = rows;  // the buffer keeps its size
    const size_t bytes = k6::packed_plan_bytes(p);
    int *d_cu, *d_err, err = -1;
    char *d_plan;
    if (cudaMalloc(&d_cu, cu.size() * 4) || cudaMalloc(&d_err, 4) || cudaMalloc(&d_plan, bytes)) return 2;
    cudaMemcpy(d_cu, cu.data(), cu.size() * 4, cudaMemcpyHostToDevice);
    cudaMemset(d_err, 0, 4);
    cudaMemset(d_plan, 255, bytes);
    if (k6::launch_packed_plan(p, d_cu, d_cu + n + 1, d_plan, d_err, 0)) return 3;
    if (cudaDeviceSynchronize()) return 4;
    std::vector<int> plan(bytes / 4);
    cudaMemcpy(&err, d_err, 4, cudaMemcpyDeviceToHost);
    cudaMemcpy(plan.data(), d_plan, bytes, cudaMemcpyDeviceToHost);
    const k6::PackedPlan at = k6::packed_plan_at(nullptr, p);
    printf("%d %d %d %d %d %zu %zu %zu %zu %zu %zu\n", err, p.tpt, p.cap_rows, p.cap_slots, p.cap_merge, (size_t)at.count / 4,
           (size_t)at.merge / 4, (size_t)at.fwd / 4, (size_t)at.sched / 4, (size_t)at.q / 4, (size_t)at.k / 4);
    for (int x : plan) printf("%d\n", x);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib = B.build()
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cu").write_text(SOURCE)
    cmd = [B.NVCC, *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "plan.cu"), "-o", str(d / "plan"), lib,
           "-Xlinker", "-rpath," + os.path.dirname(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(d / "plan")


Head = collections.namedtuple("Head", "magic n_seq H Hkv block Tq Tk n_fwd n_merge n_q n_k stream slot_step q_lo q_hi k_lo "
                                      "k_hi bad")


def offsets(lens, first=0):
    out = [first]
    for x in lens:
        out.append(out[-1] + x)
    return out


def made(program, q, k, H, kv, block, rows=0, sms=152, first=0):
    cq, ck = offsets(q, first), offsets(k, first)
    text = f"{H} {kv} {block} {cq[-1] + 2} {ck[-1] + 2} {sms} {rows} {len(q)} " + " ".join(map(str, cq + ck))
    r = subprocess.run([program], input=text, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    lines = r.stdout.split("\n")
    return list(map(int, lines[0].split())), list(map(int, lines[1:-1])), cq, ck


def check(program, q, k, H, kv, block, stream, sms=152):
    (err, tpt, cap_rows, cap_slots, cap_merge, count, merge, fwd, sched, at_q, at_k), w, cq, ck = made(program, q, k, H, kv,
                                                                                                       block, sms=sms, first=3)
    h = Head(*w[:18])
    G = H // kv
    assert err == 0 and not h.bad and h.stream == stream and tpt == 128 // G
    assert (h.q_lo, h.q_hi, h.k_lo, h.k_hi) == (cq[0], cq[-1], ck[0], ck[-1])
    # what every tile of the batch must be covered by: its first token -> (tokens, first key row, keys, position, key tiles)
    tiles = {}
    for s, (lq, lk) in enumerate(zip(q, k)):
        for t in range(0, lq, tpt):
            n = min(tpt, lq - t)
            hi = (limit(t + n - 1 + lk - lq, lk, block) + 127) // 128
            tiles[cq[s] + t] = (n, ck[s], lk, t + lk - lq, hi)
    item = lambda base, i: w[base + 8 * i:base + 8 * i + 8]  # noqa: E731
    # forward: pieces of each (tile, key head)
    pieces = collections.defaultdict(list)

    def take(it, hk):
        tok0, n_hk, krow0, lk, pos0, a, b, slot = it
        assert (n_hk & 255, krow0, lk, pos0) == tiles[tok0][:4]
        pieces[tok0, hk].append((a, b, slot))

    if stream:
        for sm in range(sms):
            assert 0 <= w[count + sm] <= cap_rows
            for i in range(w[count + sm]):
                it = item(fwd, sm * cap_rows + i)
                take(it, it[1] >> 8)
    else:
        units = [w[sched + i] for i in range(-(-h.n_fwd * kv // sms) * sms)]
        assert sorted(u for u in units if u >= 0) == list(range(h.n_fwd * kv))
        for u in units:
            if u >= 0:
                take(item(fwd, u % h.n_fwd), u // h.n_fwd)
    assert set(pieces) == {(t, hk) for t in tiles for hk in range(kv)}
    slots, joins = set(), {}
    for i in range(h.n_merge):
        tok0, n_hk, slot0, n = w[merge + 4 * i:merge + 4 * i + 4]
        joins[tok0, n_hk >> 8] = (n_hk & 255, slot0, n)
    assert len(joins) == h.n_merge <= cap_merge
    for (tok0, hk), got in pieces.items():
        got.sort()
        hi = tiles[tok0][4]
        assert got[0][0] == 0 and got[-1][1] == hi and all(x[1] == y[0] for x, y in zip(got, got[1:]))
        if len(got) == 1:
            assert got[0][2] == -1 and (tok0, hk) not in joins
            continue
        n, slot0, m = joins.pop((tok0, hk))
        assert (n, m) == (tiles[tok0][0], len(got))
        # the place of a piece's partial, as the attention kernel and the join find it
        mine = [slot * h.slot_step + (hk if h.slot_step > 1 else 0) for _, _, slot in got]
        assert mine == [slot0 + c * h.slot_step for c in range(m)]
        assert all(0 <= x < cap_slots for x in mine) and not slots & set(mine)
        slots |= set(mine)
    assert not joins
    # backward: query tiles and key tiles, unsplit
    got = {}
    for i in range(h.n_q):
        tok0, n, krow0, lk, pos0, a, b, slot = item(at_q, i)
        got[tok0] = (n, krow0, lk, pos0, b)
        assert a == 0 and slot == -1
    assert got == tiles and h.n_q == len(tiles)
    want, got = {}, {}
    for s, (lq, lk) in enumerate(zip(q, k)):
        for t in range(0, lk, 128):
            first = 0 if block == 0 else max(0, t // block * block - (lk - lq))
            hi = -(-lq // tpt)
            want[ck[s] + t] = (min(128, lk - t), t, cq[s], lq, lk - lq, min(first // tpt, hi), hi)
    for i in range(h.n_k):
        krow0, *rest = item(at_k, i)
        got[krow0] = tuple(rest)
    assert got == want and h.n_k == len(want)
    return h


LONG = [1, 52360, 300, 8192, 129, 26440, 5000, 4352, 1000, 3152, 12345, 20000]


@pytest.mark.parametrize("q,k,H,kv,block", [
    ([77, 1, 130], [77, 1, 130], 24, 8, 1), ([1] * 12, LONG, 24, 4, 1), ([432, 432], [3024, 10800], 24, 8, 432),
    ([4352, 3152, 1081, 257, 77, 1], [4352, 3152, 1081, 257, 77, 1], 24, 8, 1), ([300, 0, 2], [10, 40, 1], 6, 6, 7),
    ([0, 5, 0], [0, 0, 9], 4, 2, 0), ([3152, 1081], [3152, 1081], 24, 1, 0), ([1], [1], 128, 1, 0),
])
def test_stretches(program, q, k, H, kv, block):
    check(program, q, k, H, kv, block, stream=1)


@pytest.mark.parametrize("q,k,H,kv,block", [
    ([25920], [25920], 24, 8, 1620), ([512] * 30 + [9000], [512] * 30 + [9000], 24, 24, 1),
    ([3, 0, 9] * 500 + [2], [4, 1, 9] * 500 + [20000], 4, 2, 1), ([16000], [16000], 24, 3, 0),
])
def test_dealt_out(program, q, k, H, kv, block):
    check(program, q, k, H, kv, block, stream=0)


def test_a_plan_without_room_is_a_bad_one(program):
    """The lists' sizes are upper bounds; were one too short after all, its items must not go missing silently."""
    q = [4352, 3152, 1081, 257, 77, 1]
    head, w, *_ = made(program, q, q, 24, 8, 1, rows=2)
    assert head[2] == 2 and Head(*w[:18]).bad == 1 and head[0] == 4  # the error word: a bad plan
    head, w, *_ = made(program, q, q, 24, 8, 1)
    assert Head(*w[:18]).bad == 0 and head[0] == 0
