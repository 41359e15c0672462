"""The lists that the paged plan wrote, read back: every query tile of every key
head is covered once over the keys it sees, its own and those its group shares;
partials and joins stay within what the host allots; every new token has its place."""
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
#include "k6_paged.cuh"
// H kv block q_tokens page max_pages n_pages sms n_seq n_groups, then cu_q, k_lens, cu_groups and shared (with groups).
// Stream s's pages are s * max_pages and on.  Prints the error word, the geometry and places, then the plan's words.
int main() {
    int H, kv, block, page, cols, sms, n, groups;
    long q, pages;
    if (scanf("%d %d %d %ld %d %d %ld %d %d %d", &H, &kv, &block, &q, &page, &cols, &pages, &sms, &n, &groups) != 10) return 1;
    std::vector<int> x(n + 1 + n + (groups ? groups + 1 + groups : 0)), table((size_t)n * cols);
    for (int &y : x)
        if (scanf("%d", &y) != 1) return 1;
    for (size_t i = 0; i < table.size(); i++) table[i] = (int)i;
    k6::Geom g = {};
    g.H = H, g.d = 128;
    const k6attn_paged b = {n, kv, block, page, cols, groups, pages, q};
    const k6::PagedGeom p = k6::paged_geom(g, b, sms);
    const size_t bytes = k6::paged_plan_bytes(p);
    int *d_x, *d_t, *d_err, err = -1;
    char *d_plan;
    if (cudaMalloc(&d_x, x.size() * 4) || cudaMalloc(&d_t, table.size() * 4) || cudaMalloc(&d_err, 4) || cudaMalloc(&d_plan, bytes))
        return 2;
    cudaMemcpy(d_x, x.data(), x.size() * 4, cudaMemcpyHostToDevice);
    cudaMemcpy(d_t, table.data(), table.size() * 4, cudaMemcpyHostToDevice);
    cudaMemset(d_err, 0, 4);
    cudaMemset(d_plan, 255, bytes);
    int *cg = groups ? d_x + 2 * n + 1 : nullptr;
    if (k6::launch_paged_plan(p, d_x, d_x + n + 1, d_t, cg, groups ? cg + groups + 1 : nullptr, d_plan, d_err, 0)) return 3;
    if (cudaDeviceSynchronize()) return 4;
    std::vector<int> plan(bytes / 4);
    cudaMemcpy(&err, d_err, 4, cudaMemcpyDeviceToHost);
    cudaMemcpy(plan.data(), d_plan, bytes, cudaMemcpyDeviceToHost);
    const k6::PagedPlan at = k6::paged_plan_at(nullptr, p);
    printf("%d %d %d %d %d %ld %zu %zu %zu %zu %zu %zu %zu\n", err, p.g.tpt, p.g.cap_rows, p.g.cap_merge, p.cap_prefix, p.cap_part,
           (size_t)at.count / 4, (size_t)at.first / 4, (size_t)at.merge / 4, (size_t)at.prefix / 4, (size_t)at.fwd / 4,
           (size_t)at.sched / 4, (size_t)at.slot / 4);
    for (int y : plan) printf("%d\n", y);
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
                                      "k_hi bad page n_pages max_pages n_groups")


def check(program, q, k, H, kv, block, stream, groups=(), taken=(), page=16, sms=152, first=2):
    """taken: for each group the key tiles that the plan should take together, 0 for none."""
    cols = max(-(-x // page) for x in k) + 1
    cq = [first]
    for x in q:
        cq.append(cq[-1] + x)
    cg = [0]
    for n, _ in groups:
        cg.append(cg[-1] + n)
    numbers = cq + k + (cg + [x for _, x in groups] if groups else [])
    text = f"{H} {kv} {block} {cq[-1] + 3} {page} {cols} {len(q) * cols} {sms} {len(q)} {len(groups)} " + " ".join(map(str, numbers))
    r = subprocess.run([program], input=text, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    lines = r.stdout.split("\n")
    err, tpt, cap_rows, cap_merge, cap_prefix, cap_part, count, at_first, merge, prefix, fwd, sched, slot = map(int, lines[0].split())
    w = list(map(int, lines[1:-1]))
    h = Head(*w[:22])
    G = H // kv
    assert err == 0 and not h.bad and h.stream == stream and (h.q_lo, h.q_hi) == (cq[0], cq[-1])
    # what must be covered: (row of the table, first token) -> tokens, keys, key tiles, and of a group
    lo = [0] * len(q)
    group_of = [None] * len(q)
    tiles = {}
    for g, ((n, _), t) in enumerate(zip(groups, taken)):
        members = range(cg[g], cg[g + 1])
        if not t:
            continue
        row = next(s for s in members if q[s])
        for s in members:
            lo[s], group_of[s] = t, g
        total = cq[cg[g + 1]] - cq[cg[g]]
        for i in range(0, total, tpt):
            tiles["shared", g, cq[cg[g]] + i] = (min(tpt, total - i), row, t * 128, None, 0, t)
    for s, (lq, lk) in enumerate(zip(q, k)):
        for i in range(0, lq, tpt):
            n = min(tpt, lq - i)
            hi = (limit(i + n - 1 + lk - lq, lk, block) + 127) // 128
            assert hi >= lo[s]
            tiles["own", s, cq[s] + i] = (n, s, lk, i + lk - lq, lo[s], hi)
    item = lambda base, i: w[base + 8 * i:base + 8 * i + 8]  # noqa: E731
    pieces = collections.defaultdict(list)

    def take(it, hk):
        tok0, n_hk, row, lk, pos0, a, b, at = it
        key = next(x for x in tiles if x[2] == tok0 and (x[0] == "shared") == (pos0 == 1 << 29) and tiles[x][1] == row)
        n, _, keys, pos, *_ = tiles[key]
        assert (n_hk & 255, lk) == (n, keys) and pos in (pos0, None)
        pieces[key, hk].append((a, b, at))

    if stream:
        for sm in range(sms):
            assert 0 <= w[count + sm] <= cap_rows
            for i in range(w[count + sm]):
                it = item(fwd, sm * cap_rows + i)
                take(it, it[1] >> 8)
                if i == 0:
                    assert item(at_first, sm) == it
    else:
        units = [w[sched + i] for i in range(-(-h.n_fwd * kv // sms) * sms)]
        assert sorted(u for u in units if u >= 0) == list(range(h.n_fwd * kv))
        for i, u in enumerate(units):
            if u >= 0:
                it = item(fwd, u % h.n_fwd)
                take(it, u // h.n_fwd)
                if i < sms:
                    assert item(at_first, i) == [it[0], it[1] | u // h.n_fwd << 8, *it[2:]]
    assert set(pieces) == {(t, hk) for t in tiles for hk in range(kv)}
    rows = set()

    def partials(key, hk):
        """Rows of a tile's partials, by piece in key order."""
        got = sorted(pieces[key, hk])
        assert got[0][0] == tiles[key][4] and got[-1][1] == tiles[key][5] and all(x[1] == y[0] for x, y in zip(got, got[1:]))
        if got[0][2] == -1:
            assert len(got) == 1
            return []
        at = [x + (0 if stream else hk * tiles[key][0] * G) for _, _, x in got]
        return at

    shared_rows = {}
    for key, hk in pieces:
        mine = partials(key, hk)
        for r in mine:
            block_ = set(range(r, r + tiles[key][0] * G))
            assert min(block_) >= 0 and max(block_) < cap_part and not block_ & rows
            rows |= block_
        if key[0] == "shared":
            assert mine
            shared_rows[key[1], key[2], hk] = mine
    # the joins: which partials each row of a tile takes up
    joined = {}
    assert h.n_merge <= cap_merge
    for i in range(h.n_merge):
        tok0, n_hk, pre, group_q0, row, n, step, r0, srow, sn, sstep, _ = w[merge + 12 * i:merge + 12 * i + 12]
        for r in range(r0, min(r0 + 16, (n_hk & 255) * G)):
            own = [row + c * step + r for c in range(n)]
            above = [srow + c * sstep + r for c in range(sn)]
            if pre >= 0:
                x = tok0 + r // G - group_q0
                p = prefix + 4 * ((n_hk >> 8) * cap_prefix + pre + x // tpt)
                above = [w[p] + c * w[p + 2] + x % tpt * G + r % G for c in range(w[p + 1])]
            assert (tok0, n_hk >> 8, r) not in joined
            joined[tok0, n_hk >> 8, r] = above + own
    for key, hk in pieces:
        if key[0] == "shared":
            continue
        kind, s, tok0 = key
        own = partials(key, hk)
        g = group_of[s]
        for r in range(tiles[key][0] * G):
            want = []
            if g is not None:
                i = tok0 + r // G - cq[cg[g]]
                want += [x + i % tpt * G + r % G for x in shared_rows[g, cq[cg[g]] + i // tpt * tpt, hk]]
            want += [x + r for x in own]
            if want:
                assert joined.pop((tok0, hk, r)) == want
            else:
                assert (tok0, hk, r) not in joined
    assert not joined
    # the places of the new tokens
    want = [-1] * (cq[-1] + 3)
    for s, (lq, lk) in enumerate(zip(q, k)):
        for i in range(lq):
            if lk - lq + i >= 0:
                p = lk - lq + i
                want[cq[s] + i] = (s * cols + p // page) * page + p % page
    assert w[slot:slot + len(want)] == want


LONG = [1, 52360, 300, 8192, 129, 26440, 5000, 4352, 1000, 3152, 12345, 20000]


@pytest.mark.parametrize("q,k,H,kv,block", [
    ([77, 1, 130], [77, 1, 130], 24, 8, 1), ([1] * 12, LONG, 24, 4, 1), ([432, 432], [3024, 10800], 24, 8, 432),
    ([300, 0, 2], [10, 40, 1], 6, 6, 7), ([0, 5, 0], [0, 0, 9], 4, 2, 0), ([1], [1], 128, 1, 0), ([1], [300], 24, 8, 1),
])
def test_stretches(program, q, k, H, kv, block):
    check(program, q, k, H, kv, block, stream=1)


@pytest.mark.parametrize("q,k,H,kv,block", [
    ([5000], [25920], 24, 8, 1620), ([512] * 30 + [9000], [512] * 30 + [9000], 24, 24, 1),
    ([3, 0, 9] * 400 + [2], [4, 1, 9] * 400 + [20000], 4, 2, 1),
])
def test_dealt_out(program, q, k, H, kv, block):
    check(program, q, k, H, kv, block, stream=0, page=64)


@pytest.mark.parametrize("q,k,H,kv,block,groups,taken", [
    # thirty-two tokens over a clip; a prefix that ends inside a tile; a group whose tiles are not halved (42 tokens a tile);
    # one that saves too little; no keys shared; a stream that sees less of it, one that has nothing new, one nothing at all
    ([1] * 32, [25921 + 37 * n for n in range(32)], 24, 8, 1, [(32, 25920)], [202]),
    ([5] * 14, [4357, 4500, 5000, 4400, 4700, 4900, 6000, 4358, 1086, 1100, 1500, 1200, 1300, 2500], 24, 4, 1,
     [(8, 4352), (5, 1081), (1, 0)], [34, 8, 0]),
    ([432] * 6, [3456, 3888, 4320, 3456, 5184, 3456], 24, 8, 432, [(6, 3024)], [0]),
    ([1] * 3, [400] * 3, 24, 8, 1, [(3, 399)], [0]),
    ([1, 0, 1, 0, 1, 1], [1000, 1000, 1001, 0, 300, 1000], 6, 2, 1, [(6, 999)], [0]),  # (4 - 1) * 2 tiles saved: below 8
    ([1, 0, 1, 0, 1, 1], [1000, 1000, 1001, 0, 700, 1000], 6, 2, 1, [(6, 999)], [5]),
    ([1] * 4 + [200] + [1] * 4, [900] * 9, 6, 2, 1, [(9, 890)], [5]),
    ([1] * 90, [1300 + n for n in range(90)], 6, 6, 0, [(90, 1290)], [10]),
    ([1] * 5, [513] * 5, 6, 2, 1, [(5, 512)], [4]),
])
def test_groups(program, q, k, H, kv, block, groups, taken):
    check(program, q, k, H, kv, block, 1, groups, taken)


def test_groups_dealt_out(program):
    """Among more streams than are cut into stretches."""
    q = [1, 2, 0, 1] * 300
    k = [30 + s % 7 for s in range(40)] + [2000 + s for s in range(60)] + [40] * 1100
    check(program, q, k, 4, 2, 1, 0, [(40, 0), (60, 1990)], [0, 15])
