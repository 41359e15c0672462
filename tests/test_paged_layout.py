"""Host-side arithmetic of the paged calls, from the library's own code: where a
plan's parts lie, which boxes of which pages make up a tile of keys (and what a bad
page becomes), and when pools overlap."""
import itertools
import os
import random
import subprocess

import pytest

from video_dit_long_gb300 import build as B

SOURCE = r"""
#include <cstdio>
#include "k6_paged.cuh"
#include "k6_packed_api.cu"
// "geom": H kv n_seq q_tokens page max_pages n_groups sms;  "tile": page n_pages Lk kt page_named;
// "div": page x;  "pools": Hkv page n_pages, three strides, three strides, distance (elements)
int main() {
    char what[16];
    while (scanf("%15s", what) == 1) {
        if (what[0] == 'g') {
            int H, kv, n, page, max_pages, groups, sms;
            long q;
            if (scanf("%d %d %d %ld %d %d %d %d", &H, &kv, &n, &q, &page, &max_pages, &groups, &sms) != 8) return 1;
            k6::Geom g = {};
            g.H = H, g.d = 128;
            const k6attn_paged b = {n, kv, 1, page, max_pages, groups, 1000, q};
            const k6::PagedGeom p = k6::paged_geom(g, b, sms);
            const k6::PagedPlan at = k6::paged_plan_at(nullptr, p);
            k6attn_handle h;
            h.g = g, h.g.dtype = K6ATTN_BF16, h.sms = sms, h.device = 5;  // never the current one
            printf("%zu %zu %zu %zu %zu %zu %zu %zu %zu %d %d %d %ld %d %d %zu %zu %zu %zu %zu\n", k6::paged_plan_bytes(p),
                   k6::packed_plan_common_bytes(sms), (size_t)at.count, (size_t)at.merge, (size_t)at.prefix, (size_t)at.units,
                   (size_t)at.fwd, (size_t)at.sched, (size_t)at.slot, p.g.cap_q, p.g.cap_merge, p.cap_prefix, p.cap_part,
                   p.g.cap_slots, 1 << p.box_log2, k6attn_paged_plan_bytes(&h, &b), k6attn_paged_workspace_bytes(&h, &b),
                   k6::paged_fwd_workspace(p), sizeof(k6::PagedMerge), sizeof(k6::PagedUnits));
        } else if (what[0] == 'd') {
            k6::PagedGeom p = {};
            unsigned x;
            if (scanf("%d %u", &p.page, &x) != 2) return 1;
            k6::paged_set_page(p, p.page);
            printf("%llu %u\n", (unsigned long long)x * p.page_mul >> p.page_shift, p.page_shift);
        } else if (what[0] == 't') {
            k6::PagedGeom p = {};
            int Lk, kt, named;
            if (scanf("%d %d %d %d %d", &p.page, &p.n_pages, &Lk, &kt, &named) != 5) return 1;
            k6::paged_set_page(p, p.page);
            const int n = k6::paged_boxes(p, Lk, kt), span = p.page / 8 + 3;
            printf("%d %d %d %d %d %d", 1 << p.box_log2, n, k6::paged_page(p, named), k6::paged_group(p, span, named, 16 % p.page), span,
                   k6::paged_groups(p, span));
            for (int i = 0; i < n; i++) {
                int column;
                const int tok = k6::paged_box(p, kt, i, column);
                printf(" %d %d", column, tok);
            }
            printf("\n");
        } else {
            k6::PagedGeom p = {};
            int n_pages;
            long a[3], b[3], d;
            if (scanf("%d %d %d %ld %ld %ld %ld %ld %ld %ld", &p.g.Hkv, &p.page, &n_pages, a, a + 1, a + 2, b, b + 1, b + 2,
                      &d) != 10)
                return 1;
            p.n_pages = n_pages;
            char *base = reinterpret_cast<char *>(1ul << 40);
            const k6attn_pages x = {base, a[0], a[1], a[2]}, y = {base + 2 * d, b[0], b[1], b[2]};
            Pool px, py;
            const int sx = check_pool("t", "x", &x, p, &px), sy = check_pool("t", "y", &y, p, &py);
            printf("%d %d %d\n", sx, sy, sx || sy ? -1 : (int)share(px, py));
        }
    }
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    lib = B.build()
    d = tmp_path_factory.mktemp("paged")
    (d / "layout.cu").write_text(SOURCE)
    cmd = [B.NVCC, *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "layout.cu"), "-o", str(d / "layout"), lib,
           "-Xlinker", "-rpath," + os.path.dirname(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(lines):
        r = subprocess.run([str(d / "layout")], input="\n".join(lines), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        out = [list(map(int, x.split())) for x in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return out

    return run


def test_plan_layout_and_room(run):
    cases = [(H, kv, n, q, page, cols, groups, sms) for (H, kv), (n, q), (page, cols), groups, sms in itertools.product(
        [(1, 1), (4, 2), (24, 8), (24, 24), (128, 1)], [(1, 0), (1, 1), (12, 12), (2000, 9000), (3, 52360)],
        [(16, 1), (16, 4000), (128, 500), (4096, 100)], [0, 1, 3], [152, 7, 512])]
    for c, r in zip(cases, run(["geom " + " ".join(map(str, c)) for c in cases])):
        H, kv, n, q, page, cols, groups, sms = c
        (total, common, count, merge, prefix, units, fwd, sched, slot, cap_q, cap_merge, cap_prefix, cap_part, cap_slots, box,
         asked, ws_asked, ws, merge_size, units_size) = r
        G, rows = H // kv, 128 // (H // kv) * (H // kv)
        assert count == 256
        assert 0 < merge < prefix <= units <= fwd <= sched <= slot and total == slot + 4 * q
        assert all(x % 16 == 0 for x in (merge, prefix, units, fwd, sched, slot))
        # what the join reads of a plan before the header has shown whose it is: its first `sms` entries
        assert merge == count + (sms * 4 + 15) // 16 * 16 + sms * 32
        assert prefix - merge >= sms * merge_size and units - prefix == cap_prefix * kv * 16
        assert fwd - units == (n + groups) * units_size
        assert asked == total and ws_asked == ws and (ws >= cap_part * 516 if cap_part else ws == 0)
        assert page % box == 0 and 128 % box == 0 and box >= 16
        # units of a batch whose groups all are taken together: at most two tiles of each stream, one over its prefix
        assert cap_q >= q // (128 // G) + n + cap_prefix and cap_prefix == (n if groups else 0)
        # joins of 16 rows: of tiles that are cut, and of the rows of every stream that a group may share
        assert cap_merge >= cap_slots // 2 * -(-rows // 16)
        if groups:
            tiles = min(2 * n, q // (128 // G) + n)
            assert cap_merge >= cap_slots // 2 * -(-rows // 16) + kv * (min(tiles * rows, q * G) // 16 + tiles)
            assert cap_part >= cap_slots * rows + min(2 * n * kv * rows, q * H) + min(n * kv * rows, q * H)


def test_the_bound_on_tiles_of_groups_taken_together():
    """A group is taken together where that at least halves its query tiles: then its streams have at most two tiles
    each on average, and its prefix at most one for each of them."""
    rng = random.Random(0)
    taken = 0
    for _ in range(20000):
        tpt, n = rng.choice([1, 3, 5, 16, 42, 128]), rng.randint(1, 12)
        q = [rng.choice([0, 1, 1, rng.randint(0, 3 * tpt)]) for _ in range(n)]
        own, together = sum(-(-x // tpt) for x in q), -(-sum(q) // tpt)
        if own and 2 * together <= own:
            taken += 1
            assert own <= 2 * n and together <= n
    assert taken > 1000


def test_boxes_of_a_tile(run):
    rng = random.Random(1)
    cases = []
    for _ in range(400):
        page = 16 * rng.choice([1, 2, 3, 4, 7, 8, 16, 24, 27, 100])
        Lk = rng.randint(1, 3000)
        cases.append((page, rng.randint(0, 50), Lk, rng.randint(0, (Lk + 127) // 128 - 1),
                      rng.choice([0, 3, 49, 50, 51, -1, -2 ** 31, 2 ** 31 - 1])))
        if cases[-1][1] == 0:
            cases[-1] = (page, 1, *cases[-1][2:])
    for (page, n_pages, Lk, kt, named), (box, n, got, group, span, groups, *at) in zip(cases, run(["tile " + " ".join(map(str, c)) for c in cases])):
        assert got == (named if 0 <= named < n_pages else n_pages)
        # the group that a copy begins at: inside the page's own; of a page that is none, behind the last group
        assert groups == (n_pages - 1) * span + page // 8
        assert group == (named * span + 16 % page // 8 if 0 <= named < n_pages else groups)
        rows = []
        for column, tok in zip(at[::2], at[1::2]):
            assert 0 <= tok and tok + box <= page and column <= (Lk - 1) // page
            rows += [column * page + tok + i for i in range(box)]
        assert len(at) == 2 * n and len(rows) <= 128
        assert rows == list(range(kt * 128, kt * 128 + len(rows)))  # in order, from the tile's first key
        assert len(rows) == 128 or len(rows) >= Lk - kt * 128       # all keys; none skipped but those behind the last


def test_division_by_the_page(run):
    rng = random.Random(3)
    cases = []
    for _ in range(3000):
        page = 16 * rng.choice([1, 2, 3, 7, rng.randint(1, 1 << 20), (1 << 20) - 1])
        q = rng.randint(0, (2 ** 29 - 1) // page)
        cases.append((page, max(0, min(2 ** 29 - 1, rng.choice([q * page, q * page - 1, q * page + page - 1, 2 ** 29 - 1])))))
    for (page, x), (q, shift) in zip(cases, run([f"div {page} {x}" for page, x in cases])):
        assert q == x // page and shift < 64


def test_pools_that_interleave_and_pools_that_overlap(run):
    """Against sets of rows, in units of 128 elements."""
    rng = random.Random(2)
    cases, want = [], []
    for _ in range(4000):
        n = [rng.randint(1, 3) for _ in range(3)]  # heads, tokens, pages
        order = rng.sample(range(3), 3)
        w, stride = 1, [0, 0, 0]
        for i in order:  # from the densest axis on, with a gap now and then
            stride[i] = w * rng.choice([1, 1, 1, 2, 2, 3])
            w = stride[i] * n[i]
        other = list(stride) if rng.random() < 0.9 else [s * rng.choice([1, 2]) for s in stride]
        d = rng.choice([rng.randint(-2 * w, 2 * w), rng.choice(stride) // 2, w])
        rows = lambda s, at: {at + h * s[0] + t * s[1] + p * s[2] for h in range(n[0]) for t in range(n[1])  # noqa: E731
                              for p in range(n[2])}
        want.append((rows(stride, 0), rows(other, d), n[0] * n[1] * n[2]))
        cases.append("pools " + " ".join(map(str, (*n, *(128 * s for s in stride[::-1]), *(128 * s for s in other[::-1]),
                                                   128 * d))))
    seen = {True: 0, False: 0}
    made = run(cases)
    assert sum(r[0] == 0 for r in made) > 1000
    for c, (a, b, size), (sx, sy, shared) in zip(cases, want, made):
        assert (sx == 0) <= (len(a) == size) and (sy == 0) <= (len(b) == size), c
        assert sx == 0, c  # strides made without overlap
        if sy == 0:
            assert shared or not a & b, c  # never missed
            seen[bool(shared)] += 1
    assert min(seen.values()) > 200
    # the parts of one tensor, whichever axis the two kinds lie on: not taken for overlapping
    H, t, n = 4, 16, 10
    rows = 128 * H
    for strides, d in (((2 * t * rows, rows, 128), t * rows), ((2 * t * rows, 2 * rows, 128), rows),
                       ((2 * t * rows, 2 * rows, 256), 128), ((t * rows, rows, 128), n * t * rows)):
        line = " ".join(map(str, (H, t, n, *strides, *strides)))
        assert run([f"pools {line} {d}", f"pools {line} {-d}", f"pools {line} {d + 64}"]) in (
            [[0, 0, 0], [0, 0, 0], [0, 0, 1]], [[0, 0, 0], [0, 0, 0], [0, 0, 0]])
    assert run([f"pools {H} {t} {n} 0 {rows} 128 0 {rows} 128 0", f"pools {H} {t} {n} {t * rows} {rows} 64 1 1 1 0",
                f"pools {H} {t} {n} {t * rows + 4} {rows} 128 1 1 1 0"]) == [[1, 1, -1], [1, 1, -1], [1, 1, -1]]
