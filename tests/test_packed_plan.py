"""Host-side model of how the forward plan cuts a batch into one stretch per SM
(k6_packed_plan.cu): the units (query tiles of a key head) lie end to end, each
costing its key tiles and a constant; every SM takes one stretch of equal cost;
cuts that would leave a piece of a few tiles move to the unit's border.

Checked over random batches: the pieces of a unit cover its key tiles once and in
order, no piece is shorter than allowed, each SM's list has no hole and no entry
written twice, and lists, partials and joins stay within what the host allots.
"""
import random

import pytest

MIN_PIECE, ITEM_COST, STREAM_MOST = 4, 2, 256


def limit(pos, keys, block):
    if block == 0:
        return keys
    return 0 if pos < 0 else min(keys, (pos // block + 1) * block)


def plan(q, k, kv, G, block, sms):
    """(cost per SM, largest load, mean load), or None where the batch is dealt out as a list instead."""
    tpt, n, Tq, Tk = 128 // G, len(q), sum(q), sum(k)
    extra = -(-sms // kv) if Tk > (2 * MIN_PIECE - 1) * 128 else 0
    cap_slots = 2 * max(extra * kv, sms) if extra else 0
    most = ((Tq // tpt + n) * kv * ((Tk + 127) // 128 + 1 + ITEM_COST) + sms - 1) // sms
    cap_rows = min(most, STREAM_MOST) // (ITEM_COST + 1) + 8
    one = []
    for lq, lk in zip(q, k):
        for t in range(-(-lq // tpt)):
            last = min((t + 1) * tpt, lq) - 1
            one.append((limit(last + lk - lq, lk, block) + 127) // 128)
    total = kv * sum(max(w, 1) + ITEM_COST for w in one)
    if total > sms * STREAM_MOST:
        return None
    assert most > 0 or not one
    Q = max(1, -(-total // sms))
    units, a = [], 0
    for w in one * kv:
        units.append((a, a + max(w, 1) + ITEM_COST, w))
        a = units[-1][1]

    def cut(c, a, w):
        x = max(0, c * Q - a - ITEM_COST)
        if Q < MIN_PIECE:
            x -= x % MIN_PIECE
        return 0 if x < MIN_PIECE else w if w - x < MIN_PIECE else x

    first = {}
    for u, (a, b, w) in enumerate(units):
        for c in range(-(-a // Q), min(sms, -(-b // Q))):
            assert c not in first
            first[c] = u + (cut(c, a, w) >= max(w, 1))
    cells, load, slots, merges = {}, {}, 0, 0
    for u, (a, b, w) in enumerate(units):
        c0, c1 = -(-a // Q), min(sms, -(-b // Q))
        pieces, at = 1, 0
        for c in range(c0, c1):
            x = cut(c, a, w)
            if at < x < w:
                pieces, at = pieces + 1, x
        if pieces > 1:
            slots, merges = slots + pieces, merges + 1
        at, got, owner = 0, [], min(sms - 1, a // Q)
        for c in range(c0, c1 + 1):
            x = cut(c, a, w) if c < c1 else w
            if c < c1 and x >= w > 0:
                continue
            if c < c1 and x == at:
                owner = c
                continue
            i = u - first[owner]
            assert 0 <= i < cap_rows and (owner, i) not in cells
            cells[owner, i] = u
            load[owner] = load.get(owner, 0) + x - at + ITEM_COST
            got.append((at, x))
            at, owner = x, c
        assert len(got) == pieces and got[0][0] == 0 and got[-1][1] == w
        assert all(l[1] == r[0] for l, r in zip(got, got[1:]))
        assert pieces == 1 or all(y - x >= MIN_PIECE for x, y in got)
    for sm in load:
        assert sorted(i for s, i in cells if s == sm) == list(range(sum(s == sm for s, _ in cells)))
    assert slots <= cap_slots and merges <= cap_slots // 2
    return Q, max(load.values(), default=0), total / sms


@pytest.mark.parametrize("seed", range(4))
def test_stretches_cover_every_unit_once(seed):
    rng = random.Random(seed)
    done = 0
    for _ in range(250):
        n, m = int(10 ** rng.uniform(0, 2)), 10 ** rng.uniform(0, 4)
        k = [int(m ** rng.random()) for _ in range(n)]
        q = list(k) if rng.random() < 0.5 else [rng.choice([0, 1, 1, rng.randint(0, 600)]) for _ in k]
        r = plan(q, k, rng.choice([1, 2, 3, 4, 8, 24]), rng.choice([1, 3, 5, 6, 24, 128]), rng.choice([0, 1, 7, 432]),
                 rng.choice([152, 148, 7]))
        if r:
            done += 1
            # a stretch ends at most a short piece and an item's cost behind its border
            assert r[1] <= r[0] + 2 * (MIN_PIECE + ITEM_COST)
    assert done > 100


def test_stretches_of_new_tokens_over_long_caches_are_even():
    Q, most, mean = plan([1] * 12, [1, 52360, 300, 8192, 129, 26440, 5000, 4352, 1000, 3152, 12345, 20000], 4, 6, 1, 152)
    assert most <= 1.4 * mean and most <= Q + MIN_PIECE + ITEM_COST


def test_the_model_has_the_kernels_constants():
    import pathlib
    import re
    src = (pathlib.Path(__file__).parent.parent / "video_dit_long_gb300/csrc/k6_packed_plan.cu").read_text()
    for name in ("MIN_PIECE", "ITEM_COST", "STREAM_MOST"):
        assert int(re.search(rf"constexpr int {name} = (\d+);", src).group(1)) == globals()[name]
