"""Host-side model of the waits of the packed attention kernel
(k6_packed_attn.cu): a persistent CTA that runs one item after another, the K/V
ring of the joint kernel (modelled in test_ring_protocol.py) carried from item
to item, and one Q buffer that an item's first S waits for.

Added to that model, in program order:
- the producer issues an item's Q before its first K, once the last S of the
  item before is done;
- the first S of an item waits for its Q;
- each softmax group posts its row sums after its last tile of an item, once the
  epilogue has read those of the item before, and goes on at once;
- the epilogue reads both posts, waits for the item's last P.V, takes O and
  stores it, one item after another;
- the first P.V of an item waits for the epilogue before to have read O.
Checked over sequences of items of 1-7 key tiles: every slot is freed by
someone, no wait cycle, no wait that an earlier phase of its slot could match.
"""
import itertools

from .test_ring_protocol import NSTAGE, acyclic, ancestors, model

CASES = [list(Ts) for k in range(1, 5) for Ts in itertools.product((1, 2, 3, 4, 5, 7), repeat=k)] + \
    [[1] * 12, [2] * 9, [3] * 7, [17, 1, 17], [1, 2, 1, 2, 1, 2, 1], [6, 6, 6, 6]]


def packed_model(Ts, q_first=True):
    loads, idx, deps, consumer, N = model(Ts, 2)
    first = 0
    for u, T in enumerate(Ts):
        last = first + T - 1
        deps[("S_release", first)].add(("Q", u))  # waited for before anything else of the item
        deps[("stored", u)].add(("read_O", u))
        # tile n belongs to group n % 2; a group without a tile of the item posts all the same
        for g in (0, 1):
            mine = [n for n in range(first, first + T) if n % 2 == g]
            if mine:
                deps[("post", u, g)].add(("P", mine[-1]))
            if u:
                deps[("post", u, g)] |= {("post", u - 1, g), ("read_sums", u - 1)}
                for n in mine[:1]:
                    deps[("wake", n)].add(("post", u - 1, g))
            deps[("read_sums", u)].add(("post", u, g))
        if u:
            deps[("read_sums", u)].add(("stored", u - 1))
        deps[("read_O", u)] |= {("PV_done", last), ("read_sums", u)}
        if u:
            deps[("Q", u)].add(("S", first - 1))
            prev = max(idx[("K", first - 1)], idx[("V", first - 1)])
            if q_first:
                deps[("Q", u)].add(("load", prev))
                deps[("load", prev + 1)].add(("Q", u))
            else:  # Q issued after the first two K tiles
                deps[("Q", u)].add(("load", prev + min(2, T)))
                deps[("load", prev + min(2, T) + 1)].add(("Q", u))
            deps[("wait_O", first)].add(("read_O", u - 1))
            deps[("PV", first)].add(("wait_O", first))
        first += T
    return loads, deps, consumer


def test_no_wait_cycle_over_items():
    for Ts in CASES:
        _, deps, _ = packed_model(Ts)
        assert acyclic(deps), Ts


def test_no_wait_can_match_an_earlier_phase():
    for Ts in CASES:
        loads, deps, consumer = packed_model(Ts)
        for i, (kind, n) in enumerate(loads):
            if i >= NSTAGE:
                wait = ("wait_K" if kind == "K" else "wait_V", n)
                assert consumer[i - NSTAGE] in ancestors(deps, wait), (Ts, loads[i], loads[i - NSTAGE])


def test_q_behind_the_first_k_tiles_would_deadlock():
    # a K of a later item takes the slot of a V that only that item's first S frees, which waits for its Q
    assert not all(acyclic(packed_model(Ts, q_first=False)[1]) for Ts in CASES)
