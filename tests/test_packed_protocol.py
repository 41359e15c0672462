"""Host-side model of the waits of the packed attention kernel
(k6_packed_attn.cu): a persistent CTA that runs one item after another.

In program order, as a dependency graph over the items' key tiles n:
- one producer loads an item's first K, then its Q (once the last S of the item
  before is done), then its other K tiles, K(n) into slot n % 3; another loads
  V(n) into slot n % 3 of a ring of its own;
- the Q.K^T warp issues S(n) once K(n) has landed and the softmax has read
  S(n-2), whose buffer it takes;
- tile n belongs to softmax group n % 2, which frees K(n)'s slot when it sees
  S(n), waits for the maximum after tile n-1, reads S(n), posts its own maximum,
  and writes P(n) once P(n-2).V, which read the same buffer, is done (and
  P(n-1).V, where it rescales the output);
- the P.V warp issues P(n).V once V(n) has landed and P(n) is there; V(n)'s slot
  is freed when it is done; the first of an item also waits until the epilogue
  has taken the output of the item before;
- each group posts its row sums after its last tile of an item, once the
  epilogue has read those of the item before;
- the epilogue reads both posts, waits for the item's last P.V and takes O.
Checked over sequences of items: no wait cycle, and no wait that an earlier phase
of its barrier could match.
"""
import collections
import itertools

from .test_ring_protocol import acyclic, ancestors

SLOTS = 3

CASES = [list(Ts) for k in range(1, 5) for Ts in itertools.product((1, 2, 3, 4, 5, 7), repeat=k)] + \
    [[1] * 12, [2] * 9, [3] * 7, [17, 1, 17], [1, 2, 1, 2, 1, 2, 1], [6, 6, 6, 6]]


def packed_model(Ts, k_before_q=1):
    deps = collections.defaultdict(set)
    N = sum(Ts)
    first = [sum(Ts[:u]) for u in range(len(Ts))]
    item_of = {n: u for u, T in enumerate(Ts) for n in range(first[u], first[u] + T)}
    order = []  # of the K and Q producer
    for u, T in enumerate(Ts):
        ks = [("load_K", n) for n in range(first[u], first[u] + T)]
        order += ks[:k_before_q] + [("Q", u)] + ks[k_before_q:]
    for a, b in zip(order, order[1:]):
        deps[b].add(a)
    for n in range(N):
        u = item_of[n]
        at_start = n == first[u]
        if n:
            deps[("load_V", n)].add(("load_V", n - 1))
        if n >= SLOTS:
            deps[("load_K", n)].add(("wake", n - SLOTS))
            deps[("load_V", n)].add(("PV_done", n - SLOTS))
        # Q.K^T warp
        if n:
            deps[("wait_K", n)].add(("S", n - 1))
        if n >= 2:
            deps[("wait_K", n)].add(("read_S", n - 2))
        if at_start:
            deps[("wait_K", n)].add(("Q", u))
        deps[("S", n)] |= {("wait_K", n), ("load_K", n)}
        # softmax group n % 2
        deps[("wake", n)].add(("S", n))
        if n >= 2:
            deps[("wake", n)].add(("P", n - 2))
        deps[("read_S", n)] |= {("wake", n)} | ({("max", n - 1)} if n else set())
        deps[("max", n)].add(("read_S", n))
        deps[("P", n)].add(("max", n))
        if n >= 2:
            deps[("P", n)].add(("PV_done", n - 2))
        if not at_start:
            deps[("P", n)].add(("PV_done", n - 1))
        # P.V warp
        if n:
            deps[("wait_V", n)].add(("PV", n - 1))
        deps[("PV", n)] |= {("wait_V", n), ("load_V", n), ("P", n)}
        if at_start and u:
            deps[("PV", n)].add(("read_O", u - 1))
        deps[("PV_done", n)].add(("PV", n))
    for u, T in enumerate(Ts):
        last = first[u] + T - 1
        if u:
            deps[("Q", u)].add(("S", first[u] - 1))
        for g in (0, 1):
            mine = [n for n in range(first[u], last + 1) if n % 2 == g]
            if mine:
                deps[("post", u, g)].add(("P", mine[-1]))
            if u:
                deps[("post", u, g)] |= {("post", u - 1, g), ("read_sums", u - 1)}
                for n in mine[:1]:
                    deps[("wake", n)].add(("post", u - 1, g))
            deps[("read_sums", u)].add(("post", u, g))
        if u:
            deps[("read_sums", u)].add(("read_O", u - 1))
        deps[("read_O", u)] |= {("PV_done", last), ("read_sums", u)}
    return deps, N


def test_no_wait_cycle_over_items():
    for Ts in CASES:
        assert acyclic(packed_model(Ts)[0]), Ts


def test_no_wait_can_match_an_earlier_phase():
    """A barrier's phase is told by its parity, so its completion before must be known when a wait starts."""
    for Ts in CASES:
        deps, N = packed_model(Ts)
        for n in range(N):
            if n >= SLOTS:  # K and V slots: the consumer's use of the load before
                assert ("S", n - SLOTS) in ancestors(deps, ("wait_K", n)), (Ts, n)
                assert ("PV", n - SLOTS) in ancestors(deps, ("wait_V", n)), (Ts, n)
            if n >= 3:
                # a group waits for P(n-2).V in turn; where it rescales it then waits for P(n-1).V, whose
                # barrier's completion before is P(n-3).V
                assert ("PV", n - 3) in ancestors(deps, ("PV_done", n - 2)), (Ts, n)


def test_two_k_tiles_ahead_of_q_would_deadlock_in_a_two_slot_ring():
    """The order matters: a K ahead of its item's Q may need a slot that a later tile frees only after that Q."""
    global SLOTS
    SLOTS, was = 2, SLOTS
    try:
        assert not all(acyclic(packed_model(Ts, k_before_q=3)[0]) for Ts in CASES)
    finally:
        SLOTS = was
