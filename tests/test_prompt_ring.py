"""The barriers of prompt attention's block, over every order of events.

A block's roles (hand out items, load, multiply, clear, softmax) are modelled as lists of steps, each a wait followed by
what the role does before its next wait; loads land in any order, a batch of products commits in order.  All
interleavings are walked.  The ring's order and the ragged tiles' barriers are csrc/prompt_ring.hpp's own, compiled here
for the host.  An error is an arrival at a barrier whose phase has none outstanding, a wait that a wrong phase's parity
lets through, a value tile that is used before its tail is cleared, and a state that nothing can leave."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "event_tensor_task_b200", "csrc")
SHIM = """
#include "%s/prompt_ring.hpp"
extern "C" {
int tails() { return mk::kTails; }
int slot(int c) { return mk::tail_slot(c); }
int parity(int c) { return mk::tail_parity(c); }
int k_at(int apart, int j) { return apart ? mk::ring_k<true>(j) : mk::ring_k<false>(j); }
int v_at(int apart, int j, int n) { return apart ? mk::ring_v<true>(j, n) : mk::ring_v<false>(j, n); }
int is_v(int apart, int i, int n) { return apart ? mk::ring_is_v<true>(i, n) : mk::ring_is_v<false>(i, n); }
int tile(int apart, int i, int n) { return apart ? mk::ring_tile<true>(i, n) : mk::ring_tile<false>(i, n); }
}
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "shim.cpp").write_text(SHIM % CSRC)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", str(d / "shim.so"), str(d / "shim.cpp")], check=True)
    return ctypes.CDLL(str(d / "shim.so"))


def roles(ring, apart, stages, items, slot, parity):
    """The roles' steps for `items` of (key tiles, ends ragged): a step is (wait or None, actions), a wait (barrier,
    phase, parity), an action (kind, barrier or item)."""
    hand, load, multiply, clear, softmax = [], [], [], [], []
    it = tails = 0
    phase = lambda bar, n: (bar, n, n & 1)
    took = lambda k: (phase(("item_full", k & 1), k >> 1), [("arrive", ("item_empty", k & 1))])
    full = {}   # place in the ring -> wait for its tile
    tail = {}   # item -> (barrier, phase, parity)
    uses = {}
    for k, (n, ragged) in enumerate(items):
        if ragged:
            bar = ("tail", slot(tails))
            tail[k] = (bar, uses.get(bar, 0), parity(tails))
            uses[bar] = uses.get(bar, 0) + 1
            tails += 1
    for k, (n, ragged) in enumerate(items):
        # items
        if k:
            hand.append((phase(("item_empty", (k - 1) & 1), (k - 1) >> 1), [("arrive", ("item_full", k & 1))]))
        else:
            hand.append((None, [("arrive", ("item_full", 0))]))
        # loads
        load.append(took(k))
        load.append((phase("q_empty", k - 1) if k else None, [("arm", "q_full")]))
        for i in range(2 * n):
            at = it + i
            stage = at % stages
            ends = ragged and ring.is_v(apart, i, n) and ring.tile(apart, i, n) == n - 1
            full[at] = phase(("kv_full", stage), at // stages)
            load.append((phase(("kv_empty", stage), at // stages - 1) if at >= stages else None,
                         [("arm", tail[k][0] if ends else ("kv_full", stage))]))
        # products
        multiply.append(took(k))
        multiply.append((phase("q_full", k), []))
        base = sum(m for m, _ in items[:k])  # S and P tiles before this item

        def scores(j):
            at = it + ring.k_at(apart, j)
            multiply.append((full[at], []))
            done = [("commit", "s_full"), ("commit", ("kv_empty", at % stages))] + ([("commit", "q_empty")] if j + 1 == n else [])
            # (where P lies over S, its product is issued before)
            multiply.append((phase("s_read", base + j - 1) if apart and base + j else None, done))

        scores(0)
        for j in range(n):
            at = it + ring.v_at(apart, j, n)
            if apart and j + 1 < n:
                scores(j + 1)
            multiply.append((full[at], [("cleared", k)] if ragged and j == n - 1 else []))
            multiply.append((phase("p_full", base + j), [("commit", "pv_done")]))
            if not apart and j + 1 < n:
                scores(j + 1)
            multiply[-1][1].append(("commit", ("kv_empty", at % stages)))
        # tails
        clear.append(took(k))
        if ragged:
            at = it + ring.v_at(apart, n - 1, n)
            clear.append((tail[k], [("clear", k), ("arrive", ("kv_full", at % stages))]))
        # softmax
        softmax.append(took(k))
        for j in range(n):
            softmax.append((phase("s_full", base + j), [("arrive", "s_read")] if apart else []))
            softmax.append((phase("pv_done", base + j - 1) if apart and j else None, [("arrive", "p_full")]))
        softmax.append((phase("pv_done", base + n - 1), []))
        it += 2 * n
    return [hand, load, multiply, clear, softmax]


def walk(programs):
    """Every interleaving; the first error as a text, or the number of states."""
    names = sorted({b for p in programs for w, acts in p for b in [w and w[0]] + [a[1] for a in acts if a[0] in ("arrive", "arm", "commit")]
                    if b is not None}, key=str)
    index = {b: i for i, b in enumerate(names)}
    count = [4 if b[0] == "item_empty" else 1 for b in names]
    #        places of the roles, (phases, outstanding arrivals, bytes on the way) of each barrier, loads on the way,
    #        commits on the way, items whose tail is cleared
    start = ((0,) * len(programs), tuple((0, c, 0) for c in count), (), (), frozenset())
    seen, todo = {start}, [start]

    def settle(bars, i, arrive, tx):
        done, pending, flying = bars[i]
        if arrive and pending == 0:
            return f"{names[i]}: an arrival too many"
        pending, flying = pending - arrive, flying + tx
        bars[i] = (done + 1, count[i], 0) if pending == 0 and flying == 0 else (done, pending, flying)
        return None

    while todo:
        place, bars, loads, commits, cleared = todo.pop()
        after = []
        for r, program in enumerate(programs):
            if place[r] == len(program):
                continue
            wait, acts = program[place[r]]
            if wait is not None:
                done = bars[index[wait[0]]][0]
                if done & 1 == wait[2]:
                    continue
                if done != wait[1] + 1:
                    return f"{wait[0]}: the wait for phase {wait[1]} ends in phase {done}"
            b, l, c, z = list(bars), loads, commits, cleared
            for kind, what in acts:
                bad = None
                if kind == "arrive":
                    bad = settle(b, index[what], 1, 0)
                elif kind == "arm":
                    bad = settle(b, index[what], 1, 1)
                    l = tuple(sorted(l + (index[what],)))
                elif kind == "commit":
                    c = c + (index[what],)
                elif kind == "clear":
                    z = z | {what}
                elif what not in z:
                    bad = f"item {what}: values used before they are cleared"
                if bad:
                    return bad
            after.append((place[:r] + (place[r] + 1,) + place[r + 1:], tuple(b), l, c, z))
        for i in set(loads):
            b = list(bars)
            settle(b, i, 0, -1)
            at = loads.index(i)
            after.append((place, tuple(b), loads[:at] + loads[at + 1:], commits, cleared))
        if commits:
            b = list(bars)
            bad = settle(b, commits[0], 1, 0)
            if bad:
                return bad
            after.append((place, tuple(b), loads, commits[1:], cleared))
        if not after and any(p != len(programs[r]) for r, p in enumerate(place)):
            return "a state that nothing leaves"
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return len(seen)


@pytest.mark.parametrize("apart,stages", [(1, 5), (0, 4)])
def test_ring_order_both_ways(ring, apart, stages):
    for n in range(1, 12):
        places = [(0, ring.k_at(apart, j), j) for j in range(n)] + [(1, ring.v_at(apart, j, n), j) for j in range(n)]
        assert sorted(p for _, p, _ in places) == list(range(2 * n))
        for v, p, j in places:
            assert bool(ring.is_v(apart, p, n)) == bool(v) and ring.tile(apart, p, n) == j
        for j in range(n):  # a tile's keys come before its values
            assert ring.k_at(apart, j) < ring.v_at(apart, j, n)


ITEMS = [
    [(1, True)] * 4,                                    # short prompts, one after the other
    [(1, True), (1, False), (1, True), (1, True)],
    [(2, True), (1, True), (1, True)],
    [(1, True), (2, True), (1, True)],
    [(3, True), (1, True)],
    [(3, True), (2, False), (1, True), (1, True), (2, True), (1, True)],
]


@pytest.mark.parametrize("apart,stages", [(1, 5), (0, 4)])
@pytest.mark.parametrize("items", ITEMS, ids=str)
def test_no_order_of_events_arms_a_barrier_twice(ring, apart, stages, items):
    found = walk(roles(ring, apart, stages, items, ring.slot, ring.parity))
    assert isinstance(found, int), found


@pytest.mark.parametrize("apart,stages", [(1, 5), (0, 4)])
def test_the_walk_finds_a_barrier_that_all_ragged_tiles_share(ring, apart, stages):
    found = walk(roles(ring, apart, stages, [(1, True)] * 2, lambda c: 0, lambda c: c & 1))
    assert isinstance(found, str)  # an arrival too many, or a phase that goes by before the clearing warp has seen it
