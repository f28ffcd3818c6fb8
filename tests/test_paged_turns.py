"""The two slots of an attention CTA never wait for each other in a circle: every wait and arrival of its warps, walked
through on the CPU for all starts and ends of the slots' tiles, with the rules and stage counts that the kernel is built
from.  No GPU needed."""
import ctypes
import itertools
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hash_sparse_kv_b200", "csrc")
SOURCE = """
#include "attend_paged_turns.h"
using namespace hkv::pa;
extern "C" {
int k_stages() { return kKStages; }
int v_stages() { return kVStages; }
void turns(const int* mine, const int* other, int both, int* out) {
  const Turns t = turns_of(Run{mine[0], mine[1], mine[2]}, Run{other[0], other[1], other[2]}, both != 0);
  out[0] = t.from, out[1] = t.n;
}
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    (d / "turns.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "turns.cpp"), "-o", str(d / "turns.so")],
                   check=True, capture_output=True, text=True)
    return ctypes.CDLL(str(d / "turns.so"))


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def over(self, parity):  # the phase of this parity has ended
        return self.phase & 1 != parity


def _loader(t0, t1, full, empty, lag):
    """K or V tiles; with `lag` a tile's arrival is told when the next one has been issued, or before a wait."""
    pending, stages = None, len(full)
    for i, _ in enumerate(range(t0, t1)):
        b, parity = empty[i % stages], (i // stages & 1) ^ 1
        if not b.over(parity) and pending:
            pending.arrive()
            pending = None
        yield b, parity
        if pending:
            pending.arrive()
            pending = None
        if lag:
            pending = full[i % stages]
        else:
            full[i % stages].arrive()
    if pending:
        pending.arrive()


def _products(s, both, t0, t1, run, k_full, k_empty, v_full, v_empty, s_full, p_half, p_full, o_done):
    at = [0]

    def stage(bars):
        return bars[at[0] % len(bars)], at[0] // len(bars) & 1

    def passing(a, b):
        for _ in range(a, b):
            yield stage(k_full)
            stage(k_empty)[0].arrive()
            yield stage(v_full)
            stage(v_empty)[0].arrive()
            at[0] += 1

    first, last, step = run
    if both:
        yield from passing(t0, min(t1, first))
    elif s == 1:
        at[0] += 1
    if first < last:
        yield stage(k_full)
        s_full[s].arrive(), stage(k_empty)[0].arrive()
    for done, n in enumerate(range(first, last, step)):
        yield stage(v_full)
        v_free = stage(v_empty)[0]
        at[0] += step
        more = n + step < last
        if more:
            yield stage(k_full)
        yield p_half[s], done & 1
        yield p_full[s], done & 1
        v_free.arrive(), o_done[s].arrive()
        if more:
            s_full[s].arrive(), stage(k_empty)[0].arrive()
    if both:
        yield from passing(max(last, first), t1)


def _softmax(s, run, turns, rescale, s_full, p_half, p_full, o_done, turn):
    done = 0
    for done, _ in enumerate(range(*run)):
        yield s_full[s], done & 1
        if rescale and done:
            yield o_done[s], (done - 1) & 1
        in_turn = turns[0] <= done < turns[0] + turns[1]
        if in_turn and (s == 1 or done > turns[0]):
            yield turn[s], (done - turns[0] - (0 if s else 1)) & 1
        p_half[s].arrive()
        if in_turn:
            turn[1 - s].arrive()
        p_full[s].arrive()
    if len(range(*run)):
        yield o_done[s], done & 1


def _ends(rules, both, t0, t1, runs, lag, rescale, order):
    k, v = rules.k_stages(), rules.v_stages()
    k_full, v_full = [Barrier(1) for _ in range(k)], [Barrier(1) for _ in range(v)]
    k_empty, v_empty = [Barrier(1 + both) for _ in range(k)], [Barrier(1 + both) for _ in range(v)]
    s_full, p_half, p_full, o_done, turn = ([Barrier(1), Barrier(1)] for _ in range(5))
    turns = []
    for s in range(2):
        out = (ctypes.c_int * 2)()
        rules.turns((ctypes.c_int * 3)(*runs[s]), (ctypes.c_int * 3)(*runs[1 - s]), int(both), out)
        turns.append(tuple(out))
    roles = [_loader(t0, t1, k_full, k_empty, lag), _loader(t0, t1, v_full, v_empty, lag)]
    roles += [_products(s, both, t0, t1, runs[s], k_full, k_empty, v_full, v_empty, s_full, p_half, p_full, o_done)
              for s in range(2)]
    roles += [_softmax(s, runs[s], turns[s], rescale, s_full, p_half, p_full, o_done, turn) for s in range(2)]
    roles = [roles[i] for i in order]
    waits = [next(r, None) for r in roles]
    moved = True
    while moved:
        moved = False
        for i, r in enumerate(roles):
            while waits[i] is not None and waits[i][0].over(waits[i][1]):
                waits[i], moved = next(r, None), True
    return all(w is None for w in waits)


ORDERS = [(0, 1, 2, 3, 4, 5), (5, 3, 1, 0, 2, 4), (4, 2, 0, 1, 3, 5)]


@pytest.mark.parametrize("lag", [False, True])
def test_slots_that_share_their_tiles(rules, lag):
    """All starts and ends of both runs within eleven tiles, slots without a tile and runs cut off by a split among them."""
    top = 11
    runs = [(a, b, 1) for a in range(top + 1) for b in range(a, top + 1)]
    stuck = []
    for i, (r0, r1) in enumerate(itertools.product(runs, runs)):
        if min(r0[0], r1[0]) > 0 and i % 3:  # the first tile that anyone works on is the CTA's first
            continue
        t0 = 0 if i % 3 == 0 else min(r0[0], r1[0])
        if not _ends(rules, True, t0, top, (r0, r1), lag, i % 2 == 0, ORDERS[i % 3]):
            stuck.append((r0[:2], r1[:2]))
    assert not stuck, f"{len(stuck)} pairs of runs end in a circle, the first {stuck[0]}"


@pytest.mark.parametrize("rescale", [False, True])
@pytest.mark.parametrize("lag", [False, True])
def test_slots_that_take_every_other_tile(rules, lag, rescale):
    for n in range(15):
        for order in ORDERS:
            assert _ends(rules, False, 0, n, ((0, n, 2), (1, n, 2)), lag, rescale, order), n
