"""The many-row attention kernel's notes of non-finite values, replayed on the host (csrc/paged_notes.h).

Two parties share the notes of a thread block: the cleaning warps write those
of item i while they prepare its tiles, the softmax warps read and clear them
at the item's end, which is phase i of a barrier.  A wait for a phase sees its
parity alone, and the tiles of item i can be there as soon as the weights of
item i - 2 are done.  The rules (which phase, and when) are compiled alone; every
order of events of small batches is gone through:
  * an item's end finds the notes of that item, all of them and no others;
  * no order ends with a party waiting for ever.
"""
import itertools
import os
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "recurrent_memory_transformer_gb300", "csrc")
ITEMS, TILES = 6, 2

PROGRAM = r"""
#include <cstdio>
#include "paged_notes.h"
int main() {
  for (int i = 0; i < %d; ++i)
    for (int count = 1; count <= %d; ++count)
      for (int t = 0; t < count; ++t)
        std::printf("%%d %%d %%d %%d %%d\n", i, count, t, armt::notes_phase(i), (int)armt::notes_hold_back(i, t, count));
}
""" % (ITEMS, TILES)


@pytest.fixture(scope="module")
def rules():
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    with tempfile.TemporaryDirectory() as td:
        src, exe = os.path.join(td, "a.cpp"), os.path.join(td, "a")
        with open(src, "w") as f:
            f.write(PROGRAM)
        subprocess.run([cxx, "-std=c++17", "-I", CSRC, src, "-o", exe], check=True)
        lines = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")
    out = {}
    for line in lines:
        if line:
            i, count, t, phase, hold = map(int, line.split())
            out[i, count, t] = phase, bool(hold)
    return out


def passes(ended, phase):
    """A wait for `phase` by parity, when phases 0 .. ended - 1 are over: the current phase has the other parity."""
    return phase < 0 or (ended & 1) != (phase & 1)


def faults(counts, rules):
    """Goes through all orders; returns the kinds of fault met.

    State: cleaning warps at (item, tile, step: 0 before the choice to note, 1
    about to note, 2 about to hand over); tiles handed over; softmax at (item,
    weights done); the notes' owners."""
    n = len(counts)
    found, seen = set(), set()
    start = (0, 0, 0, 0, 0, False, frozenset(), frozenset())
    todo = [start]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        ci, ct, step, handed, si, weighed, notes, due = state
        moves = []
        if ci < n:
            phase, hold = rules[ci, counts[ci], ct]
            there = ci < 2 or si > ci - 2 or (si == ci - 2 and weighed)
            if step == 0 and there:
                moves.append((ci, ct, 1, handed, si, weighed, notes, due))
                moves.append((ci, ct, 2, handed, si, weighed, notes, due))
            elif step == 1 and passes(si, phase):
                moves.append((ci, ct, 2, handed, si, weighed, notes | {ci}, due | {ci}))
            elif step == 2 and (not hold or passes(si, phase)):
                nxt = (ci, ct + 1) if ct + 1 < counts[ci] else (ci + 1, 0)
                moves.append(nxt + (0, handed + 1, si, weighed, notes, due))
        if si < n:
            if not weighed:
                moves.append((ci, ct, step, handed, si, True, notes, due))
            elif handed >= sum(counts[:si + 1]):
                if notes - {si}:
                    found.add("notes of a later item")
                if (si in due) != (si in notes):
                    found.add("notes lost")
                moves.append((ci, ct, step, handed, si + 1, False, frozenset(), due - {si}))
        if not moves and (ci < n or si < n):
            found.add("waits for ever")
        todo += moves
    return found


def test_every_item_end_finds_its_own_notes(rules):
    for counts in itertools.product(range(1, TILES + 1), repeat=ITEMS):
        assert not faults(counts, rules), counts


def test_the_replay_sees_a_wait_that_comes_too_early(rules):
    # without the wait before the last tile, a wait by parity finds the phase before the last one
    lazy = {k: (phase, False) for k, (phase, hold) in rules.items()}
    assert "notes of a later item" in faults((1,) * ITEMS, lazy)
    # waiting for the end of the item before that at every item's beginning can miss it: the phase after has come
    early = {k: (phase if k[0] < 2 else phase - 1, k[2] == 0) for k, (phase, hold) in rules.items()}
    assert "waits for ever" in faults((1,) * ITEMS, early)
