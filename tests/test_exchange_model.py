"""A model of how the CTAs of a cluster sum the bins of a split (sampling's
searches): every CTA sums its share of the bins and sends the sums around.

Each CTA has a group of threads for each CTA of the cluster.  In a round, group
g of CTA c (1) meets the other groups at a barrier, (2) sends CTA g this CTA's
counts of the bins that CTA g sums, (3) waits until all CTAs' counts are here,
(4) reads them and sends their sum to CTA g, (5) waits until all sums are here,
reads them and meets the other groups again.  Only the order of these steps is
modelled, every order of them that the barriers and waits allow: no array may
be written while a group has yet to read what is in it."""
import os
import re

import pytest

from conftest import ROOT

SOURCE = os.path.join(ROOT, "parity_binade_chunked_gb300", "csrc", "sample_kernel.cu")
BEGIN, SEND, READ_PARTS, READ_TOTALS, END = range(5)   # a group's next step in its round


def violations(size, rounds, slots):
    """Which arrays some order of the steps overwrites too early, where a CTA has `slots` arrays of parts in turn."""
    start = ((0, BEGIN),) * (size * size)
    seen, todo, found = {start}, [start], set()
    while todo:
        state = todo.pop()
        at = lambda c, g: state[c * size + g]
        for c in range(size):
            for g in range(size):
                r, step = at(c, g)
                if r == rounds:
                    continue
                if step == BEGIN and any(at(c, o) < (r, BEGIN) for o in range(size)):
                    continue
                if step == READ_PARTS and any(at(o, c) <= (r, SEND) for o in range(size)):
                    continue
                if step == READ_TOTALS and any(at(o, c) <= (r, READ_PARTS) for o in range(size)):
                    continue
                if step == END and any(at(c, o) < (r, END) for o in range(size)):
                    continue
                if step == SEND:         # to parts[r % slots] of CTA g: were all its groups through with round r - slots?
                    if r >= slots and any(at(g, o) <= (r - slots, READ_PARTS) for o in range(size)):
                        found.add("parts")
                if step == READ_PARTS:   # to the sums of CTA g: were all its groups through with those of the round before?
                    if r >= 1 and any(at(g, o) <= (r - 1, READ_TOTALS) for o in range(size)):
                        found.add("totals")
                n = list(state)
                n[c * size + g] = (r, step + 1) if step < END else (r + 1, BEGIN)
                n = tuple(n)
                if n not in seen:
                    seen.add(n)
                    todo.append(n)
    return found


def test_one_array_of_parts_is_not_enough():
    assert violations(2, 2, 1) == {"parts"}


@pytest.mark.parametrize("rounds", [2, 3, 4])
def test_two_in_turn_are(rounds):
    assert violations(2, rounds, 2) == set()


def test_the_kernel_takes_two_in_turn():
    source = open(SOURCE).read()
    slots = re.search(r"uint64_t part\[(\d+)\]\[\w+\];", source)
    assert slots and violations(2, 3, int(slots[1])) == set()
    assert "uint64_t *part = sh.part[parity];" in source
