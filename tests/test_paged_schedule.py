"""Models of two barrier schedules of the paged attention kernels under random interleavings.

Waits on an mbarrier are by parity: waiting for phase i passes if the number of completed
phases differs from i in its last bit, which is right only while a waiter is at most one
phase away.  Each model steps its actors in random order, checks every buffer it fills or
reads, and is shown to catch the arrangement that failed on the hardware or would have.
"""
import random

import pytest


def passes(done, phase):
    return (done & 1) != (phase & 1)


def raw_ring(stages, tiles, rng):
    """Two producers (K: even tiles, V: odd ones) fill the raw stages of one ring, two groups of
    widening warps empty them, each tensor in its own order; returns "ok" or the first fault."""
    full, empty, held = [0] * stages, [0] * stages, [None] * stages
    loaded, read = {0: 0, 1: 0}, {0: 0, 1: 0}
    while min(read.values()) < tiles:
        acts = []
        for kv in (0, 1):
            c = 2 * loaded[kv] + kv
            if loaded[kv] < tiles and (c < stages or passes(empty[c % stages], c // stages - 1)):
                acts.append((True, kv, c))
            c = 2 * read[kv] + kv
            if read[kv] < tiles and full[c % stages] > 0 and passes(full[c % stages], c // stages):
                acts.append((False, kv, c))
        if not acts:
            return "nothing can go on"
        load, kv, c = rng.choice(acts)
        st = c % stages
        if load:
            if held[st] is not None:
                return f"tile {c} over {held[st]}"
            held[st] = c
            full[st] += 1
            loaded[kv] += 1
        else:
            if held[st] != c:
                return f"{held[st]} read for {c}"
            held[st] = None
            empty[st] += 1
            read[kv] += 1
    return "ok"


@pytest.mark.parametrize("stages", [2, 4, 6])
def test_raw_ring_of_two_producers_needs_an_even_number_of_stages(stages):
    assert all(raw_ring(stages, 12, random.Random(s)) == "ok" for s in range(400))


def test_raw_ring_model_catches_shared_stages():
    assert any(raw_ring(3, 12, random.Random(s)) != "ok" for s in range(400))


def few_rows(slots, ahead, steps, rng):
    """The kernel for few rows: the MMA thread issues S `ahead` steps before P V, two softmax groups
    take alternate steps, P is announced on `slots` barriers.  P(g) goes to one of 4 buffers."""
    s_done, ready, pv = 0, [0] * slots, 0          # S complete up to, P announced, P V issued
    done = [0, 0]                                  # steps each group has finished
    buffer = [None] * 4
    while pv < steps:
        acts = []
        if s_done < min(steps, pv + ahead):
            acts.append(("s", s_done))
        for x in (0, 1):
            g = 2 * done[x] + x
            if g < min(steps, s_done):
                acts.append(("p", g))
        if s_done > pv and passes(ready[pv % slots], pv // slots):
            acts.append(("pv", pv))
        if not acts:
            return "nothing can go on"
        what, g = rng.choice(acts)
        if what == "s":
            s_done += 1
        elif what == "p":
            if buffer[g % 4] is not None:
                return f"P({g}) over P({buffer[g % 4]})"
            buffer[g % 4] = g
            ready[g % slots] += 1
            done[g % 2] += 1
        else:
            if buffer[g % 4] != g:
                return f"P V({g}) reads {buffer[g % 4]}"
            buffer[g % 4] = None
            pv += 1
    return "ok"


@pytest.mark.parametrize("ahead", [2, 3])
def test_few_rows_schedule_with_a_barrier_per_buffer(ahead):
    assert all(few_rows(4, ahead, 40, random.Random(s)) == "ok" for s in range(400))


def test_few_rows_model_catches_a_group_two_steps_ahead_of_one_barrier_per_group():
    assert any(few_rows(2, 3, 40, random.Random(s)) != "ok" for s in range(400))
