"""The order of waits of the persistent commit kernel warp by warp, on the CPU.

The model of test_commit_protocol.py with two or four producer warps a group (bf16 and float32 nodes)
and a group's four warps as actors of their own: each waits and arrives for itself, so that they may
be anywhere between the first and the last of them."""
import random

import pytest

from tests.test_commit_protocol import BUFS, SLOTS, Barrier, Wrong

WARPS = 4


class Model:
    """One CTA.  chunks[i]: slots of head number i.  ``arrivals``: how many warps of a group a slot
    or a buffer waits for before it is filled again."""

    def __init__(self, chunks, producers, rng, state_first=False, all_ahead=False, arrivals=WARPS):
        self.chunks, self.producers, self.rng = chunks, producers, rng
        self.state_first, self.all_ahead, self.arrivals = state_first, all_ahead, arrivals
        self.state_full = [Barrier(1) for _ in range(BUFS)]
        self.state_empty = [Barrier(arrivals) for _ in range(BUFS)]
        self.full = [[Barrier(producers) for _ in range(SLOTS)] for _ in range(2)]
        self.empty = [[Barrier(arrivals) for _ in range(SLOTS)] for _ in range(2)]
        self.buffer, self.copies = [None] * BUFS, []
        self.slot = [[{} for _ in range(SLOTS)] for _ in range(2)]

    def producer(self, grp, part):
        """Brings its part of every slot; the first of a group also asks for the states."""
        my, following = len(self.chunks), grp

        def states(upto, may):
            nonlocal following
            while part == 0 and following < my and following <= may:
                i, use = following, following // BUFS
                if use:
                    ready = lambda: self.state_empty[i % BUFS].done((use - 1) & 1)  # noqa: E731
                    if i <= upto:
                        while not ready():
                            yield
                    elif not ready():
                        return
                self.state_full[i % BUFS].arrive(copies=1)
                self.copies.append((i % BUFS, i))
                following += 2
                yield

        ahead = my if self.all_ahead else 2
        yield from states(grp, grp + ahead)
        number = 0
        for i in range(grp, my, 2):
            for c in range(self.chunks[i]):
                yield from states(i, i + (ahead if self.all_ahead else 0))
                to = number % SLOTS
                while number >= SLOTS and not self.empty[grp][to].done((number // SLOTS - 1) & 1):
                    yield
                yield from states(i, i + ahead)
                self.slot[grp][to][part] = (i, c)
                yield
                self.full[grp][to].arrive()
                number += 1
                yield

    def group_warp(self, grp, warp):
        number = 0

        def nodes():
            while not self.full[grp][number % SLOTS].done((number // SLOTS) & 1):
                yield

        for i in range(grp, len(self.chunks), 2):
            if not self.state_first:
                yield from nodes()
            buf = i % BUFS
            while not self.state_full[buf].done((i // BUFS) & 1):
                yield
            for _ in range(2):
                if self.buffer[buf] != i:
                    raise Wrong("head %d reads the state of %s" % (i, self.buffer[buf]))
                yield
            if warp < self.arrivals:
                self.state_empty[buf].arrive()
            for c in range(self.chunks[i]):
                yield from nodes()
                for _ in range(self.rng.randint(1, 4)):
                    if self.slot[grp][number % SLOTS] != {p: (i, c) for p in range(self.producers)}:
                        raise Wrong("slot")
                    yield
                if warp < self.arrivals:
                    self.empty[grp][number % SLOTS].arrive()
                number += 1

    def run(self):
        rng = self.rng
        warps = [self.producer(g, p) for g in (0, 1) for p in range(self.producers)]
        warps += [self.group_warp(g, w) for g in (0, 1) for w in range(WARPS)]
        speed = [rng.random() ** 3 + 0.01 for _ in warps]
        memory = rng.random() ** 3 + 0.005
        for _ in range(1000000):
            if not warps:
                break
            if self.copies and rng.random() < memory:
                buf, i = self.copies.pop(rng.randrange(len(self.copies)))
                self.buffer[buf] = i
                self.state_full[buf].copied()
            k = rng.choices(range(len(warps)), speed)[0]
            try:
                next(warps[k])
            except StopIteration:
                del warps[k], speed[k]
        if warps or self.copies:
            raise Wrong("it does not end")


def fails(seed, producers, **order):
    rng = random.Random(1000 * producers + seed)
    chunks = [rng.choice([1, 1, 1, 2, 2, 3, 8]) for _ in range(rng.randint(1, 12))]
    try:
        Model(chunks, producers, rng, **order).run()
    except Wrong:
        return True
    return False


@pytest.mark.parametrize("producers", [2, 4])
def test_the_kernels_order(producers):
    assert not any(fails(seed, producers) for seed in range(80))


@pytest.mark.parametrize("producers", [2, 4])
@pytest.mark.parametrize("order", [dict(state_first=True), dict(all_ahead=True), dict(arrivals=1)])
def test_orders_that_are_wrong_are_seen(order, producers):
    """A group that waits for its state before its nodes; states asked for as far ahead as the
    barriers seem to allow; slots and buffers that are free when one of the four warps is done."""
    assert any(fails(seed, producers, **order) for seed in range(60))
