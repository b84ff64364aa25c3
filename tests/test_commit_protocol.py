"""The order of waits of the persistent commit kernel, on the CPU.

A model of its barriers (a phase ends when all arrivals and copies of it are in; a wait tells a
phase only from the one before it) run in random interleavings: every head's state is read whole and
not overwritten under its reader, no barrier gets more arrivals than a phase has, and all ends.
Two orders that the kernel must not have are caught by the same model."""
import random

import pytest

BUFS, SLOTS = 3, 2


class Wrong(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.copies = self.phase = 0

    def arrive(self, copies=0):
        if self.pending <= 0:
            raise Wrong("more arrivals than the phase has")
        self.copies += copies
        self.pending -= 1
        self.settle()

    def copied(self):
        self.copies -= 1
        self.settle()

    def settle(self):
        if self.pending == 0 and self.copies == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, parity):
        return (self.phase & 1) != parity


class Model:
    """One CTA: two groups, two producer warps each; chunks[i] slots for head number i."""

    def __init__(self, chunks, rng, state_first=False, all_ahead=False):
        self.chunks, self.rng = chunks, rng
        self.state_first, self.all_ahead = state_first, all_ahead
        self.state_full = [Barrier(1) for _ in range(BUFS)]
        self.state_empty = [Barrier(1) for _ in range(BUFS)]
        self.full = [[Barrier(2) for _ in range(SLOTS)] for _ in range(2)]
        self.empty = [[Barrier(1) for _ in range(SLOTS)] for _ in range(2)]
        self.buffer, self.copies = [None] * BUFS, []
        self.slot = [[{} for _ in range(SLOTS)] for _ in range(2)]

    def producer(self, grp, half):
        my, following = len(self.chunks), grp

        def states(upto, may):
            nonlocal following
            while half == 0 and following < my and following <= may:
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
                self.slot[grp][to][half] = (i, c)
                yield
                self.full[grp][to].arrive()
                number += 1
                yield

    def group(self, grp):
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
            self.state_empty[buf].arrive()
            for c in range(self.chunks[i]):
                yield from nodes()
                for _ in range(self.rng.randint(1, 6)):
                    if self.slot[grp][number % SLOTS] != {0: (i, c), 1: (i, c)}:
                        raise Wrong("slot")
                    yield
                self.empty[grp][number % SLOTS].arrive()
                number += 1

    def run(self):
        rng = self.rng
        warps = [self.producer(g, h) for g in (0, 1) for h in (0, 1)]
        warps += [self.group(0), self.group(1)]
        speed = [rng.random() ** 3 + 0.01 for _ in warps]
        memory = rng.random() ** 3 + 0.005
        for _ in range(400000):
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


def failures(seeds, **order):
    n = 0
    for seed in range(seeds):
        rng = random.Random(seed)
        chunks = [rng.choice([1, 1, 1, 2, 2, 3, 8]) for _ in range(rng.randint(1, 16))]
        try:
            Model(chunks, rng, **order).run()
        except Wrong:
            n += 1
    return n


def test_the_kernels_order():
    assert failures(150) == 0


@pytest.mark.parametrize("order", [dict(state_first=True), dict(all_ahead=True)])
def test_orders_that_are_wrong_are_seen(order):
    """A group that waits for its state before its nodes; states asked for as far ahead as the
    barriers seem to allow."""
    assert failures(60, **order) > 0
