"""The barriers of the block-scaled products, modelled on the CPU: agents that run in any order, copies that end in any
order, and barriers that tell phases by their parity alone, as the hardware's do.

The model has what the kernels have: a loader that fills a ring of stages, two issuing warps that take K blocks in turn
(or one half of every block each), accumulator slots and a promoting side that takes blocks in order.  Every step
asserts what the kernel relies on: the stage that is multiplied holds its block and no copy is under way, a slot that is
written has been read, a barrier is armed only when its last phase is over."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_gemm_dequant_gb300", "csrc",
                   "block", "hq_gemm_block.cuh")


class Broken(Exception):
    pass


class Barrier:
    def __init__(self, count=1):
        self.count, self.left, self.done = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def passes(self, parity):  # a wait for the phase of this parity: over when the current phase has the other one
        return self.done & 1 != parity


def simulate(seed, stages, slots, tiles, slot_first=True, halves=1, late=0.0):
    """tiles: K blocks of each tile.  Raises Broken where a step finds something else than it relies on."""
    rng = random.Random(seed)
    full, empty = [Barrier() for _ in range(stages)], [Barrier(halves) for _ in range(stages)]
    dfull, dempty = [Barrier() for _ in range(slots)], [Barrier() for _ in range(slots)]
    held, flying, acc = [None] * stages, {}, [None] * slots
    depth = slots // halves
    blocks = [(t, b) for t, n in enumerate(tiles) for b in range(n)]
    base = [sum(tiles[:t]) for t in range(len(tiles))]

    def loader():
        for n, _ in enumerate(blocks):
            s, f = n % stages, n // stages
            yield lambda: empty[s].passes((f & 1) ^ 1)
            if full[s].done != f or s in flying:
                raise Broken("a stage's barrier is armed while a phase is open")
            flying[s] = n

    def copies():
        while True:
            yield lambda: bool(flying)
            s = rng.choice(list(flying)) if rng.random() < 0.7 or late == 0 else max(flying, key=flying.get)
            held[s] = flying.pop(s)
            full[s].arrive()

    def issuer(w):
        phase = [0] * slots
        todo = []  # MMAs under way: (stage, slot, block), in order
        for t, n in enumerate(tiles):
            for b in range(w if halves == 1 else 0, n, 2 if halves == 1 else 1):
                i = base[t] + b
                s, f = i % stages, i // stages
                d = (b % depth) * halves + (w if halves == 2 else 0)
                waits = [lambda: dempty[d].passes(phase[d] ^ 1), lambda: full[s].passes(f & 1)]
                for k in (0, 1) if slot_first else (1, 0):
                    yield waits[k]
                phase[d] ^= 1
                if held[s] != i or s in flying:
                    raise Broken("a stage is multiplied that does not hold its block")
                if acc[d] is not None:
                    raise Broken("a slot is written that has not been read")
                todo.append((s, d, i))
                yield lambda: True
                s, d, i = todo.pop(0)
                acc[d] = i
                empty[s].arrive()
                dfull[d].arrive()

    def promoter(h):
        phase = [0] * slots
        for t, n in enumerate(tiles):
            for b in range(n):
                d = (b % depth) * halves + h
                yield lambda: dfull[d].passes(phase[d])
                phase[d] ^= 1
                if acc[d] != base[t] + b:
                    raise Broken("a slot does not hold the block that is promoted")
                acc[d] = None
                dempty[d].arrive()

    agents = [loader(), copies(), issuer(0), issuer(1)] + [promoter(h) for h in range(halves)]
    weights = [rng.choice([1, 1, 4, 30]) for _ in agents]
    ready = [next(a, None) for a in agents]
    idle = 0
    while any(r is not None for k, r in enumerate(ready) if k != 1):
        k = rng.choices(range(len(agents)), weights)[0]
        if ready[k] is None or not ready[k]():
            idle += 1
            if idle > 20000:
                raise Broken("nobody can go on")
            continue
        idle = 0
        ready[k] = next(agents[k], None)


def _constants():
    s = open(SRC).read()
    few = dict(zip((16, 32, 64, 128), map(int, re.search(
        r"STAGES = BT == 16 \? (\d+) : \(BT == 32 \? (\d+) : \(BT == 64 \? (\d+) : (\d+)\)\)", s).groups())))
    pair = dict(zip((256, 128), map(int, re.search(r"STAGES = BN == 256 \? (\d+) : (\d+)", s).groups())))
    assert re.search(r"SLOTS = 4;", s) and re.search(r"SLOTS = 512 / SN", s) and re.search(r"SN = 128;", s)
    return few, pair


def test_few_tokens():
    few, _ = _constants()
    for stages in few.values():
        assert stages % 2 == 0
        for seed in range(300):
            simulate(seed, stages, 4, [random.Random(seed).choice([1, 2, 3, 5, 7, 8, 20, 57])], late=0.3)


def test_pairs():
    _, pair = _constants()
    for seed in range(300):
        rng = random.Random(seed)
        tiles = [rng.choice([1, 2, 3, 5, 8, 13])] * rng.choice([1, 2, 5])
        simulate(seed, pair[256], 4, tiles, halves=2, late=0.3)
        simulate(seed, pair[128], 4, tiles, late=0.3)


@pytest.mark.parametrize("slot_first,stages,tiles", [(False, 5, [57])])
def test_the_model_sees_an_odd_ring_with_the_stage_awaited_first(slot_first, stages, tiles):
    """A warp that takes every second fill of a stage passes on the fill before, once in a while."""
    with pytest.raises(Broken):
        for seed in range(3000):
            simulate(seed, stages, 4, tiles, slot_first=slot_first, late=0.5)
