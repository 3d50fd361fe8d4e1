"""A model of the copies, the two converting warpgroups and the consumer of the 8-bit chunk kernel
(csrc/qg_chunk.cu, heads of 256) that meet on phase-parity barriers, run under random orders.

A barrier knows only the parity of the phase it is in: a wait for a phase whose predecessor is still
open returns at once.  Nothing orders the arrival of copies, so the model lets them land in any order."""
import random

import pytest

AREAS = SLOTS = 3  # NRAW, NS
GROUPS = 2         # NCONV


class Barrier:
    def __init__(self):
        self.done = 0  # phases completed

    def passes(self, phase):
        return (self.done & 1) != (phase & 1)


def run(units, barriers, rng):
    """Steps the model in random order to the end; units of codes read before they had landed, or None
    where nothing could move any more."""
    full, empty = [Barrier() for _ in range(barriers)], [Barrier() for _ in range(AREAS)]
    tile_full, tile_empty = [Barrier() for _ in range(SLOTS)], [Barrier() for _ in range(SLOTS)]
    landed, flight, wrong = [], [], []
    copied, used, conv = 0, 0, list(range(GROUPS))  # next unit of the copies, the consumer, each group
    past = [False] * GROUPS                         # the group's wait for codes is over, that for the slot not yet
    bias = [rng.random() ** 3 for _ in range(4)]
    while used < units:
        moves = []
        if copied < units and (copied < AREAS or empty[copied % AREAS].passes(copied // AREAS - 1)):
            moves.append(0)
        if flight:
            moves.append(1)
        ready = [g for g in range(GROUPS) if conv[g] < units and
                 ((conv[g] < SLOTS or tile_empty[conv[g] % SLOTS].passes(conv[g] // SLOTS - 1)) if past[g] else
                  full[conv[g] % barriers].passes(conv[g] // barriers))]
        if ready:
            moves.append(2)
        if tile_full[used % SLOTS].passes(used // SLOTS):
            moves.append(3)
        if not moves:
            return None
        m = rng.choices(moves, [0.02 + bias[i] for i in moves])[0]
        if m == 0:
            flight.append(copied)
            copied += 1
        elif m == 1:  # any copy in flight may land first
            u = flight.pop(rng.randrange(len(flight)))
            landed.append(u)
            full[u % barriers].done += 1
        elif m == 2:
            g = rng.choice(ready)
            past[g] = not past[g]
            if past[g]:
                continue
            if conv[g] not in landed:
                wrong.append(conv[g])
            empty[conv[g] % AREAS].done += 1
            tile_full[conv[g] % SLOTS].done += 1
            conv[g] += GROUPS
        else:
            tile_empty[used % SLOTS].done += 1
            used += 1
    return wrong


@pytest.mark.parametrize("seed", range(8))
def test_barriers_of_one_warpgroup_each_never_mislead(seed):
    rng = random.Random(seed)
    for _ in range(300):
        assert run(rng.randrange(1, 40), AREAS * GROUPS, rng) == []


def test_the_model_sees_the_fault_of_shared_barriers():
    rng = random.Random(1)
    results = [run(40, AREAS, rng) for _ in range(300)]
    assert any(r is None or r for r in results)


def test_the_kernel_has_a_barrier_per_area_and_warpgroup():
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gguf_block_quantized_quant_gb300", "csrc", "qg_chunk.cu")
    with open(path) as f:
        text = f.read()
    assert re.search(r"NRAWBAR = NRAW \* \(NCONV > 1 \? NCONV : 1\)", text)
    assert "raw_full(units % Cfg::NRAWBAR)" in text and "raw_full(n % Cfg::NRAWBAR), (n / Cfg::NRAWBAR) & 1" in text
