"""A model of the ring of raw tiles between the loader and the expanders of the attention kernel for
many query rows (CPU only): whatever the order in which copies land, an expander reads a slot only
after its own fill has landed there."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_expert_ffn_b200", "csrc", "kv_attn_tc.cu")


class Barrier:
    """An mbarrier: a phase ends when its arrivals and bytes are in; a wait for a parity is over when
    the phase under way has the other parity."""

    def __init__(self, count):
        self.count, self.left, self.tx, self.phase = count, count, 0, 0

    def _end(self):
        if self.left == 0 and self.tx == 0:
            self.phase, self.left = self.phase + 1, self.count

    def arrive(self, tx=0):
        assert self.left > 0, "more arrivals than the phase takes"
        self.left, self.tx = self.left - 1, self.tx + tx
        self._end()

    def landed(self, tx):
        self.tx -= tx
        self._end()

    def passed(self, parity):
        return (self.phase & 1) != parity


def run(slots, bars, tiles, seed, slow):
    """Fills 2t (K) and 2t + 1 (V) of slot n % slots, announced on barrier n % bars, read by an
    expander of each kind. Copies land in random order, each in `slow` of the steps only. Returns what
    goes wrong first, or None."""
    rng = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(bars)], [Barrier(1) for _ in range(slots)]
    holds, flying, n_fill, done = [None] * slots, [], 0, [0, 0]
    while min(done) < tiles:
        what = rng.choice(["load", "land", "K", "V", "V", "K"])
        if what == "load" and n_fill < 2 * tiles:
            if empty[n_fill % slots].passed(((n_fill // slots) & 1) ^ 1):
                try:
                    full[n_fill % bars].arrive(tx=1)
                except AssertionError as e:
                    return str(e)
                flying.append(n_fill)
                n_fill += 1
        elif what == "land" and flying and rng.random() < slow:
            n = flying.pop(rng.randrange(len(flying)))
            holds[n % slots] = n
            full[n % bars].landed(1)
        elif what in "KV":
            kind = "KV".index(what)
            n = 2 * done[kind] + kind
            if done[kind] < tiles and full[n % bars].passed((n // bars) & 1):
                if holds[n % slots] != n:
                    return f"fill {n} read from slot {n % slots} which holds {holds[n % slots]}"
                done[kind] += 1
                empty[n % slots].arrive()
    return None


def kernel_ring():
    text = open(SRC).read()
    slots = [int(x) for x in re.search(r"raw_slots = D == 128 \? (\d+) : (\d+);", text).groups()]
    twice = re.search(r"raw_bars = raw_slots % 2 \? 2 \* raw_slots : raw_slots;", text) is not None
    return sorted({(n, 2 * n if twice and n % 2 else n) for n in slots})


@pytest.mark.parametrize("slots,bars", kernel_ring())
def test_no_expander_reads_a_fill_that_has_not_landed(slots, bars):
    for seed in range(400):
        assert run(slots, bars, 12, seed, 0.3) is None, seed


def test_the_model_finds_a_barrier_shared_by_both_kinds():
    assert any(run(3, 3, 12, seed, 0.3) for seed in range(400))
    assert not any(run(n, n, 12, seed, 0.3) for n in (2, 4, 8) for seed in range(100))
