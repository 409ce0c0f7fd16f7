"""The barrier protocol of the tcgen05 attention kernels (fc_attention_tc.cu, fc_attention_tc_vjp.cu) under random
schedules.

A parity wait passes whenever the last completed phase has that parity, so that a waiter who is two phases behind
passes early.  The model steps the roles of a block (copies, matrix products, an in-order tensor pipe, two groups of
four row warps) in random order, with some of them much slower than others, and records every wait that passes before
the phase it means is complete."""
import random

import pytest


class Barrier:
    def __init__(self, count=1):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1


def early_waits(tiles, stages, bufs, ahead, outputs, last, seed):
    """bufs: score tiles in tensor memory; ahead: how many tiles the scores are issued before the weights are needed;
    outputs: "groups" (one output and barrier per group: forward) or "tiles" (a barrier per score tile: gradient);
    last: what the row warps wait for at the end, "drain" or "product"."""
    rng, early = random.Random(seed), []
    full = [Barrier() for _ in range(stages)]
    scored = [Barrier() for _ in range(bufs)]
    weighed = [Barrier(4) for _ in range(bufs)]
    product = [Barrier() for _ in range(2 if outputs == "groups" else bufs)]
    drain, pipe, finished = Barrier(), [], [0]
    of = (lambda i: (product[i & 1], i >> 1)) if outputs == "groups" else (lambda i: (product[i % bufs], i // bufs))

    def wait(who, bar, phase):
        while (bar.phase & 1) == (phase & 1):     # the phase of this parity is not the last completed one
            yield
        if bar.phase <= phase:
            early.append(who)

    def copies():
        for i in range(tiles):
            while finished[0] < i - stages + 1:
                yield
            full[i % stages].arrive()
            yield

    def scores(i):
        yield from wait("products: tile", full[i % stages], i // stages)
        pipe.append(("score", scored[i % bufs]))
        yield

    def products():
        for i in range(min(ahead, tiles)):
            yield from scores(i)
        for i in range(tiles):
            yield from wait("products: weights", weighed[i % bufs], i // bufs)
            yield
            pipe.append(("product", of(i)[0]))
            yield
            if i + ahead < tiles:
                # the columns of the next scores: those of tile i (gradient), of tile i - 1 (forward)
                old = i + ahead - bufs
                if old >= 0:
                    yield from wait("products: columns", *of(old))
                yield from scores(i + ahead)
        pipe.append(("drain", drain))

    def tensor():
        while not drain.phase:
            if pipe:
                kind, bar = pipe.pop(0)
                bar.arrive()
                finished[0] += kind == "product"
            yield

    def rows(group):
        for i in range(group, tiles, 2):
            yield from wait("rows: tile", full[i % stages], i // stages)
            yield from wait("rows: scores", scored[i % bufs], i // bufs)
            if outputs == "groups" and i >= 2 and rng.random() < 0.3:    # the reference is raised
                yield from wait("rows: rescale", *of(i - 2))
            yield
            weighed[i % bufs].arrive()
        if outputs == "groups" and tiles <= group:
            return
        mine = tiles - 1 if outputs == "tiles" or (tiles - 1) % 2 == group else tiles - 2
        yield from wait("rows: end", *((drain, 0) if last == "drain" else of(mine)))

    run = [copies(), products(), tensor()] + [rows(g) for g in (0, 1) for _ in range(4)]
    speed = [rng.choice([1, 1, 10, 100]) for _ in run]
    while run:
        k = rng.choices(range(len(run)), speed)[0]
        try:
            next(run[k])
        except StopIteration:
            del run[k], speed[k]
    return early


FORWARD = dict(bufs=4, ahead=3, outputs="groups")
PROTOCOLS = {"forward": dict(FORWARD, stages=8), "forward, wide": dict(FORWARD, stages=5),
             "gradient": dict(bufs=3, ahead=3, outputs="tiles", stages=6),
             "gradient, wide": dict(bufs=3, ahead=3, outputs="tiles", stages=4),
             "key and value gradient, wide": dict(bufs=2, ahead=2, outputs="tiles", stages=4)}


@pytest.mark.parametrize("name", list(PROTOCOLS))
def test_no_wait_passes_early(name):
    for seed in range(120):
        assert early_waits(1 + seed % 14, last="drain", seed=seed, **PROTOCOLS[name]) == [], seed


@pytest.mark.parametrize("name", list(PROTOCOLS))
def test_the_model_sees_a_wait_on_a_barrier_of_several_phases(name):
    """Waiting at the end for the barrier of the last product can pass a phase early: a group is done with its last
    tile while the products of the one before are open."""
    found = set()
    for seed in range(120):
        found.update(early_waits(1 + seed % 14, last="product", seed=seed, **PROTOCOLS[name]))
    assert found == {"rows: end"}
