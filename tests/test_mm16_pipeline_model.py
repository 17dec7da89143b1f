"""CPU: a model of the 16-bit products' barrier protocol under random interleavings.

The persistent kernel (csrc/mm16_tc.cu) runs, over a ring of stages whose waits test only a phase's
parity: two TMA producers in each CTA of the tile, one of each operand (one CTA, or the two of a pair, whose copies all
report to the leader's full barrier, perhaps before its A producer has announced their bytes), the thread that issues the MMAs (the leader's; its commits complete in issue
order and release the stage in every CTA), for ragged reductions a cleaner that passes every stage,
clears a tile's last one where the group ends inside a step of 16, and has to arrive on the stage's empty
barrier too, and the epilogue warps of every CTA, which hand accumulators back to the leader. Two accumulators
take turns (several to a tile where the result is fp32), or lie side by side and are handed back one by one.

`simulate` asserts for every wait that its barrier is at the phase waited for or the next one (two phases off,
the parity would answer wrongly), for every arrival and copy that it lands in its own phase, and that the run ends.
A cleaner that goes straight to the stages it clears, as a first version of the kernel did, is caught.
"""
import random

import pytest

from test_gemm_pipeline_model import Bar, Violation

WARPS = 3  # epilogue warps per CTA (the kernel has eight: the count does not matter to the protocol)


def simulate(seed, ctas, stages, tiles, ragged=False, seg=None, side_by_side=False, eager_cleaner=False):
    """tiles: (stages, ends inside a step) of each; seg: stages that one accumulator takes."""
    rng = random.Random(seed)
    full = [Bar(f"full[{i}]", 1) for i in range(stages)]
    empty = [[Bar(f"empty[{c}][{i}]", 2 if ragged and not eager_cleaner else 1) for i in range(stages)] for c in range(ctas)]
    clean = [Bar(f"clean[{i}]", 1) for i in range(stages)]
    acc_full = [[Bar(f"acc_full[{c}][{i}]", 1) for i in range(2)] for c in range(ctas)]
    acc_empty = [Bar(f"acc_empty[{i}]", WARPS * ctas) for i in range(2)]
    landing, mma_queue = [], []  # copies in flight; commits in issue order

    def wait(bar, k):
        bar.check_wait(k)
        while not bar.done(k):
            yield
        bar.check_wait(k)

    def producer(c, of_a):
        g = 0
        for n, _ in tiles:
            for _ in range(n):
                s, use = g % stages, g // stages
                yield from wait(empty[c][s], use - 1)
                if c == 0 and of_a:
                    full[s].arrive(use, tx=2 * ctas)
                yield
                landing.append((full[s], use))
                g += 1

    def mma():
        g, acc, cleaned = 0, 0, [0] * stages
        for t, (n, tail) in enumerate(tiles):
            in_seg = 0
            for k in range(n):
                s, use = g % stages, g // stages
                if in_seg == 0:
                    if side_by_side:
                        yield from wait(acc_empty[0 if k == 0 else 1], t - 1)
                    else:
                        yield from wait(acc_empty[acc % 2], acc // 2 - 1)
                yield from wait(full[s], use)
                if ragged and tail and k == n - 1:
                    yield from wait(clean[s], cleaned[s])
                    cleaned[s] += 1
                mma_queue.append([(empty[c][s], use) for c in range(ctas)])
                g += 1
                in_seg += 1
                if k == n - 1 or (not side_by_side and in_seg == seg):
                    i, phase = (0, t) if side_by_side else (acc % 2, acc // 2)
                    mma_queue.append([(acc_full[c][i], phase) for c in range(ctas)])
                    acc += 1
                    in_seg = 0
                elif in_seg == seg:
                    in_seg = 0
                yield

    def cleaner():
        g, cleaned = 0, [0] * stages
        for n, tail in tiles:
            for k in range(n):
                s, use = g % stages, g // stages
                g += 1
                last = tail and k == n - 1
                if eager_cleaner and not last:
                    continue
                yield from wait(full[s], use)
                yield
                if last:
                    clean[s].arrive(cleaned[s])
                    cleaned[s] += 1
                if not eager_cleaner:
                    empty[0][s].arrive(use)

    def epilogue(c):
        acc = 0
        for t, (n, _) in enumerate(tiles):
            for _ in range(1 if side_by_side or not seg else -(-n // seg)):
                if side_by_side:
                    yield from wait(acc_full[c][0], t)
                    yield
                    acc_empty[0].arrive(t)
                    yield
                    acc_empty[1].arrive(t)
                else:
                    yield from wait(acc_full[c][acc % 2], acc // 2)
                    yield
                    acc_empty[acc % 2].arrive(acc // 2)
                acc += 1

    actors = [producer(c, of_a) for c in range(ctas) for of_a in (True, False)] + [mma()] + [epilogue(c) for c in range(ctas) for _ in range(WARPS)]
    if ragged:
        actors.append(cleaner())
    weight = [rng.choice((1, 1, 5)) for _ in actors]  # some actors run far more often than others
    idle = 0
    while actors or landing or mma_queue:
        before = (len(actors), len(landing), len(mma_queue), sum(b.phase + b.arrived for b in full + clean + acc_empty))
        kind = rng.random()
        if kind < 0.15 and landing:
            bar, use = landing.pop(rng.randrange(len(landing)))
            bar.land(use)
        elif kind < 0.3 and mma_queue:
            for bar, use in mma_queue.pop(0):
                bar.arrive(use)
        elif actors:
            i = rng.choices(range(len(actors)), weight)[0]
            try:
                next(actors[i])
            except StopIteration:
                del actors[i], weight[i]
        after = (len(actors), len(landing), len(mma_queue), sum(b.phase + b.arrived for b in full + clean + acc_empty))
        idle = 0 if before != after else idle + 1
        if idle > 20000:
            raise Violation("nothing moves any more")


def tiles_of(rng, most, count):
    return [(rng.randint(1, most), rng.random() < 0.7) for _ in range(count)]


@pytest.mark.parametrize("ctas,stages", [(1, 4), (1, 2), (2, 6), (2, 5), (1, 12)])
@pytest.mark.parametrize("seed", range(12))
def test_stages_and_two_accumulators(ctas, stages, seed):
    simulate(seed, ctas, stages, tiles_of(random.Random(seed), 9, 14))


@pytest.mark.parametrize("stages", [2, 4, 9])
@pytest.mark.parametrize("seed", range(25))
def test_ragged_reductions(stages, seed):
    simulate(seed, 1, stages, tiles_of(random.Random(seed), 7, 18), ragged=True)
    simulate(seed, 1, stages, tiles_of(random.Random(seed), 17, 8), ragged=True, seg=8)


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("seed", range(12))
def test_several_accumulators_a_tile(ctas, seed):
    simulate(seed, ctas, 4, tiles_of(random.Random(seed), 20, 8), seg=6)


@pytest.mark.parametrize("seed", range(12))
def test_accumulators_side_by_side(seed):
    rng = random.Random(seed)
    half = rng.randint(3, 9)
    simulate(seed, 1, 4, [(2 * half - rng.randint(0, 1), False)] * 9, seg=half, side_by_side=True)


def test_a_cleaner_that_skips_stages_is_caught():
    caught = 0
    for seed in range(60):
        rng = random.Random(seed)
        try:
            simulate(seed, 1, 4, [(rng.choice((2, 3, 9)), rng.random() < 0.5) for _ in range(30)], ragged=True, eager_cleaner=True)
        except Violation:
            caught += 1
    assert caught > 10
