"""CPU: a model of the 16-bit products' barriers where a pair of CTAs sums up ragged groups, and where tiles wider than one
accumulator take both (csrc/mm16_tc.cu).

Ragged pairs: both CTAs' copies report to the leader's full barrier, but those of a ragged end each to its own CTA's, where
its cleaner waits for them, clears the end and arrives at the leader, whose MMA waits for both cleaners. The leader's
cleaner passes every stage and takes part in its release, so that the ring cannot lap it; the other CTA's full barriers
see nothing but ragged ends, so that its cleaner may skip the rest.

Wide tiles: the MMA waits for both accumulators and commits both; the epilogue waits for both and hands both back; narrower
tiles before and after go on taking turns.

The rules are those of the other model: every wait's barrier is at the phase waited for or the next one, every arrival
lands in its own phase, and the run ends.
"""
import random

import pytest

from test_gemm_pipeline_model import Bar

WARPS = 3


def run(actors, queues, rng):
    """actors: generators; queues: (list, in order) of things that complete by themselves."""
    weight = [rng.choice((1, 1, 5)) for _ in actors]
    for step in range(60000):
        live = [i for i, a in enumerate(actors) if a is not None]
        if not live and not any(q for q, _ in queues):
            return
        waiting = [(q, ordered) for q, ordered in queues if q]
        if waiting and (not live or rng.random() < 0.3):
            q, ordered = rng.choice(waiting)
            q.pop(0 if ordered else rng.randrange(len(q)))()
            continue
        i = rng.choices(live, [weight[j] for j in live])[0]
        try:
            next(actors[i])
        except StopIteration:
            actors[i] = None
    raise AssertionError("the run did not end")


def wait(bar, k):
    bar.check_wait(k)
    while not bar.done(k):
        yield
    bar.check_wait(k)


def ragged_pair(seed, stages, tiles, forgets=False):
    """tiles: (stages, ends inside a step of 16). forgets: the leader's cleaner visits ragged ends alone."""
    rng = random.Random(seed)
    full = [[Bar(f"full[{c}][{i}]", 1) for i in range(stages)] for c in range(2)]
    empty = [[Bar(f"empty[{c}][{i}]", 1 if c or forgets else 2) for i in range(stages)] for c in range(2)]
    clean = [Bar(f"clean[{i}]", 2) for i in range(stages)]
    acc_full = [[Bar(f"acc_full[{c}][{i}]", 1) for i in range(2)] for c in range(2)]
    acc_empty = [Bar(f"acc_empty[{i}]", 2 * WARPS) for i in range(2)]
    landing, commits = [], []

    def walk():
        """(stage, its use, ragged ends in it before, whether this one is) in turn"""
        g, ends = 0, [0] * stages
        for n, tail in tiles:
            for k in range(n):
                s, last = g % stages, tail and k == n - 1
                yield s, g // stages, ends[s], last
                ends[s] += last
                g += 1

    def producer(c, of_a):
        for s, use, ends, last in walk():
            yield from wait(empty[c][s], use - 1)
            to, phase = (full[1][s], ends) if c and last else (full[0][s], use)
            if of_a and (c == 0 or last):
                to.arrive(phase, tx=2 if last else 4)
            yield
            landing.append(lambda to=to, phase=phase: to.land(phase))

    def cleaner(c):
        for s, use, ends, last in walk():
            if (c or forgets) and not last:
                continue
            yield from wait(full[c][s], ends if c else use)
            yield
            if last:
                clean[s].arrive(ends)
            if c == 0 and not forgets:
                empty[0][s].arrive(use)

    def mma():
        turn = walk()
        for acc, (n, _) in enumerate(tiles):
            yield from wait(acc_empty[acc % 2], acc // 2 - 1)
            for _ in range(n):
                s, use, ends, last = next(turn)
                yield from wait(full[0][s], use)
                if last:
                    yield from wait(clean[s], ends)
                commits.append(lambda s=s, use=use: [empty[c][s].arrive(use) for c in range(2)])
                yield
            commits.append(lambda acc=acc: [acc_full[c][acc % 2].arrive(acc // 2) for c in range(2)])

    def epilogue(c):
        for acc in range(len(tiles)):
            yield from wait(acc_full[c][acc % 2], acc // 2)
            yield
            acc_empty[acc % 2].arrive(acc // 2)

    actors = [producer(c, a) for c in range(2) for a in (True, False)] + [cleaner(0), cleaner(1), mma()] + [epilogue(c) for c in range(2) for _ in range(WARPS)]
    run(actors, [(landing, False), (commits, True)], rng)


def wide_tiles(seed, stages, tiles, half_commit=False):
    """tiles: (stages, wide). half_commit: a wide tile that commits only its first accumulator."""
    rng = random.Random(seed)
    empty = [Bar(f"empty[{i}]", 1) for i in range(stages)]
    full = [Bar(f"full[{i}]", 1) for i in range(stages)]
    acc_full = [[Bar(f"acc_full[{c}][{i}]", 1) for i in range(2)] for c in range(2)]
    acc_empty = [Bar(f"acc_empty[{i}]", 2 * WARPS) for i in range(2)]
    commits = []

    def uses():
        """(accumulators, the use of each) of every tile, as the MMA and the epilogue count them"""
        buf, count, out = 0, [0, 0], []
        for _, wide in tiles:
            mine = (0, 1) if wide else (buf,)
            out.append([(b, count[b]) for b in mine])
            for b in mine:
                count[b] += 1
            if not wide:
                buf ^= 1
        return out

    def producer():
        for g in range(sum(n for n, _ in tiles)):
            yield from wait(empty[g % stages], g // stages - 1)
            full[g % stages].arrive(g // stages)
            yield

    def mma():
        g = 0
        for (n, wide), mine in zip(tiles, uses()):
            for b, use in mine:
                yield from wait(acc_empty[b], use - 1)
            for _ in range(n):
                s, use = g % stages, g // stages
                yield from wait(full[s], use)
                commits.append(lambda s=s, use=use: empty[s].arrive(use))
                g += 1
                yield
            for b, use in mine[:1] if half_commit else mine:
                commits.append(lambda b=b, use=use: [acc_full[c][b].arrive(use) for c in range(2)])

    def epilogue(c):
        for mine in uses():
            for b, use in mine[:1] if half_commit else mine:
                yield from wait(acc_full[c][b], use)
            yield
            for b, use in mine:
                acc_empty[b].arrive(use)
                yield

    run([producer(), mma()] + [epilogue(c) for c in range(2) for _ in range(WARPS)], [(commits, True)], rng)


@pytest.mark.parametrize("stages", [1, 2, 4, 6])
@pytest.mark.parametrize("seed", range(8))
def test_ragged_pairs_end_without_a_false_wait(seed, stages):
    rng = random.Random(100 + seed)
    ragged_pair(seed, stages, [(rng.choice((1, 2, 4, 5, 9)), rng.random() < 0.7) for _ in range(25)])


@pytest.mark.parametrize("stages", [2, 4, 5])
@pytest.mark.parametrize("seed", range(6))
def test_wide_tiles_end_without_a_false_wait(seed, stages):
    rng = random.Random(200 + seed)
    wide_tiles(seed, stages, [(rng.choice((1, 3, 8)), rng.random() < 0.4) for _ in range(30)])


def test_the_model_sees_a_leaders_cleaner_that_skips_stages_and_a_commit_that_is_missing():
    caught = 0
    for seed in range(40):
        rng = random.Random(seed)
        try:
            ragged_pair(seed, 4, [(rng.choice((2, 3, 9)), rng.random() < 0.5) for _ in range(30)], forgets=True)
        except AssertionError:  # (a Violation is one)
            caught += 1
    assert caught > 5
    with pytest.raises(AssertionError):
        for seed in range(4):
            wide_tiles(seed, 3, [(2, True), (1, False), (1, False), (2, True)] * 6, half_commit=True)
