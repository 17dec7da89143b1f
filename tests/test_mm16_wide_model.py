"""CPU: a model of the 16-bit products' barriers where tiles wider than one accumulator take both (csrc/mm16_tc.cu).

The MMA waits for both accumulators and commits both; the epilogue waits for both and hands both back; narrower tiles
before and after go on taking turns. The rules are those of the other model: every wait's barrier is at the phase
waited for or the next one, every arrival lands in its own phase, and the run ends.
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


@pytest.mark.parametrize("stages", [2, 4, 5])
@pytest.mark.parametrize("seed", range(6))
def test_wide_tiles_end_without_a_false_wait(seed, stages):
    rng = random.Random(200 + seed)
    wide_tiles(seed, stages, [(rng.choice((1, 3, 8)), rng.random() < 0.4) for _ in range(30)])


def test_the_model_sees_a_commit_that_is_missing():
    with pytest.raises(AssertionError):
        for seed in range(4):
            wide_tiles(seed, 3, [(2, True), (1, False), (1, False), (2, True)] * 6, half_commit=True)
