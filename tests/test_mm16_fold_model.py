"""CPU: a model of how the 16-bit products share two accumulators between short and long reductions.

Tiles with a short reduction take the accumulators in turn. A tile whose reduction is summed up piece by piece
(csrc/mm16_tc.cu, fold_acc) keeps its accumulator for every piece, and the epilogue holds the running sum in the place
of the other one; the tile after it keeps the same accumulator too, because its wait for that one is what says that the
sum has been read. `simulate` replays the MMA's thread, its commits in issue order and the epilogue warps of every CTA
under random interleavings. It asserts what the barriers' parities allow (Bar), and that every epilogue warp finds in its
own part of each accumulator what it expects there: the piece it waited for, the sum of all pieces before it, and at the
end still that sum, after any number of steps in which the MMA's thread may have gone on.
"""
import random

import pytest

from test_gemm_pipeline_model import Bar, Violation

WARPS = 3


def simulate(seed, ctas, tiles, turn_after_long=False):
    """tiles: the pieces of each tile (0: an empty sum, without an accumulator). turn_after_long: the rule that would not do."""
    rng = random.Random(seed)
    acc_full = [[Bar(f"acc_full[{c}][{i}]", 1) for i in range(2)] for c in range(ctas)]
    acc_empty = [Bar(f"acc_empty[{i}]", WARPS * ctas) for i in range(2)]
    held = {(c, w, i): None for c in range(ctas) for w in range(WARPS) for i in range(2)}
    queue, out = [], []

    def wait(bar, k):
        bar.check_wait(k)
        while not bar.done(k):
            yield
        bar.check_wait(k)

    def fill(buf, what):
        for c in range(ctas):
            for w in range(WARPS):
                held[c, w, buf] = what

    def mma():
        buf, uses = 0, [0, 0]
        for t, pieces in enumerate(tiles):
            for j in range(pieces):
                yield from wait(acc_empty[buf], uses[buf] - 1)
                fill(buf, "being written")
                queue.append((buf, uses[buf], ("piece", t, j)))
                uses[buf] += 1
                if pieces == 1 or (turn_after_long and j == pieces - 1):
                    buf ^= 1
                yield

    def epilogue(c, w):
        buf, uses = 0, [0, 0]

        def expect(i, what):
            if held[c, w, i] != what:
                raise Violation(f"warp {w} of {c} finds {held[c, w, i]} where {what} should be")

        for t, pieces in enumerate(tiles):
            own = buf
            for j in range(pieces):
                yield from wait(acc_full[c][buf], uses[buf])
                use, uses[buf] = uses[buf], uses[buf] + 1
                if pieces > 1:
                    yield
                    expect(buf, ("piece", t, j))
                    if j:
                        expect(buf ^ 1, ("sum", t, j))
                    held[c, w, buf ^ 1] = ("sum", t, j + 1)
                if j + 1 < pieces:
                    acc_empty[buf].arrive(use)
                    yield
                    continue
                for _ in range(rng.randrange(4)):  # the results leave bit by bit
                    yield
                    expect(*((buf ^ 1, ("sum", t, pieces)) if pieces > 1 else (buf, ("piece", t, 0))))
                out.append((c, w, t))
                acc_empty[buf].arrive(use)
                own = buf if pieces > 1 and not turn_after_long else buf ^ 1
                yield
            buf = own

    actors = [mma()] + [epilogue(c, w) for c in range(ctas) for w in range(WARPS)]
    weight = [rng.choice((1, 1, 6)) for _ in actors]
    idle = 0
    while actors or queue:
        if queue and (not actors or rng.random() < 0.3):
            buf, use, what = queue.pop(0)
            fill(buf, what)
            for c in range(ctas):
                acc_full[c][buf].arrive(use)
            idle = 0
            continue
        i = rng.choices(range(len(actors)), weight)[0]
        try:
            next(actors[i])
        except StopIteration:
            del actors[i], weight[i]
        idle += 1
        if idle > 20000:
            raise Violation("nothing moves any more")
    assert len(out) == ctas * WARPS * sum(1 for p in tiles if p)


@pytest.mark.parametrize("ctas", [1, 2])
@pytest.mark.parametrize("seed", range(60))
def test_long_tiles_among_short_ones(ctas, seed):
    rng = random.Random(1000 + seed)
    simulate(seed, ctas, [rng.choice((0, 1, 1, 1, 2, 2, 3, 7)) for _ in range(25)])


@pytest.mark.parametrize("tiles", [[1] * 20, [2] * 12, [5] * 6, [1, 4] * 6, [4, 1, 1] * 5, [0, 3, 0, 1], [9]])
def test_patterns(tiles):
    for seed in range(30):
        simulate(seed, 2, tiles)


def test_taking_turns_after_a_long_tile_is_caught():
    caught = 0
    for seed in range(60):
        rng = random.Random(seed)
        try:
            simulate(seed, 1, [rng.choice((1, 1, 2, 3)) for _ in range(25)], turn_after_long=True)
        except Violation:
            caught += 1
    assert caught > 20
