"""CPU: a model of how the 16-bit products' kernel ends when one of its waits gives up.

Every wait on an mbarrier is bounded (csrc/tc_ptx.cuh, mbar_wait): it returns false when its time is up, raising the CTA's
abort flag, or when another warp of the CTA has raised it. What follows must still bring every warp of every CTA
to the end, through the named barriers that the epilogue warps of a half share, the cluster barrier at which a split's
sums change hands and the cluster's last one. `run` lets one arrival go missing, anywhere, and asserts that all
actors end, that the members of a named barrier meet at the same place of their programs, that a cluster barrier is
reached by every warp of every CTA the same number of times.
Time runs out only when nothing else can move, for one waiting warp at a time, in any order.
"""
import random

import pytest

STAGES, CHUNKS, WARPS = 3, 2, 4  # (four epilogue warps to a half, as in the kernel)


class Stuck(AssertionError):
    pass


class Mbar:
    def __init__(self, expected):
        self.expected, self.phase, self.arrived = expected, 0, 0

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.expected:
            self.phase, self.arrived = self.phase + 1, 0


class Meeting:
    """A barrier of a fixed number of warps; every generation has one tag."""

    def __init__(self, name, members):
        self.name, self.members = name, members
        self.gen, self.here, self.tag, self.all_ok = 0, 0, None, True
        self.results = []

    def enter(self, tag, ok=True):
        if self.here and tag != self.tag:
            raise Stuck(f"{self.name}: {tag} meets {self.tag}")
        self.tag = tag
        self.here += 1
        self.all_ok &= ok
        gen = self.gen
        if self.here == self.members:
            self.results.append(self.all_ok)
            self.gen, self.here, self.all_ok = self.gen + 1, 0, True
        return gen


def run(seed, ctas, split, tiles, lose, early_leave=False):
    """tiles: (stages of each seg, ...) per tile; lose: the arrival (counted over the run) that never comes.
    early_leave: a rule that would not do, a split's warps leaving before the sums change hands."""
    rng = random.Random(seed)
    pair = ctas == 2 and not split
    full = [[Mbar(1) for _ in range(STAGES)] for _ in range(ctas)]
    empty = [[Mbar(1) for _ in range(STAGES)] for _ in range(ctas)]
    acc_full = [[Mbar(1) for _ in range(2)] for _ in range(ctas)]
    acc_empty = [[Mbar(2 * WARPS * (2 if pair else 1)) for _ in range(2)] for _ in range(ctas)]
    halves = [[Meeting(f"half {h} of {c}", WARPS) for h in range(2)] for c in range(ctas)]
    per_cta = 3 + 2 * WARPS  # one producer warp, the MMA's warp, an idle one, the epilogue
    cluster = Meeting("cluster", ctas * per_cta)
    last = Meeting("end", ctas * per_cta) if ctas == 2 else None
    abort, count, timed = [False] * ctas, [0], []
    waiting = {}  # actor id -> CTA, of the waits that only time can end

    def arrive(bar):
        count[0] += 1
        if count[0] != lose:
            bar.arrive()

    def wait(me, c, bar, k):
        while not (k < 0 or bar.phase > k):
            if abort[c]:
                return False
            waiting[me] = c
            yield
            waiting.pop(me, None)
            if me in timed:
                timed.remove(me)
                if k < 0 or bar.phase > k:
                    break
                abort[c] = True
                return False
        return True

    def meet(m, tag, ok=True):
        gen = m.enter(tag, ok)
        while m.gen == gen:
            yield
        return m.results[gen]

    def leave(me, c, epilogue):
        if split and not epilogue:
            yield from meet(cluster, "sums")
        if last:
            yield from meet(last, "end")

    def producer(me, c):
        g, ok = 0, True
        for tile in tiles:
            for n in tile:
                for _ in range(n):
                    ok = yield from wait(me, c, empty[c][g % STAGES], g // STAGES - 1)
                    if not ok:
                        break
                    yield
                    if not pair or c == 0:
                        arrive(full[c][g % STAGES])  # (of a pair both CTAs' copies, on the leader's barrier)
                    g += 1
                if not ok:
                    break
            if not ok:
                break
        yield from leave(me, c, False)

    def mma(me, c):
        g, buf, uses, ok = 0, 0, [0, 0], not (pair and c)
        for tile in tiles if ok else ():
            for n in tile:
                ok = yield from wait(me, c, acc_empty[c][buf], uses[buf] - 1)
                for _ in range(n):
                    ok = ok and (yield from wait(me, c, full[c][g % STAGES], g // STAGES))
                    if not ok:
                        break
                    yield
                    for peer in range(ctas) if pair else (c,):
                        arrive(empty[peer][g % STAGES])
                    g += 1
                if not ok:
                    break
                for peer in range(ctas) if pair else (c,):
                    arrive(acc_full[peer][buf])
                uses[buf] += 1
                if len(tile) == 1:
                    buf ^= 1
            if not ok:
                break
        yield from leave(me, c, False)

    def idle(me, c):
        yield
        yield from leave(me, c, False)

    def epilogue(me, c, h, w):
        buf, uses = 0, [0, 0]
        owner = 0 if pair else c
        for t, tile in enumerate(tiles):
            ok = True
            for j in range(len(tile)):
                ok = yield from wait(me, c, acc_full[c][buf], uses[buf])
                uses[buf] += 1
                if ok and j + 1 < len(tile):
                    arrive(acc_empty[owner][buf])
                    continue
                break
            ok = yield from meet(halves[c][h], ("go", t), ok)
            if split:
                if early_leave and not ok:
                    break
                yield from meet(cluster, "sums")
                if c > 0:
                    ok = False
            if not ok:
                break
            for chunk in range(CHUNKS):
                yield from meet(halves[c][h], ("staged", t, chunk))
                yield from meet(halves[c][h], ("stored", t, chunk))
            arrive(acc_empty[owner][buf])
            if len(tile) == 1:
                buf ^= 1
        yield from leave(me, c, True)

    actors = {}
    for c in range(ctas):
        for make in (producer, mma, idle):
            me = len(actors)
            actors[me] = make(me, c)
        for h in range(2):
            for w in range(WARPS):
                me = len(actors)
                actors[me] = epilogue(me, c, h, w)
    still = 0
    while actors:
        before = (count[0], len(actors), sum(m.gen * 100 + m.here for row in halves for m in row), cluster.gen * 100 + cluster.here,
                  last and last.here, tuple(abort), len(waiting))
        me = rng.choice(list(actors))
        try:
            next(actors[me])
        except StopIteration:
            del actors[me]
            waiting.pop(me, None)
        after = (count[0], len(actors), sum(m.gen * 100 + m.here for row in halves for m in row), cluster.gen * 100 + cluster.here,
                 last and last.here, tuple(abort), len(waiting))
        still = 0 if before != after else still + 1
        if still > 60 * len(actors) + 200:
            late = [m for m in waiting if m in actors]
            if not late:
                raise Stuck(f"{len(actors)} warps wait for each other")
            timed.append(rng.choice(late))
            still = 0
    if split:
        assert cluster.gen == 1 and cluster.here == 0
    return count[0], any(abort)


TILES = {"short": [(2,), (4,), (1,)], "long": [(2, 2, 1), (3,), (2, 2)], "one": [(5,)], "one long": [(2, 2, 2)]}


@pytest.mark.parametrize("ctas,split,tiles", [(1, False, "short"), (1, False, "long"), (2, False, "short"), (2, False, "long"),
                                              (2, True, "one"), (2, True, "one long"), (4, True, "one long")])
def test_every_warp_ends_whatever_arrival_is_lost(ctas, split, tiles):
    total, gave_up = run(0, ctas, split, TILES[tiles], lose=-1)
    assert not gave_up
    rng = random.Random(7)
    gave = 0
    for lose in range(1, total + 1):
        gave += run(rng.random(), ctas, split, TILES[tiles], lose)[1]
    assert gave > total // 4  # (the last uses' arrivals are waited for by nobody)


def test_leaving_before_the_sums_change_hands_is_caught():
    total, _ = run(0, 2, True, TILES["one"], lose=-1)
    caught = 0
    for lose in range(1, total + 1):
        try:
            run(lose, 2, True, TILES["one"], lose, early_leave=True)
        except Stuck:
            caught += 1
    assert caught > 3
