"""The hand-offs of csrc/paged_attend_tc.cu after a bounded wait has run out, as
a model on the CPU.

Every warp of a CTA is a coroutine that goes through the waits and arrivals of
its role, under a scheduler that picks the next one at random; named barriers
count warps, mbarriers have a phase and are waited for by parity, and the tensor
pipe completes commits in order, some time later or, once it is stuck, never.
Any mbarrier wait may run out.  Whatever the order, every warp has to reach the
end, and no warp may arrive twice in one phase of a named barrier.

With `lockstep` the feeders of the issuing warp do what the kernel does: where
their mbarrier wait has run out, they wait for the issuer's count of finished
tiles, from then on (softmax: whenever any wait has run out before).  Without it they go on at once, and get two arrivals
ahead of the issuer: that has to be seen.
"""
import random

import pytest

PROD, SOFT, LOAD = 4, 4, 3


class Stop(Exception):
    pass


class Named:
    """bar.arrive / bar.sync of `size` warps."""
    arrivals = 0   # of all

    def __init__(self, size):
        self.size, self.phase, self.here = size, 0, []

    def arrive(self, who):
        if who in self.here:
            raise Stop(f"{who} arrives twice in a phase")
        self.here.append(who)
        Named.arrivals += 1
        if len(self.here) == self.size:
            self.here, self.phase = [], self.phase + 1

    def sync(self, who):
        at = self.phase
        self.arrive(who)
        while self.phase == at:
            yield "blocked"


class Mbar:
    def __init__(self, count=1):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Cta:
    def __init__(self, seed, items, lockstep, p_timeout, stuck_after):
        self.r = random.Random(seed)
        self.items, self.lockstep, self.p = items, lockstep, p_timeout
        self.stuck_after = stuck_after
        self.abort = False
        self.finished_tiles = 0
        self.k = [Named(PROD + 1) for _ in range(2)]
        self.v = [Named(PROD + 1) for _ in range(2)]
        self.pb = [[Named(SOFT + 1) for _ in range(3)] for _ in range(2)]
        self.group = [Named(SOFT) for _ in range(2)]
        self.loaders = Named(LOAD)
        self.s_done, self.pv_done = [Mbar(), Mbar()], [Mbar(), Mbar()]
        self.k_free, self.v_free = [Mbar(), Mbar()], [Mbar(), Mbar()]
        self.q_ready, self.q_free, self.drain = Mbar(LOAD), Mbar(), Mbar()
        self.pipe, self.commits = [], 0
        self.poisoned = [{}, {}]   # item -> its rows are marked as lost
        self.stored = [0, 0]

    def wait(self, bar, parity):
        """The kernel's bounded wait: false when it runs out or another has given up."""
        while True:
            yield "poll"
            if bar.done(parity):
                return True
            if self.abort:
                return False
            if self.r.random() < self.p:
                self.abort = True
                return False

    def follow(self, tiles):
        while self.finished_tiles < tiles:
            yield "poll"

    def softmax(self, g, n):
        who, u = ("soft", n, g), 0
        for item, tiles in enumerate(self.items):
            for _ in range(tiles):
                if n == 0:
                    gone = self.abort
                    got = yield from self.wait(self.s_done[g], u & 1)
                    if self.lockstep and (gone or not got):
                        yield from self.follow(u)
                yield from self.group[g].sync(who)
                for part in range(3):
                    yield "step"
                    self.pb[g][part].arrive(who)
                u += 1
            if n == 0:
                yield from self.wait(self.pv_done[g], item & 1)
            yield from self.group[g].sync(who)
            if n == 0:
                self.poisoned[g][item] = self.abort
                self.stored[g] += 1

    def producer(self, n):
        who, ok = ("prod", n), True
        for u in range(sum(self.items)):
            st, par = u & 1, ((u >> 1) - 1) & 1
            for free, ready in ((self.k_free, self.k), (self.v_free, self.v)):
                if u >= 2:
                    if ok or not self.lockstep:
                        ok = (yield from self.wait(free[st], par)) and ok
                    if self.lockstep and not ok:
                        yield from self.follow(u - 1)
                yield "step"
                ready[st].arrive(who)

    def loader(self, n):
        who, par, ok = ("load", n), 0, True
        for item in range(len(self.items)):
            if item > 0:
                ok = ok and (yield from self.wait(self.q_free, par))
                par ^= 1
            yield from self.loaders.sync(who)
            yield from self.loaders.sync(who)
            self.q_ready.arrive()
            yield "step"

    def commit(self, bar):
        self.pipe.append(bar)

    def issuer(self):
        who, u, q_par, ok = ("mma",), 0, 0, True

        def s(g, st, last):
            self.commit(self.s_done[g])
            if g == 1:
                self.commit(self.k_free[st])
                if last:
                    self.commit(self.q_free)

        for tiles in self.items:
            yield from self.k[u & 1].sync(who)
            ok = (yield from self.wait(self.q_ready, q_par)) and ok
            q_par ^= 1
            if ok:
                s(0, u & 1, False)
                s(1, u & 1, tiles == 1)
            for t in range(tiles):
                st, last = u & 1, t + 1 == tiles
                ok = ok and not self.abort
                for g in range(2):
                    yield from self.pb[g][0].sync(who)
                    if g == 0:
                        yield from self.v[st].sync(who)
                    yield from self.pb[g][1].sync(who)
                    yield from self.pb[g][2].sync(who)
                    if ok:
                        if last:
                            self.commit(self.pv_done[g])
                        if g == 1:
                            self.commit(self.v_free[st])
                    if not last:
                        if g == 0:
                            yield from self.k[st ^ 1].sync(who)
                        if ok:
                            s(g, st ^ 1, t + 2 == tiles)
                    yield "step"
                u += 1
                self.finished_tiles = u
        self.commit(self.drain)
        while not self.drain.done(0):   # limited by the clock alone
            yield "poll"
            if self.stuck():
                break

    def stuck(self):
        return self.stuck_after is not None and self.commits >= self.stuck_after

    def run(self):
        warps = [self.issuer()] + [self.producer(n) for n in range(PROD)] + [self.loader(n) for n in range(LOAD)]
        warps += [self.softmax(g, n) for g in range(2) for n in range(SOFT)]
        asleep, steps = set(), 0
        while warps:
            steps += 1
            if steps > 1_000_000:
                raise Stop("no end")
            if self.pipe and not self.stuck() and self.r.random() < 0.2:
                self.pipe.pop(0).arrive()
                self.commits += 1
            w, before = self.r.choice(warps), Named.arrivals
            try:
                state = next(w)
            except StopIteration:
                warps.remove(w)
                asleep.clear()
                continue
            if state == "blocked" and Named.arrivals == before:
                asleep.add(w)
                if len(asleep) == len(warps):
                    raise Stop("every warp is blocked")
            else:
                asleep.clear()


SHAPES = ([1], [2], [3], [7], [1, 1, 1, 1], [3, 1, 2, 5], [1, 4, 1, 1, 6, 2])


def trial(seed, lockstep):
    r = random.Random(seed)
    items = r.choice(SHAPES)
    stuck = r.choice([None, 0, r.randrange(8 * sum(items))])
    p = r.choice([0.0, 0.002, 0.02, 0.3]) if stuck is None else r.choice([0.002, 0.02, 0.3])
    cta = Cta(seed, items, lockstep, p, stuck)
    cta.run()
    return cta


@pytest.mark.parametrize("part", range(8))
def test_every_warp_reaches_the_end(part):
    lost = 0
    for seed in range(part * 250, part * 250 + 250):
        cta = trial(seed, True)
        assert cta.stored == [len(cta.items)] * 2
        lost += any(any(p.values()) for p in cta.poisoned)
        if not cta.abort:
            assert not any(any(p.values()) for p in cta.poisoned)
    assert lost > 50   # the waits did run out


def test_feeders_that_go_on_at_once_are_caught():
    caught = 0
    for seed in range(300):
        try:
            trial(seed, False)
        except Stop:
            caught += 1
    assert caught > 30
