"""A model of the grouped product's roles (csrc/grouped.cu), checked on the CPU.

Each CTA, alone or one of a pair, has a loading thread, a multiplying one (the pair's
leader), a warp that cuts stages at a group's end, and writer warps.  They pass stages
through mbarriers (full, or whole and cut; empty) and accumulators through two more
(done, free).  The model runs the roles' orders of operations under random
interleavings, with copies and products that complete at random times, for random
units of work: empty sums, few and many K blocks, stages that are cut.  Some runs lose
a copy, so that a wait runs out.  It asserts:

  * no barrier is over-arrived, no wait passes before the phase that it means;
  * no stage is filled while it is read, no accumulator written while it is read;
  * without a loss every unit is written out by every writer;
  * with one every role still ends, in both CTAs, behind at most a few waits that ran
    out, and nothing is in flight at the exit.

The planted mistakes are orders of operations that the kernel must not have.
"""
import random

import pytest

WRITERS = 2


class Wrong(AssertionError):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count = name, count
        self.phase, self.pending, self.tx = 0, count, 0

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def arrive(self):
        self.pending -= 1
        if self.pending < 0:
            raise Wrong(f"{self.name}: over-arrived")
        self.settle()

    def expect(self, n):
        self.tx += n
        self.arrive()

    def bytes(self, n):
        self.tx -= n
        self.settle()

    def ready(self, phase):
        """The hardware knows the parity alone: the model asks for the phase itself."""
        if self.phase > phase + 1:
            raise Wrong(f"{self.name}: two phases ahead of a wait")
        return self.phase == phase + 1


class Cta:
    def __init__(self, stages, cg):
        self.full = [Bar("full", 1) for _ in range(stages)]
        self.empty = [Bar("empty", 1) for _ in range(stages)]
        self.whole = [Bar("whole", 1) for _ in range(stages)]
        self.cut = [Bar("cut", cg) for _ in range(stages)]
        self.done = [Bar("done", 1) for _ in range(2)]
        self.free = [Bar("free", WRITERS * cg) for _ in range(2)]
        self.drain = Bar("drain", 1)
        self.turns = Bar("named", WRITERS)     # the writers' named barrier
        self.abort = False
        self.reading = [0] * stages            # products that read a stage


class Run:
    """units: lists of K blocks, each True where its stage is cut; [] is an empty sum."""

    def __init__(self, rng, cg, stages, units, lose=None, mistake=None):
        self.rng, self.cg, self.stages, self.units, self.mistake = rng, cg, stages, units, mistake
        self.ctas = [Cta(stages, cg) for _ in range(cg)]
        self.copies, self.products = [], []     # in flight; products complete in order
        self.lose, self.copied = lose, 0
        self.written = [[[0] * len(units) for _ in range(WRITERS)] for _ in range(cg)]
        self.read_bufs = [[0, 0] for _ in range(cg)]
        self.timeouts, self.exits, self.at_sync = 0, 0, [0, 0]
        self.grad = any(any(u) for u in units)

    # ---- a wait: yields until its barrier is ready; False where it gave up
    def wait(self, cta, bar, phase, abortable=True):
        why = yield ("wait", cta, bar, phase, abortable)
        return why == "ready"

    def load(self, rank):
        cta, lead = self.ctas[rank], self.ctas[0]
        st = turn = 0
        self.used[rank] = {}
        for unit in self.units:
            for cut in unit:
                if turn > 0 and self.mistake != "no empty" and \
                        not (yield from self.wait(cta, cta.empty[st], turn - 1)):
                    return
                bar = lead.full[st]
                if cut:
                    bar = cta.whole[st]
                    self.used[rank]["whole", st] = bar.phase
                    bar.expect(1)
                elif rank == 0:
                    self.used[rank]["full", st] = bar.phase
                    bar.expect(self.cg)
                yield "step"
                if any(c[0] is cta and c[1] == st for c in self.copies) or cta.reading[st]:
                    raise Wrong("a stage is filled while it is in use")
                lost = self.copied == self.lose
                self.copied += 1
                self.copies.append((cta, st, bar, lost))
                yield "step"
                st += 1
                if st == self.stages:
                    st, turn = 0, turn + 1

    def multiply(self):
        cta = self.ctas[0]
        st = acc = 0
        fulls, cuts = [0] * self.stages, [0] * self.stages
        for unit in self.units:
            if not unit:
                continue
            buf = acc & 1
            if acc >= 2 and self.mistake != "no free" and \
                    not (yield from self.wait(cta, cta.free[buf], acc // 2 - 1)):
                return
            acc += 1
            for kb, cut in enumerate(unit):
                kind, n = (cta.cut, cuts) if cut else (cta.full, fulls)
                if not (yield from self.wait(cta, kind[st], n[st])):
                    return
                n[st] += 1
                for c in range(self.cg):
                    if self.read_bufs[c][buf]:
                        raise Wrong("an accumulator is written while it is read")
                    self.ctas[c].reading[st] += 1
                self.products.append((st, buf if kb + 1 == len(unit) else None))
                yield "step"
                st = (st + 1) % self.stages

    def cutter(self, rank):
        cta = self.ctas[rank]
        st, turns = 0, [0] * self.stages
        for unit in self.units:
            for cut in unit:
                if cut:
                    if not (yield from self.wait(cta, cta.whole[st], turns[st])):
                        return
                    turns[st] += 1
                    yield "step"
                    if self.mistake != "one cut" or rank == 0:
                        self.ctas[0].cut[st].arrive()
                st = (st + 1) % self.stages

    def write(self, rank, warp):
        cta = self.ctas[rank]
        acc, tile, dead = 0, 0, False
        for i, unit in enumerate(self.units):
            # the named barrier is no mbarrier: nothing lets a warp give it up
            phase = tile
            tile += 1
            cta.turns.arrive()
            yield ("named", cta, cta.turns, phase, False)
            buf = acc & 1
            if unit and not dead:
                dead = not (yield from self.wait(cta, cta.done[buf], acc // 2))
                acc += 1
            if not dead:
                if unit:
                    self.read_bufs[rank][buf] += 1
                yield "step"
                self.written[rank][warp][i] += 1
                if unit:
                    self.read_bufs[rank][buf] -= 1
                    self.ctas[0].free[buf].arrive()

    def sync(self, which):
        self.at_sync[which] += 1
        yield ("sync", which)

    def role(self, body, rank, kind):
        yield from body
        yield from self.sync(0)
        cta = self.ctas[rank]
        if cta.abort:
            if kind == "load":
                for (name, st), phase in self.used[rank].items():
                    bar = cta.full[st] if name == "full" else cta.whole[st]
                    if bar.phase == phase:
                        yield from self.wait(cta, bar, phase, False)
            if kind == "multiply":
                self.products.append(("drain", None))
                yield from self.wait(cta, cta.drain, 0, False)
        yield from self.sync(1)
        self.exits += 1

    def complete(self):
        """One copy or the oldest product ends."""
        landing = [i for i, c in enumerate(self.copies) if not c[3]]
        if self.products and (not landing or self.rng.random() < 0.5):
            st, done = self.products.pop(0)
            for cta in self.ctas:
                if st == "drain":
                    cta.drain.arrive()
                    continue
                cta.reading[st] -= 1
                cta.empty[st].arrive()
                if done is not None:
                    cta.done[done].arrive()
        elif landing:
            _, _, bar, _ = self.copies.pop(self.rng.choice(landing))
            bar.bytes(1)

    def go(self):
        self.used = [{} for _ in range(self.cg)]
        roles = [(0, "multiply", self.multiply())]
        for r in range(self.cg):
            roles.append((r, "load", self.load(r)))
            if self.grad:
                roles.append((r, "cutter", self.cutter(r)))
            roles += [(r, "write", self.write(r, w)) for w in range(WRITERS)]
        live = {i: [self.role(body, rank, kind), None, None] for i, (rank, kind, body) in
                enumerate(roles)}
        count = len(live)
        for i in list(live):
            live[i][1] = next(live[i][0])
        while live:
            ready = []
            for i, (_, want, _) in live.items():
                if want == "step":
                    ready.append((i, None))
                elif want[0] == "sync":
                    if self.at_sync[want[1]] == count:
                        ready.append((i, None))
                elif want[2].ready(want[3]):
                    ready.append((i, "ready"))
                elif want[4] and want[1].abort:
                    ready.append((i, "abort"))
            flying = self.products or any(not c[3] for c in self.copies)
            if flying and (not ready or self.rng.random() < 0.3):
                self.complete()
                continue
            if not ready:   # two seconds pass
                late = [i for i, (_, want, _) in live.items() if want[0] == "wait"]
                if not late:
                    raise Wrong("deadlock")
                self.timeouts += 1
                i = self.rng.choice(late)
                live[i][1][1].abort = True
                ready = [(i, "late")]
            i, why = self.rng.choice(ready)
            try:
                live[i][1] = live[i][0].send(why)
            except StopIteration:
                del live[i]
        if self.products or any(not c[3] for c in self.copies):
            raise Wrong("in flight at the exit")
        return self


def units_of(rng, cut):
    units = []
    for _ in range(rng.randint(1, 9)):
        u = [False] * rng.choice([0, 1, 1, 2, 3, 7])
        if u and cut and rng.random() < 0.6:
            u[-1] = True                       # the last block of a group's rows
        units.append(u)
    return units


def run(seed, cg, cut, lose=False, mistake=None):
    rng = random.Random(seed)
    units = units_of(rng, cut)
    blocks = sum(len(u) for u in units) * cg
    r = Run(rng, cg, rng.randint(2, 5), units, rng.randrange(blocks) if lose and blocks else None,
            mistake)
    return r.go(), bool(lose and blocks)


@pytest.mark.parametrize("cg", [1, 2])
@pytest.mark.parametrize("cut", [False, True])
def test_every_unit_is_written(cg, cut):
    for seed in range(400):
        r, _ = run(seed, cg, cut)
        assert r.timeouts == 0
        assert all(n == 1 for cta in r.written for warp in cta for n in warp)


@pytest.mark.parametrize("cg", [1, 2])
@pytest.mark.parametrize("cut", [False, True])
def test_a_lost_copy_ends_the_launch(cg, cut):
    for seed in range(400):
        r, lost = run(seed, cg, cut, lose=True)
        assert (r.timeouts > 0) == lost
        # in each CTA one wait that starts the way out, and the drain's for what was lost
        assert r.timeouts <= 2 * cg + 1


@pytest.mark.parametrize("mistake", ["no empty", "no free", "one cut"])
def test_planted_mistakes_are_reported(mistake):
    """A stage filled without waiting for its products, an accumulator written over
    without waiting for its writers, and a pair's stage cut in one CTA alone."""
    with pytest.raises(AssertionError):
        for seed in range(400):
            r, _ = run(seed, 2, True, mistake=mistake)
            assert r.timeouts == 0
