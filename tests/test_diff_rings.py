"""The barriers of the two-SM differential attention kernel as a model on the
CPU: loaders, issuing threads and softmax warps of both CTAs pass key, value and
query tiles, scores, weights and accumulators to each other through mbarriers
whose waiters know a phase by its parity alone. Every schedule of the model has
to end, and everyone has to find in a slot what was meant for him. The number of
stages is read from the kernel's source; who waits for and arrives at what is
restated here. Softmax warps are fewer than the kernel's: two groups of rows of
two parts in either CTA."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_decode_18_gb300", "csrc", "pa_diff_tc.cu")
GROUPS, PARTS = 2, 2
CTAS = (0, 1)


def stages():
    with open(SOURCE) as f:
        return int(re.search(r"constexpr int kMaxStagesT = (\d+);", f.read()).group(1))


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, "more arrivals than the barrier expects"
        if self.left == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passed(self, parity):    # mbarrier.try_wait.parity
        return (self.phase & 1) != parity


class Model:
    """One cluster. An agent is a generator that yields a (barrier, parity) to wait
    for, or None where others may come between."""

    def __init__(self, runs, ring, rng, p_barriers=2, sloppy_end=False):
        self.n = sum(runs)
        self.first = set()
        at = 0
        for r in runs:                       # runs: key tiles of each map of each piece
            self.first.add(at)
            at += r
        self.run = [sum(f <= i for f in self.first) - 1 for i in range(self.n)]
        self.ring, self.rng, self.p_barriers, self.sloppy_end = ring, rng, p_barriers, sloppy_end
        both = lambda k, count=1: {c: [Bar(count) for _ in range(k)] for c in CTAS}  # noqa: E731
        warps = GROUPS * PARTS * 2
        self.qfull = [Bar(3) for _ in range(2)]           # the leader's announcement, two copies
        self.kfull = [Bar(3) for _ in range(ring)]
        self.vfull = [Bar(3) for _ in range(ring)]
        self.vempty, self.vseen = both(ring), both(1)
        self.kempty, self.qempty = both(ring), both(2)
        self.sfull, self.pfree = both(1), both(2)
        self.sempty = Bar(GROUPS * 2)
        self.pfull = [Bar(warps) for _ in range(p_barriers)]
        self.xch = {(c, g): Bar(PARTS) for c in CTAS for g in range(GROUPS)}
        self.vote = {(c, g): Bar(PARTS) for c in CTAS for g in range(GROUPS)}
        self.k, self.v, self.q = {}, {}, {}
        self.scores, self.held = None, set()              # tile in S; who holds it in registers
        self.p = [{}, {}]
        self.o, self.flushed = [], {}                     # tiles in O; runs written out, per warp
        self.s_done, self.pv_done = -1, -1
        self.flying, self.s_queue, self.pv_queue = [], [], []
        self.agents = {f"k{c}": self.load_k(c) for c in CTAS}
        self.agents |= {f"v{c}": self.load_v(c) for c in CTAS}
        self.agents |= {"s": self.issue_s(), "pv": self.issue_pv(), "s pipe": self.s_pipe(),
                        "pv pipe": self.pv_pipe(), "copies": self.land()}
        self.agents |= {f"w{c}{g}{p}": self.softmax(c, g, p)
                        for c in CTAS for g in range(GROUPS) for p in range(PARTS)}

    # copies land in any order
    def land(self):
        total = self.n * 4 + (max(self.run) + 1) * 2
        for _ in range(total):
            while not self.flying:
                yield
            slot, key, tile, bar = self.flying.pop(self.rng.randrange(len(self.flying)))
            slot[key] = tile
            bar.arrive()
            yield

    def load_k(self, c):
        for i in range(self.n):
            if i in self.first:
                r = self.run[i]
                if r >= 2:
                    yield self.qempty[c][r & 1], ((r >> 1) - 1) & 1
                if c == 0:
                    self.qfull[r & 1].arrive()
                self.flying.append((self.q, (c, r & 1), r, self.qfull[r & 1]))
                yield
            st, use = i % self.ring, i // self.ring
            if use > 0:
                yield self.kempty[c][st], (use - 1) & 1
            if c == 0:
                self.kfull[st].arrive()
            self.flying.append((self.k, (c, st), i, self.kfull[st]))
            yield

    def load_v(self, c):
        for i in range(self.n):
            st, use = i % self.ring, i // self.ring
            if use > 0:
                yield self.vempty[c][st], (use - 1) & 1
            if c == 0:
                self.vfull[st].arrive()
            self.flying.append((self.v, (c, st), i, self.vfull[st]))
            yield

    def issue_s(self):
        for i in range(self.n):
            if i in self.first:
                r = self.run[i]
                yield self.qfull[r & 1], (r >> 1) & 1
            yield self.kfull[i % self.ring], (i // self.ring) & 1
            if i >= 1:
                yield self.sempty, (i - 1) & 1
            if i >= 2:
                yield self.pfree[0][i & 1], ((i >> 1) - 1) & 1
            self.s_queue.append(i)
            yield

    def s_pipe(self):
        for i in range(self.n):
            while not self.s_queue:
                yield
            assert self.s_queue.pop(0) == i
            for c in CTAS:
                assert self.k[c, i % self.ring] == i, "another tile's keys"
                assert self.q[c, self.run[i] & 1] == self.run[i], "another map's queries"
            if i:
                assert len(self.held) == GROUPS * PARTS * 2, "scores that a warp has not read"
            self.scores, self.held = i, set()
            yield
            self.s_done = i
            for c in CTAS:
                self.sfull[c][0].arrive()
                self.kempty[c][i % self.ring].arrive()
                if i + 1 == self.n or i + 1 in self.first:
                    self.qempty[c][self.run[i] & 1].arrive()
            yield

    def issue_pv(self):
        for i in range(self.n):
            b = i % self.p_barriers
            yield self.vfull[i % self.ring], (i // self.ring) & 1
            if self.cleaned(i):
                for c in CTAS:
                    self.vseen[c][0].arrive()
                    yield
            yield self.pfull[b], (i // self.p_barriers) & 1
            self.pv_queue.append(i)
            yield

    def pv_pipe(self):
        for i in range(self.n):
            while not self.pv_queue:
                yield
            assert self.pv_queue.pop(0) == i
            assert len(self.p[i & 1]) == GROUPS * PARTS * 2
            assert set(self.p[i & 1].values()) == {i}, "weights of another tile"
            for c in CTAS:
                assert self.v[c, i % self.ring] == i, "another tile's values"
            if i in self.first:
                if i:
                    done = self.flushed.values()
                    assert len(self.flushed) == GROUPS * PARTS * 2 and \
                        set(done) == {self.run[i] - 1}, "an accumulator not yet written out"
                self.o = []
            yield
            self.o.append(i)
            self.pv_done = i
            for c in CTAS:
                self.vempty[c][i % self.ring].arrive()
                self.pfree[c][i & 1].arrive()
            yield

    # tiles with values that not every query sees, and tiles that move a reference
    def cleaned(self, i):
        return i % 4 == 2 or i + 1 == self.n or i + 1 in self.first

    def moves(self, i):
        return i in self.first or i % 3 == 1

    def softmax(self, c, g, part):
        me, phase, seen, pending = (c, g, part), 0, 0, None
        for i in range(self.n):
            yield self.sfull[c][0], i & 1
            assert self.scores == i and self.s_done == i, "another tile's scores"
            self.held.add(me)
            self.vote[c, g].arrive()
            yield self.vote[c, g], i & 1
            if part == 0:
                self.sempty.arrive()
                yield
            if self.moves(i):
                self.xch[c, g].arrive()
                yield self.xch[c, g], phase & 1
                phase += 1
            assert self.pv_done >= i - 2, "weights that a product still reads"
            self.p[i & 1][me] = i
            yield
            if pending is not None or (i not in self.first and self.moves(i)):
                yield self.pfree[c][(i - 1) & 1], ((i - 1) >> 1) & 1
                assert self.pv_done == i - 1, "an accumulator under a product"
            if pending is not None:
                self.xch[c, g].arrive()     # the parts' sums
                yield self.xch[c, g], phase & 1
                phase += 1
                self.flushed[me] = pending
                pending = None
            if self.cleaned(i):
                yield self.vseen[c][0], seen & 1
                seen += 1
                assert self.v[c, i % self.ring] == i
            self.pfull[i % self.p_barriers].arrive()
            if i + 1 == self.n or i + 1 in self.first:
                pending = self.run[i]
            yield
        if self.sloppy_end:      # one barrier of all products in the place of two
            while self.pv_done < self.n - 2 and not self.rng.random() < 0.5:
                yield
        else:
            yield self.pfree[c][(self.n - 1) & 1], ((self.n - 1) >> 1) & 1
        assert self.o and self.pv_done == self.n - 1, "an accumulator under a product"

    def go(self, slow=None):
        waits = {name: None for name in self.agents}
        idle = 0
        while self.agents:
            names = [n for n in self.agents if n != slow or self.rng.random() < 0.05]
            if not names:
                continue
            name = self.rng.choice(names)
            w = waits[name]
            if w is not None and not w[0].passed(w[1]):
                idle += 1
                assert idle < 200000, f"stuck: {sorted(self.agents)}"
                continue
            idle = 0
            try:
                waits[name] = next(self.agents[name])
            except StopIteration:
                del self.agents[name], waits[name]


RUNS = [[1], [2], [3], [1, 1], [2, 2, 1], [5, 5], [7, 4, 4, 1, 1, 3], [1] * 9, [12, 12, 5]]
NAMES = ["k0", "k1", "v0", "v1", "s", "pv", "s pipe", "pv pipe", "copies", "w000", "w011", "w100",
         "w111"]


@pytest.mark.parametrize("runs", RUNS, ids=lambda r: "-".join(map(str, r)))
@pytest.mark.parametrize("ring", [2, 3])
def test_every_schedule_ends_and_finds_its_tiles(runs, ring):
    assert stages() == 3   # and two, where a long plan leaves no room
    for seed in range(25):
        Model(runs, ring, random.Random(seed)).go()
    for k, slow in enumerate(NAMES):
        Model(runs, ring, random.Random(100 + k)).go(slow)


def caught(**kw):
    for seed in range(300):
        rng = random.Random(seed)
        try:
            Model([5, 5, 3], 3, rng, **kw).go(rng.choice([None] + NAMES))
        except AssertionError:
            return True
    return False


def test_the_model_sees_a_single_barrier_of_weights():
    # a warp through with the next tile would arrive in the place of a late one
    assert caught(p_barriers=1)


def test_the_model_sees_an_end_that_does_not_wait():
    assert caught(sloppy_end=True)
