"""The rings of the tcgen05 weights kernel as a model on the CPU: its loaders,
issuing threads, converter and epilogue groups pass K tiles, query tiles and
accumulators to each other through mbarriers whose waiters know a phase by its
parity alone. Every schedule of the model has to end, and everyone has to find
in a slot what was meant for him. The ring sizes and arrival counts are read
from the kernel's source; who waits for and arrives at what is restated here."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_decode_18_gb300", "csrc")


def source():
    with open(os.path.join(CSRC, "pa_weights_tc.cu")) as f:
        return f.read()


def layout(q8, split):
    """The sizes of Lay<FMT, SPLIT> and the issuing threads' share in a query
    tile's release."""
    text = source()
    env = {"q8": q8, "SPLIT": split}

    def value(name):
        e = re.search(rf"constexpr int {name} = ([^;]+);", text).group(1)
        m = re.fullmatch(r"(.+) \? (\d+) : (\d+)", e)
        if not m:
            return int(e)
        cond = m.group(1).replace("&&", "and").replace("!", "not ")
        return int(m.group(2) if eval(cond, {}, env) else m.group(3))

    both = re.search(r"mbar_init\(bar\(B_QEMPTY \+ i\), \(SPLIT \? (\d)u : (\d)u\) \+ "
                     r"kEpiWarps \* 32u\)", text)
    return {"stages": value("kStages"), "raw": value("kRawStages"), "qbufs": value("kQBufs"),
            "dbufs": value("kDBufs"), "parts": value("kPartSlots"), "scales": value("kScaleSlots"),
            "issuers": int(both.group(1 if split else 2))}


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


def plan(seqs, qtb):
    """Items in the order of a CTA: (item of its head, key tiles, query tiles,
    first query tile)."""
    out = []
    for c, lq in seqs:
        nt, nq = -(-c // 128), -(-lq // qtb)
        for _head in range(2):
            for i in range(nt):
                kt = nt - 1 - (i >> 1) if i & 1 else i >> 1
                out.append((i, nt, nq, max(0, kt * 128 - (c - lq)) // qtb if nq > 1 else 0))
    return out


class Model:
    """One CTA. An agent is a generator that yields a (barrier, parity) to wait
    for, or None where others may come between."""

    def __init__(self, q8, split, seqs, qtb, issuers=None):
        self.L = L = layout(q8, split)
        if issuers is not None:
            L["issuers"] = issuers
        self.q8, self.split, self.items = q8, split, plan(seqs, qtb)
        self.kfull = [Bar(1) for _ in range(L["stages"])]
        self.kempty = [Bar(2 if split else 1) for _ in range(L["stages"])]
        self.rfull = [Bar(1) for _ in range(L["raw"])]
        self.rempty = [Bar(1) for _ in range(L["raw"])]
        self.qfull = [Bar(1) for _ in range(L["qbufs"])]
        self.qempty = [Bar(L["issuers"] + 2) for _ in range(L["qbufs"])]
        self.dfull = [Bar(2) for _ in range(L["dbufs"])]
        self.dempty = [Bar(2 if split else 1) for _ in range(L["dbufs"])]
        self.bpart = [Bar(1) for _ in range(L["parts"])]
        self.k, self.rawt, self.q, self.d, self.part, self.scale = {}, {}, {}, {}, {}, {}
        self.queue = []          # the tensor pipe: products and commits, in order
        self.summed = {0: [], 1: []}
        self.agents = {"k": self.load_k(), "q": self.load_q(), "mma0": self.issue(0),
                       "mma1": self.issue(1), "epi0": self.epilogue(0), "epi1": self.epilogue(1),
                       "pipe": self.pipe()}
        if q8:
            self.agents["conv"] = self.convert()

    def fresh(self, x):
        i, _, nq, _ = self.items[x]
        return nq > 1 or i == 0 or x == 0

    def last_use(self, x):
        i, nt, nq, _ = self.items[x]
        return nq > 1 or i == nt - 1 or x + 1 == len(self.items)

    def load_k(self):
        full, empty, slot = ((self.rfull, self.rempty, self.rawt) if self.q8 else
                             (self.kfull, self.kempty, self.k))
        ring = len(full)
        for n in range(len(self.items)):
            if n >= ring:
                yield empty[n % ring], (n // ring - 1) & 1
            slot[n % ring] = n
            full[n % ring].arrive()
            yield

    def convert(self):
        raw, st = self.L["raw"], self.L["stages"]
        for n in range(len(self.items)):
            yield self.rfull[n % raw], (n // raw) & 1
            assert self.rawt[n % raw] == n
            self.rempty[n % raw].arrive()
            if n >= st:
                yield self.kempty[n % st], (n // st - 1) & 1
            self.scale[n % self.L["scales"]] = n
            self.k[n % st] = n
            self.kfull[n % st].arrive()
            yield

    def load_q(self):
        nb, qn = self.L["qbufs"], 0
        for x, (_, _, nq, first) in enumerate(self.items):
            if not self.fresh(x):
                continue
            for _ in range(first, nq):
                if qn >= nb:
                    yield self.qempty[qn % nb], (qn // nb - 1) & 1
                self.q[qn % nb] = qn
                self.qfull[qn % nb].arrive()
                qn += 1
                yield

    def issue(self, me):
        L, qn, dn = self.L, 0, 0
        for n, (_, _, nq, first) in enumerate(self.items):
            st, mine = n % L["stages"], (n & 1) == me
            if self.split or mine:
                yield self.kfull[st], (n // L["stages"]) & 1
            for _ in range(first, nq):
                if self.fresh(n):
                    yield self.qfull[qn % L["qbufs"]], (qn // L["qbufs"]) & 1
                    qn += 1
                qb, db = (qn - 1) % L["qbufs"], dn % L["dbufs"]
                if ((dn & 1) != me) if self.split else not mine:
                    if self.last_use(n) and L["issuers"]:
                        if self.split:
                            self.qempty[qb].arrive()
                        else:
                            self.queue.append(("commit", self.qempty[qb]))
                    dn += 1
                    yield
                    continue
                if dn >= L["dbufs"]:
                    yield self.dempty[db], (dn // L["dbufs"] - 1) & 1
                self.queue.append(("mma", (st, n, qb, qn - 1, db, dn)))
                self.queue.append(("commit", self.dfull[db]))
                self.dfull[db].arrive()
                if not self.split and self.last_use(n):
                    self.queue.append(("commit", self.qempty[qb]))
                dn += 1
                yield
            if self.split or mine:
                self.queue.append(("commit", self.kempty[st]))
            yield

    def pipe(self):
        while True:
            if self.queue:
                what, x = self.queue.pop(0)
                if what == "commit":
                    x.arrive()
                else:
                    st, n, qb, qn, db, dn = x
                    assert self.k[st] == n and self.q[qb] == qn
                    self.d[db] = dn
                yield
            else:
                yield "idle"

    def epilogue(self, group):
        L, qn, dn = self.L, 0, 0
        for n, (_, _, nq, first) in enumerate(self.items):
            mine = 0 if self.split else n & 1
            for _ in range(first, nq):
                if self.fresh(n):
                    yield self.qfull[qn % L["qbufs"]], (qn // L["qbufs"]) & 1
                    qn += 1
                qb, db = (qn - 1) % L["qbufs"], dn % L["dbufs"]
                assert self.q[qb] == qn - 1          # its log-sum-exps and limits
                if self.split or mine == group:
                    yield self.dfull[db], (dn // L["dbufs"]) & 1
                    assert self.d[db] == dn and self.q[qb] == qn - 1
                    if self.q8:
                        assert self.scale[n % L["scales"]] == n
                    self.summed[group].append(dn)
                    self.dempty[db].arrive()
                    yield
                if self.last_use(n):
                    self.qempty[qb].arrive()
                dn += 1
                yield
            if self.split:
                p = n % L["parts"]
                if group == 1:
                    self.part[p] = n
                    self.bpart[p].arrive()
                else:
                    yield self.bpart[p], (n // L["parts"]) & 1
                    assert self.part[p] == n
                yield

    def run(self, pick):
        """Names of the agents left waiting for ever ([]: all came to their end);
        pick chooses who goes next."""
        at = {}
        for a, g in self.agents.items():
            at[a] = next(g, "end")
        while True:
            able = [a for a, w in at.items() if w != "end" and
                    (w is None or (w == "idle" and self.queue) or
                     (isinstance(w, tuple) and w[0].passed(w[1])))]
            if not able:
                return [a for a, w in at.items() if w not in ("end", "idle")]
            a = pick(able)
            at[a] = next(self.agents[a], "end")


def schedules(names):
    """Each agent as the slowest, as the fastest, and some at random."""
    names = list(names)
    for slow in names:
        for turn in range(len(names)):
            order = [a for a in names[turn:] + names[:turn] if a != slow]
            yield lambda able, o=order + [slow]: min(able, key=o.index)
    for seed in range(40):
        rng = random.Random(seed)
        order = names[:]
        rng.shuffle(order)
        yield lambda able, o=order, r=rng: (r.choice(able) if r.random() < 0.3 else
                                            min(able, key=o.index))


def stuck(q8, split, seqs, qtb, **kw):
    names = Model(q8, split, seqs, qtb).agents
    return [m for m in (Model(q8, split, seqs, qtb, **kw).run(p) for p in schedules(names)) if m]


# windows of one tile, of several, of both in turn, and of several with a short
# one between (contexts and window lengths)
ONE = [(900, 60), (128, 1), (1300, 64)]
SEVERAL = [(700, 400), (513, 513), (300, 129)]
MIXED = [(500, 300), (900, 20), (260, 200), (64, 64), (1500, 65)]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("split,seqs", [(False, ONE), (True, ONE), (True, SEVERAL), (True, MIXED)])
def test_every_schedule_ends(q8, split, seqs):
    assert not stuck(q8, split, seqs, 64)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("seqs", [SEVERAL, MIXED])
def test_windows_longer_than_announced_end_too(q8, seqs):
    # a launch for windows of one tile that meets longer ones
    assert not stuck(q8, False, seqs, 64)


def test_the_model_finds_a_lost_phase():
    # an issuing thread that does not hold back the query tiles it leaves to the
    # other one can find two phases gone by at once, which looks like none
    assert stuck(False, True, SEVERAL, 64, issuers=0)


@pytest.mark.parametrize("q8,split", [(False, False), (False, True), (True, False), (True, True)])
def test_every_tile_is_summed_once(q8, split):
    m = Model(q8, split, MIXED if split else ONE, 64)
    assert m.run(lambda able: able[0]) == []
    tiles = sum(nq - first for _, _, nq, first in m.items)
    if split:
        assert m.summed[0] == m.summed[1] == list(range(tiles))
    else:
        assert sorted(m.summed[0] + m.summed[1]) == list(range(tiles))
