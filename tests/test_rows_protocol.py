"""Host model of the rows kernel's mbarrier protocol (csrc/rows_kernel.cuh).

One CTA: the warp that walks the plan, the TMA producer, the MMA issuer and
the softmax warps of each row tile (two stand for the four), replayed under
random interleavings.  TMA loads land in any order, MMAs and their commits
complete in issue order, an agent advances whenever its wait is satisfied.
Items follow one another in all their forms: two tiles of rows that share the
key blocks, one tile alone, split keys (both tiles hold the same rows, with the
blocks in turn), items without keys, and, with head_dim 256, one tile with two
score slots and key blocks of two ring tiles each.

Checked at every step:
- a parity wait for phase k starts when k - 1 has completed, so that it passes
  on its own phase (as in test_pipeline_protocol.py);
- no ring stage is loaded while an MMA may still read it, none zeroed while one
  may read or before it has landed, and every MMA reads the block meant for it;
- scores are overwritten only after every warp has read them and the value MMA
  of the P that took their place has been issued before;
- O is rescaled, or read, only while no value MMA of its tile is in flight,
  and a new item's first value MMA waits for the last one's epilogue;
- nothing stands still, and nothing is in flight when the CTA ends.

With one wait that runs out, whichever and whenever, every agent still ends
and no load is left in flight.  And no wait takes longer than the blocks of the
items in the ring, which is what a wait is allowed beside its timeout.
"""
import random
from collections import namedtuple

import pytest

RING = 4    # items handed out ahead
WARPS = 2   # softmax warps of a tile

# blocks, kind ("two", "lone", "split"), whether its last block ends inside (V past the end is zeroed)
Item = namedtuple("Item", "n kind tail")
# tiles of a CTA, ring tiles of a key block, stages of the K and of the V ring
Shape = namedtuple("Shape", "nt tpb nsk nsv")
SHAPES = {64: Shape(2, 1, 4, 4), 128: Shape(2, 1, 2, 2), 256: Shape(1, 2, 2, 2)}


class Violation(Exception):
    pass


class GaveUp(Exception):
    """This agent's wait ran out, or another's did."""


class Bar:
    def __init__(self, arrivals=1):
        self.arrivals, self.pending, self.c = arrivals, arrivals, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.c = self.arrivals, self.c + 1


class Cta:
    def __init__(self, shape, items, rng, give_up_at=None, mistake=None):
        self.shape, self.items, self.rng, self.mistake = shape, items, rng, mistake
        self.nt = shape.nt
        self.k_full, self.k_empty = [Bar() for _ in range(shape.nsk)], [Bar() for _ in range(shape.nsk)]
        self.v_full, self.v_empty = [Bar() for _ in range(shape.nsv)], [Bar() for _ in range(shape.nsv)]
        self.q_full, self.q_empty = [Bar() for _ in range(self.nt)], [Bar() for _ in range(self.nt)]
        self.s_full, self.o_full = [Bar(), Bar()], [Bar(), Bar()]
        self.p_half, self.p_full = [Bar(WARPS), Bar(WARPS)], [Bar(WARPS), Bar(WARPS)]
        self.drain = Bar()
        self.item_full = [Bar() for _ in range(RING)]
        self.item_empty = [Bar(self.nt * WARPS + 2) for _ in range(RING)]
        self.item_ring = [None] * RING
        self.landing = []                        # loads in flight: (barrier, the dict of the stage, its content)
        self.mma = []                            # MMAs and commits in issue order
        self.stage = {k: [dict(holds=None, loading=False, readers=0, zeroed=True) for _ in range(n)]
                      for k, n in (("K", shape.nsk), ("V", shape.nsv), ("Q", self.nt))}
        self.scores = [dict(unread=0, p_pending=False) for _ in range(2)]     # by S slot
        self.o = [dict(in_flight=0, unread=0) for _ in range(self.nt)]        # by tile
        self.abort, self.waits, self.give_up_at = False, 0, give_up_at
        self.pv_done = 0                         # blocks whose value MMA has been issued
        self.longest_wait = 0                    # ... during one wait of a softmax warp, at most

    # ------------------------------------------------------------ primitives
    def wait(self, bar, k, what, bounded=True):
        """Generator step: yields until the hardware's predicate (completed phases have the other parity) holds."""
        self.waits += 1
        if bounded and self.waits == self.give_up_at:
            self.abort = True
            raise GaveUp
        start = self.pv_done
        while True:
            if (bar.c & 1) != (k & 1):
                if bar.c != k + 1:
                    raise Violation(f"{what}: wait for phase {k} passed at {bar.c}")
                if what.startswith("softmax"):
                    self.longest_wait = max(self.longest_wait, self.pv_done - start)
                return
            if bar.c >= k + 2:
                raise Violation(f"{what}: wait for phase {k} blocks at {bar.c}")
            if bounded and self.abort:
                raise GaveUp
            yield

    def load(self, kind, slot, bar, content):
        st = self.stage[kind][slot]
        if st["loading"] or st["readers"]:
            raise Violation(f"{kind} stage {slot} loaded with {content} while in use")
        st.update(loading=True, holds=None)
        self.landing.append((bar, st, content))

    def next_item(self, n, what):
        yield from self.wait(self.item_full[n % RING], n // RING, what)
        it = self.item_ring[n % RING]
        if it[0] != n:
            raise Violation(f"{what}: item {it[0]} in the place of {n}")
        self.item_empty[n % RING].arrive()
        return it[1]

    def slots_of(self, it):
        return 2 if it.kind == "two" else 1

    # ---------------------------------------------------------------- agents
    def planner(self):
        try:
            for n in range(len(self.items) + 1):
                if n >= RING:
                    yield from self.wait(self.item_empty[n % RING], n // RING - 1, f"planner item {n}")
                self.item_ring[n % RING] = (n, self.items[n] if n < len(self.items) else None)
                self.item_full[n % RING].arrive()
                yield
        except GaveUp:
            self.abort = True

    def producer(self):
        sh, t = self.shape, dict(K=0, V=0, Q=0)

        def load_block(kind, n_item, blk):
            full, empty, ns = ((self.k_full, self.k_empty, sh.nsk) if kind == "K" else
                               (self.v_full, self.v_empty, sh.nsv))
            for hf in range(sh.tpb):
                n = t[kind]
                if n >= ns:
                    yield from self.wait(empty[n % ns], n // ns - 1, f"producer {kind}")
                self.load(kind, n % ns, full[n % ns], (n_item, blk, hf))
                t[kind] += 1

        gave_up = False
        try:
            n = 0
            while True:
                it = yield from self.next_item(n, "producer item")
                if it is None:
                    break
                if it.n > 0:
                    for slot in range(self.slots_of(it)):
                        s = t["Q"] % self.nt
                        if t["Q"] >= self.nt:
                            yield from self.wait(self.q_empty[s], t["Q"] // self.nt - 1, "producer Q")
                        self.load("Q", s, self.q_full[s], (n, slot, 0))
                        t["Q"] += 1
                    yield from load_block("K", n, 0)
                    for i in range(it.n):
                        if i + 1 < it.n:
                            yield from load_block("K", n, i + 1)
                        yield from load_block("V", n, i)
                n += 1
        except GaveUp:
            self.abort = gave_up = True
        if self.mistake == "loads awaited only by a producer that gave up" and not gave_up:
            return
        # of every stage, the last load: all before it have landed
        for kind, full, ns in (("K", self.k_full, sh.nsk), ("V", self.v_full, sh.nsv), ("Q", self.q_full, self.nt)):
            for u in range(max(0, t[kind] - ns), t[kind]):
                yield from self.wait(full[u % ns], u // ns, f"drain {kind}", bounded=False)

    def reads(self, kind, slot, content):
        st = self.stage[kind][slot]
        if st["loading"] or st["holds"] != content:
            raise Violation(f"an MMA reads {kind} stage {slot} with {st['holds']}, not {content}")
        if kind == "V" and not st["zeroed"]:
            raise Violation(f"an MMA reads V {content} before the rows past the end are zeros")
        st["readers"] += 1
        return st

    def issuer(self):
        sh, nt = self.shape, self.nt
        u = uq = n = 0
        g = [0, 0]
        try:
            while True:
                it = yield from self.next_item(n, "issuer item")
                if it is None:
                    break
                if it.n == 0:
                    n += 1
                    continue
                slots = self.slots_of(it)
                two = slots == 2
                for s in range(slots):
                    yield from self.wait(self.q_full[(uq + s) % nt], (uq + s) // nt, "issuer Q")
                steps = 2 * it.n if two else it.n
                ahead = 1 if nt == 1 else (2 if it.kind in ("two", "split") else 1)

                def slot_of(j):
                    return (u + j) & 1 if nt == 1 else (j & 1 if ahead == 2 else 0)

                def qk(j):
                    slot, i = slot_of(j), j >> 1 if two else j
                    read = []
                    for hf in range(sh.tpb):
                        m = (u + i) * sh.tpb + hf
                        if not two or slot == 0:
                            yield from self.wait(self.k_full[m % sh.nsk], m // sh.nsk, "issuer K")
                        read.append(self.reads("K", m % sh.nsk, (n, i, hf)))
                    q = self.reads("Q", (uq + (slot if two else 0)) % nt, (n, slot if two else 0, 0))
                    s = self.scores[slot]
                    if s["unread"] or s["p_pending"]:
                        raise Violation("scores overwritten before they were used")
                    s.update(unread=WARPS, p_pending=True)
                    self.mma.append(("read", read + [q]))
                    self.mma.append(("arrive", self.s_full[slot]))
                    if not two or slot == 1:
                        for hf in range(sh.tpb):
                            self.mma.append(("arrive", self.k_empty[((u + i) * sh.tpb + hf) % sh.nsk]))
                    if j + 1 == steps:
                        for s2 in range(slots):
                            self.mma.append(("arrive", self.q_empty[(uq + s2) % nt]))

                def pv(j):
                    slot, i = slot_of(j), j >> 1 if two else j
                    tile = 0 if nt == 1 else slot
                    first = j < (1 if nt == 1 else ahead)
                    if sh.tpb == 1 and (not two or slot == 0):
                        m = u + i
                        yield from self.wait(self.v_full[m % sh.nsv], m // sh.nsv, "issuer V")
                    read = []
                    for part in range(1 if nt == 1 else 2):
                        half = nt == 2 and part == 0
                        yield from self.wait((self.p_half if half else self.p_full)[slot], g[slot], "issuer P")
                        for hf in range(sh.tpb):
                            m = (u + i) * sh.tpb + hf
                            if sh.tpb > 1:
                                yield from self.wait(self.v_full[m % sh.nsv], m // sh.nsv, "issuer V")
                            read.append(self.reads("V", m % sh.nsv, (n, i, hf)))
                        o = self.o[tile]
                        if first and part == 0:
                            if o["unread"]:
                                raise Violation("O overwritten before the epilogue read it")
                            o["unread"] = WARPS
                        if part == 0:
                            o["in_flight"] += 1
                    if self.scores[slot]["unread"]:
                        raise Violation("a value MMA of scores that were not read")
                    g[slot] += 1
                    self.scores[slot]["p_pending"] = False
                    self.pv_done += 1
                    self.mma.append(("read", read))
                    self.mma.append(("pv", tile))
                    self.mma.append(("arrive", self.o_full[slot]))
                    if not two or slot == 1:
                        for hf in range(sh.tpb):
                            self.mma.append(("arrive", self.v_empty[((u + i) * sh.tpb + hf) % sh.nsv]))

                for j in range(-ahead, steps):
                    if nt == 1:
                        if j + 1 < steps:
                            yield from qk(j + 1)
                        if j >= 0:
                            yield from pv(j)
                    elif self.mistake == "QK before PV":
                        if j + ahead < steps:
                            yield from qk(j + ahead)
                        if j >= 0:
                            yield from pv(j)
                    else:
                        if j >= 0:
                            yield from pv(j)
                        if j + ahead < steps:
                            yield from qk(j + ahead)
                u += it.n
                uq += slots
                n += 1
        except GaveUp:
            self.abort = True
        self.mma.append(("arrive", self.drain))
        yield from self.wait(self.drain, 0, "drain", bounded=False)

    def softmax(self, t, warp):
        sh, nt = self.shape, self.nt
        g = u = n = 0
        o = self.o[t]

        def wait_pv(k, what):
            if nt == 2:
                yield from self.wait(self.o_full[t], k, what)
            else:
                yield from self.wait(self.o_full[k & 1], k >> 1, what)

        try:
            while True:
                it = yield from self.next_item(n, "softmax item")
                if it is None:
                    return
                n, u0, u = n + 1, u, u + it.n
                split = it.kind == "split"
                if not split and t >= self.slots_of(it):
                    continue
                i0, step = (t, 2) if split else (0, 1)
                for i in range(i0, it.n, step):
                    slot = t if nt == 2 else g & 1
                    yield from self.wait(self.s_full[slot], g if nt == 2 else g >> 1, "softmax S")
                    if i == it.n - 1 and it.tail and (t == 0 or split):
                        if nt == 1 and g >= 1 and self.mistake != "zeros without waiting for the block before":
                            yield from wait_pv(g - 1, "softmax zeros")
                        for hf in range(sh.tpb):
                            m = (u0 + i) * sh.tpb + hf
                            yield from self.wait(self.v_full[m % sh.nsv], m // sh.nsv, "softmax V")
                            st = self.stage["V"][m % sh.nsv]
                            if st["holds"] != (n - 1, i, hf) or st["readers"]:
                                raise Violation("rows of another block zeroed, or of one in use")
                            st["zeros"] = st.get("zeros", 0) + 1
                            if st["zeros"] == WARPS:
                                st["zeroed"] = True
                    self.scores[slot]["unread"] -= 1
                    yield
                    if i > i0 and self.rng.random() < 0.4:   # this warp rescales O
                        if self.mistake != "rescale without waiting":
                            yield from wait_pv(g - 1, "softmax rescale")
                        if o["in_flight"]:
                            raise Violation("O rescaled under a value MMA")
                        yield
                    if nt == 2:
                        self.p_half[slot].arrive()
                        yield
                    self.p_full[slot].arrive()
                    g += 1
                if i0 < it.n:
                    yield from wait_pv(g - 1, "softmax epilogue")
                    if o["in_flight"]:
                        raise Violation("O read under a value MMA")
                    yield
                    o["unread"] -= 1
        except GaveUp:
            self.abort = True

    # ------------------------------------------------------------- execution
    def run(self):
        agents = {"planner": self.planner(), "producer": self.producer(), "issuer": self.issuer()}
        for t in range(self.nt):
            for w in range(WARPS):
                agents[f"softmax {t}.{w}"] = self.softmax(t, w)
        idle = 0
        while agents or self.landing or self.mma:
            before = (self.waits, len(self.landing), len(self.mma), len(agents), self.pv_done)
            moves = list(agents) + ["land"] * bool(self.landing) + ["mma"] * bool(self.mma)
            move = self.rng.choice(moves)
            if move == "land":
                bar, st, content = self.landing.pop(self.rng.randrange(len(self.landing)))
                last = self.items[content[0]]
                st.update(loading=False, holds=content, zeros=0,
                          zeroed=not (last.tail and content[1] == last.n - 1))
                bar.arrive()
            elif move == "mma":
                kind, x = self.mma.pop(0)
                if kind == "read":
                    for st in x:
                        st["readers"] -= 1
                elif kind == "pv":
                    self.o[x]["in_flight"] -= 1
                else:
                    x.arrive()
            else:
                try:
                    next(agents[move])
                except StopIteration:
                    del agents[move]
            after = (self.waits, len(self.landing), len(self.mma), len(agents), self.pv_done)
            idle = 0 if before != after else idle + 1
            if idle > 3000:
                raise Violation(f"stands still: {sorted(agents)}")
            if not agents and self.landing:
                raise Violation("the CTA ends with loads in flight")


def _items(rng, nt, most=6):
    kinds = ["two", "lone", "split"] if nt == 2 else ["lone"]
    items = []
    for _ in range(rng.randint(1, 9)):
        n = 0 if rng.random() < 0.2 else rng.randint(1, most)
        items.append(Item(n, rng.choice(kinds), rng.random() < 0.5))
    return items


@pytest.mark.parametrize("d", [64, 128, 256])
def test_protocol_holds(d):
    rng = random.Random(d)
    for _ in range(250):
        Cta(SHAPES[d], _items(rng, SHAPES[d].nt), rng).run()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_wait_that_runs_out_ends_every_role(d):
    rng = random.Random(2 * d)
    for _ in range(250):
        items = _items(rng, SHAPES[d].nt, 4)
        whole = Cta(SHAPES[d], items, rng)
        whole.run()
        cta = Cta(SHAPES[d], items, rng, give_up_at=rng.randint(1, whole.waits))
        cta.run()


def test_waits_take_no_longer_than_the_items_in_the_ring():
    """The second tile's warps leave items of one tile at once.  Their next wait then spans the items that the first
    tile still works on: more than one item (so that a timeout of one must not be all they have), but never more
    blocks than RING items hold, and the few that are under way."""
    rng = random.Random(5)
    longest = 0
    for _ in range(40):
        items = [Item(rng.choice([25, 30]), rng.choice(["lone", "lone", "lone", "two"]), False) for _ in range(12)]
        cta = Cta(SHAPES[128], items, rng)
        cta.run()
        longest = max(longest, cta.longest_wait)
    assert 2 * 30 < longest <= RING * 30 + 4


@pytest.mark.parametrize("d,mistake,found", [
    (128, "QK before PV", "scores overwritten"), (256, "rescale without waiting", "O rescaled"),
    (256, "zeros without waiting for the block before", "softmax V: wait"),
    (64, "loads awaited only by a producer that gave up", "in flight"),
    (256, "loads awaited only by a producer that gave up", "in flight")])
def test_the_model_finds_mistakes(d, mistake, found):
    rng = random.Random(7)
    seen = set()
    for _ in range(400):
        items = _items(rng, SHAPES[d].nt)
        give_up = None
        if "gave up" in mistake:
            whole = Cta(SHAPES[d], items, rng)
            whole.run()
            give_up = rng.randint(1, whole.waits)
        try:
            Cta(SHAPES[d], items, rng, give_up, mistake).run()
        except Violation as e:
            seen.add(str(e))
    assert any(found in s for s in seen), seen
