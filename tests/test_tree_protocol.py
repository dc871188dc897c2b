"""Host model of the rows kernel's mbarrier protocol over paged keys (csrc/rows_kernel.cuh).

What differs from test_rows_protocol, whose checks these are: V may have a producer of
its own; at head_dim 64 three S slots that the steps take in turn, with two QKs ahead of the PV at hand and the
barriers of a tile's steps three in turn; at head_dim 128, where the rows fit one
tile, one tile with two S slots, two Q slots and three stages of V; at head_dim 256
halves of K's and V's blocks given back each after its own MMAs.  There the block that
ends inside is any one of an item's, as items may take their blocks from the middle on.
"""
import random
from collections import namedtuple

import pytest

from tests.test_rows_protocol import RING, WARPS, Bar, Cta, GaveUp, Item, Shape, Violation

Form = namedtuple("Form", "shape nq three")
FORMS = {64: Form(Shape(2, 1, 4, 4), 2, True), 128: Form(Shape(1, 1, 2, 3), 2, False), 256: Form(Shape(1, 2, 2, 2), 1, False)}


class Paged(Cta):
    def __init__(self, form, items, rng, give_up_at=None, mistake=None, loaders=2):
        super().__init__(form.shape, items, rng, give_up_at, mistake)
        self.nq, self.three, self.by_half = form.nq, form.three, form.shape.tpb == 2
        self.tails = [rng.randrange(it.n) if it.n and it.tail else -1 for it in items]
        self.turn = 2 if mistake == "two barriers in turn" else 3
        self.o_turn = 1 if mistake == "one barrier for O" else self.turn
        self.q_full, self.q_empty = [Bar() for _ in range(self.nq)], [Bar() for _ in range(self.nq)]
        self.stage["Q"] = [dict(holds=None, loading=False, readers=0, zeroed=True) for _ in range(self.nq)]
        self.halves = form.shape.tpb == 1 and not form.three
        self.loaders = loaders
        self.item_empty = [Bar(self.nt * WARPS + 1 + loaders) for _ in range(RING)]
        if self.three:
            n = self.turn * self.nt
            self.s_full, self.o_full = [Bar() for _ in range(n)], [Bar() for _ in range(self.o_turn * self.nt)]
            self.p_half, self.p_full = [Bar(WARPS) for _ in range(n)], [Bar(WARPS) for _ in range(n)]
            self.scores = [dict(unread=0, p_pending=False) for _ in range(3)]

    def reads(self, kind, slot, content):
        st = self.stage[kind][slot]
        if self.by_half and kind == "V":  # (the base has it that the last block ends inside)
            st["zeroed"] = content[1] != self.tails[content[0]] or st.get("zeros") == WARPS
        return super().reads(kind, slot, content)

    def producer(self):
        """One warp, or two, of Q and K and of V, in any order."""
        warps = [self.loads("QK"), self.loads("V")] if self.loaders == 2 else [self.loads("QKV")]
        while warps:
            warp = self.rng.choice(warps)
            try:
                next(warp)
            except StopIteration:
                warps.remove(warp)
            yield

    def loads(self, kinds):
        sh, t = self.shape, dict(K=0, V=0, Q=0)
        rings = dict(K=(self.k_full, self.k_empty, sh.nsk), V=(self.v_full, self.v_empty, sh.nsv),
                     Q=(self.q_full, self.q_empty, self.nq))

        def load(kind, content):
            full, empty, ns = rings[kind]
            n = t[kind]
            if n >= ns:
                yield from self.wait(empty[n % ns], n // ns - 1, f"producer {kind}")
            self.load(kind, n % ns, full[n % ns], content)
            t[kind] += 1

        try:
            n = 0
            while True:
                it = yield from self.next_item(n, "producer item")
                if it is None:
                    break
                if it.n > 0 and "Q" in kinds:
                    for slot in range(self.slots_of(it)):
                        yield from load("Q", (n, slot, 0))
                for i in range(-1, it.n):
                    for kind, blk in (("K", i + 1), ("V", i)):
                        for hf in range(sh.tpb if kind in kinds and 0 <= blk < it.n else 0):
                            yield from load(kind, (n, blk, hf))
                n += 1
        except GaveUp:
            self.abort = True
        for kind in kinds:
            full, _, ns = rings[kind]
            for u in range(max(0, t[kind] - ns), t[kind]):
                yield from self.wait(full[u % ns], u // ns, f"drain {kind}", bounded=False)

    def issuer(self):
        sh, nt, three = self.shape, self.nt, self.three
        u = uq = n = us = 0
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
                    yield from self.wait(self.q_full[(uq + s) % self.nq], (uq + s) // self.nq, "issuer Q")
                steps = 2 * it.n if two else it.n
                both = nt == 2 and it.kind in ("two", "split")

                def tile_of(j):
                    return j & 1 if both else 0

                def slot_of(j):
                    return (us + j) % 3 if three else (u + j) & 1

                def count_of(j):
                    return g[tile_of(j)] + (j >> 1 if both else j)

                def set_of(j):
                    return self.turn * tile_of(j) + count_of(j) % self.turn if three else slot_of(j)

                def halves(kind, full, empty, ns, i, last):
                    """The MMAs of a block's halves; `last` goes with the second's."""
                    for hf in range(sh.tpb):
                        m = (u + i) * sh.tpb + hf
                        yield from self.wait(full[m % ns], m // ns, f"issuer {kind}")
                        st = self.reads(kind, m % ns, (n, i, hf))
                        self.mma.append(("read", [st] + (last if hf + 1 == sh.tpb else [])))
                        if self.mistake == "given back by the warp" and kind == "V":
                            empty[m % ns].arrive()
                        else:
                            self.mma.append(("arrive", empty[m % ns]))

                def qk(j):
                    slot, tile, i = slot_of(j), tile_of(j), j >> 1 if two else j
                    read = []
                    for hf in range(0 if self.by_half else sh.tpb):
                        m = (u + i) * sh.tpb + hf
                        if not two or tile == 0:
                            yield from self.wait(self.k_full[m % sh.nsk], m // sh.nsk, "issuer K")
                        read.append(self.reads("K", m % sh.nsk, (n, i, hf)))
                    q = self.reads("Q", (uq + (tile if two else 0)) % self.nq, (n, tile if two else 0, 0))
                    s = self.scores[slot]
                    if s["unread"] or s["p_pending"]:
                        raise Violation("scores overwritten before they were used")
                    s.update(unread=WARPS, p_pending=True)
                    if self.by_half:
                        yield from halves("K", self.k_full, self.k_empty, sh.nsk, i, [q])
                    else:
                        self.mma.append(("read", read + [q]))
                    self.mma.append(("arrive", self.s_full[set_of(j)]))
                    if not self.by_half and (not two or tile == 1):
                        for hf in range(sh.tpb):
                            self.mma.append(("arrive", self.k_empty[((u + i) * sh.tpb + hf) % sh.nsk]))
                    if j + 1 == steps:
                        for s2 in range(slots):
                            self.mma.append(("arrive", self.q_empty[(uq + s2) % self.nq]))

                def pv(j):
                    slot, tile, i = slot_of(j), tile_of(j), j >> 1 if two else j
                    the_set, first = set_of(j), j < (2 if both else 1)
                    phase = count_of(j) // self.turn if three else g[slot]
                    if sh.tpb == 1 and (not two or tile == 0):
                        m = u + i
                        yield from self.wait(self.v_full[m % sh.nsv], m // sh.nsv, "issuer V")
                    read = []
                    for part in range(2 if self.halves else 1):
                        half = self.halves and part == 0
                        yield from self.wait((self.p_half if half else self.p_full)[the_set], phase, "issuer P")
                        for hf in range(0 if self.by_half else sh.tpb):
                            m = (u + i) * sh.tpb + hf
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
                    if not three:
                        g[slot] += 1
                    self.scores[slot]["p_pending"] = False
                    self.pv_done += 1
                    if self.by_half:
                        yield from halves("V", self.v_full, self.v_empty, sh.nsv, i, [])
                    else:
                        self.mma.append(("read", read))
                    self.mma.append(("pv", tile))
                    o_set = self.o_turn * tile + count_of(j) % self.o_turn if three else slot
                    self.mma.append(("arrive", self.o_full[o_set]))
                    if not self.by_half and (not two or tile == 1):
                        for hf in range(sh.tpb):
                            self.mma.append(("arrive", self.v_empty[((u + i) * sh.tpb + hf) % sh.nsv]))

                ahead = 2 if three else 1
                for j in range(-ahead, steps):
                    if j + ahead < steps:
                        yield from qk(j + ahead)
                    if j >= 0:
                        yield from pv(j)
                if three:
                    g[0] += (steps + 1) // 2 if both else steps
                    g[1] += steps // 2 if both else 0
                    us += steps
                u += it.n
                uq += slots
                n += 1
        except GaveUp:
            self.abort = True
        self.mma.append(("arrive", self.drain))
        yield from self.wait(self.drain, 0, "drain", bounded=False)

    def softmax(self, t, warp):
        sh, nt, three = self.shape, self.nt, self.three
        g = u = n = us = 0
        o = self.o[t]

        def wait_pv(k, what):
            if three:
                yield from self.wait(self.o_full[self.o_turn * t + k % self.o_turn], k // self.o_turn, what)
            else:
                yield from self.wait(self.o_full[k & 1], k >> 1, what)

        try:
            while True:
                it = yield from self.next_item(n, "softmax item")
                if it is None:
                    return
                n, u0, u = n + 1, u, u + it.n
                split, two = it.kind == "split", self.slots_of(it) == 2
                us0, us = us, us + (2 * it.n if two else it.n)
                if not split and t >= self.slots_of(it):
                    continue
                i0, step = (t, 2) if split else (0, 1)
                for i in range(i0, it.n, step):
                    slot = (us0 + (2 * i + t if two else i)) % 3 if three else g & 1
                    the_set = self.turn * t + g % self.turn if three else slot
                    yield from self.wait(self.s_full[the_set], g // self.turn if three else g >> 1, "softmax S")
                    if (i == self.tails[n - 1] if self.by_half else i == it.n - 1 and it.tail) and (t == 0 or split):
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
                        yield from wait_pv(g - 1, "softmax rescale")
                        if o["in_flight"]:
                            raise Violation("O rescaled under a value MMA")
                        yield
                    if self.halves:
                        self.p_half[the_set].arrive()
                        yield
                    self.p_full[the_set].arrive()
                    g += 1
                if i0 < it.n:
                    yield from wait_pv(g - 1, "softmax epilogue")
                    if o["in_flight"]:
                        raise Violation("O read under a value MMA")
                    yield
                    o["unread"] -= 1
        except GaveUp:
            self.abort = True


def _items(rng, nt, most=7):
    """Of one launch: all split, or tiles in pairs with a lone one where the last group has no more."""
    kinds = rng.choice([["split"], ["two", "two", "lone"], ["lone"]]) if nt == 2 else ["lone"]
    return [Item(0 if rng.random() < 0.2 else rng.randint(1, most), rng.choice(kinds), rng.random() < 0.5)
            for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("loaders", [1, 2])
def test_protocol_holds(d, loaders):
    rng = random.Random(d)
    for _ in range(250):
        Paged(FORMS[d], _items(rng, FORMS[d].shape.nt), rng, loaders=loaders).run()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("loaders", [1, 2])
def test_a_wait_that_runs_out_ends_every_role(d, loaders):
    rng = random.Random(2 * d)
    for _ in range(250):
        items = _items(rng, FORMS[d].shape.nt, 4)
        whole = Paged(FORMS[d], items, rng, loaders=loaders)
        whole.run()
        Paged(FORMS[d], items, rng, give_up_at=rng.randint(1, whole.waits), loaders=loaders).run()


def test_waits_take_no_longer_than_the_items_in_the_ring():
    rng = random.Random(5)
    for _ in range(30):
        items = [Item(rng.choice([25, 30]), rng.choice(["lone", "lone", "lone", "two"]), False) for _ in range(12)]
        cta = Paged(FORMS[64], items, rng)
        cta.run()
        assert cta.longest_wait <= RING * 30 + 6


@pytest.mark.parametrize("d,mistake,found", [
    (64, "two barriers in turn", "softmax S"), (64, "one barrier for O", "softmax"),
    (256, "given back by the warp", "while in use"), (256, "zeros without waiting for the block before", "softmax V")])
def test_the_model_finds_mistakes(d, mistake, found):
    rng = random.Random(7)
    seen = set()
    for _ in range(400):
        try:
            Paged(FORMS[d], _items(rng, FORMS[d].shape.nt), rng, mistake=mistake).run()
        except Violation as e:
            seen.add(str(e))
    assert any(found in s for s in seen), seen
