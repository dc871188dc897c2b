"""Host model of how a CTA of the decode kernel ends when a wait runs out.

The roles of test_pipeline_protocol.py (producer, score-MMA issuer, value-MMA
issuer, softmax warpgroup) under random interleavings, with one wait, whichever
and whenever, that gives up: it raises the CTA's abort flag, which every other
wait sees.  Every role must end, an issuer not before its MMAs have completed,
and the CTA must not end while a TMA load is still on its way into it: it would
write the shared memory of whichever CTA comes next.
"""
import random

import pytest

from tests.test_pipeline_protocol import Bar, Violation, random_items, split_rings


class GaveUp(Exception):
    pass


def run_cta(ns, items, rng, give_up_at=None, always_drain=True):
    """One CTA over `items` (block counts); returns the waits that were begun."""
    G = sum(items)
    k_slot, v_slot = split_rings(ns)
    full, empty = [Bar() for _ in range(ns)], [Bar() for _ in range(ns)]
    q_full, q_empty = [Bar(), Bar()], [Bar(), Bar()]
    s_full, s_empty, p_full, p_empty = ([Bar(), Bar()] for _ in range(4))
    drains = {"qk": Bar(), "pv": Bar()}
    landing, mma = [], {"qk": [], "pv": []}
    state = dict(waits=0, abort=False)

    def wait(bar, k, bounded=True):
        state["waits"] += 1
        if bounded and state["waits"] == give_up_at:
            raise GaveUp
        while (bar.c & 1) == (k & 1):
            if bounded and state["abort"]:
                raise GaveUp
            yield
        if bar.c != k + 1:
            raise Violation(f"wait for phase {k} passed at {bar.c}")

    def producer():
        last, kq, gave_up = {}, 0, False

        def load(slot):
            stage, phase = slot
            if phase > 0:
                yield from wait(empty[stage], phase - 1)
            landing.append(full[stage])
            last[stage] = (full[stage], phase)

        try:
            g = 0
            for n in items:
                if n == 0:
                    continue
                if kq >= 2:
                    yield from wait(q_empty[kq % 2], kq // 2 - 1)
                landing.append(q_full[kq % 2])
                last["Q", kq % 2] = (q_full[kq % 2], kq // 2)
                kq += 1
                for _ in range(n):
                    yield from load(k_slot(g, G))
                    if g > 0:
                        yield from load(v_slot(g - 1, G))
                    g += 1
            if G > 0:
                yield from load(v_slot(G - 1, G))
        except GaveUp:
            state["abort"] = gave_up = True
        if gave_up or always_drain:
            for bar, phase in last.values():
                yield from wait(bar, phase, bounded=False)

    def issuer(which):
        try:
            g = kq = 0
            for n in items:
                if n and which == "qk":
                    yield from wait(q_full[kq % 2], kq // 2)
                for i in range(n):
                    sl = g & 1
                    if which == "qk":
                        if g >= 2:
                            yield from wait(s_empty[sl], (g >> 1) - 1)
                        stage, phase = k_slot(g, G)
                        yield from wait(full[stage], phase)
                        mma["qk"] += [s_full[sl], empty[stage]] + ([q_empty[kq % 2]] if i == n - 1 else [])
                    else:
                        yield from wait(p_full[sl], g >> 1)
                        stage, phase = v_slot(g, G)
                        yield from wait(full[stage], phase)
                        mma["pv"] += [p_empty[sl], empty[stage]]
                    g += 1
                kq += n > 0
        except GaveUp:
            state["abort"] = True
        mma[which].append(drains[which])
        yield from wait(drains[which], 0, bounded=False)

    def softmax():
        try:
            for g in range(G):
                sl = g & 1
                yield from wait(s_full[sl], g >> 1)
                s_empty[sl].c += 1
                if g >= 2:
                    yield from wait(p_empty[sl], (g >> 1) - 1)
                p_full[sl].c += 1
            if G > 0:
                yield from wait(p_empty[(G - 1) & 1], (G - 1) >> 1)
        except GaveUp:
            state["abort"] = True

    agents = {"producer": producer(), "qk": issuer("qk"), "pv": issuer("pv"), "softmax": softmax()}
    for _ in range(200000):
        if not agents:
            if landing or any(mma.values()):
                raise Violation("the CTA ends with work in flight")
            return state["waits"]
        move = rng.choice(list(agents) + ["land"] * bool(landing) + [("mma", q) for q in mma if mma[q]])
        if move == "land":
            landing.pop(rng.randrange(len(landing))).c += 1
        elif isinstance(move, tuple):
            mma[move[1]].pop(0).c += 1
        else:
            try:
                next(agents[move])
            except StopIteration:
                del agents[move]
    raise Violation("no progress")


@pytest.mark.parametrize("ns", [4, 5, 6, 12])
def test_a_wait_that_runs_out_ends_every_role(ns):
    rng = random.Random(ns)
    for _ in range(400):
        items = random_items(rng, rng.randint(1, 12))
        run_cta(ns, items, rng, rng.randint(1, run_cta(ns, items, rng)))


def test_loads_in_flight_are_found():
    """The model sees a producer that has issued its last load and does not wait for it."""
    rng = random.Random(9)
    with pytest.raises(Violation, match="in flight"):
        for _ in range(400):
            items = random_items(rng, rng.randint(1, 12))
            run_cta(6, items, rng, rng.randint(1, run_cta(6, items, rng)), always_drain=False)
