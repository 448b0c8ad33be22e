"""Randomized models of the hand-off protocols of the paged attention kernels, checked on the CPU.

`chunks`: csrc/swska_extend_tc.cu. Three producer warps load K (with Q), V0 and V1 of every key tile into one four-slot
ring; the MMA warp issues S_h and P V_h; two softmax warpgroups read which pages exist (`have`, four entries, handed over by
the `known` barriers), clear value rows on some tiles after waiting for their slot, hand over P in two halves, and end each
unit with its output rows. Units may be empty (no tile) and every role skips them alike.

`few`: csrc/swska_extend_few.cu. Two producer warps load the halves of a stage, one warp per head uses it and frees it.

Every read is checked against the data that it must see, and no buffer may be overwritten before its readers are done.
Planted mistakes must be caught."""
import random

import pytest

from .barrier_model import Bar, simulate

NSLOT = 4


def chunks(units, seed, mistake=None):
    """units: (key tiles, whether the unit clears value rows) in a CTA's order."""
    full = [Bar(1) for _ in range(NSLOT)]
    empty = [Bar(1) for _ in range(NSLOT)]
    known = [Bar(1) for _ in range(4)]
    qfull, qempty = Bar(1), Bar(1)
    sfull, phalf, pfull, odone = ([Bar(n), Bar(n)] for n in (1, 128, 128, 1))
    slot, slot_reads = [None] * NSLOT, [0] * NSLOT
    have = [None] * 4
    st = {"q": None, "q_reads": 0}
    S, S_reading, P, O = [None, None], [False, False], [[None, None], [None, None]], [None, None]
    rows_done = [set(), set()]
    pipe, copies = [], []
    rnd = random.Random(seed)

    def producer(which):
        nq = tiles = 0
        for un, (n_it, _) in enumerate(units):
            if n_it == 0:
                continue
            if which == 0:
                if nq > 0:
                    yield ("wait", qempty, (nq - 1) & 1)
                qfull.expect_tx(2)
                copies.append(("q", None, un, qfull, 2))
                nq += 1
            for j in range(n_it):
                L = 3 * tiles + which
                s, use = L % NSLOT, L // NSLOT
                if use > 0 and mistake != "slot_without_empty":
                    yield ("wait", empty[s], (use - 1) & 1)
                if which == 0:
                    k = tiles & 3
                    if mistake == "one_entry":
                        k = 0
                    have[k] = (un, j)
                    known[tiles & 3].arrive()
                full[s].expect_tx(1)
                copies.append(("slot", s, ("K", un, j) if which == 0 else ("V", which - 1, un, j), full[s], 1))
                tiles += 1
                yield ("step",)
        # the waits before the CTA leaves end, and the copies they are for have landed
        if nq:
            yield ("wait", qfull, (nq - 1) & 1)
        for t in range(max(0, tiles - 2), tiles):
            L = 3 * t + which
            if L + NSLOT >= 3 * tiles:
                yield ("wait", full[L % NSLOT], (L // NSLOT) & 1)

    def issuer():
        Lb = tb = done = 0
        for un, (n_it, _) in enumerate(units):
            if n_it == 0:
                continue
            yield ("wait", qfull, done & 1)
            yield ("wait", full[Lb % NSLOT], (Lb // NSLOT) & 1)
            pipe.extend([("S", 0, un, 0, Lb % NSLOT), ("C", sfull[0]), ("S", 1, un, 0, Lb % NSLOT), ("C", sfull[1]),
                         ("C", empty[Lb % NSLOT])])
            if n_it == 1:
                pipe.append(("C", qempty))
            for j in range(n_it):
                more, Lj, tj = j + 1 < n_it, Lb + 3 * j, tb + j
                for h in (0, 1):
                    Lv = Lj + 1 + h
                    yield ("wait", full[Lv % NSLOT], (Lv // NSLOT) & 1)
                    yield ("wait", phalf[h], tj & 1)
                    pipe.append(("PV", h, un, j, 0, Lv % NSLOT))
                    yield ("wait", pfull[h], tj & 1)
                    pipe.extend([("PV", h, un, j, 1, Lv % NSLOT), ("C", empty[Lv % NSLOT])])
                    if not more:
                        pipe.append(("C", odone[h]))
                        continue
                    Lk = Lj + 3
                    if h == 0:
                        yield ("wait", full[Lk % NSLOT], (Lk // NSLOT) & 1)
                    pipe.extend([("S", h, un, j + 1, Lk % NSLOT), ("C", sfull[h])])
                    if h == 1:
                        pipe.append(("C", empty[Lk % NSLOT]))
                        if j + 2 == n_it:
                            pipe.append(("C", qempty))
            Lb += 3 * n_it
            tb += n_it
            done += 1

    def softmax(h):
        Lb = tb = done = 0
        for un, (n_it, clears) in enumerate(units):
            for j in range(n_it):
                yield ("wait", sfull[h], (tb + j) & 1)
                assert S[h] == (un, j), f"softmax {h} read S {S[h]}, expected {(un, j)}"
                yield ("wait", known[(tb + j) & 3], ((tb + j) >> 2) & 1)
                k = 0 if mistake == "one_entry" else (tb + j) & 3
                assert have[k] == (un, j), f"softmax {h} read the pages of {have[k]}, expected {(un, j)}"
                S_reading[h] = True
                yield ("step",)
                S_reading[h] = False
                if clears and j in (0, n_it - 1):
                    Lv = Lb + 3 * j + 1 + h
                    if mistake != "clear_without_wait":
                        yield ("wait", full[Lv % NSLOT], (Lv // NSLOT) & 1)
                    assert slot[Lv % NSLOT] == ("V", h, un, j), f"rows of {slot[Lv % NSLOT]} cleared for {(h, un, j)}"
                    assert slot_reads[Lv % NSLOT] == 0, "rows cleared after their product"
                P[h][0] = (un, j)
                phalf[h].arrive(128)
                yield ("step",)
                P[h][1] = (un, j)
                pfull[h].arrive(128)
            if n_it:
                yield ("wait", odone[h], done & 1)
                assert O[h] == (un, 2 * n_it), f"rows of unit {un}, head {h} saw O {O[h]}"
                yield ("step",)
                Lb += 3 * n_it
                tb += n_it
                done += 1
            rows_done[h].add(un)

    def execute(op):
        if op[0] == "C":
            op[1].arrive()
        elif op[0] == "S":
            _, h, un, j, s = op
            assert st["q"] == un and slot[s] == ("K", un, j), f"S{h}{(un, j)} read Q {st['q']}, {slot[s]}"
            assert not S_reading[h], "S overwritten while the softmax reads it"
            S[h], P[h] = (un, j), [None, None]
            slot_reads[s] += 1
            st["q_reads"] += 1
        else:
            _, h, un, j, half, s = op
            assert P[h][half] == (un, j) and slot[s] == ("V", h, un, j), f"PV{h}{(un, j)} read P {P[h][half]}, {slot[s]}"
            if j == 0 and half == 0:
                earlier = [x for x in range(un) if units[x][0]]
                assert not earlier or earlier[-1] in rows_done[h], "O reset before the last unit's rows were read"
                O[h] = (un, 1)
            else:
                assert O[h] == (un, 2 * j + half), f"PV{h}{(un, j, half)} accumulates onto {O[h]}"
                O[h] = (un, 2 * j + half + 1)
            slot_reads[s] += 1

    def land(copy):
        kind, s, what, bar, nbytes = copy
        if kind == "q":
            before = [units[x][0] for x in range(what) if units[x][0]]
            assert st["q_reads"] == (2 * before[-1] if before else 0), "Q overwritten before its score products ran"
            st["q"], st["q_reads"] = what, 0
        else:
            assert slot[s] is None or slot_reads[s] == 2, f"slot {s} overwritten: {slot[s]}"
            slot[s], slot_reads[s] = what, 0
        bar.complete_tx(nbytes)

    actors = {"K": producer(0), "V0": producer(1), "V1": producer(2), "issuer": issuer(), "softmax0": softmax(0), "softmax1": softmax(1)}
    simulate(seed, actors, [pipe], copies, execute, land)
    assert rnd and all(len(rows_done[h]) == len(units) for h in (0, 1)) and not copies


def _units(seed, at_least=1):
    rnd = random.Random(seed)
    return [(rnd.choice([0, 1, 1, 2, 3, 5, 12]), rnd.random() < 0.6) for _ in range(rnd.randint(at_least, 6))]


def test_chunks_protocol_over_random_units():
    for seed in range(300):
        chunks(_units(seed), seed)


@pytest.mark.parametrize("mistake,least", [("slot_without_empty", 150), ("one_entry", 30), ("clear_without_wait", 5)])
def test_chunks_model_catches_planted_mistakes(mistake, least):
    """The last one shows only where a value tile lands after its head's scores are read."""
    caught = 0
    for seed in range(300):
        try:
            chunks([(5, True)] + _units(seed, 2), seed, mistake)
        except AssertionError:
            caught += 1
    assert caught >= least, f"{mistake}: caught in {caught} of 300 runs"


def few(tiles, heads, stages, seed, mistake=None):
    full = [Bar(2) for _ in range(stages)]
    empty = [Bar(heads) for _ in range(stages)]
    held = [[None, None] for _ in range(stages)]  # tile whose half is there
    reads = [0] * stages
    mask = [None] * stages
    copies, used = [], [0] * heads

    def producer(half):
        for t in range(tiles):
            s, use = t % stages, t // stages
            if use > 0 and not (mistake == "one_half_waits" and half == 1):
                yield ("wait", empty[s], (use - 1) & 1)
            if half == 0:
                mask[s] = t
            full[s].expect_tx(1)
            copies.append((s, half, t))
            yield ("step",)
        for t in range(max(0, tiles - stages), tiles):
            yield ("wait", full[t % stages], (t // stages) & 1)

    def head(h):
        for t in range(tiles):
            s = t % stages
            yield ("wait", full[s], (t // stages) & 1)
            assert held[s] == [t, t] and mask[s] == t, f"head {h} read {held[s]}, {mask[s]}, expected {t}"
            yield ("step",)
            assert held[s] == [t, t], "stage overwritten while it is read"
            reads[s] += 1
            used[h] += 1
            empty[s].arrive()

    def land(copy):
        s, half, t = copy
        assert held[s][half] is None or mistake or reads[s] >= heads * (t // stages), f"stage {s} overwritten early"
        held[s][half] = t
        full[s].complete_tx(1)

    simulate(seed, {**{f"p{i}": producer(i) for i in (0, 1)}, **{f"h{i}": head(i) for i in range(heads)}}, [], copies, None, land)
    assert used == [tiles] * heads


def test_few_protocol():
    for seed in range(200):
        rnd = random.Random(seed)
        few(rnd.randint(0, 20), rnd.randint(1, 8), rnd.randint(2, 5), seed)


def test_few_model_catches_a_producer_that_does_not_wait():
    caught = 0
    for seed in range(60):
        try:
            few(20, 3, 3, seed, "one_half_waits")
        except AssertionError:
            caught += 1
    assert caught >= 30
