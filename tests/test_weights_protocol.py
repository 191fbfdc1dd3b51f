"""A model of cache_weights_kernel's mbarrier protocol, run under random
interleavings of its warp roles (CPU only).

Roles as in ``tiled_attention_25_b200/csrc/weights_sm100.cu``: the TMA warp
publishes units and loads the first K tile of each and its Q tiles, a second
TMA warp the second K tile; the column warps fill in each Q
slot's LSE and limits (one arrival here); the MMA warp forms the scores of one
or two key tiles per Q tile into two buffers each; a warpgroup to each buffer sums
them, and the two of a tile join their sums.  A Q tile may stay for the next
unit, and a unit may have no queries.

Checks: no deadlock, no aliasing, and with any one wait of any role running
out, every role ends with no copy or product in flight.
"""
import pytest

from protocol_sim import Sim


COLS = 4  # slots of the columns' ring
UNITS_AHEAD = 4  # units published ahead


def roles(sim, units, kbufs, qslots, gathered=False):
    """units: (Q tiles, key tiles, new_q, keep_q)."""
    full, empty, drain = sim.full, sim.empty, sim.drain
    for i in range(UNITS_AHEAD):
        sim.bar(f"unit_full{i}", 1)
        sim.bar(f"unit_empty{i}", 7)
    for i in range(2):
        sim.bar(f"j_full{i}", 2)
        sim.bar(f"j_empty{i}", 1)
        for t in range(2):
            sim.bar(f"s_full{t}{i}", 1)
            sim.bar(f"s_empty{t}{i}", 1)
    for t in range(2):
        for i in range(kbufs[t]):
            sim.bar(f"k_full{t}{i}", 1)
            sim.bar(f"k_empty{t}{i}", 1)
    for i in range(qslots):
        sim.bar(f"q_full{i}", 1)
        sim.bar(f"q_empty{i}", 1)
    for i in range(COLS):
        sim.bar(f"c_full{i}", 1)
        sim.bar(f"c_empty{i}", 4)
    sim.bar("drain", 1)
    walk = list(units) + [None]

    def tma():
        kn = ql = 0

        def body():
            nonlocal kn, ql
            for it, u in enumerate(walk):
                if not (yield empty(f"unit_empty{it % UNITS_AHEAD}", it // UNITS_AHEAD)):
                    return
                sim.arrive(f"unit_full{it % UNITS_AHEAD}")
                if u is None:
                    return
                n, _, new, _ = u
                if n:
                    if not (yield empty(f"k_empty0{kn % kbufs[0]}", kn // kbufs[0])):
                        return
                    sim.load(f"k_full0{kn % kbufs[0]}")
                    kn += 1
                for _ in range(0 if new else 1, 0 if gathered else n):
                    if not (yield empty(f"q_empty{ql % qslots}", ql // qslots)):
                        return
                    sim.load(f"q_full{ql % qslots}")
                    ql += 1
        yield from body()
        for s in range(kbufs[0]):
            if (uses := (kn + kbufs[0] - 1 - s) // kbufs[0]):
                yield drain(f"k_full0{s}", uses - 1)
        for s in range(qslots):
            if (uses := (ql + qslots - 1 - s) // qslots):
                yield drain(f"q_full{s}", uses - 1)

    def tma2():
        kn = 0
        for it, u in enumerate(walk):
            if not (yield full(f"unit_full{it % UNITS_AHEAD}", it // UNITS_AHEAD)):
                break
            sim.arrive(f"unit_empty{it % UNITS_AHEAD}")
            if u is None:
                break
            if u[0] and u[1] > 1:
                if not (yield empty(f"k_empty1{kn % kbufs[1]}", kn // kbufs[1])):
                    break
                sim.load(f"k_full1{kn % kbufs[1]}")
                kn += 1
        for s in range(kbufs[1]):
            if (uses := (kn + kbufs[1] - 1 - s) // kbufs[1]):
                yield drain(f"k_full1{s}", uses - 1)

    def columns():
        ql = 0
        for it, u in enumerate(walk):
            if not (yield full(f"unit_full{it % UNITS_AHEAD}", it // UNITS_AHEAD)):
                return
            sim.arrive(f"unit_empty{it % UNITS_AHEAD}")
            if u is None:
                return
            for _ in range(0 if u[2] else 1, u[0]):
                if not (yield empty(f"c_empty{ql % COLS}", ql // COLS)):
                    return
                if gathered and not (yield empty(f"q_empty{ql % qslots}", ql // qslots)):
                    return
                sim.arrive(f"c_full{ql % COLS}")
                ql += 1

    def mma():
        def body():
            kn, ql, sc = [0, 0], 0, [0, 0]
            for it, u in enumerate(walk):
                if not (yield full(f"unit_full{it % UNITS_AHEAD}", it // UNITS_AHEAD)):
                    return
                sim.arrive(f"unit_empty{it % UNITS_AHEAD}")
                if u is None:
                    return
                n, tiles, new, keep = u
                if n == 0:
                    continue
                for j in range(n):
                    ql += j > 0 or new
                    ring, of = ("c_full", COLS) if gathered else ("q_full", qslots)
                    if not (yield full(f"{ring}{(ql - 1) % of}", (ql - 1) // of)):
                        return
                    for t in range(tiles):
                        k = kn[t]
                        if j == 0 and not (yield full(f"k_full{t}{k % kbufs[t]}", k // kbufs[t])):
                            return
                        if not (yield empty(f"s_empty{t}{sc[t] & 1}", sc[t] >> 1)):
                            return
                        sim.commit(f"s_full{t}{sc[t] & 1}")
                        sc[t] += 1
                        if j == n - 1:
                            sim.commit(f"k_empty{t}{k % kbufs[t]}")
                    if j < n - 1 or not keep:
                        sim.commit(f"q_empty{(ql - 1) % qslots}")
                kn[0] += 1
                kn[1] += tiles > 1
        yield from body()
        sim.commit("drain")
        yield drain("drain", 0)

    def sums(t, sb):
        ql = sc = joins = 0
        for it, u in enumerate(walk):
            if not (yield full(f"unit_full{it % UNITS_AHEAD}", it // UNITS_AHEAD)):
                return
            sim.arrive(f"unit_empty{it % UNITS_AHEAD}")
            if u is None:
                return
            n, tiles, new, keep = u
            owner = (sc + max(n, 1) - 1) % 2 == sb
            for j in range(n):
                ql += j > 0 or new
                if not (yield full(f"c_full{(ql - 1) % COLS}", (ql - 1) // COLS)):
                    return
                if t < tiles:
                    if sc % 2 == sb:
                        if not (yield full(f"s_full{t}{sb}", sc >> 1)):
                            return
                        sim.arrive(f"s_empty{t}{sb}")
                    sc += 1
                if j < n - 1 or not keep:
                    sim.arrive(f"c_empty{(ql - 1) % COLS}")
            if t < tiles and n > 1:
                if joins and not (yield full(f"j_empty{t}", joins - 1)):
                    return
                sim.arrive(f"j_full{t}")
                if owner:
                    if not (yield full(f"j_full{t}", joins)):
                        return
                    sim.arrive(f"j_empty{t}")
                joins += 1

    return {"tma": tma(), "tma2": tma2(), "columns": columns(), "mma": mma(),
            **{f"sums{t}{sb}": sums(t, sb) for t in range(2) for sb in range(2)}}


UNITS = {
    "prompt": [(5, 2, 1, 0), (3, 2, 1, 0), (1, 1, 1, 0)],
    "draft": [(1, 2, 1, 1), (1, 2, 0, 1), (1, 1, 0, 0), (1, 2, 1, 1), (1, 1, 0, 0), (1, 1, 1, 0)],
    "half": [(6, 1, 1, 0), (1, 1, 1, 0), (4, 2, 1, 0)],
    "no queries": [(0, 2, 0, 0), (0, 1, 0, 0), (1, 2, 1, 0), (0, 2, 0, 0)],
    "nothing": [],
}


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("bufs", [((2, 2), 2), ((3, 2), 1), ((3, 2), 2), ((4, 4), 4)])
@pytest.mark.parametrize("name", sorted(UNITS))
def test_weights_protocol_never_deadlocks_or_aliases(name, bufs, gathered):
    for seed in range(120):
        sim = Sim(seed)
        stuck = sim.run(roles(sim, UNITS[name], *bufs, gathered))
        assert stuck is None, f"{name}, seed {seed}: {stuck}"
        assert sim.in_flight_at_exit == 0


@pytest.mark.parametrize("role", ["tma", "tma2", "columns", "mma", "sums00", "sums01", "sums11"])
def test_a_wait_that_runs_out_ends_every_role(role):
    for name in ("prompt", "draft", "half"):
        for at in range(20):
            for seed in range(8):
                sim = Sim(seed)
                stuck = sim.run(roles(sim, UNITS[name], (2, 2), 2), give_up=(role, at))
                assert stuck is None, f"{role} wait {at}, seed {seed}: {stuck}"
                assert sim.in_flight_at_exit == 0, f"{role} wait {at}, seed {seed}: {sim.pending_at_exit}"


def joins_of_a_key_tile(sim, units, ctas, warps=2):
    """The sums' barriers alone, warp by warp: two warpgroups to each CTA of a
    cluster, any speed of each warp.  units: the steps of each CTA."""
    for c in range(ctas):
        sim.bar(f"j_full{c}", 2 * warps)
        sim.bar(f"j_empty{c}", warps)
        sim.bar(f"x_empty{c}", 2 * warps)
    sim.bar("x_full", (ctas - 1) * 2 * warps)
    joined, handed = {}, {}  # what lies in the buffers, and who has read it

    def warp(c, sb, w):
        sc = joins = 0
        for it, steps in enumerate(units):
            n = steps[c]
            owner = (sc + max(n, 1) - 1) % 2 == sb
            sc += n
            if n > 1:
                if joins and not (yield sim.full(f"j_empty{c}", joins - 1)):
                    return
                if not owner:
                    joined[c, w] = it
                sim.arrive(f"j_full{c}")
                if owner:
                    if not (yield sim.full(f"j_full{c}", joins)):
                        return
                    assert joined[c, w] == it
                    sim.arrive(f"j_empty{c}")
                joins += 1
            if ctas > 1 and c > 0:
                if it and not (yield sim.full(f"x_empty{c}", it - 1)):
                    return
                if owner:
                    handed[c, w] = it
                sim.arrive("x_full")
            elif ctas > 1:
                if not (yield sim.full("x_full", it)):
                    return
                if owner:
                    assert all(handed[x, w] == it for x in range(1, ctas))
                for x in range(1, ctas):
                    sim.arrive(f"x_empty{x}")

    return {f"cta{c} sums{sb} warp{w}": warp(c, sb, w) for c in range(ctas) for sb in range(2) for w in range(warps)}


@pytest.mark.parametrize("ctas", [1, 2, 4])
@pytest.mark.parametrize("most", [1, 2, 3, 5])
def test_sums_meet_once_a_unit(ctas, most):
    """Units of many and of few steps, and of none for some CTAs: no warp takes
    one phase of the sums' barriers for another, or reads another unit's sum."""
    for seed in range(250):
        sim = Sim(seed)
        units = [[sim.rng.randint(0 if c else 1, most) for c in range(ctas)] for _ in range(6)]
        stuck = sim.run(joins_of_a_key_tile(sim, units, ctas))
        assert stuck is None, f"seed {seed}, {units}: {stuck}"
