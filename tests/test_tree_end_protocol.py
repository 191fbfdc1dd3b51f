"""A model of the end of a piece in attn_tree_kernel, warp by warp, under random
interleavings (CPU only).

Roles as in ``tiled_attention_25_b200/csrc/tree_sm100.cu``: the walk publishes
pieces in two buffers, the MMA warp completes a piece's O once all warps have
read the last piece's, and the eight softmax warps (two warpgroups) exchange
(m, l), stage O in rounds through two buffers, and, for a piece of a cut item,
count it in and learn from one thread whether theirs was the last.  A yield on
``tick`` is no wait, only a place where another warp may come in between.

Checks: no deadlock, no aliasing of phases, every read finds what its piece and
round wrote, and with any one wait of any role running out every role ends.
"""
import pytest

from protocol_sim import Sim

WARPS = 4  # of a warpgroup


def roles(sim, pieces, rounds):
    """pieces: True where the item is cut; rounds: of staging, per piece."""
    full, empty = sim.full, sim.empty
    tick = empty("tick", 0)
    sim.bar("tick", 1)
    for b in range(2):
        sim.bar(f"list_full{b}", 1)
        sim.bar(f"list_empty{b}", 1 + 2 * WARPS)
        sim.bar(f"staged{b}", WARPS)
    for name, count in (("o_final", 1), ("epi_done", 2 * WARPS), ("ml_ready", 2 * WARPS), ("written", 2 * WARPS), ("counted", 1)):
        sim.bar(name, count)
    walk = list(pieces) + [None]
    published, o, last = {}, {}, {}
    stage = {}  # (warpgroup, buffer, warp): what the warp's part of the buffer holds
    ml = {}     # (warpgroup, warp of either): (m, l), in the first part of the warpgroup's first buffer

    def put_stage(t, buf, w, tag):
        stage[t, buf, w] = tag
        if buf == 0 and w == 0:
            for x in range(2 * WARPS):
                ml[t, x] = None

    def put_ml(t, x, tag):
        ml[t, x] = tag
        stage[t, 0, 0] = None

    def producer():
        for u, cut in enumerate(walk):
            if not (yield empty(f"list_empty{u & 1}", u >> 1)):
                return
            published[u & 1] = u
            sim.arrive(f"list_full{u & 1}")

    def mma():
        for u, cut in enumerate(walk):
            if not (yield full(f"list_full{u & 1}", u >> 1)) or cut is None:
                return
            if not (yield empty("epi_done", u)):
                return
            o["piece"] = u
            sim.commit("o_final")
            sim.arrive(f"list_empty{u & 1}")

    def warp(t, w):
        n_rounds = cuts = 0
        for u, cut in enumerate(walk):
            if not (yield full(f"list_full{u & 1}", u >> 1)) or cut is None:
                return
            assert published[u & 1] == u
            if not (yield full("o_final", u)):
                return
            for region in range(2):
                put_ml(region, t * WARPS + w, u)
                yield tick
            sim.arrive("ml_ready")
            if not (yield full("ml_ready", u)):
                return
            for x in range(2 * WARPS):
                assert ml[t, x] == u, f"piece {u}: (m, l) of {ml[t, x]}"
                if x % 3 == 0:
                    yield tick
            for k in range(rounds):
                buf = (k & 1) ^ 1
                assert o["piece"] == u
                put_stage(t, buf, w, (u, k))
                yield tick
                sim.arrive(f"staged{t}")
                if not (yield full(f"staged{t}", n_rounds)):
                    return
                n_rounds += 1
                for x in range(WARPS):
                    assert stage[t, buf, x] == (u, k), f"piece {u} round {k}: {stage[t, buf, x]}"
                    if x & 1:
                        yield tick
            if cut:
                sim.arrive("written")
                if not (yield full("written", cuts)):
                    return
                if t == 0 and w == 0:
                    last["of"] = cuts
                    sim.arrive("counted")
                if not (yield full("counted", cuts)):
                    return
                yield tick
                assert last["of"] == cuts
                cuts += 1
                yield tick
                assert published[u & 1] == u  # the join reads the piece's record
            sim.arrive("epi_done")
            sim.arrive(f"list_empty{u & 1}")

    return {"walk": producer(), "mma": mma(), **{f"softmax{t}{w}": warp(t, w) for t in range(2) for w in range(WARPS)}}


PIECES = {"whole": [False] * 4, "cut": [True] * 4, "mixed": [True, False, False, True, True, False], "one": [True], "none": []}


@pytest.mark.parametrize("rounds", [2, 4])
@pytest.mark.parametrize("name", sorted(PIECES))
def test_the_end_of_a_piece(name, rounds):
    for seed in range(150):
        sim = Sim(seed)
        stuck = sim.run(roles(sim, PIECES[name], rounds))
        assert stuck is None, f"{name}, seed {seed}: {stuck}"
        assert sim.in_flight_at_exit == 0


@pytest.mark.parametrize("role", ["walk", "mma", "softmax00", "softmax03", "softmax10"])
def test_a_wait_that_runs_out_ends_every_role(role):
    for at in range(60):
        for seed in range(4):
            sim = Sim(seed)
            stuck = sim.run(roles(sim, PIECES["mixed"], 2), give_up=(role, at))
            assert stuck is None, f"{role} wait {at}, seed {seed}: {stuck}"


def test_a_single_buffer_would_be_overwritten():
    """Why there are two: a fast warp would overwrite what a slow one still reads."""
    found = 0
    for seed in range(60):
        sim = Sim(seed)
        try:
            sim.run(one_buffer(sim, 3))
        except AssertionError:
            found += 1
    assert found > 0


def one_buffer(sim, rounds):
    """The staging rounds of one warpgroup with a single buffer."""
    sim.bar("staged", WARPS)
    sim.bar("tick", 1)
    stage = {}

    def warp(w):
        for k in range(rounds):
            stage[w] = k
            sim.arrive("staged")
            if not (yield sim.full("staged", k)):
                return
            for x in range(WARPS):
                assert stage[x] == k
                yield sim.empty("tick", 0)

    return {f"warp{w}": warp(w) for w in range(WARPS)}
