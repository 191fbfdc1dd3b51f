"""A model of attn_tree_kernel's mbarrier protocol, run under random
interleavings of its warp roles (CPU only).

Roles as in ``tiled_attention_25_b200/csrc/tree_sm100.cu``, with its barrier
counts and phases (a group of warps that arrive together is one arrival):

* one TMA warp publishes pieces (a number of 128-key steps) and streams K
  through its ring, a second streams V, a third loads each piece's Q;
* the MMA warp issues S(j) and O(j) alternately for the two softmax
  warpgroups, which take the even and the odd steps;
* on a step with missing keys a softmax warpgroup first waits for that step's
  V itself (it zeroes rows of it); at the end of a piece the two exchange
  their running values and join O, which the next piece's first O waits for.

Checks: no deadlock, no aliasing, and with any one wait of any role running
out, every role ends with no copy or product in flight.
"""
import pytest

from protocol_sim import Sim


def roles(sim, pieces, partial, stages):
    """pieces: steps of each; stages: of the K and the V ring; partial: the (piece, step) whose V is zeroed in part."""
    full, empty, drain = sim.full, sim.empty, sim.drain
    for b in range(2):
        sim.bar(f"list_full{b}", 1)
        sim.bar(f"list_empty{b}", 5)
        sim.bar(f"s_full{b}", 1)
        sim.bar(f"p_full{b}", 1)
        sim.bar(f"o_full{b}", 1)
    for name, count in (("q_full", 1), ("q_empty", 1), ("o_final", 1), ("epi_done", 2), ("ml_ready", 2), ("drain", 1)):
        sim.bar(name, count)
    stages = dict(zip("kv", stages))
    for kv in "kv":
        for s in range(stages[kv]):
            sim.bar(f"{kv}_full{s}", 1)
            sim.bar(f"{kv}_empty{s}", 1)
    walk = list(pieces) + [None]

    def copies(kv, n, done):
        for _ in range(n):
            if not (yield empty(f"{kv}_empty{done[0] % stages[kv]}", done[0] // stages[kv])):
                return False
            sim.load(f"{kv}_full{done[0] % stages[kv]}")
            done[0] += 1
        return True

    def drain_ring(kv, done):
        for s in range(stages[kv]):
            if (uses := (done[0] + stages[kv] - 1 - s) // stages[kv]):
                yield drain(f"{kv}_full{s}", uses - 1)

    def tma():
        done = [0]

        def body():
            for u, n in enumerate(walk):
                if not (yield empty(f"list_empty{u & 1}", u >> 1)):
                    return
                sim.arrive(f"list_full{u & 1}")
                if n is None or not (yield from copies("k", n, done)):
                    return
        yield from body()
        yield from drain_ring("k", done)

    def tma_q():
        loads = 0
        for u, n in enumerate(walk):
            if not (yield full(f"list_full{u & 1}", u >> 1)):
                break
            sim.arrive(f"list_empty{u & 1}")
            if n is None or not (yield empty("q_empty", u)):
                break
            sim.load("q_full")
            loads += 1
        if loads:
            yield drain("q_full", loads - 1)

    def tma_v():
        done = [0]
        for u, n in enumerate(walk):
            if not (yield full(f"list_full{u & 1}", u >> 1)):
                break
            sim.arrive(f"list_empty{u & 1}")
            if n is None or not (yield from copies("v", n, done)):
                break
        yield from drain_ring("v", done)

    def mma():
        kn, vn, p_cnt = 0, 0, [0, 0]

        def body():
            nonlocal kn, vn
            for u, n in enumerate(walk):
                if not (yield full(f"list_full{u & 1}", u >> 1)) or n is None:
                    return
                if not (yield full("q_full", u)):
                    return
                for i in range(n + 2):
                    t = i & 1
                    if i >= 2 and i - 2 < n:
                        if i == 2 and not (yield empty("epi_done", u)):
                            return
                        if not (yield full(f"v_full{vn % stages['v']}", vn // stages["v"])):
                            return
                        if not (yield full(f"p_full{t}", p_cnt[t])):
                            return
                        p_cnt[t] += 1
                        sim.commit(f"o_full{t}")
                        sim.commit(f"v_empty{vn % stages['v']}")
                        vn += 1
                    if i < n:
                        if not (yield full(f"k_full{kn % stages['k']}", kn // stages["k"])):
                            return
                        sim.commit(f"s_full{t}")
                        sim.commit(f"k_empty{kn % stages['k']}")
                        if i == n - 1:
                            sim.commit("q_empty")
                        kn += 1
                sim.commit("o_final")
                sim.arrive(f"list_empty{u & 1}")
        yield from body()
        sim.commit("drain")
        yield drain("drain", 0)

    def softmax(t):
        s_cnt = base = 0
        for u, n in enumerate(walk):
            if not (yield full(f"list_full{u & 1}", u >> 1)) or n is None:
                return
            for j in range(t, n, 2):
                if not (yield full(f"s_full{t}", s_cnt)):
                    return
                s_cnt += 1
                if j > 1 and sim.rng.random() < 0.3:  # the maximum moved: O is rescaled
                    if not (yield full(f"o_full{t}", s_cnt - 2)):
                        return
                if (u, j) in partial:
                    if not (yield full(f"v_full{(base + j) % stages['v']}", (base + j) // stages["v"])):
                        return
                sim.arrive(f"p_full{t}")
            base += n
            if not (yield full("o_final", u)):
                return
            sim.arrive("ml_ready")
            if not (yield full("ml_ready", u)):
                return
            sim.arrive("epi_done")
            sim.arrive(f"list_empty{u & 1}")

    return {"tma": tma(), "tma_v": tma_v(), "tma_q": tma_q(), "mma": mma(), "softmax0": softmax(0), "softmax1": softmax(1)}


PIECES = {"one": [1], "two": [2], "long": [17], "short": [1, 1, 1, 1, 1], "mixed": [3, 1, 2, 8, 1, 5], "none": []}


@pytest.mark.parametrize("stages", [(3, 2), (6, 5)])
@pytest.mark.parametrize("name", sorted(PIECES))
def test_tree_protocol_never_deadlocks_or_aliases(name, stages):
    pieces = PIECES[name]
    for seed in range(150):
        sim = Sim(seed)
        partial = {(u, n - 1) for u, n in enumerate(pieces)} | {(u, n - 2) for u, n in enumerate(pieces) if seed & 1}
        stuck = sim.run(roles(sim, pieces, partial, stages))
        assert stuck is None, f"{name}, seed {seed}: {stuck}"
        assert sim.in_flight_at_exit == 0


@pytest.mark.parametrize("role", ["tma", "tma_v", "tma_q", "mma", "softmax0", "softmax1"])
def test_a_wait_that_runs_out_ends_every_role(role):
    for at in range(25):
        for seed in range(12):
            sim = Sim(seed)
            stuck = sim.run(roles(sim, PIECES["mixed"], {(0, 2), (3, 7)}, (3, 2)), give_up=(role, at))
            assert stuck is None, f"{role} wait {at}, seed {seed}: {stuck}"
            assert sim.in_flight_at_exit == 0, f"{role} wait {at}, seed {seed}: {sim.pending_at_exit}"

