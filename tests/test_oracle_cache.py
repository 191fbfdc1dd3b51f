"""Pins of the cache oracle: closed forms and identities (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import cache as oc


def make(rng, lens, Hkv, D, page):
    n = -(-max(lens) // page)
    P = len(lens) * n + 1
    table = rng.permutation(P)[: len(lens) * n].reshape(len(lens), n)
    return rng.standard_normal((P, Hkv, page, D)), rng.standard_normal((P, Hkv, page, D)), table


def test_ancestors():
    keep = oc.ancestors([-1, 0, 0, 2, 9, -7, 3], 7)
    assert [np.flatnonzero(r).tolist() for r in keep] == [[0], [0, 1], [0, 2], [0, 2, 3], [4], [5], [0, 2, 3, 6]]
    assert np.array_equal(oc.ancestors(None, 5), np.tri(5, dtype=bool))


@pytest.mark.parametrize("softcap", [None, 3.0])
def test_a_chain_is_causal_attention(softcap):
    rng = np.random.default_rng(1)
    n, T, Hq, Hkv, D = 21, 6, 4, 2, 8
    k, v, table = make(rng, [n], Hkv, D, 16)
    q, kn, vn = rng.standard_normal((1, Hq, T, D)), rng.standard_normal((1, Hkv, T, D)), rng.standard_normal((1, Hkv, T, D))
    O, L, A = oc.tree_attention(q, kn, vn, k, v, table, [n], None, None, 0.3, softcap)
    full = [np.stack([np.concatenate([oc.slots(p, table[0], n, h), x[0, h]]) for h in range(Hkv)])[None]
            for p, x in ((k, kn), (v, vn))]
    qq = np.concatenate([np.zeros((1, Hq, n, D)), q], 2)
    if softcap is None:
        O2, L2 = oracle.attention_forward(qq, *full, 0.3, oracle.MOD_CAUSAL)
        assert np.allclose(O, O2[:, :, n:]) and np.allclose(L, L2[:, :, n:])
    assert (np.abs(O) <= A + 1e-12).all()
    # appended, the chain is the cache
    lens = oc.append(kn, vn, k, v, table, [n], None, None)
    assert lens[0] == n + T
    O3, L3, _ = oc.tree_attention(q[:, :, -1:], None, None, k, v, table, lens, None, None, 0.3, softcap)
    assert np.allclose(O3[:, :, 0], O[:, :, -1]) and np.allclose(L3[:, :, 0], L[:, :, -1])
    # and each query's weights sum to one over what it saw
    w, add = oc.slot_weights(q, L, k, table, lens, None, None, None, 0.3, softcap)
    assert np.allclose(w[0, :, : n + T].sum(-1), T * Hq / Hkv) and np.allclose(w[0, :, :n], add[0, :, :n])
    one, _ = oc.slot_weights(q[:, :1], L[:, :1], k[:, :1], table, lens, None, [[T - 1]], [1], 0.3, softcap)
    assert np.allclose(one[0, 0, : n + T].sum(), 1.0)


def test_a_path_of_the_tree_is_its_chain():
    rng = np.random.default_rng(2)
    n, T, D = 10, 5, 4
    k, v, table = make(rng, [n], 1, D, 16)
    q, kn, vn = (rng.standard_normal((1, 1, T, D)) for _ in range(3))
    parents = [[-1, 0, 0, 2, 1]]
    O, L, _ = oc.tree_attention(q, kn, vn, k, v, table, [n], parents, None, 0.5)
    path = [0, 2, 3]
    O2, L2, _ = oc.tree_attention(q[:, :, path], kn[:, :, path], vn[:, :, path], k, v, table, [n], None, None, 0.5)
    assert np.allclose(O[:, :, path], O2) and np.allclose(L[:, :, path], L2)


def test_equal_weights_and_empty_rows():
    k = v = np.ones((1, 1, 16, 4))
    O, L, _ = oc.tree_attention(np.zeros((2, 1, 1, 4)), None, None, k, v, [[0], [0]], [8, 0], None, None, 1.0)
    assert np.allclose(O[0], 1) and np.isclose(L[0, 0, 0], np.log(8)) and (O[1] == 0).all() and np.isneginf(L[1]).all()


def test_plan_and_compact():
    w = np.array([[[5.0, 1.0, 3.0, 1.0, 0.0, 2.0, 9.0, 1.0]]])
    pos = np.arange(8)[None, None]
    moves, n = oc.evict_plan(w, pos, [8], [8], 4, 0, 0)
    assert n[0, 0] == 2 and moves[0, 0, :2].tolist() == [[1, 5], [3, 6]] and (moves[0, 0, 2:] == -1).all()
    moves, n = oc.evict_plan(w, pos, [8], [8], 4, 1, 1)  # 0 and 7 protected, then 9, 3
    assert moves[0, 0, : n[0, 0]].tolist() == [[1, 6], [3, 7]]
    moves, n = oc.evict_plan(np.ones_like(w), pos, [8], [8], 4, 0, 0)  # ties to the lower slot: nothing moves
    assert n[0, 0] == 0
    w[0, 0, 6] = np.nan
    moves, n = oc.evict_plan(w, pos, [8], [8], 7, 0, 0)
    assert moves[0, 0, : n[0, 0]].tolist() == [[6, 7]]
    k = np.arange(8.0)[None, None, :, None].repeat(16, 2)[:, :, :16].copy()
    k = np.arange(16.0)[None, None, :, None].copy()
    v = -k
    lens = oc.compact(np.array([[[[1, 5], [3, 6]]]]), np.array([[2]]), 4, k, v, [[0]], np.array([8]))
    assert lens[0] == 4 and k[0, 0, :5, 0].tolist() == [0, 5, 2, 6, 4] and v[0, 0, 1, 0] == -5
    assert sorted(k[0, 0, :4, 0]) == [0, 2, 5, 6]


def test_append_writes_the_path():
    rng = np.random.default_rng(3)
    k, v, table = make(rng, [20], 2, 4, 16)
    kn, vn = rng.standard_normal((1, 2, 5, 4)), rng.standard_normal((1, 2, 5, 4))
    pos = np.full((1, 2, 32), -1)
    lens = oc.append(kn, vn, k, v, table, [14], [[0, 3, 4, 9, 9]], [3], pos, [100])
    assert lens[0] == 17 and pos[0, 1, 13:18].tolist() == [-1, 100, 101, 102, -1]
    assert np.array_equal(oc.slots(k, table[0], 17, 1)[14:], kn[0, 1, [0, 3, 4]])
