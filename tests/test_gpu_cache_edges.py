"""KV-cache operators at the ends of their ranges, against their definitions."""
import numpy as np
import pytest
import torch

import oracle
from cache_common import CacheCase, check_tree, i32

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def ta():
    import tiled_attention_25_b200 as m
    return m


@pytest.mark.parametrize("cap,page,lens", [
    (796672, 128, [3000, 999, 40000]), (800000, 128, [3000, 1001]), (850048, 128, [5000]), (900096, 128, [3000, 2000]),
    (1 << 20, 1 << 14, [3000, 1000, 1 << 20]),
])
def test_plan_of_long_tables_and_many_heads(ta, cap, page, lens):
    """More heads than half the SMs over tables of up to the longest capacity,
    short and full rows: a plan follows the filled slots, not the table."""
    B, budget, first, recent = 80, 1000, 3, 100
    rng = np.random.default_rng(cap)
    rows = np.full(B, 7)
    rows[rng.permutation(B)[: len(lens)]] = lens
    w, pos = torch.zeros(B, 1, cap, device="cuda"), torch.zeros(B, 1, cap, dtype=torch.int32, device="cuda")
    moves = torch.full((B, 1, budget, 2), 9, dtype=torch.int32, device="cuda")
    count = torch.full((B, 1), 9, dtype=torch.int32, device="cuda")
    host = {}
    for b, n in enumerate(rows):
        x = rng.exponential(size=n).astype(np.float32)
        x[rng.random(n) < 0.3] = 0.5
        host[b] = x, rng.permutation(n)
        w[b, 0, :n], pos[b, 0, :n] = torch.from_numpy(x).cuda(), i32(host[b][1])
    seen = rows + 3
    pool = torch.zeros(1, 1, page, 64, dtype=torch.bfloat16, device="cuda")  # a plan reads no K or V
    cache = ta.AttnCache(pool, pool, i32(rows), torch.zeros(B, cap // page, dtype=torch.int32, device="cuda"))
    ta.attn_evict_plan(cache, w, pos, i32(seen), moves, count, budget, first, recent)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    for b, n in enumerate(rows):
        want, wn = oracle.cache.evict_plan(host[b][0][None, None], host[b][1][None, None], seen[b:b + 1], rows[b:b + 1], budget,
                                           first, recent)
        assert int(count[b, 0]) == wn[0, 0], (b, n)
        assert np.array_equal(moves[b].cpu().numpy(), want[0]), (b, n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,Hq", [(1, 4), (9, 8), (40, 4)])
def test_scores_that_are_not_finite(ta, D, T, Hq):
    """A visible key whose score is NaN or +inf leaves a row without a softmax:
    O and LSE are NaN.  A score of -inf is a weight of zero."""
    lens = [300, 128, 20000, 5]  # whole items, and one cut into pieces
    c = CacheCase(T + D, lens, Hq, 2, D, 128, T)
    ws = ta.new_tree_workspace(Hq, 2, T, D)

    def call():
        out, lse = torch.empty_like(c.q_t), torch.empty(4, Hq, T, device="cuda")
        ta.attn_tree_fwd(c.q_t, c.k_new_t, c.v_new_t, c.cache, out, lse, ws, scale=c.scale)
        torch.cuda.synchronize()
        return out, lse

    place = lambda b, slot: (int(c.table[b, slot // 128]), 0, slot % 128)  # head 0
    good_out, good_lse = call()
    for b, slot in ((0, 17), (2, 11111), (3, 4)):
        c.k_t[place(b, slot)] = NAN
    out, lse = call()
    hit = torch.zeros(4, Hq, T, dtype=torch.bool, device="cuda")
    hit[[0, 2, 3], : Hq // 2] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    assert torch.equal(lse[~hit], good_lse[~hit]) and torch.equal(out[~hit], good_out[~hit])
    for b, slot in ((0, 17), (2, 11111), (3, 4)):
        c.k_t[place(b, slot)] = 0.0
        c.k[place(b, slot)] = 0.0
        c.k_t[place(b, slot)][3] = float("inf")
        c.k[place(b, slot)][3] = np.inf
    out, lse = call()
    hit &= c.q_t[..., 3] > 0
    assert hit.any() and not hit[:, : Hq // 2].all()
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    want = oracle.cache.tree_attention(c.q, c.k_new, c.v_new, c.k, c.v, c.table, c.lens, None, None, c.scale)
    for x in want:
        x[hit.cpu().numpy()] = np.nan  # no definition
    check_tree(out, lse, want)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("bad", [-1, 1 << 30])
@pytest.mark.parametrize("storage", ["head", "row"])
def test_moves_from_and_into_a_page_outside_the_pool(ta, bad, storage):
    """Such a move is left out whole: weight and position stay with the row's
    K and V."""
    c = CacheCase(5, [256, 200], 2, 2, 64, 64, storage=storage)
    c.table[0, 3] = c.table[1, 0] = bad
    c.load()
    w = c.rng.exponential(size=(2, 2, c.cap)).astype(np.float32)
    pos = np.tile(np.arange(c.cap), (2, 2, 1))
    moves = np.array([[[5, 200], [6, 130], [70, 191]], [[5, 130], [66, 150], [7, 199]]], dtype=np.int32)
    moves = np.repeat(moves[:, None], 2, axis=1)  # row 0 reads the bad page once, row 1 writes it twice
    w_t, pos_t = torch.from_numpy(w).cuda(), i32(pos)
    ta.attn_cache_compact(c.cache, i32(moves), i32(np.full((2, 2), 3)), 3, weights=w_t, positions=pos_t)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
    done = np.full((2, 2, 3, 2), -1)
    done[0, :, :2], done[1, :, :1] = moves[0, :, 1:], moves[1, :, 1:2]
    new = oracle.cache.compact(done, np.array([[2, 2], [1, 1]]), 3, c.k, c.v, c.table, c.lens, w, pos)
    assert np.array_equal(c.k_t.float().cpu().double().numpy(), c.k, equal_nan=True)
    assert np.array_equal(c.v_t.float().cpu().double().numpy(), c.v, equal_nan=True)
    assert np.array_equal(w_t.cpu().numpy(), w) and np.array_equal(pos_t.cpu().numpy(), pos)
    assert np.array_equal(c.lens_t.cpu().numpy(), new)


@pytest.mark.parametrize("which", ["seen", "counts", "lens"])
def test_new_lengths_in_the_place_of_an_argument(ta, which):
    """lens_out may be an array that the call reads: every block has read it by then."""
    B, T = 6, 900
    counts = np.array([T, 0, 13, 500, 1, T])
    c = CacheCase(6, [0, 30, 129, 7, 64, 1], 2, 2, 64, 64, T, room=T)
    seen = c.lens + 1000
    args = {"seen": i32(seen), "counts": i32(counts), "lens": c.lens_t}
    pos = np.full((B, 2, c.cap), -1)
    pos_t = i32(pos)
    ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t, args[which], counts=args["counts"], positions=pos_t, seen=args["seen"])
    want = oracle.cache.append(c.k_new, c.v_new, c.k, c.v, c.table, c.lens, None, counts, pos, seen)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    assert np.array_equal(c.k_t.float().cpu().double().numpy(), c.k, equal_nan=True)
    assert np.array_equal(pos_t.cpu().numpy(), pos)
    for name, before in (("seen", seen), ("counts", counts), ("lens", c.lens)):
        assert np.array_equal(args[name].cpu().numpy(), want if name == which else before), name
