"""KV-cache operators at the ends of their ranges, against their definitions."""
import numpy as np
import pytest
import torch

import oracle
from cache_common import CacheCase, check_tree, i32, random_tree, tree_reference
from test_gpu_cache_ops import check_weights, weights_case

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


# ------------------------------------------------------------------ every form of the kernels


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,T", [(6, 3), (10, 10), (40, 4), (4, 130)])
@pytest.mark.parametrize("softcap", [None, 2.0])
def test_tree_of_any_number_of_query_rows(ta, D, Hq, T, softcap):
    """9, 50 and 80 rows to a tile, and several tiles, with and without softcap:
    whole items, and some cut into pieces."""
    lens = [300, 5000, 0, 129]
    c = CacheCase(Hq + T, lens, Hq, 2, D, 64, T, counts=[T, T, (T + 1) // 2, 1])
    parents = random_tree(c.rng, 4, T)
    kw = dict(mod_kind=ta.MOD_SOFTCAP, mod_params=ta.ModParams(softcap=softcap)) if softcap else {}
    out, lse = torch.zeros_like(c.q_t), torch.zeros(4, Hq, T, device="cuda")
    ta.attn_tree_fwd(c.q_t, c.k_new_t, c.v_new_t, c.cache, out, lse, ta.new_tree_workspace(Hq, 2, T, D), parents=i32(parents),
                     counts=i32(c.counts), scale=c.scale, **kw)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    check_tree(out, lse, tree_reference(c, parents, softcap=softcap), f"{Hq} heads, {T} tokens")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,counts,T,Hq,Hkv,path", [
    ([700, 300, 17], [9, 1, 4], 9, 6, 2, True),       # one Q tile of 27 rows, two slots to hold it
    ([600, 129], [11, 12], 12, 16, 2, True),          # one Q tile of 96 rows
    ([900, 257, 640], [70, 3, 41], 70, 8, 2, True),   # gathered tiles that stream
    ([700, 257], None, 257, 4, 2, False),             # tiles that stream, shared by clusters
    ([1500], None, 1100, 8, 1, False),
])
def test_weights_with_softcap(ta, D, lens, counts, T, Hq, Hkv, path):
    c, p, lse, w = weights_case(T + D, lens, counts, T, Hq, Hkv, D, 64, path, softcap=2.0)
    check_weights(ta, c, p, lse, w, softcap=2.0)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_weights_of_one_token_and_many_long_rows(ta, D):
    """A plain decode loop's call, without a path."""
    lens = [4000 + 37 * b for b in range(24)]
    c, p, lse, w = weights_case(D, lens, None, 1, 8, 2, D, 128, False)
    check_weights(ta, c, p, lse, w, inplace=True)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("path", [False, True])
def test_weights_of_many_rows_and_query_tiles(ta, path):
    """More rows than a warp looks at together, more than one Q tile to a row."""
    rng = np.random.default_rng(3)
    lens = rng.integers(40, 900, 70)
    counts = rng.integers(0, 41, 70)
    c, p, lse, w = weights_case(3, lens, counts, 40, 8, 2, 64, 64, path)
    check_weights(ta, c, p, lse, w)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,n", [(300, 2000), (130, 0)])
def test_chunks_of_a_prompt(ta, D, T, n):
    """A chunk over a filled cache: attention as a chain, its rows appended, its
    weights; each of its queries spreads a weight of one."""
    Hq, Hkv, page = 8, 2, 128
    c = CacheCase(T, [n, n // 3], Hq, Hkv, D, page, T, room=T)
    out, lse = torch.zeros_like(c.q_t), torch.zeros(2, Hq, T, device="cuda")
    ta.attn_tree_fwd(c.q_t, c.k_new_t, c.v_new_t, c.cache, out, lse, ta.new_tree_workspace(Hq, Hkv, T, D), scale=c.scale)
    ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t)
    w = torch.rand(2, Hkv, c.cap, device="cuda")
    base = w.clone()
    ta.attn_cache_weights(c.q_t, lse, c.cache, w, w, scale=c.scale)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    check_tree(out, lse, tree_reference(c, None))
    lens = oracle.cache.append(c.k_new, c.v_new, c.k, c.v, c.table, c.lens, None, None)
    want, add = oracle.cache.slot_weights(c.q, lse.cpu().double().numpy(), c.k, c.table, lens, base.double().cpu().numpy(), None,
                                          None, c.scale)
    got, live = w.cpu().double().numpy(), ~np.isnan(want)
    # each exponential to 1e-4 relative (scores up to ~8 in fp32), the sum and the base rounded in fp32
    assert (np.abs(got - want) <= 1e-4 * add + 1e-6 * np.abs(want))[live].all()
    for b in range(2):
        old = int(c.lens[b])
        mass = got[b, :, : int(lens[b])].sum(-1) - base[b, :, :old].double().sum(-1).cpu().numpy()
        # the weights of the tree's own LSE: 1e-4 each of the LSE and of the exponentials; fp32 totals
        assert np.abs(mass - Hq // Hkv * T).max() <= 2e-4 * (Hq // Hkv) * T + 1e-6 * want[b][:, : int(lens[b])].sum()


@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 64), (64, 6, 6, 16)])
def test_an_accepted_path_spreads_a_weight_of_one(ta, D, Hq, Hkv, page):
    """Rounds of drafting, accepting and evicting: the tree's LSE of an accepted
    node is over just the slots that its weights go to, so each accepted query
    adds one per head."""
    B, T, budget, G = 3, 7, 90, Hq // Hkv
    cache = ta.new_attn_cache(B, Hkv, 128, D, page_size=page)
    cap = cache.capacity
    rng, g = np.random.default_rng(D), torch.Generator(device="cuda").manual_seed(D)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    w, pos = torch.zeros(B, Hkv, cap, device="cuda"), torch.zeros(B, Hkv, cap, dtype=torch.int32, device="cuda")
    moves = torch.empty(B, Hkv, budget, 2, dtype=torch.int32, device="cuda")
    n_moves, seen = torch.empty(B, Hkv, dtype=torch.int32, device="cuda"), i32([0] * B)
    ws = ta.new_tree_workspace(Hq, Hkv, T, D)
    for step in range(60):  # about two tokens each
        q, k, v = rnd(B, Hq, T, D), rnd(B, Hkv, T, D), rnd(B, Hkv, T, D)
        parents = random_tree(rng, B, T)
        out, lse = torch.empty_like(q), torch.empty(B, Hq, T, device="cuda")
        ta.attn_tree_fwd(q, k, v, cache, out, lse, ws, parents=i32(parents))
        path, accepted = np.zeros((B, T), dtype=np.int32), np.zeros(B, dtype=np.int32)
        for b in range(B):
            node, up = int(rng.integers(0, T)), []
            while node >= 0:
                up.append(node)
                node = int(parents[b, node])
            accepted[b] = len(up)
            path[b, : len(up)] = up[::-1]
        acc_t, live = i32(accepted), torch.arange(cap, device="cuda")[None, :] < cache.lens[:, None]
        before = torch.where(live[:, None], w, 0.0).double().sum(-1)
        ta.attn_cache_append(cache, k, v, path=i32(path), counts=acc_t, positions=pos, seen=seen)
        ta.attn_cache_weights(q, lse, cache, w, w, path=i32(path), counts=acc_t)
        seen += acc_t
        live = torch.arange(cap, device="cuda")[None, :] < cache.lens[:, None]
        after = torch.where(live[:, None], w, 0.0).double().sum(-1)
        # 1e-4 each of the LSE and of the exponentials; fp32 totals
        want = G * acc_t.double()[:, None]
        assert ((after - before - want).abs() <= 2e-4 * want + 1e-6 * after).all(), step
        ta.attn_evict_plan(cache, w, pos, seen, moves, n_moves, budget, 1, 16)
        ta.attn_cache_compact(cache, moves, n_moves, budget, weights=w, positions=pos)
    assert torch.equal(cache.lens, seen.clamp(max=budget)) and (seen > budget).all() and ta.attn_get_status() == 0


# ------------------------------------------------------------------ layouts and offsets


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("T,Hq", [(5, 4), (70, 8)])
def test_weights_of_strided_views(ta, D, path, T, Hq):
    """q as [B][T][H][D] storage with room between its rows, pools as [page][row][head][D]."""
    c, p, lse, w = weights_case(T, [300, T + 40], [T, T - 3], T, Hq, 2, D, 32, path)
    check_weights(ta, c, p, lse, w)
    wide = torch.full((2, T, Hq, D + 24), NAN, dtype=torch.bfloat16, device="cuda")
    wide[..., 8: 8 + D] = c.q_t.permute(0, 2, 1, 3)
    c.q_t = wide[..., 8: 8 + D].permute(0, 2, 1, 3)
    c.storage = "row"
    c.load()
    check_weights(ta, c, p, lse, w)
    assert ta.attn_get_status() == 0


def test_append_weights_and_compact_beyond_32_bit_offsets(ta):
    """Pages that start past 2^32 elements of the pool."""
    page, D, T = 128, 64, 5
    stride = 1 << 31  # elements between pages: the third page starts at 2^32
    flat = torch.empty(2 * stride + page * D, dtype=torch.bfloat16, device="cuda")
    pool = flat.as_strided((3, 1, page, D), (stride, page * D, D, 1))
    c = CacheCase(16, [300], 4, 1, D, page, T, spare=0, room=T)
    pool.copy_(c.k_t)
    c.k_t = pool
    c.cache = ta.AttnCache(pool, c.v_t, c.lens_t, c.table_t)
    ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t)
    c.lens = oracle.cache.append(c.k_new, c.v_new, c.k, c.v, c.table, c.lens, None, None).astype(np.int32)
    torch.cuda.synchronize()
    assert np.array_equal(pool.float().cpu().double().numpy(), c.k, equal_nan=True)
    lse = np.full((1, 4, T), 5.0, dtype=np.float32)
    check_weights(ta, c, None, lse, np.ones((1, 1, c.cap), dtype=np.float32))
    moves = np.array([[[[3, 290], [140, 301], [200, 10]]]], dtype=np.int32)
    ta.attn_cache_compact(c.cache, i32(moves), i32([[3]]), 3)
    oracle.cache.compact(moves, np.array([[3]]), 3, c.k, c.v, c.table, c.lens)
    torch.cuda.synchronize()
    assert np.array_equal(pool.float().cpu().double().numpy(), c.k, equal_nan=True)
    assert np.array_equal(c.v_t.float().cpu().double().numpy(), c.v, equal_nan=True) and ta.attn_get_status() == 0


@pytest.mark.parametrize("budget", [128, 500])
def test_a_budget_that_nothing_exceeds(ta, budget):
    """At the capacity and above it: no moves, and the lengths stay."""
    c = CacheCase(3, [128, 77], 2, 2, 64, 64)
    w, pos = torch.rand(2, 2, c.cap, device="cuda"), torch.zeros(2, 2, c.cap, dtype=torch.int32, device="cuda")
    moves, n = torch.full((2, 2, budget, 2), 9, dtype=torch.int32, device="cuda"), i32(np.full((2, 2), 9))
    ta.attn_evict_plan(c.cache, w, pos, i32([128, 77]), moves, n, budget, 4, 20)
    ta.attn_cache_compact(c.cache, moves, n, budget, weights=w, positions=pos)
    torch.cuda.synchronize()
    assert (moves == -1).all() and (n == 0).all() and c.lens_t.tolist() == [128, 77] and ta.attn_get_status() == 0
    assert np.array_equal(c.k_t.float().cpu().double().numpy(), c.k, equal_nan=True)


@pytest.mark.parametrize("T", [1, 3])
def test_tree_over_thousands_of_rows(ta, T):
    rng = np.random.default_rng(T)
    lens = rng.integers(0, 90, 2100)
    lens[rng.random(2100) < 0.3] = 0
    c = CacheCase(T, lens, 2, 1, 64, 32, T, counts=rng.integers(0, T + 1, 2100))
    out, lse = torch.zeros_like(c.q_t), torch.zeros(2100, 2, T, device="cuda")
    ta.attn_tree_fwd(c.q_t, c.k_new_t, c.v_new_t, c.cache, out, lse, ta.new_tree_workspace(2, 1, T, 64), counts=i32(c.counts),
                     scale=c.scale)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    check_tree(out, lse, tree_reference(c, None))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("T,Hq", [(6, 4), (150, 8)])
def test_weights_of_values_that_are_not_finite(ta, D, path, T, Hq):
    """A NaN key reaches its own slot's total alone, a NaN LSE the slots that its query sees."""
    lens, counts = [400, T + 9], [T, T - 2]
    c, p, lse, w = weights_case(T + D, lens, counts, T, Hq, 2, D, 64, path)

    def call(lse):
        out = torch.full((2, 2, c.cap), 7.0, device="cuda")
        ta.attn_cache_weights(c.q_t, torch.from_numpy(lse).cuda(), c.cache, torch.from_numpy(w).cuda(), out, path=i32(p),
                              counts=i32(counts), scale=c.scale)
        torch.cuda.synchronize()
        return out.cpu()

    good = call(lse)
    hit = torch.zeros(2, 2, c.cap, dtype=torch.bool)
    for b, slot in ((0, 33), (0, 399), (1, T + 4)):  # an old one, the newest, one that only some queries see
        c.k_t[int(c.table[b, slot // 64]), 1, slot % 64, 5] = NAN
        hit[b, 1, slot] = True
    got = call(lse)
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], good[~hit])
    i = T // 2  # the accepted query whose LSE goes
    lse = lse.copy()
    lse[0, 0, i if p is None else int(p[0, i])] = NAN
    hit[0, 0, : lens[0] - counts[0] + i + 1] = True
    got = call(lse)
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], good[~hit])
    assert ta.attn_get_status() == 0
