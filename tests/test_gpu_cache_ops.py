"""Append, accumulated weights, eviction plan and compaction against their definitions."""
import numpy as np
import pytest
import torch

import oracle
from cache_common import CacheCase, bf16, dev16, i32

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def ta():
    import tiled_attention_25_b200 as m
    return m


def f64(t):
    return t.float().cpu().double().numpy()


# ------------------------------------------------------------------ append


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,storage", [(16, "head"), (64, "row"), (256, "head")])
@pytest.mark.parametrize("T", [1, 5, 70, 600])
def test_append(ta, D, page, storage, T):
    rng = np.random.default_rng(T + page)
    counts = [T, 0, int(rng.integers(0, T + 1))]
    for path in (False, True):
        c = CacheCase(T, [0, 30, 129], 2, 2, D, page, T, counts, room=T, storage=storage)
        c.k_new_t, c.v_new_t = torch.nan_to_num(c.k_new_t), torch.nan_to_num(c.v_new_t)
        c.k_new, c.v_new = np.nan_to_num(c.k_new), np.nan_to_num(c.v_new)
        p = rng.integers(0, T, size=(3, T)) if path else None  # the same node may go in twice
        seen = np.array([5, 1000, 129])
        pos = np.full((3, 2, c.cap), -1)
        pos_t, lens_out = i32(pos), torch.empty(3, dtype=torch.int32, device="cuda")
        ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t, lens_out, path=i32(p), counts=i32(c.counts), positions=pos_t,
                             seen=i32(seen))
        want = oracle.cache.append(c.k_new, c.v_new, c.k, c.v, c.table, c.lens, p, counts, pos, seen)
        torch.cuda.synchronize()
        assert ta.attn_get_status() == 0
        assert np.array_equal(f64(c.k_t), c.k, equal_nan=True) and np.array_equal(f64(c.v_t), c.v, equal_nan=True)
        assert np.array_equal(pos_t.cpu().numpy(), pos) and np.array_equal(lens_out.cpu().numpy(), want)
        assert np.array_equal(c.lens_t.cpu().numpy(), c.lens)  # the cache's own lengths stay
        ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t, path=i32(p), counts=i32(c.counts))  # in place
        torch.cuda.synchronize()
        assert np.array_equal(c.lens_t.cpu().numpy(), want)


def test_append_default_positions_and_strided(ta):
    c = CacheCase(3, [10, 20], 2, 2, 128, 64, 4, room=4)
    k = c.k_new_t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    pos = np.full((2, 2, c.cap), -1)
    pos_t = i32(pos)
    ta.attn_cache_append(c.cache, k, c.v_new_t, positions=pos_t, lens_out=c.lens_t)
    want = oracle.cache.append(c.k_new, c.v_new, c.k, c.v, c.table, c.lens, None, None, pos)
    torch.cuda.synchronize()
    assert np.array_equal(f64(c.k_t), c.k, equal_nan=True)
    assert np.array_equal(pos_t.cpu().numpy(), pos) and np.array_equal(c.lens_t.cpu().numpy(), want)


def test_append_bad_values(ta):
    """A full row, nodes out of range, a page outside the pool: nothing is written there."""
    c = CacheCase(4, [60, 64, 10, 10], 2, 2, 64, 64, 8, spare=3)
    c.table[3, 0] = -1
    c.load()
    path = np.tile(np.arange(8), (4, 1))
    path[2, 3], path[2, 4] = -1, 8
    pos = np.full((4, 2, c.cap), -1)
    pos_t, out = i32(pos), torch.empty(4, dtype=torch.int32, device="cuda")
    ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t, out, path=i32(path), positions=pos_t)
    want = oracle.cache.append(c.k_new, c.v_new, c.k, c.v, c.table, c.lens, path, None, pos)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
    assert np.array_equal(f64(c.k_t), c.k, equal_nan=True) and np.array_equal(f64(c.v_t), c.v, equal_nan=True)
    assert np.array_equal(out.cpu().numpy(), want) and list(want) == [64, 64, 18, 18]
    assert np.array_equal(pos_t.cpu().numpy(), pos)


# ------------------------------------------------------------------ weights


def weights_case(seed, lens, counts, T, Hq, Hkv, D, page, path, softcap=None):
    c = CacheCase(seed, lens, Hq, Hkv, D, page, T, counts)
    rng = c.rng
    p = np.sort(rng.permuted(np.tile(np.arange(T), (c.B, 1)), axis=1), axis=1) if path else None
    if path:
        for b in range(c.B):
            m = T if counts is None else int(c.counts[b])
            p[b] = 0
            p[b, :m] = np.sort(rng.choice(T, size=m, replace=False))
    # LSE of each query over what it sees, and NaN for the queries that are not used
    lse = np.full((c.B, Hq, T), np.nan)
    for b in range(c.B):
        n, m = int(c.lens[b]), T if counts is None else int(c.counts[b])
        for h in range(Hq):
            kk = oracle.cache.slots(c.k, c.table[b], n, h // (Hq // Hkv))
            for i in range(m):
                node = i if p is None else int(p[b, i])
                s = kk[: n - m + i + 1] @ c.q[b, h, node] * c.scale
                s = softcap * np.tanh(s / softcap) if softcap else s
                lse[b, h, node] = s.max() + np.log(np.exp(s - s.max()).sum())
    lse = lse.astype(np.float32)
    w = np.abs(rng.standard_normal((c.B, Hkv, c.cap))).astype(np.float32) * 3
    return c, p, lse, w


def check_weights(ta, c, p, lse, w, softcap=None, inplace=False, no_base=False):
    kw = dict(mod_kind=ta.MOD_SOFTCAP, mod_params=ta.ModParams(softcap=softcap)) if softcap else {}
    w_t = torch.from_numpy(w).cuda()
    for b in range(c.B):  # whatever lies in the new slots and behind is not read
        w_t[b, :, max(0, int(c.lens[b]) - (c.T if c.counts is None else int(c.counts[b]))):] = NAN
    out = w_t.clone() if inplace else torch.full_like(w_t, 7.0)
    ta.attn_cache_weights(c.q_t, torch.from_numpy(lse).cuda(), c.cache, None if no_base else (out if inplace else w_t), out,
                          path=i32(p), counts=i32(c.counts), scale=c.scale, **kw)
    torch.cuda.synchronize()
    want, add = oracle.cache.slot_weights(c.q, lse.astype(np.float64), c.k, c.table, c.lens, None if no_base else w, p,
                                          c.counts, c.scale, softcap)
    got = out.cpu().double().numpy()
    sel = ~np.isnan(want)
    assert np.isfinite(got[sel]).all()
    # each exponential to 1e-4 relative (scores up to ~8 in fp32), the sum and the base rounded in fp32
    over = np.abs(got - want)[sel] - (1e-4 * add[sel] + 1e-6 * np.abs(want[sel]))
    assert over.size == 0 or over.max() <= 0, f"off by {over.max():.3e}"
    rest = got[~sel]
    assert np.isnan(rest).all() if inplace else (rest == 7.0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (15, 3), (16, 1)])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_weights_of_accepted_tokens(ta, D, Hq, Hkv, T):
    rng = np.random.default_rng(T + Hq)
    counts = [T, 1, int(rng.integers(0, T + 1)), 0]
    c, p, lse, w = weights_case(Hq + T, [T, 129, 300, 50], counts, T, Hq, Hkv, D, 16, True)
    check_weights(ta, c, p, lse, w)
    check_weights(ta, c, p, lse, w, inplace=True)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,extra", [(128, 0), (130, 0), (257, 3), (500, 200)])
def test_weights_of_a_prompt(ta, D, T, extra):
    c, p, lse, w = weights_case(T + D, [T + extra], None, T, 4, 2, D, 64, False)
    check_weights(ta, c, p, lse, w, no_base=extra == 0)
    assert ta.attn_get_status() == 0


def test_weights_softcap_and_many_heads(ta):
    c, p, lse, w = weights_case(5, [300, 17], [5, 2], 5, 8, 2, 128, 64, True, softcap=2.0)
    check_weights(ta, c, p, lse, w, softcap=2.0)
    c, p, lse, w = weights_case(6, [200, 140], [2, 1], 2, 160, 1, 64, 128, True)
    check_weights(ta, c, p, lse, w)


@pytest.mark.parametrize("Hq,Hkv,lens,T", [(8, 1, [700], 700), (8, 1, [1500], 1100), (4, 2, [300, 260], 257), (16, 4, [600], 550)])
def test_weights_of_a_prompt_shared_by_clusters(ta, Hq, Hkv, lens, T):
    """Few heads: 2 to 8 CTAs share a unit's queries; several units to a cluster, and CTAs without a query."""
    c, p, lse, w = weights_case(T, lens, None, T, Hq, Hkv, 64, 64, False)
    check_weights(ta, c, p, lse, w)
    outs = []
    for _ in range(3):
        out = torch.zeros(c.B, Hkv, c.cap, device="cuda")
        ta.attn_cache_weights(c.q_t, torch.from_numpy(lse).cuda(), c.cache, None, out, scale=c.scale)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    counts = [max(1, T // 5)] * len(lens)
    c, p, lse, w = weights_case(T + 1, lens, counts, T, Hq, Hkv, 64, 128, True)
    check_weights(ta, c, p, lse, w)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("D,page", [(64, 64), (128, 16)])
@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hkv", [(15, 28, 28, 4), (3, 70, 8, 2), (30, 40, 8, 1)])
def test_weights_of_uneven_counts(ta, D, page, B, T, Hq, Hkv, path):
    """More than one Q tile, few new tokens, long rows: many units to a CTA or to a
    cluster, some with queries for its first CTA only."""
    lens = [561 + 1031 * b // max(1, B - 1) for b in range(B)]
    counts = [1 + (5 * b + T // 2) % T for b in range(B)]
    c, p, lse, w = weights_case(B + T, lens, counts, T, Hq, Hkv, D, page, path)
    check_weights(ta, c, p, lse, w)
    outs = []
    for _ in range(4):
        out = torch.zeros(c.B, Hkv, c.cap, device="cuda")
        ta.attn_cache_weights(c.q_t, torch.from_numpy(lse).cuda(), c.cache, None, out, path=i32(p), counts=i32(counts),
                              scale=c.scale)
        outs.append(out)
    assert all(torch.equal(outs[0], x) for x in outs[1:])
    assert ta.attn_get_status() == 0


def test_weights_of_many_rows(ta):
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 256, 257] * 4
    counts = [min(n, 2) for n in lens]
    c, p, lse, w = weights_case(7, lens, counts, 3, 4, 2, 64, 32, True)
    check_weights(ta, c, p, lse, w)


def test_weights_bad_values(ta):
    """Counts above the length are clamped, nodes out of range count for nothing, a bad page is zeros."""
    c, p, lse, w = weights_case(8, [5, 200], [4, 4], 6, 4, 2, 64, 64, True)
    p[1, 2] = 6
    c.counts = np.array([6, 4], dtype=np.int32)  # row 0 has 5 slots
    p[0] = np.arange(6)
    lse[0] = 3.0
    check_weights(ta, c, p, lse, w)
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
    c, p, lse, w = weights_case(9, [200], [2], 2, 4, 2, 64, 64, True)
    c.table[0, 1] = 1 << 20
    c.load()
    check_weights(ta, c, p, lse, w)
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX


def test_weights_sum_to_the_queries(ta):
    """Every query spreads a weight of one over what it sees."""
    c, p, lse, w = weights_case(10, [400], None, 300, 8, 2, 128, 64, False)
    out = torch.zeros(1, 2, c.cap, device="cuda")
    ta.attn_cache_weights(c.q_t, torch.from_numpy(lse).cuda(), c.cache, None, out, scale=c.scale)
    assert np.allclose(out[0, :, :400].double().sum(-1).cpu().numpy(), 4 * 300, rtol=1e-4)


# ------------------------------------------------------------------ plan


def plan_case(seed, lens, Hkv, budget, recent, cap=None, ties=0.2, page=64):
    rng = np.random.default_rng(seed)
    B = len(lens)
    n = max(1, -(-max(cap or 0, max(lens)) // page))
    w = rng.exponential(size=(B, Hkv, n * page)).astype(np.float32)
    w[rng.random(w.shape) < ties] = 0.0
    w[rng.random(w.shape) < ties] = 0.5
    pos = rng.permuted(np.tile(np.arange(n * page), (B, Hkv, 1)), axis=2)
    seen = np.array([max(1, x) for x in lens]) + 3
    return w, pos, seen, n


def plan_check(ta, w, pos, seen, lens, n, budget, first, recent, page=64, unaligned=False):
    B, Hkv, cap = w.shape
    pool = torch.zeros(B * n, Hkv, page, 64, dtype=torch.bfloat16, device="cuda")
    cache = ta.AttnCache(pool, pool, i32(lens))
    moves = torch.full((B, Hkv, budget, 2), 9, dtype=torch.int32, device="cuda")
    count = torch.full((B, Hkv), 9, dtype=torch.int32, device="cuda")
    w_t, pos_t = torch.from_numpy(w).cuda(), i32(pos)
    if unaligned:  # 4 bytes behind a 16-byte boundary
        off = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
        w_t, pos_t = off(w_t), off(pos_t)
    ta.attn_evict_plan(cache, w_t, pos_t, i32(seen), moves, count, budget, first, recent)
    torch.cuda.synchronize()
    want, wn = oracle.cache.evict_plan(w, pos, seen, lens, budget, first, recent)
    assert np.array_equal(count.cpu().numpy(), wn)
    assert np.array_equal(moves.cpu().numpy(), want)


@pytest.mark.parametrize("budget", [1, 7, 64, 300])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_plan(ta, budget, Hkv):
    lens = [0, 1, budget - 1, budget, budget + 1, 2 * budget, 5 * budget + 3, 1000]
    for ties in (0.0, 0.3, 1.0):
        w, pos, seen, n = plan_case(budget, lens, Hkv, budget, 0, ties=ties)
        for first, recent in ((0, 0), (min(2, budget), 0), (budget // 4, budget // 2), (0, budget)):
            plan_check(ta, w, pos, seen, lens, n, budget, first, recent)
    assert ta.attn_get_status() == 0


@pytest.mark.parametrize("n,budget", [(5000, 4096), (20000, 1000), (33333, 32768), (9000, 8999)])
def test_plan_long(ta, n, budget):
    w, pos, seen, pages = plan_case(n, [n, n - 1], 2, budget, 0)
    plan_check(ta, w, pos, seen, [n, n - 1], pages, budget, 4, budget // 8)
    plan_check(ta, w, pos, seen, [n, n - 1], pages, budget, 0, 5, unaligned=True)


def test_plan_many_heads_and_ranks_that_do_not_fit(ta):
    """More heads than SMs, so one CTA to each, and a row too long for its shared memory; and the full capacity."""
    lens = [5] * 299 + [60000]
    w, pos, seen, pages = plan_case(5, lens, 1, 300, 0)
    plan_check(ta, w, pos, seen, lens, pages, 300, 4, 100)
    lens = [1 << 20, 100]
    w, pos, seen, pages = plan_case(6, lens, 1, 5000, 0, page=1 << 14)
    plan_check(ta, w, pos, seen, lens, pages, 5000, 0, 17, page=1 << 14)


def test_plan_strange_weights(ta):
    """Infinities, NaN, zeros of both signs, negative and denormal weights."""
    w, pos, seen, n = plan_case(3, [256, 256], 2, 100, 0)
    rng = np.random.default_rng(3)
    odd = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, -1.0, 1e-42, -1e-42, 3e38, 1.0], dtype=np.float32)
    w[:] = odd[rng.integers(0, len(odd), size=w.shape)]
    for budget in (1, 20, 100, 255):
        plan_check(ta, w, pos, seen, [256, 256], n, budget, 0, 0)
        plan_check(ta, w, pos, seen, [256, 256], n, budget, 0, min(budget, 9))


def test_plan_bad_length(ta):
    w, pos, seen, n = plan_case(4, [64], 1, 10, 0)
    pool = torch.zeros(1, 1, 64, 64, dtype=torch.bfloat16, device="cuda")
    moves, count = torch.zeros(1, 1, 10, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for raw, n_used in ((-3, 0), (1 << 30, 64)):
        ta.attn_evict_plan(ta.AttnCache(pool, pool, i32([raw])), torch.from_numpy(w).cuda(), i32(pos), i32(seen), moves, count, 10)
        torch.cuda.synchronize()
        assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
        want, wn = oracle.cache.evict_plan(w, pos, seen, [n_used], 10, 0, 0)
        assert np.array_equal(moves.cpu().numpy(), want) and np.array_equal(count.cpu().numpy(), wn)


# ------------------------------------------------------------------ compact


@pytest.mark.parametrize("D,page,storage", [(64, 16, "head"), (128, 64, "row"), (128, 256, "head")])
def test_plan_and_compact(ta, D, page, storage):
    lens, budget = [700, 400, 399, 3], 400
    c = CacheCase(D + page, lens, 3, 3, D, page, storage=storage)
    w = c.rng.exponential(size=(4, 3, c.cap)).astype(np.float32)
    pos = c.rng.permuted(np.tile(np.arange(c.cap), (4, 3, 1)), axis=2)
    seen = np.array(lens)
    w_t, pos_t = torch.from_numpy(w).cuda(), i32(pos)
    moves = torch.empty(4, 3, budget, 2, dtype=torch.int32, device="cuda")
    count = torch.empty(4, 3, dtype=torch.int32, device="cuda")
    ta.attn_evict_plan(c.cache, w_t, pos_t, i32(seen), moves, count, budget, 2, 50)
    ta.attn_cache_compact(c.cache, moves, count, budget, weights=w_t, positions=pos_t)
    want, wn = oracle.cache.evict_plan(w, pos, seen, lens, budget, 2, 50)
    new = oracle.cache.compact(want, wn, budget, c.k, c.v, c.table, c.lens, w, pos)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    assert np.array_equal(f64(c.k_t), c.k, equal_nan=True) and np.array_equal(f64(c.v_t), c.v, equal_nan=True)
    assert np.array_equal(w_t.cpu().numpy(), w) and np.array_equal(pos_t.cpu().numpy(), pos)
    assert np.array_equal(c.lens_t.cpu().numpy(), new) and list(new) == [400, 400, 399, 3]


def test_compact_bad_moves(ta):
    c = CacheCase(5, [200], 1, 1, 64, 64)
    moves = np.array([[[[3, 150], [-1, 160], [4, c.cap], [1 << 30, 5], [6, 199]]]], dtype=np.int32)
    ta.attn_cache_compact(c.cache, i32(moves), i32([[5]]), 5)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
    oracle.cache.compact(moves[:, :, [0, 4]], np.array([[2]]), 5, c.k, c.v, c.table, c.lens)
    assert np.array_equal(f64(c.k_t), c.k, equal_nan=True) and int(c.lens_t[0]) == 5
    ta.attn_cache_compact(c.cache, i32(moves), i32([[77]]), 5)  # more moves than there is room for
    torch.cuda.synchronize()
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX


def test_refusals(ta):
    c = CacheCase(6, [100], 2, 2, 64, 64, 2, room=2)
    w, pos = torch.zeros(1, 2, c.cap, device="cuda"), torch.zeros(1, 2, c.cap, dtype=torch.int32, device="cuda")
    mv, cnt = torch.zeros(1, 2, 50, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    seen, lse = i32([100]), torch.zeros(1, 2, 2, device="cuda")
    for f in (lambda: ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t[:, :1]),
              lambda: ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t, positions=pos[..., :5]),
              lambda: ta.attn_cache_append(c.cache, c.k_new_t, c.v_new_t, seen=seen.cpu()),
              lambda: ta.attn_cache_weights(c.q_t, lse, c.cache, w.double(), w),
              lambda: ta.attn_cache_weights(c.q_t, lse[..., :1], c.cache, w, w),
              lambda: ta.attn_evict_plan(c.cache, w, pos, seen, mv, cnt, 49),
              lambda: ta.attn_evict_plan(c.cache, w, pos.float(), seen, mv, cnt, 50),
              lambda: ta.attn_cache_compact(c.cache, mv.float(), cnt, 50),
              lambda: ta.AttnCache(c.k_t, c.v_t[:1], c.lens_t, c.table_t),
              lambda: ta.AttnCache(c.k_t, c.v_t, c.lens_t.long(), c.table_t),
              lambda: ta.AttnCache(c.k_t, c.v_t, c.lens_t, c.table_t[0])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ta.attn_evict_plan(c.cache, w, pos, seen, mv, cnt, 50, first=-1),
              lambda: ta.attn_evict_plan(c.cache, w, pos, seen, mv, cnt, 50, first=20, recent=31),
              lambda: ta.attn_cache_weights(c.q_t, lse, c.cache, w, w, mod_kind=ta.MOD_ALIBI)):
        with pytest.raises(ta.AttnError):
            f()
