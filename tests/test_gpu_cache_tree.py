"""Attention of new tokens over a paged cache (attn_tree_fwd) against fp64."""
import numpy as np
import pytest
import torch

import oracle
from cache_common import CacheCase, check_tree, dev16, i32, random_tree, tree_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ta():
    import tiled_attention_25_b200 as m
    return m


def call(ta, c, parents, out=None, lse=None, with_new=True, ws=None, stream=None, **kw):
    if out is None:
        out = torch.full_like(c.q_t, 7.0)
    if lse is None:
        lse = torch.full(c.q_t.shape[:3], 7.0, device="cuda")
    ws = ta.new_tree_workspace(c.Hq, c.Hkv, c.T, c.D) if ws is None else ws
    ta.attn_tree_fwd(c.q_t, c.k_new_t if with_new else None, c.v_new_t if with_new else None, c.cache, out, lse, ws,
                     parents=i32(parents), counts=i32(c.counts), scale=c.scale, stream=stream, **kw)
    return out, lse


def run_and_check(ta, c, parents, what="", with_new=True, softcap=None):
    kw = {}
    if softcap:
        kw = dict(mod_kind=ta.MOD_SOFTCAP, mod_params=ta.ModParams(softcap=softcap))
    out, lse = call(ta, c, parents, with_new=with_new, **kw)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0
    check_tree(out, lse, tree_reference(c, parents, with_new, softcap), what)
    if c.counts is not None:  # rows behind counts stay as they were
        for b in range(c.B):
            assert (out[b, :, c.counts[b]:] == 7.0).all() and (lse[b, :, c.counts[b]:] == 7.0).all()
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 384])
@pytest.mark.parametrize("n", [1, 127, 128, 129, 300, 1000])
def test_one_token(ta, D, page, n):
    run_and_check(ta, CacheCase(n + page, [n, 1, max(1, n - 5)], 8, 2, D, page), None, f"D={D} page={page} len={n}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (4, 4), (10, 2), (16, 1), (21, 3)])
@pytest.mark.parametrize("T", [1, 2, 7, 33])
def test_trees_and_heads(ta, D, Hq, Hkv, T):
    c = CacheCase(100 * T + Hq, [37, 0, 200], Hq, Hkv, D, 16, T)
    run_and_check(ta, c, random_tree(c.rng, 3, T), f"D={D} heads {Hq}/{Hkv} T={T}")


@pytest.mark.parametrize("Hq,Hkv", [(192, 1), (130, 1), (256, 2)])
def test_many_heads_share_one(ta, Hq, Hkv):
    c = CacheCase(Hq, [150, 5], Hq, Hkv, 64, 64, 2)
    run_and_check(ta, c, random_tree(c.rng, 2, 2), f"heads {Hq}/{Hkv}")


@pytest.mark.parametrize("T", [64, 128, 129, 200, 300])
@pytest.mark.parametrize("tree", [True, False])
def test_long_drafts_and_chains(ta, T, tree):
    c = CacheCase(T, [130, 0], 4, 2, 128, 32, T)
    run_and_check(ta, c, random_tree(c.rng, 2, T, 9) if tree else None, f"T={T}")


@pytest.mark.parametrize("T", [1, 8, 40])
def test_ragged_counts(ta, T):
    rng = np.random.default_rng(T)
    counts = [T, 0, 1, int(rng.integers(0, T + 1)), T]
    c = CacheCase(T, [0, 100, 0, 259, 64], 8, 2, 128, 64, T, counts)
    run_and_check(ta, c, random_tree(rng, 5, T), f"T={T}")


@pytest.mark.parametrize("Hq,Hkv,T", [(40, 1, 1024), (2, 1, 1024), (100, 2, 130)])
def test_more_query_tiles_than_sms(ta, Hq, Hkv, T):
    """342 tiles, one to a CTA; two; tiles whose tokens only some rows have."""
    c = CacheCase(T + Hq, [70, 3], Hq, Hkv, 64, 64, T, counts=[T, T // 3])
    run_and_check(ta, c, random_tree(c.rng, 2, T) if T < 1000 else None, f"heads {Hq}/{Hkv} T={T}")


def test_no_queries_at_all(ta):
    c = CacheCase(4, [300, 0], 4, 2, 128, 64, 3, counts=[0, 0])
    run_and_check(ta, c, None)


def test_more_rows_than_one_window(ta):
    """130 rows: items above and below the number of SMs, rows without queries among them."""
    rng = np.random.default_rng(21)
    for lens, Hkv in ((rng.integers(0, 40, 130), 1), (rng.integers(0, 700, 100), 2)):
        counts = rng.integers(0, 3, len(lens))
        c = CacheCase(22, lens, 2 * Hkv, Hkv, 64, 16, 2, counts)
        run_and_check(ta, c, random_tree(rng, len(lens), 2))


def test_cuts_of_many_items(ta):
    """More items than SMs, some long, so that the stream is cut inside and near the ends of items."""
    rng = np.random.default_rng(23)
    lens = [int(x) for x in rng.integers(1, 200, 36)] + [9000, 5000, 1200, 640]
    c = CacheCase(24, lens, 8, 4, 64, 128, 2)
    a, la = run_and_check(ta, c, None)
    b, lb = call(ta, c, None)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_one_workspace_serves_other_shapes(ta):
    """The counters at its head are zero after every call."""
    ws = ta.new_tree_workspace(32, 1, 64, 128)
    for seed, (lens, Hq, Hkv, D, T) in enumerate([([3000], 8, 1, 128, 3), ([900, 4000], 4, 2, 64, 20), ([6000], 32, 1, 64, 4)]):
        c = CacheCase(30 + seed, lens, Hq, Hkv, D, 64, T)
        out, lse = call(ta, c, None, ws=ws)
        torch.cuda.synchronize()
        check_tree(out, lse, tree_reference(c, None), str(lens))
        assert (ws[:1024] == 0).all()


def test_every_root_and_a_deep_chain(ta):
    """All nodes siblings (no one sees another), and one path through all."""
    c = CacheCase(5, [70, 128], 4, 1, 128, 64, 60)
    run_and_check(ta, c, np.full((2, 60), -1, dtype=np.int32), "siblings")
    chain = np.tile(np.arange(60, dtype=np.int32) - 1, (2, 1))
    a = run_and_check(ta, c, chain, "chain")
    b = run_and_check(ta, c, None, "chain by default")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_the_cache_alone_and_empty_rows(ta):
    c = CacheCase(6, [0, 90, 256, 1], 6, 3, 128, 128, 3)
    out, lse = run_and_check(ta, c, None, "cache alone", with_new=False)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [1.5, 20.0])
def test_softcap(ta, D, softcap):
    c = CacheCase(int(softcap) + D, [333, 128], 8, 2, D, 64, 5)
    run_and_check(ta, c, random_tree(c.rng, 2, 5), "softcap", softcap=softcap)


def test_many_rows_and_all_lengths(ta):
    """Every length around the 128-slot steps, in one call."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385] * 3
    c = CacheCase(8, lens, 4, 2, 64, 16, 3)
    run_and_check(ta, c, random_tree(c.rng, len(lens), 3))


@pytest.mark.parametrize("Hkv,n", [(1, 20000), (2, 9001)])
def test_a_long_row_is_split(ta, Hkv, n):
    c = CacheCase(n, [n, 3], 4 * Hkv, Hkv, 128, 128, 2)
    a, la = run_and_check(ta, c, None, f"len={n}")
    b, lb = call(ta, c, None)
    assert torch.equal(a, b) and torch.equal(la, lb)  # the same bits on every run


def test_large_scores_and_one_key_takes_all(ta):
    """Scores of hundreds, growing along the row, so that the running maximum moves often."""
    c = CacheCase(9, [700], 2, 1, 128, 64, 1)
    ramp = np.linspace(0.0, 6.0, 704, dtype=np.float32).reshape(11, 64)
    u = c.q[0, 0, 0] / np.linalg.norm(c.q[0, 0, 0])
    k = c.k.astype(np.float32)
    for i, p in enumerate(c.table[0]):
        k[p, 0] = k[p, 0] * 0.1 + (ramp[i][:, None] * u * 8).astype(np.float32)
    from cache_common import bf16
    c.k_bits, c.k = bf16(k)
    c.load()
    run_and_check(ta, c, None)


@pytest.mark.parametrize("storage", ["head", "row"])
def test_strided_views(ta, storage):
    c = CacheCase(11, [200, 77], 8, 4, 128, 64, 5, storage=storage)
    parents = random_tree(c.rng, 2, 5)
    ref = call(ta, c, parents)
    for name in ("q_t", "k_new_t", "v_new_t"):  # [B][T][H][D] storage
        t = getattr(c, name)
        setattr(c, name, t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3))
    wide = torch.full((2, 5, 8, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[..., 8:136].permute(0, 2, 1, 3)
    got = call(ta, c, parents, out=out)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert (wide[..., :8] == 7.0).all() and (wide[..., 136:] == 7.0).all()


def test_no_lse_and_contiguous_cache(ta):
    """One page per row without a table: the same bits as pages of 64."""
    c = CacheCase(12, [300, 180], 8, 2, 128, 64, 4)
    parents = random_tree(c.rng, 2, 4)
    ref, _ = call(ta, c, parents)
    cap = 384
    pools = []
    for x in (c.k_t, c.v_t):
        t = torch.full((2, 2, cap, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        for b in range(2):
            for j in range(0, int(c.lens[b]), 64):
                m = min(64, int(c.lens[b]) - j)
                t[b, :, j:j + m] = x[int(c.table[b, j // 64]), :, :m]
        pools.append(t)
    c.cache = ta.AttnCache(*pools, c.lens_t)
    out = torch.empty_like(c.q_t)
    ws = ta.new_tree_workspace(8, 2, 4, 128)
    ta.attn_tree_fwd(c.q_t, c.k_new_t, c.v_new_t, c.cache, out, None, ws, parents=i32(parents), scale=c.scale)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_bad_indices_are_recorded_and_harmless(ta):
    """A page outside the pool reads as zeros, a parent out of range is the
    root, lengths and counts are clamped; the status says so, once."""
    c = CacheCase(13, [200, 100], 4, 2, 128, 64, 6, counts=[6, 4])
    parents = random_tree(c.rng, 2, 6)
    good = c.table.copy()
    for bad in (-1, 1 << 30, -(1 << 31)):
        c.table = good.copy()
        c.table[0, 1] = bad
        c.load()
        out, lse = call(ta, c, parents)
        torch.cuda.synchronize()
        assert ta.attn_get_status() == ta.ATTN_ERR_INDEX and ta.attn_get_status() == 0
        check_tree(out, lse, tree_reference(c, parents), "bad page")
    c.table = good
    c.load()
    for bad in (4, 6, 100000, -2):
        p = parents.copy()
        p[1, 3] = bad
        out, lse = call(ta, c, p)
        torch.cuda.synchronize()
        assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
        check_tree(out, lse, tree_reference(c, p), "bad parent")
    c.lens_t[1] = -5
    c.lens_t[0] = c.cap + 1000
    c.lens = np.array([c.cap, 0], dtype=np.int32)
    finite = torch.where(torch.isnan(c.k_t), 0.0, c.k_t), torch.where(torch.isnan(c.v_t), 0.0, c.v_t)
    c.cache = ta.AttnCache(*finite, c.lens_t, c.table_t)
    c.k, c.v = np.nan_to_num(c.k), np.nan_to_num(c.v)
    out, lse = call(ta, c, parents)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == ta.ATTN_ERR_INDEX
    check_tree(out, lse, tree_reference(c, parents), "clamped")


def test_shared_pages(ta):
    """Two rows that share their first pages."""
    c = CacheCase(14, [256, 256], 4, 2, 64, 64, 3)
    c.table[1, :3] = c.table[0, :3]
    c.load()
    run_and_check(ta, c, random_tree(c.rng, 2, 3))


def test_graph_follows_lens_and_two_streams(ta):
    """A captured call replays with the lengths, table and counts of the day;
    two calls with a workspace each run at once on two streams."""
    c = CacheCase(15, [500, 380, 40], 8, 2, 128, 64, 4, counts=[4, 4, 4])
    parents = random_tree(c.rng, 3, 4)
    par_t, cnt_t = i32(parents), i32(c.counts)
    out, lse = torch.full_like(c.q_t, 7.0), torch.full(c.q_t.shape[:3], 7.0, device="cuda")
    ws = ta.new_tree_workspace(8, 2, 4, 128)
    go = lambda o, l, w: ta.attn_tree_fwd(c.q_t, c.k_new_t, c.v_new_t, c.cache, o, l, w, parents=par_t, counts=cnt_t,  # noqa: E731
                                          scale=c.scale)
    go(out, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(out, lse, ws)
    for lens, counts in (([500, 380, 40], [4, 4, 4]), ([129, 0, 3], [1, 4, 2]), ([0, 1, 40], [4, 3, 0])):
        c.lens, c.counts = np.array(lens, dtype=np.int32), np.array(counts, dtype=np.int32)
        c.lens_t.copy_(i32(c.lens))
        cnt_t.copy_(i32(c.counts))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check_tree(out, lse, tree_reference(c, parents), f"replay {lens}")
    c.lens, c.counts = np.array([500, 380, 40], dtype=np.int32), np.array([4, 4, 4], dtype=np.int32)
    c.lens_t.copy_(i32(c.lens))
    cnt_t.copy_(i32(c.counts))
    go(out, lse, ws)
    torch.cuda.synchronize()
    outs = [(torch.zeros_like(out), torch.zeros_like(lse), ta.new_tree_workspace(8, 2, 4, 128)) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s, (o, l, w) in zip(streams, outs):
            with torch.cuda.stream(s):
                go(o, l, w)
    torch.cuda.synchronize()
    for o, l, _ in outs:
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert ta.attn_get_status() == 0


def test_pool_beyond_32_bit_offsets(ta):
    """Pages that start past 2^32 elements of the pool."""
    page, Hkv, D = 128, 1, 128
    stride = 1 << 31  # elements between pages: the third page starts at 2^32
    flat = torch.empty(2 * stride + Hkv * page * D, dtype=torch.bfloat16, device="cuda")
    pool = flat.as_strided((3, Hkv, page, D), (stride, page * D, D, 1))
    c = CacheCase(16, [300], 4, 1, D, page, 2, spare=0)
    pool.copy_(c.k_t)
    c.cache = ta.AttnCache(pool, c.v_t, c.lens_t, c.table_t)
    run_and_check(ta, c, None)


def test_agrees_with_the_whole_sequence_forward(ta):
    """The last T tokens of a causal sequence: attn_fwd over everything and
    the cache's form differ by no more than both bounds."""
    S, T, B, Hq, Hkv, D = 640, 128, 1, 4, 2, 128
    c = CacheCase(17, [S - T], Hq, Hkv, D, 64, T)
    out, lse = run_and_check(ta, c, None)
    k = torch.empty(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for x, pool, new in ((k, c.k_t, c.k_new_t), (v, c.v_t, c.v_new_t)):
        x[:, :, S - T:] = new
        for j in range(0, S - T, 64):
            x[0, :, j:j + 64] = pool[int(c.table[0, j // 64])]
    q = torch.zeros(B, Hq, S, D, dtype=torch.bfloat16, device="cuda")
    q[:, :, S - T:] = c.q_t
    o2, l2 = torch.empty_like(q), torch.empty(B, Hq, S, device="cuda")
    ta.attn_fwd(q, k, v, o2, l2, mod_kind=ta.MOD_CAUSAL)
    torch.cuda.synchronize()
    assert (o2[:, :, S - T:].float() - out.float()).abs().max() <= 4e-2
    assert (l2[:, :, S - T:] - lse).abs().max() <= 1e-3 + 1e-4


def test_refusals(ta):
    c = CacheCase(18, [100], 4, 2, 128, 64, 2)
    out, lse = torch.empty_like(c.q_t), torch.empty(1, 4, 2, device="cuda")
    ws = ta.new_tree_workspace(4, 2, 2, 128)
    go = lambda **kw: ta.attn_tree_fwd(**{**dict(q=c.q_t, k_new=c.k_new_t, v_new=c.v_new_t, cache=c.cache, out=out, lse=lse,  # noqa: E731
                                                 workspace=ws), **kw})
    for bad in (dict(q=c.q_t.float()), dict(out=out[..., :64]), dict(lse=lse[..., :1]), dict(lse=lse.double()),
                dict(k_new=c.k_new_t[:, :1]), dict(parents=torch.zeros(1, 2, device="cuda")),
                dict(parents=torch.zeros(1, 3, dtype=torch.int32, device="cuda")),
                dict(counts=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(counts=torch.zeros(1, dtype=torch.int32)), dict(q=c.q_t.cpu()), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            go(**bad)
    for bad in (dict(v_new=None), dict(k_new=None, v_new=None, parents=torch.zeros(1, 2, dtype=torch.int32, device="cuda")),
                dict(scale=0.0), dict(mod_kind=ta.MOD_SOFTCAP), dict(mod_kind=ta.MOD_CAUSAL), dict(workspace=ws[:16])):
        with pytest.raises(ta.AttnError):
            go(**bad)
    torch.cuda.synchronize()
    assert ta.attn_get_status() == 0


def test_a_workspace_without_its_memory_is_refused(ta):
    """An expanded view has the size but not the bytes."""
    c = CacheCase(19, [5], 4, 2, 64, 16, 2)
    ws = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(ta.attn_tree_workspace_size(4, 2, 2, 64))
    with pytest.raises(ValueError):
        call(ta, c, None, ws=ws)


@pytest.mark.parametrize("Hq,T", [(8, 1), (12, 5), (24, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_the_same_bits_whatever_ran_before(ta, D, Hq, T):
    """Widely spread scores, so that running maxima move: when they do may not
    depend on the tile's unused rows, where shared memory holds what an
    earlier kernel left."""
    lens = [900 + 7 * b for b in range(80)]  # more items than SMs: pieces of many steps
    c = CacheCase(20, lens, Hq, 2, D, 64, T, scale=1.0)
    before = CacheCase(21, [9000, 8000], 128, 1, D, 64, 1)  # queries in all 128 rows
    o = [torch.empty_like(before.q_t), torch.empty(2, 128, 1, device="cuda")]
    ws = [ta.new_tree_workspace(128, 1, 1, D), ta.new_tree_workspace(Hq, 2, T, D)]
    first = None
    for size in (0.0, 1.0, 30.0, -30.0):
        before.q_t.mul_(0).add_(size)
        out, lse = torch.empty_like(c.q_t), torch.empty(80, Hq, T, device="cuda")
        call(ta, before, None, o[0], o[1], ws=ws[0])
        call(ta, c, None, out, lse, ws=ws[1])  # the next kernel
        first = first or (out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), size
