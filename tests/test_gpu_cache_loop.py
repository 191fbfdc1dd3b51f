"""The cache operators together, as a server uses them: a prompt, then rounds of
drafting, attending, accepting, totalling and evicting, against fp64."""
import numpy as np
import pytest
import torch

import oracle
from cache_common import bf16, check_tree, dev16, i32, random_tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,Hq,Hkv,page", [(128, 8, 2, 64), (64, 6, 6, 16)])
def test_serving_rounds(D, Hq, Hkv, page):
    import tiled_attention_25_b200 as ta
    rng = np.random.default_rng(D)
    B, S, T, cap, budget, first, recent = 2, 192, 6, 256, 200, 2, 32
    scale = D ** -0.5
    draw = lambda H, n: bf16(rng.standard_normal((B, H, n, D)))  # noqa: E731
    cache = ta.new_attn_cache(B, Hkv, cap, D, page_size=page)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    n_pages = cache.k.shape[0]
    k, v = (np.full((n_pages, Hkv, page, D), np.nan) for _ in range(2))
    table = np.arange(n_pages).reshape(B, -1)
    lens = np.zeros(B, dtype=np.int64)
    w_t, pos_t = torch.zeros(B, Hkv, cap, device="cuda"), torch.full((B, Hkv, cap), -1, dtype=torch.int32, device="cuda")
    pos = np.full((B, Hkv, cap), -1)
    seen = np.zeros(B, dtype=np.int64)
    ws = ta.new_tree_workspace(Hq, Hkv, T, D)
    moves = torch.empty(B, Hkv, budget, 2, dtype=torch.int32, device="cuda")
    n_moves = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")

    # the prompt: causal attention of the whole, its rows into the cache, its weights
    (qb, q), (kb, kn), (vb, vn) = draw(Hq, S), draw(Hkv, S), draw(Hkv, S)
    q_t, k_t, v_t = dev16(qb), dev16(kb), dev16(vb)
    out, lse = torch.empty_like(q_t), torch.empty(B, Hq, S, device="cuda")
    ta.attn_fwd(q_t, k_t, v_t, out, lse, scale=scale, mod_kind=ta.MOD_CAUSAL)
    ta.attn_cache_append(cache, k_t, v_t, positions=pos_t, seen=i32(seen))
    ta.attn_cache_weights(q_t, lse, cache, None, w_t, scale=scale)
    lens = oracle.cache.append(kn, vn, k, v, table, lens, None, None, pos, seen)
    seen += S
    w, _ = oracle.cache.slot_weights(q, lse.cpu().double().numpy(), k, table, lens, None, None, None, scale)
    live = ~np.isnan(w)
    # attn_fwd's LSE is good to 1e-3, and every weight follows it; the oracle was given the same LSE
    assert np.abs(w_t.cpu().double().numpy() - w)[live].max() <= 1e-4 * np.abs(w[live]).max()

    evicted = 0
    for step in range(20):
        (qb, q), (kb, kn), (vb, vn) = draw(Hq, T), draw(Hkv, T), draw(Hkv, T)
        q_t, k_t, v_t = dev16(qb), dev16(kb), dev16(vb)
        parents = random_tree(rng, B, T)
        counts = rng.integers(1, T + 1, size=B)
        out, lse = torch.zeros_like(q_t), torch.zeros(B, Hq, T, device="cuda")
        ta.attn_tree_fwd(q_t, k_t, v_t, cache, out, lse, ws, parents=i32(parents), counts=i32(counts), scale=scale)
        torch.cuda.synchronize()
        check_tree(out, lse, oracle.cache.tree_attention(q, kn, vn, k, v, table, lens, parents, counts, scale), f"step {step}")
        # accept the path to a random node
        path, accepted = np.zeros((B, T), dtype=np.int64), np.zeros(B, dtype=np.int64)
        for b in range(B):
            node, up = int(rng.integers(0, counts[b])), []
            while node >= 0:
                up.append(node)
                node = int(parents[b, node])
            accepted[b] = len(up)
            path[b, : len(up)] = up[::-1]
        p_t, a_t, seen_t = i32(path), i32(accepted), i32(seen)
        ta.attn_cache_append(cache, k_t, v_t, path=p_t, counts=a_t, positions=pos_t, seen=seen_t)
        ta.attn_cache_weights(q_t, lse, cache, w_t, w_t, path=p_t, counts=a_t, scale=scale)
        lens = oracle.cache.append(kn, vn, k, v, table, lens, path, accepted, pos, seen)
        seen = seen + accepted
        w2, _ = oracle.cache.slot_weights(q, lse.cpu().double().numpy(), k, table, lens, np.nan_to_num(w), path, accepted, scale)
        got = w_t.cpu().double().numpy()
        live = ~np.isnan(w2)
        assert np.abs(got - w2)[live].max() <= 1e-4 * np.abs(w2[live]).max()
        # the accepted tokens are a path: the LSE that the tree gave them is the one over the slots they see
        mass = got.copy()
        mass[~live] = 0
        w = np.where(live, got, np.nan)  # carry the library's own totals on, so that the plans are comparable bit for bit
        ta.attn_evict_plan(cache, w_t, pos_t, i32(seen), moves, n_moves, budget, first, recent)
        ta.attn_cache_compact(cache, moves, n_moves, budget, weights=w_t, positions=pos_t)
        want, wn = oracle.cache.evict_plan(w, pos, seen, lens, budget, first, recent)
        torch.cuda.synchronize()
        assert np.array_equal(moves.cpu().numpy(), want) and np.array_equal(n_moves.cpu().numpy(), wn)
        lens = oracle.cache.compact(want, wn, budget, k, v, table, lens, w, pos)
        evicted += int(wn.sum())
        assert np.array_equal(cache.lens.cpu().numpy(), lens)
        assert np.array_equal(cache.k.float().cpu().double().numpy(), k, equal_nan=True)
        for b in range(B):
            n = int(lens[b])
            assert np.array_equal(pos_t.cpu().numpy()[b, :, :n], pos[b, :, :n])
            # the newest tokens are always there
            for h in range(Hkv):
                if n == budget:
                    assert set(range(int(seen[b]) - recent, int(seen[b]))) <= set(pos[b, h, :n].tolist())
    assert evicted > 0 and (lens == budget).all()
    assert ta.attn_get_status() == 0


def test_a_captured_round_replays_like_the_eager_one():
    """One decode round, all operators in place, as a graph: replays advance the
    cache exactly as the same calls do eagerly."""
    import tiled_attention_25_b200 as ta
    B, Hq, Hkv, D, T, budget = 2, 8, 2, 64, 4, 40
    rng = np.random.default_rng(5)
    tokens = [dev16(bf16(rng.standard_normal((B, Hq, T, D)))[0]) for _ in range(3)]
    k_new, v_new = (dev16(bf16(rng.standard_normal((B, Hkv, T, D)))[0]) for _ in range(2))
    path, accepted = i32([[0, 2, 3, 0], [0, 1, 0, 0]]), i32([3, 2])
    parents = i32([[-1, 0, 0, 2], [-1, 0, 1, 1]])

    def setup():
        cache = ta.new_attn_cache(B, Hkv, 64, D, page_size=16)
        cache.k.zero_()
        cache.v.zero_()
        st = dict(cache=cache, q=torch.empty_like(tokens[0]), out=torch.zeros_like(tokens[0]),
                  lse=torch.zeros(B, Hq, T, device="cuda"), w=torch.zeros(B, Hkv, 64, device="cuda"),
                  pos=torch.zeros(B, Hkv, 64, dtype=torch.int32, device="cuda"), seen=i32([0, 0]),
                  moves=torch.zeros(B, Hkv, budget, 2, dtype=torch.int32, device="cuda"),
                  n=torch.zeros(B, Hkv, dtype=torch.int32, device="cuda"), ws=ta.new_tree_workspace(Hq, Hkv, T, D))
        return st

    def step(s):
        ta.attn_tree_fwd(s["q"], k_new, v_new, s["cache"], s["out"], s["lse"], s["ws"], parents=parents)
        ta.attn_cache_append(s["cache"], k_new, v_new, path=path, counts=accepted, positions=s["pos"], seen=s["seen"])
        ta.attn_cache_weights(s["q"], s["lse"], s["cache"], s["w"], s["w"], path=path, counts=accepted)
        s["seen"] += accepted
        ta.attn_evict_plan(s["cache"], s["w"], s["pos"], s["seen"], s["moves"], s["n"], budget, 1, 8)
        ta.attn_cache_compact(s["cache"], s["moves"], s["n"], budget, weights=s["w"], positions=s["pos"])

    eager, captured = setup(), setup()
    warm = setup()
    warm["q"].copy_(tokens[0])
    step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(captured)
    for i in range(24):
        for s in (eager, captured):
            s["q"].copy_(tokens[i % 3])
        step(eager)
        g.replay()
        torch.cuda.synchronize()
        for name in ("out", "lse", "w", "pos", "seen", "moves", "n"):
            assert torch.equal(eager[name], captured[name]), (i, name)
        for name in ("k", "v", "lens"):
            assert torch.equal(getattr(eager["cache"], name), getattr(captured["cache"], name)), (i, name)
    assert (eager["cache"].lens == budget).all() and ta.attn_get_status() == 0
