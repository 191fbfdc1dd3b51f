"""The serving operators on a paged KV cache, as cases to measure.

A cache holds K and V rows in pages: pools [pages][Hkv][page_size][D] bf16, a page table [B][pages of a row] and the
number of filled slots of each batch row.  Five operators work on it:

  tree     attention of T drafted tokens (a tree, given by parents) over the cache and over their own ancestors
  append   the accepted tokens' K and V rows go into the next slots
  weights  the attention weight that each cached key received is added to its running total
  plan     which slots to evict so that `budget` remain, and the moves that close the gaps
  compact  those moves, applied to K, V, the totals and the positions

The plain forms are elementary torch operations in 32 bits; `exact` is written from the definitions in 64 bits, one
batch row and head at a time.
"""
import math

import torch

own = False


def listed():
    return [
        # one new token for one short conversation: nothing but latency
        dict(name="tree_token_short", op="tree", B=1, Hq=32, Hkv=8, D=128, T=1, lo=500, hi=500, page=64),
        # a draft tree of 16 nodes for 8 conversations of uneven length
        dict(name="tree_draft16", op="tree", B=8, Hq=32, Hkv=8, D=128, T=16, lo=517, hi=4099, page=64),
        # one conversation of 100 thousand tokens: all SMs share one row's keys
        dict(name="tree_token_long", op="tree", B=1, Hq=32, Hkv=8, D=128, T=1, lo=100001, hi=100001, page=128),
        # the largest: 64 conversations, small drafts, the whole cache read once
        dict(name="tree_batch64", op="tree", B=64, Hq=32, Hkv=8, D=128, T=4, lo=4096, hi=16000, page=64),
        # 64-wide heads without sharing, small pages, odd draft length
        dict(name="tree_mha_d64", op="tree", B=6, Hq=16, Hkv=16, D=64, T=33, lo=130, hi=3001, page=16),
        # weights after a draft was accepted in part, keys read once
        dict(name="weights_accepted", op="weights", B=16, Hq=32, Hkv=8, D=128, T=8, lo=900, hi=8191, page=64, path=True),
        # weights of a whole prompt, from the prompt's own attention
        dict(name="weights_prompt", op="weights", B=2, Hq=32, Hkv=8, D=128, T=4096, lo=4096, hi=4096, page=128, path=False),
        # eviction of a few new slots in a short cache
        dict(name="plan_step", op="plan", B=4, Hkv=8, lo=1088, hi=1088, budget=1024, first=4, recent=128, page=64),
        # halving long caches
        dict(name="plan_halve", op="plan", B=4, Hkv=8, lo=30011, hi=65000, budget=16384, first=4, recent=512, page=128),
        # the moves of a halving in a batch
        dict(name="compact_halve", op="compact", B=16, Hkv=8, D=128, lo=6000, hi=8192, budget=4096, first=4, recent=256,
             page=64),
        # accepted nodes of a draft
        dict(name="append_accepted", op="append", B=16, Hkv=8, D=128, T=16, lo=300, hi=4000, page=64, path=True),
        # a long prompt
        dict(name="append_prompt", op="append", B=4, Hkv=8, D=128, T=8000, lo=0, hi=100, page=64, path=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "weights", "weights", "plan", "compact", "append"])
    page = rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    if op == "tree":
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        T = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 100)])
        B = _log(rng, 1, 64)
        hi = _log(rng, 16, max(32, min(120000, 600000 // (B * Hkv) * 8, 100_000_000 // (B * T * G * Hkv))))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, T=T, lo=rng.randint(0, hi), hi=hi, page=page)
    if op == "weights":
        G = rng.choice([1, 2, 3, 4, 7, 8])
        if rng.random() < 0.4:
            T = _log(rng, 64, 4096)
            B = rng.choice([1, 2])
            return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, T=T, lo=T, hi=T + rng.choice([0, rng.randint(1, 500)]), page=page,
                        path=False)
        T, B = _log(rng, 1, 64), _log(rng, 1, 32)
        hi = _log(rng, 2 * T + 16, max(2 * T + 32, min(60000, 400000 // (B * Hkv) * 4, 60_000_000 // (B * T * G * Hkv))))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, T=T, lo=rng.randint(T, hi), hi=hi, page=page, path=True)
    if op == "append":
        B, path = _log(rng, 1, 32), rng.random() < 0.5
        T = _log(rng, 1, 64) if path else _log(rng, 16, max(32, 32000 // B))
        return dict(op=op, B=B, Hkv=Hkv, D=D, T=T, lo=0, hi=rng.randint(1, 3000), page=page, path=path)
    B = _log(rng, 1, 16)
    hi = _log(rng, 64, max(128, (1000000 if op == "plan" else 400000) // (B * Hkv)))
    budget = rng.randint(max(2, hi // 4), hi - 1)
    c = dict(op=op, B=B, Hkv=Hkv, lo=rng.randint(max(1, budget // 2), hi), hi=hi, budget=budget, first=rng.choice([0, 4]),
             recent=rng.randint(0, budget // 4), page=page)
    return c if op == "plan" else dict(c, D=D)


# ------------------------------------------------------------------ inputs


def _lens(case):
    """The filled slots of each batch row: evenly spread over the case's range (the seed orders them)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (hi - lo) * b // max(1, B - 1) for b in range(B)]


def _counts(case):
    """How many of the T new tokens of each batch row are real (or accepted)."""
    B, T = case["B"], case["T"]
    if case["op"] == "tree":
        return [max(1, T - (7 * b) % (T // 4 + 1)) for b in range(B)]
    return [1 + (5 * b + T // 2) % T for b in range(B)] if case["path"] else [T] * B


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, B, Hkv, page = case["op"], case["B"], case["Hkv"], case["page"]
    D, T = case.get("D", 64), case.get("T", 0)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    order = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(_lens(case), device=dev, dtype=torch.int32)[order].contiguous()
    top = case["hi"] + (T if op == "append" else 0)
    n_tab = -(-top // page)
    n_pages = B * n_tab + 3
    room = lens + (T if op == "append" else 0)
    table = torch.randperm(n_pages, generator=g, device=dev)[: B * n_tab].view(B, n_tab).to(torch.int32)
    # entries behind a row's last page name no page
    used = torch.arange(n_tab, device=dev)[None, :] * page < room[:, None]
    table = torch.where(used, table, torch.full_like(table, -1)).contiguous()
    st = dict(case=case, lens=lens, table=table, page=page, B=B, Hkv=Hkv)
    if op != "plan":
        # keys share a direction with the queries, some much more than others, so that a few keys draw most weight
        u = rnd(Hkv, 1, D)
        pool = rnd(n_pages, Hkv, page, D)
        pool += 0.3 * rnd(n_pages, Hkv, page, 1) * u
        st["k"] = pool.to(torch.bfloat16)
        pool.normal_(generator=g)
        st["v"] = pool.to(torch.bfloat16)
        del pool
    if op in ("tree", "weights", "append"):
        counts = torch.tensor(_counts(case), device=dev, dtype=torch.int32)[order].contiguous()
        st["counts"] = counts
    if op in ("tree", "append"):
        st["k_new"] = (rnd(B, Hkv, T, D) + 0.3 * rnd(B, Hkv, T, 1) * u).to(torch.bfloat16)
        st["v_new"] = rnd(B, Hkv, T, D).to(torch.bfloat16)
    if op in ("weights", "append") and case["path"]:
        # the accepted nodes of each tree, ascending
        picked = torch.argsort(torch.rand(B, T, generator=g, device=dev), dim=1)
        n = torch.arange(T, device=dev)
        picked = torch.where(n[None, :] < counts[:, None], picked, torch.full_like(picked, T))
        picked = torch.sort(picked, dim=1).values
        st["path"] = torch.where(picked < T, picked, torch.zeros_like(picked)).to(torch.int32).contiguous()
    if op in ("tree", "weights"):
        Hq = case["Hq"]
        G = Hq // Hkv
        q = rnd(B, Hkv, G, T, D) + 0.5 * u[None, :, None]
        st["q"] = q.reshape(B, Hq, T, D).to(torch.bfloat16)
        st["scale"] = D ** -0.5
    if op == "tree":
        t = torch.arange(T, device=dev)
        par = t[None, :] - 1 - (torch.rand(B, T, generator=g, device=dev) * 4).to(torch.int64)
        st["parents"] = par.clamp(min=-1).to(torch.int32).contiguous()
        st["out"] = torch.zeros(B, Hq, T, D, dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.zeros(B, Hq, T, dtype=torch.float32, device=dev)
    if op == "weights":
        w = torch.rand(B, Hkv, n_tab * page, generator=g, device=dev) * 3
        st["w_in"], st["w_out"] = w, w.clone()
        scores, seen = _scores_seen(st)
        rows = torch.logsumexp(scores.masked_fill(~seen, -math.inf), -1)  # [B, Hkv, G, T] in the order of the path
        lse = torch.zeros(B, Hkv, G, T, device=dev)
        node = st["path"].to(torch.int64) if case["path"] else torch.arange(T, device=dev).expand(B, T)
        real = torch.arange(T, device=dev)[None, :] < counts[:, None]
        # rows that were not accepted keep some other value
        node = torch.where(real, node, torch.full_like(node, T))
        lse = torch.nn.functional.pad(lse, (0, 1)).scatter(3, node[:, None, None, :].expand(B, Hkv, G, T), rows)[..., :T]
        st["lse"] = lse.reshape(B, Hq, T).contiguous()
        del scores, seen, rows
    if op in ("plan", "compact"):
        cap = n_tab * page
        # running totals: heavy-tailed, and some keys that nothing ever looked at (ties)
        w = torch.exp(1.5 * rnd(B, Hkv, cap))
        st["weights"] = torch.where(torch.rand(B, Hkv, cap, generator=g, device=dev) < 0.05, torch.zeros_like(w), w)
        # earlier evictions left gaps and moved rows below the budget; what came after is in order
        seen_tok = lens.to(torch.int64) + 1000
        slot = torch.arange(cap, device=dev)
        old = torch.argsort(torch.rand(B, Hkv, case["budget"], generator=g, device=dev), dim=-1)
        pos = (slot[None, :] + (seen_tok - lens)[:, None])[:, None, :].expand(B, Hkv, cap).clone()
        pos[..., : min(cap, case["budget"])] = old[..., :cap]
        st["positions"] = pos.to(torch.int32).contiguous()
        st["seen"] = seen_tok.to(torch.int32)
        st["moves"] = torch.empty(B, Hkv, case["budget"], 2, dtype=torch.int32, device=dev)
        st["n_moves"] = torch.empty(B, Hkv, dtype=torch.int32, device=dev)
    if op == "compact":
        st["moves"], st["n_moves"] = _plan(st)
    if op == "append":
        st["positions"] = torch.full((B, Hkv, n_tab * page), -1, dtype=torch.int32, device=dev)
        st["seen"] = lens + 77
        st["lens_out"] = torch.empty_like(lens)
    if own:
        import tiled_attention_25_b200 as ta

        if op == "plan":  # reads no K or V: the smallest pool that has the table's pages
            st["k"] = st["v"] = torch.zeros(n_pages, Hkv, page, 64, dtype=torch.bfloat16, device=dev)
        st["cache"] = ta.AttnCache(st["k"], st["v"], lens, table)
        if op == "tree":
            st["ws"] = ta.new_tree_workspace(case["Hq"], Hkv, T, D, device=dev)
    return st


# ------------------------------------------------------------------ plain forms


def _gather(st, pool):
    """Pool rows in slot order: [B, Hkv, slots of the table, D] in 32 bits."""
    slot = torch.arange(st["table"].shape[1] * st["page"], device=pool.device)
    pages = st["table"].to(torch.int64).clamp(min=0)[:, slot // st["page"]]
    return pool[pages[:, None, :], torch.arange(st["Hkv"], device=pool.device)[None, :, None], (slot % st["page"])[None, None, :]].float()


def _tree(st):
    q, k_new, v_new, lens, counts = st["q"], st["k_new"], st["v_new"], st["lens"], st["counts"]
    B, Hq, T, D = q.shape
    Hkv = st["Hkv"]
    dev = q.device
    t = torch.arange(T, device=dev)
    # the ancestors of each node: (1 - P)^-1 = 1 + P + P^2 + ..., P the parent matrix; its entries are 0 and 1
    P = (st["parents"][:, :, None] == t[None, None, :]).float()
    eye = torch.eye(T, device=dev).expand(B, T, T)
    above = torch.linalg.solve_triangular(eye - P, eye, upper=False, unitriangular=True) > 0.5
    k = torch.cat([_gather(st, st["k"]), k_new.float()], 2)
    cap = k.shape[2] - T
    s = torch.matmul(q.float().view(B, Hkv, -1, D), k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, T, cap + T) * st["scale"]
    del k
    slots = (torch.arange(cap, device=dev)[None, :] < lens[:, None])[:, None, :].expand(B, T, cap)
    keep = torch.cat([slots, above], 2)[:, None, None]
    s = s.masked_fill_(~keep, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp_(s - m)
    l = p.sum(-1, keepdim=True)
    v = torch.cat([torch.where((torch.arange(cap, device=dev)[None, :] < lens[:, None])[:, None, :, None], _gather(st, st["v"]), 0.0), v_new.float()], 2)
    o = torch.matmul(p.view(B, Hkv, -1, cap + T), v).view(B, Hkv, Hq // Hkv, T, D) / l
    lse = (m + torch.log(l))[..., 0]
    real = (t[None, :] < counts[:, None])[:, None, :]
    out = torch.where(real[..., None], o.reshape(B, Hq, T, D), 0.0).to(torch.bfloat16)
    return {"out": out, "lse": torch.where(real, lse.reshape(B, Hq, T), 0.0)}


def _scores_seen(st):
    """Scores of the accepted queries [B, Hkv, G, T, slots] (in the order of the path), and which slots each sees."""
    q, lens, counts = st["q"], st["lens"], st["counts"]
    B, Hq, T, D = q.shape
    Hkv = st["Hkv"]
    if "path" in st:
        q = torch.gather(q, 2, st["path"].to(torch.int64)[:, None, :, None].expand(B, Hq, T, D))
    k = _gather(st, st["k"])
    s = torch.matmul(q.float().view(B, Hkv, -1, D), k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, T, -1) * st["scale"]
    i = torch.arange(T, device=q.device)
    end = torch.where(i[None, :] < counts[:, None], (lens - counts)[:, None] + i[None, :] + 1, 0)
    seen = (torch.arange(s.shape[-1], device=q.device)[None, None, :] < end[:, :, None])[:, None, None]
    return s, seen


def _weights(st):
    s, seen = _scores_seen(st)
    lse, lens, counts = st["lse"], st["lens"], st["counts"]
    B, Hq, T = lse.shape
    if "path" in st:
        lse = torch.gather(lse, 2, st["path"].to(torch.int64)[:, None, :].expand(B, Hq, T))
    s -= lse.view(B, st["Hkv"], -1, T, 1)
    got = torch.exp_(s.masked_fill_(~seen, -math.inf)).sum((2, 3))
    slot = torch.arange(got.shape[-1], device=s.device)[None, :]
    before = torch.where((slot < (lens - counts)[:, None])[:, None, :], st["w_in"], 0.0)
    return {"weights": torch.where((slot < lens[:, None])[:, None, :], before + got, st["w_in"])}


def _plan(st):
    case, w, pos, lens, seen = st["case"], st["weights"], st["positions"], st["lens"], st["seen"]
    budget = case["budget"]
    cap = w.shape[-1]
    slot = torch.arange(cap, device=w.device)
    valid = (slot[None, :] < lens[:, None])[:, None, :].expand_as(w)
    kept_by_age = (pos < case["first"]) | (pos >= (seen - case["recent"])[:, None, None])
    order = torch.argsort(w, dim=-1, descending=True, stable=True)
    cls = torch.where(valid, torch.where(kept_by_age, 2, 1), 0)
    order = torch.gather(order, -1, torch.argsort(torch.gather(cls, -1, order), dim=-1, descending=True, stable=True))
    kept = torch.zeros_like(valid).scatter(-1, order, (slot < budget).expand_as(valid)) & valid
    low = slot < budget
    hole, extra = ~kept & valid & low, kept & ~low
    n = torch.where((lens > budget)[:, None], hole.sum(-1), 0)
    dst = torch.argsort(hole.to(torch.int32), dim=-1, descending=True, stable=True)
    src = torch.argsort(extra.to(torch.int32), dim=-1, descending=True, stable=True)
    moves = torch.nn.functional.pad(torch.stack([dst, src], -1), (0, 0, 0, max(0, budget - cap)))[:, :, :budget]
    moves = torch.where((torch.arange(budget, device=w.device) < n[..., None])[..., None], moves, -1)
    return moves.to(torch.int32).contiguous(), n.to(torch.int32)


def _place(st, slot):
    """The page and the row in it of slots [B, n]."""
    return torch.gather(st["table"].to(torch.int64), 1, slot // st["page"]), slot % st["page"]


def _compact(st):
    budget = st["case"]["budget"]
    b, h, i = torch.nonzero(torch.arange(budget, device=st["lens"].device) < st["n_moves"][..., None], as_tuple=True)
    dst, src = st["moves"][b, h, i].to(torch.int64).unbind(-1)
    row = lambda slot: (st["table"][b, slot // st["page"]].to(torch.int64), h, slot % st["page"])  # noqa: E731
    to, at = row(dst), row(src)
    st["k"][to] = st["k"][at]
    st["v"][to] = st["v"][at]
    st["weights"][b, h, dst] = st["weights"][b, h, src]
    st["positions"][b, h, dst] = st["positions"][b, h, src]
    st["lens"].clamp_(max=budget)
    return {n: st[n] for n in ("k", "v", "weights", "positions", "lens")}


def _append(st):
    lens, counts, k_new = st["lens"], st["counts"], st["k_new"]
    B, Hkv, T, D = k_new.shape
    b, i = torch.nonzero(torch.arange(T, device=lens.device)[None, :] < counts[:, None], as_tuple=True)
    node = st["path"][b, i].to(torch.int64) if "path" in st else i
    slot = lens[b].to(torch.int64) + i
    page = st["table"][b, slot // st["page"]].to(torch.int64)
    st["k"][page, :, slot % st["page"]] = k_new[b, :, node]
    st["v"][page, :, slot % st["page"]] = st["v_new"][b, :, node]
    st["positions"][b, :, slot] = (st["seen"][b] + i).to(torch.int32)[:, None]
    st["lens_out"].copy_(lens + counts)
    return {n: st[n] for n in ("k", "v", "positions", "lens_out")}


def _run_own(st):
    import tiled_attention_25_b200 as ta

    op, cache = st["case"]["op"], st["cache"]
    if op == "tree":
        ta.attn_tree_fwd(st["q"], st["k_new"], st["v_new"], cache, st["out"], st["lse"], st["ws"], parents=st["parents"],
                         counts=st["counts"], scale=st["scale"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "weights":
        ta.attn_cache_weights(st["q"], st["lse"], cache, st["w_in"], st["w_out"], path=st.get("path"), counts=st["counts"],
                              scale=st["scale"])
        return {"weights": st["w_out"]}
    if op == "plan":
        case = st["case"]
        ta.attn_evict_plan(cache, st["weights"], st["positions"], st["seen"], st["moves"], st["n_moves"], case["budget"],
                           first=case["first"], recent=case["recent"])
        return {"moves": st["moves"], "n_moves": st["n_moves"]}
    if op == "compact":
        ta.attn_cache_compact(cache, st["moves"], st["n_moves"], st["case"]["budget"], weights=st["weights"],
                              positions=st["positions"])
        return {n: st[n] for n in ("k", "v", "weights", "positions", "lens")}
    ta.attn_cache_append(cache, st["k_new"], st["v_new"], st["lens_out"], path=st.get("path"), counts=st["counts"],
                         positions=st["positions"], seen=st["seen"])
    return {n: st[n] for n in ("k", "v", "positions", "lens_out")}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "tree":
        return _tree(state)
    if op == "weights":
        return _weights(state)
    if op == "plan":
        moves, n = _plan(state)
        return {"moves": moves, "n_moves": n}
    return _compact(state) if op == "compact" else _append(state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op, B, Hkv, D = case["op"], case["B"], case["Hkv"], case.get("D", 0)
    lens, T = _lens(case), case.get("T", 0)
    if op == "tree":
        Hq, n = case["Hq"], _counts(case)
        rows = sum(n)
        by = 4 * D * Hkv * sum(lens) + rows * (4 * D * Hkv + 4 * D * Hq + 4 * Hq + 4) + 4 * len(lens)
        # each node sees the cache and itself at least
        return {"bytes": by, "flops": 4 * D * Hq * sum(c * (x + 1) for c, x in zip(n, lens))}
    if op == "weights":
        Hq, n = case["Hq"], _counts(case)
        by = 2 * D * Hkv * sum(lens) + sum(n) * (2 * D + 4) * Hq + 8 * Hkv * sum(lens)
        pairs = sum(c * (x - c) + c * (c + 1) // 2 for c, x in zip(n, lens))
        return {"bytes": by, "flops": 2 * D * Hq * pairs}
    if op == "append":
        rows = sum(_counts(case))
        return {"bytes": rows * Hkv * (8 * D + 4) + 8 * B, "flops": 0}
    # slots beyond the budget that stay: the recent ones, and their share of the rest
    budget, recent = case["budget"], case["recent"]
    moved = sum(min(budget, x - budget, recent + (x - budget) * (budget - recent) // x) for x in lens if x > budget)
    if op == "plan":
        return {"bytes": 8 * Hkv * sum(lens) + 8 * Hkv * B * budget, "flops": 0}
    return {"bytes": moved * Hkv * (2 * (4 * D + 8) + 8) + 8 * B, "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    op = case["op"]
    if op not in ("tree", "weights"):
        return None  # whole numbers and copies
    st = prepare(case, seed)
    q, lens = st["q"].double(), st["lens"].tolist()
    counts, table, page = st["counts"].tolist(), st["table"].tolist(), st["page"]
    B, Hq, T, D = q.shape
    G = Hq // st["Hkv"]
    if op == "tree":
        out, lse = torch.zeros_like(q), torch.zeros(B, Hq, T, dtype=torch.float64, device=q.device)
        parents = st["parents"].tolist()
    else:
        w = st["w_in"].double().clone()
        node = st["path"].tolist() if "path" in st else [list(range(T))] * B
    for b in range(B):
        n, used = lens[b], table[b][: -(-lens[b] // page)]
        if op == "tree":
            see = torch.zeros(T, T, dtype=torch.bool)
            for t in range(T):
                if parents[b][t] >= 0:
                    see[t] = see[parents[b][t]]
                see[t, t] = True
            see = see.to(q.device)
        for h in range(st["Hkv"]):
            k = torch.cat([st["k"][x, h] for x in used], 0)[:n].double() if used else q.new_zeros(0, D)
            if op == "tree":
                v = torch.cat([st["v"][x, h] for x in used], 0)[:n].double() if used else q.new_zeros(0, D)
                k, v = torch.cat([k, st["k_new"][b, h].double()]), torch.cat([v, st["v_new"][b, h].double()])
                c = counts[b]
                for f in range(h * G, (h + 1) * G):
                    s = q[b, f, :c] @ k.t() * st["scale"]
                    s[:, n:][~see[:c]] = -math.inf
                    lse[b, f, :c] = torch.logsumexp(s, 1)
                    out[b, f, :c] = torch.exp(s - lse[b, f, :c, None]) @ v
            else:
                c = counts[b]
                w[b, h, n - c : n] = 0
                ends = torch.arange(n - c + 1, n + 1, device=q.device)
                hidden = torch.arange(n, device=q.device)[None, :] >= ends[:, None]
                for f in range(h * G, (h + 1) * G):
                    s = q[b, f, node[b][:c]] @ k.t() * st["scale"]
                    p = torch.exp(s - st["lse"][b, f, node[b][:c]].double()[:, None])
                    w[b, h, :n] += p.masked_fill(hidden, 0.0).sum(0)
    return {"out": out, "lse": lse} if op == "tree" else {"weights": w}
