"""fp64 definitions of the KV-cache operators, one row and head at a time.

Test infrastructure only.  A cache is given by its pools [pages][Hkv][page][D]
(float64), page table [B][n] and lens [B]; slot j of row b is row j % page of
page table[b][j // page], and a page outside the pool is rows of zeros.
"""
from __future__ import annotations

import numpy as np


def slots(pool, table_row, n, hk):
    """The first n slots of a row for one head: [n][D]."""
    P, _, page, D = pool.shape
    out = np.zeros((n, D))
    for j in range(0, n, page):
        p, end = int(table_row[j // page]), min(n, j + page)
        if 0 <= p < P:
            out[j:end] = pool[p, hk, : end - j]
    return out


def ancestors(parents, T):
    """keep[t][x]: node x is t or an ancestor of t; a parent outside [-1, t)
    counts as -1; parents None is the chain."""
    keep = np.zeros((T, T), dtype=bool)
    for t in range(T):
        p = t - 1 if parents is None else int(parents[t])
        if 0 <= p < t:
            keep[t] = keep[p]
        keep[t, t] = True
    return keep


def _modded(s, softcap):
    return softcap * np.tanh(s / softcap) if softcap else s


def tree_attention(q, k_new, v_new, k, v, table, lens, parents, counts, scale, softcap=None):
    """O, LSE and sum_j P_ij |v_j| (the size that rounding errors of P scale
    with); rows t >= counts[b] are NaN."""
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    O, A = np.full((B, Hq, T, D), np.nan), np.full((B, Hq, T, D), np.nan)
    L = np.full((B, Hq, T), np.nan)
    for b in range(B):
        n, c = int(lens[b]), T if counts is None else int(counts[b])
        keep = ancestors(None if parents is None else parents[b], T)
        for hk in range(Hkv):
            kk, vv = slots(k, table[b], n, hk), slots(v, table[b], n, hk)
            for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                for t in range(c):
                    ks, vs = kk, vv
                    if k_new is not None:
                        ks, vs = np.concatenate([kk, k_new[b, hk][keep[t]]]), np.concatenate([vv, v_new[b, hk][keep[t]]])
                    if len(ks) == 0:
                        O[b, h, t], A[b, h, t], L[b, h, t] = 0.0, 0.0, -np.inf
                        continue
                    s = _modded(ks @ q[b, h, t] * scale, softcap)
                    m = s.max()
                    p = np.exp(s - m)
                    L[b, h, t] = m + np.log(p.sum())
                    p /= p.sum()
                    O[b, h, t], A[b, h, t] = p @ vs, p @ np.abs(vs)
    return O, L, A


def append(k_new, v_new, k, v, table, lens, path, counts, positions=None, seen=None):
    """Writes k, v (and positions) in place; returns the new lens."""
    P, Hkv, page, _ = k.shape
    B, _, T, _ = k_new.shape
    cap = table.shape[1] * page
    out = np.array(lens)
    for b in range(B):
        c = T if counts is None else int(counts[b])
        for i in range(c):
            slot, node = int(lens[b]) + i, i if path is None else int(path[b][i])
            if slot >= cap or not 0 <= node < T:
                continue
            if positions is not None:
                positions[b, :, slot] = (int(lens[b]) if seen is None else int(seen[b])) + i
            p = int(table[b][slot // page])
            if 0 <= p < P:
                k[p, :, slot % page], v[p, :, slot % page] = k_new[b, :, node], v_new[b, :, node]
        out[b] = min(int(lens[b]) + c, cap)
    return out


def slot_weights(q, lse, k, table, lens, w_in, path, counts, scale, softcap=None):
    """The new totals and what this call added; entries behind lens[b] are NaN."""
    B, Hq, T, _ = q.shape
    P, Hkv, page, _ = k.shape
    cap = table.shape[1] * page
    w, add = np.full((B, Hkv, cap), np.nan), np.full((B, Hkv, cap), np.nan)
    for b in range(B):
        n = int(lens[b])
        c = min(T if counts is None else int(counts[b]), n)
        for hk in range(Hkv):
            kk = slots(k, table[b], n, hk)
            base = np.zeros(n)
            if w_in is not None:
                base[: n - c] = w_in[b, hk, : n - c]
            got = np.zeros(n)
            for i in range(c):
                node = i if path is None else int(path[b][i])
                if not 0 <= node < T:
                    continue
                see = n - c + i + 1
                for h in range(hk * (Hq // Hkv), (hk + 1) * (Hq // Hkv)):
                    got[:see] += np.exp(_modded(kk[:see] @ q[b, h, node] * scale, softcap) - lse[b, h, node])
            w[b, hk, :n], add[b, hk, :n] = base + got, got
    return w, add


def evict_plan(weights, positions, seen, lens, budget, first, recent):
    """moves [B][Hkv][budget][2] and n_moves [B][Hkv]."""
    B, Hkv, _ = weights.shape
    moves, count = np.full((B, Hkv, budget, 2), -1, dtype=np.int64), np.zeros((B, Hkv), dtype=np.int64)
    for b in range(B):
        n = int(lens[b])
        if n <= budget:
            continue
        for h in range(Hkv):
            def value(j):
                if positions[b, h, j] < first or positions[b, h, j] >= int(seen[b]) - recent:
                    return (0, 0.0, j)
                x = float(weights[b, h, j])
                return (2, 0.0, j) if np.isnan(x) else (1, -x, j)
            kept = set(sorted(range(n), key=value)[:budget])
            to = [j for j in range(budget) if j not in kept]
            frm = [j for j in range(budget, n) if j in kept]
            assert len(to) == len(frm)
            count[b, h] = len(to)
            moves[b, h, : len(to), 0], moves[b, h, : len(to), 1] = to, frm
    return moves, count


def compact(moves, n_moves, budget, k, v, table, lens, weights=None, positions=None):
    """In place; returns the new lens."""
    page = k.shape[2]
    row = lambda b, j: (int(table[b][j // page]), j % page)  # noqa: E731
    for b, h in np.ndindex(*n_moves.shape):
        for to, frm in moves[b, h, : int(n_moves[b, h])]:
            (p, r), (p2, r2) = row(b, int(to)), row(b, int(frm))
            k[p, h, r], v[p, h, r] = k[p2, h, r2], v[p2, h, r2]
            for x in (weights, positions):
                if x is not None:
                    x[b, h, to] = x[b, h, frm]
    return np.minimum(lens, budget)
