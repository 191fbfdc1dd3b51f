"""Seeded KV-cache problems: host fp64 copies for the oracle, device tensors
for the library, and the error bounds of the comparison."""
import numpy as np
import torch

import oracle
from synth_inputs import bf16_bits, bf16_bits_to_f64


def bf16(x):
    """x rounded to bf16: (bits, the rounded values in float64)."""
    bits = bf16_bits(np.ascontiguousarray(x, dtype=np.float32))
    return bits, bf16_bits_to_f64(bits)


def dev16(bits):
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda()


def i32(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def random_tree(rng, B, T, back=4):
    t = np.arange(T)
    return np.maximum(-1, t[None, :] - 1 - rng.integers(0, back, size=(B, T))).astype(np.int32)


class CacheCase:
    """A cache of B rows with lens filled slots, and T new tokens.  Everything
    that no call may use is NaN: rows behind lens, pages of no row, new tokens
    from counts[b] on (in K and V)."""

    def __init__(self, seed, lens, Hq, Hkv, D, page, T=1, counts=None, spare=2, room=0, storage="head", scale=None):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, dtype=np.int32)
        B = self.B = len(self.lens)
        self.Hq, self.Hkv, self.D, self.page, self.T = Hq, Hkv, D, page, T
        self.counts = None if counts is None else np.asarray(counts, dtype=np.int32)
        n = max(1, -(-(int(self.lens.max()) + room) // page))
        P = B * n + spare
        self.table = rng.permutation(P)[: B * n].reshape(B, n).astype(np.int32)
        self.cap = n * page
        self.scale = D ** -0.5 if scale is None else scale
        for name in ("k", "v"):
            pool = np.full((P, Hkv, page, D), np.nan, dtype=np.float32)
            for b in range(B):
                for j in range(0, int(self.lens[b]), page):
                    m = min(page, int(self.lens[b]) - j)
                    pool[self.table[b, j // page], :, :m] = rng.standard_normal((Hkv, m, D))
            bits, f64 = bf16(pool)
            setattr(self, name + "_bits", bits)
            setattr(self, name, f64)
        # entries behind a row's last page name no page, or any page
        for b in range(B):
            used = -(-(int(self.lens[b]) + room) // page)
            self.table[b, used:] = rng.choice([-1, 1 << 30, 0], size=n - used)
        for name, H in (("q", Hq), ("k_new", Hkv), ("v_new", Hkv)):
            x = rng.standard_normal((B, H, T, D)).astype(np.float32)
            if self.counts is not None and name != "q":
                for b in range(B):
                    x[b, :, self.counts[b]:] = np.nan
            bits, f64 = bf16(x)
            setattr(self, name + "_t", dev16(bits))
            setattr(self, name, f64)
        self.storage = storage
        self.load()

    def load(self):
        """(Re)load the device pools from the host copies."""
        import tiled_attention_25_b200 as ta
        def pool(bits):
            t = dev16(bits)
            if self.storage == "row":  # [page][row][head][D] storage
                t = t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            return t
        self.k_t, self.v_t = pool(self.k_bits), pool(self.v_bits)
        self.lens_t, self.table_t = i32(self.lens), i32(self.table)
        self.cache = ta.AttnCache(self.k_t, self.v_t, self.lens_t, self.table_t)


# A row's O is sum_j P_ij v_j / l with P_ij rounded to bf16 (half a step, 2^-8
# relative) before the product, the result rounded to bf16 once more; the
# fp32 arithmetic between (scores of size up to ~8 in the exponent, 2^-24
# relative each way, the softcap's tanh to 3e-7 of a cap of 20) stays below
# 1e-4 of sum_j P_ij |v_j|.
def o_bound(o_ref, size_ref):
    return 2.0 ** -8 * (1 + 2.0 ** -7) * (size_ref + np.abs(o_ref)) + 1e-4 * size_ref


# fp32 scores: 128 products of magnitude up to ~16 in all, accumulated in fp32
LSE_BOUND = 1e-4


def check_tree(out, lse, ref, what=""):
    O, L, A = ref
    sel = ~np.isnan(O)
    o = out.float().cpu().double().numpy()
    assert np.isfinite(o[sel]).all(), f"{what}: {np.sum(~np.isfinite(o[sel]))} values of O are not finite"
    over = np.abs(o[sel] - O[sel]) - o_bound(O[sel], A[sel])
    assert over.size == 0 or over.max() <= 0, f"{what}: O off its bound by {over.max():.3e}"
    if lse is not None:
        got, want = lse.cpu().double().numpy(), L
        sel = ~np.isnan(want)
        inf = np.isneginf(want) & sel
        assert np.array_equal(np.isneginf(got) & sel, inf), f"{what}: LSE of empty rows"
        d = np.abs(got[sel & ~inf] - want[sel & ~inf])
        assert d.size == 0 or d.max() <= LSE_BOUND, f"{what}: LSE off by {d.max():.3e}"


def tree_reference(c, parents, with_new=True, softcap=None):
    # the oracle must not see the NaN that no query may use: the ancestors of real nodes are real
    return oracle.cache.tree_attention(c.q, c.k_new if with_new else None, c.v_new if with_new else None, c.k, c.v, c.table,
                                       c.lens, parents, c.counts, c.scale, softcap)
