"""Argument checks of the cache entry points, before any GPU work: a valid call
gets as far as the device lookup (ATTN_ERR_DEVICE here, with no GPU)."""
import ctypes

import pytest
import torch

import tiled_attention_25_b200 as ta
from tiled_attention_25_b200 import abi

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where nothing can be launched")

GOOD = ctypes.c_void_p(1 << 32)
ODD4, ODD16 = ctypes.c_void_p((1 << 32) + 2), ctypes.c_void_p((1 << 32) + 8)
DEVICE, ARG, UNSUPPORTED, ALIGN, WORKSPACE = -7, -1, -2, -3, -4


def cache(**kw):
    f = dict(k=GOOD.value, v=GOOD.value, k_strides=abi.CStrides(8192, 8192, 128), v_strides=abi.CStrides(8192, 8192, 128),
             page_table=GOOD.value, lens=GOOD.value, B=2, Hkv=2, D=128, num_pages=9, page_size=64, max_pages=4)
    f.update(kw)
    return abi.CCache(**f)


BAD_CACHES = [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(lens=None), ARG), (dict(B=0), ARG), (dict(Hkv=0), ARG),
    (dict(num_pages=0), ARG), (dict(max_pages=0), ARG), (dict(page_size=0), ARG), (dict(page_size=-16), ARG),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=192), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(max_pages=1 << 14, page_size=128), UNSUPPORTED),
    (dict(max_pages=1 << 30, page_size=1 << 20), UNSUPPORTED), (dict(B=65536, Hkv=1), UNSUPPORTED),
    (dict(B=40000, Hkv=2), UNSUPPORTED), (dict(k=ODD16.value), ALIGN), (dict(v=ODD16.value), ALIGN),
    (dict(lens=ODD4.value), ALIGN), (dict(page_table=ODD4.value), ALIGN),
    (dict(k_strides=abi.CStrides(8192, 8192, 132)), ALIGN), (dict(v_strides=abi.CStrides(0, 8192, 128)), ALIGN),
    (dict(v_strides=abi.CStrides(-8192, 8192, 128)), ALIGN),
]
GOOD_CACHES = [{}, dict(page_table=None), dict(page_size=384), dict(page_size=1 << 20, max_pages=1), dict(D=64)]


def append(c, **kw):
    a = dict(k=GOOD, v=GOOD, lens_out=None, path=None, counts=None, T=5, lay=None, pos=None, seen=None)
    a.update(kw)
    return ta.LIB.attn_cache_append(c, a["k"], a["v"], a["lens_out"], a["path"], a["counts"], a["T"], a["lay"], a["pos"],
                                    a["seen"], None)


def tree(c, **kw):
    a = dict(q=GOOD, k=GOOD, v=GOOD, out=GOOD, lse=None, ws=GOOD, bytes=1 << 30, parents=None, counts=None, Hq=4, T=5,
             scale=0.1, mod=0, mp=None, lay=None)
    a.update(kw)
    return ta.LIB.attn_tree_fwd(a["q"], a["k"], a["v"], c, a["out"], a["lse"], a["ws"], a["bytes"], a["parents"], a["counts"],
                                a["Hq"], a["T"], a["scale"], a["mod"], a["mp"], a["lay"], None)


def weights(c, **kw):
    a = dict(q=GOOD, lse=GOOD, w_in=None, w_out=GOOD, path=None, counts=None, Hq=4, T=5, scale=0.1, mod=0, mp=None, lay=None)
    a.update(kw)
    return ta.LIB.attn_cache_weights(a["q"], a["lse"], c, a["w_in"], a["w_out"], a["path"], a["counts"], a["Hq"], a["T"],
                                     a["scale"], a["mod"], a["mp"], a["lay"], None)


def plan(c, **kw):
    a = dict(w=GOOD, pos=GOOD, seen=GOOD, moves=GOOD, n=GOOD, budget=10, first=2, recent=3)
    a.update(kw)
    return ta.LIB.attn_evict_plan(c, a["w"], a["pos"], a["seen"], a["moves"], a["n"], a["budget"], a["first"], a["recent"], None)


def compact(c, **kw):
    a = dict(moves=GOOD, n=GOOD, budget=10, w=None, pos=None)
    a.update(kw)
    return ta.LIB.attn_cache_compact(c, a["moves"], a["n"], a["budget"], a["w"], a["pos"], None)


@pytest.mark.parametrize("call", [append, tree, weights, plan, compact])
def test_caches(call):
    assert call(None) == ARG
    for kw in GOOD_CACHES:
        assert call(ctypes.byref(cache(**kw))) == DEVICE, kw
    for kw, want in BAD_CACHES:
        no_pools = call is plan and (set(kw) & {"k", "v", "k_strides", "v_strides"})
        assert call(ctypes.byref(cache(**kw))) == (DEVICE if no_pools else want), kw


SOFT = ctypes.byref(abi.CModParams(softcap=30.0))
BAD_SOFT = ctypes.byref(abi.CModParams(softcap=0.0))
BAD_LAYOUT = abi.CLayouts(q=abi.CStrides(640, 640, 100), k=abi.CStrides(640, 640, 100), v=abi.CStrides(640, 640, 128),
                          out=abi.CStrides(640, 640, 128))


@pytest.mark.parametrize("call,cases", [
    (append, [(dict(k=None), ARG), (dict(v=None), ARG), (dict(T=0), ARG), (dict(T=-3), ARG), (dict(T=(1 << 20) + 1), UNSUPPORTED),
              (dict(k=ODD16), ALIGN), (dict(path=ODD4), ALIGN), (dict(counts=ODD4), ALIGN), (dict(pos=ODD4), ALIGN),
              (dict(seen=ODD4), ALIGN), (dict(lens_out=ODD4), ALIGN), (dict(lay=ctypes.byref(BAD_LAYOUT)), ALIGN),
              (dict(path=GOOD, counts=GOOD, pos=GOOD, seen=GOOD, lens_out=GOOD), DEVICE)]),
    (tree, [(dict(q=None), ARG), (dict(out=None), ARG), (dict(ws=None), ARG), (dict(k=None), ARG), (dict(v=None), ARG),
            (dict(k=None, v=None), DEVICE), (dict(k=None, v=None, parents=GOOD), ARG), (dict(T=0), ARG),
            (dict(T=1025), UNSUPPORTED), (dict(T=1024), DEVICE), (dict(Hq=0), ARG), (dict(Hq=3), ARG),
            (dict(Hq=1 << 24), UNSUPPORTED), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
            (dict(scale=float("inf")), ARG), (dict(mod=3), ARG), (dict(mod=3, mp=BAD_SOFT), ARG), (dict(mod=3, mp=SOFT), DEVICE),
            (dict(mod=9), ARG), (dict(mod=2), UNSUPPORTED), (dict(mod=0x100), UNSUPPORTED), (dict(mod=3 | 0x200, mp=SOFT), UNSUPPORTED),
            (dict(q=ODD16), ALIGN), (dict(out=ODD16), ALIGN), (dict(lse=ODD4), ALIGN), (dict(ws=ODD16), ALIGN),
            (dict(parents=ODD4), ALIGN), (dict(counts=ODD4), ALIGN), (dict(bytes=0), WORKSPACE),
            (dict(lay=ctypes.byref(BAD_LAYOUT)), ALIGN)]),
    (weights, [(dict(q=None), ARG), (dict(lse=None), ARG), (dict(w_out=None), ARG), (dict(T=0), ARG), (dict(T=262145), UNSUPPORTED),
               (dict(T=262144), DEVICE), (dict(Hq=5), ARG), (dict(mod=2), UNSUPPORTED), (dict(mod=3, mp=SOFT), DEVICE),
               (dict(scale=-1.0), ARG), (dict(w_in=ODD4), ALIGN), (dict(w_out=ODD4), ALIGN), (dict(path=ODD4), ALIGN),
               (dict(q=ODD16), ALIGN), (dict(lay=ctypes.byref(BAD_LAYOUT)), ALIGN)]),
    (plan, [(dict(w=None), ARG), (dict(pos=None), ARG), (dict(seen=None), ARG), (dict(moves=None), ARG), (dict(n=None), ARG),
            (dict(budget=0), ARG), (dict(first=-1), ARG), (dict(recent=-1), ARG), (dict(first=11, recent=0), ARG),
            (dict(first=5, recent=6), ARG), (dict(first=5, recent=5), DEVICE), (dict(budget=(1 << 20) + 1), UNSUPPORTED),
            (dict(recent=(1 << 31) - 1), ARG), (dict(moves=ctypes.c_void_p((1 << 32) + 4)), ALIGN)]),
    (compact, [(dict(moves=None), ARG), (dict(n=None), ARG), (dict(budget=0), ARG), (dict(budget=(1 << 20) + 1), UNSUPPORTED),
               (dict(w=ODD4), ALIGN), (dict(pos=ODD4), ALIGN), (dict(moves=ctypes.c_void_p((1 << 32) + 4)), ALIGN),
               (dict(w=GOOD, pos=GOOD), DEVICE)]),
])
def test_arguments(call, cases):
    c = ctypes.byref(cache())
    for kw, want in cases:
        assert call(c, **kw) == want, kw


def test_workspace_sizes():
    f = ta.attn_tree_workspace_size
    assert f(4, 3, 1, 128) == 0 and f(4, 2, 0, 128) == 0 and f(4, 2, 1025, 128) == 0 and f(4, 2, 1, 96) == 0
    for Hq, Hkv in ((1, 1), (32, 8), (160, 1)):
        for D in (64, 128):
            sizes = [f(Hq, Hkv, T, D) for T in (1, 2, 3, 17, 64, 100, 1000, 1024)]
            assert sizes[0] > 0 and sizes == sorted(sizes)  # a workspace serves every smaller T


def test_status_text():
    assert "index" in ta.attn_strerror(ta.ATTN_ERR_INDEX)
