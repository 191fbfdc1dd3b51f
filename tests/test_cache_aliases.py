"""Arrays of one cache call that overlap, before any GPU work."""
import ctypes

import pytest
import torch

import tiled_attention_25_b200 as ta
from tiled_attention_25_b200 import abi

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers: only where nothing can be launched")
DEVICE, ARG = -7, -1
POOL, LENS, COUNTS, SEEN, OUT = 1 << 32, 2 << 32, 3 << 32, 4 << 32, 5 << 32
B = 6


def append(out, counts=COUNTS, seen=SEEN):
    st = abi.CStrides(8192, 8192, 128)
    c = abi.CCache(k=POOL, v=POOL, k_strides=st, v_strides=st, page_table=None, lens=LENS, B=B, Hkv=2, D=128, num_pages=24,
                   page_size=64, max_pages=4)
    p = ctypes.c_void_p
    return ta.LIB.attn_cache_append(ctypes.byref(c), p(POOL), p(POOL), p(out) if out else None, None, p(counts) if counts else None,
                                    5, None, None, p(seen) if seen else None, None)


def test_new_lengths_replace_an_argument_or_lie_apart():
    for out in (None, OUT, LENS, COUNTS, SEEN):
        assert append(out) == DEVICE
        assert append(out, None, None) == DEVICE
    for base in (LENS, COUNTS, SEEN):
        for off in (4, 4 * (B - 1), -4, -4 * (B - 1)):
            assert append(base + off) == ARG, (base, off)
        assert append(base + 4 * B) == DEVICE and append(base - 4 * B) == DEVICE
    assert append(COUNTS + 4, counts=None) == DEVICE and append(SEEN + 4, seen=None) == DEVICE
