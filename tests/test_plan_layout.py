"""The shared-memory layout of the eviction plan (csrc/cache_index.h), compiled
for the host: whatever the heads and the capacity, its parts lie in order
within the block's memory."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMEM, MOST_SLOTS = 227 * 1024, 1 << 20
SOURCE = r"""
#include "cache_index.h"
using namespace attn25;
extern "C" {
void layout(int heads, int cap, int sms, int fixed, int* o) { PlanLayout p = plan_layout(heads, cap, sms, fixed);
  o[0]=p.ctas; o[1]=p.share; o[2]=p.held; o[3]=p.kept; o[4]=p.bytes; }
int share(int slots, int ctas) { return plan_share(slots, ctas); }
}
"""
FIXED = (33312, 32768, 40960)  # bytes of counters: the kernel's, and others near it


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan_layout")
    src = d / "x.cpp"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "tiled_attention_25_b200", "csrc"), str(src), "-o", str(d / "x.so")], check=True)
    return ctypes.CDLL(str(d / "x.so"))


def layout(lib, heads, cap, fixed, sms=148):
    o = (ctypes.c_int * 5)()
    lib.layout(heads, cap, sms, fixed, o)
    return list(o)


@pytest.mark.parametrize("fixed", FIXED)
@pytest.mark.parametrize("heads", [1, 8, 18, 19, 37, 38, 74, 75, 80, 149, 4096, 65535])
def test_parts_lie_in_order_within_the_block(lib, heads, fixed):
    caps = set(range(16, MOST_SLOTS + 1, 4096 - 16)) | {MOST_SLOTS, MOST_SLOTS - 16, 800000, 850048, 900096, 929792, 796544, 796560}
    for cap in sorted(caps):
        ctas, share, held, kept, total = layout(lib, heads, cap, fixed)
        assert ctas in (1, 2, 4, 8) and share % 32 == 0 and ctas * share >= cap, cap
        assert 0 <= held <= share and held % 4 == 0, (cap, held)
        assert kept == fixed + 4 * held and total == kept + share // 4 <= SMEM, (cap, kept, total)
        # a row's share, whatever its length, has its flags there
        for n in (1, cap // 3 + 1, cap - 1, cap):
            assert lib.share(n, ctas) <= share


def test_ranks_are_held_where_they_fit(lib):
    assert layout(lib, 32, 65024, 33312)[:3] == [4, 16256, 16256]
    assert layout(lib, 300, 60000, 33312)[2] < 60000  # one CTA: some ranks are formed again
    assert layout(lib, 32, 1088, 33312)[:3] == [1, 1088, 1088]
