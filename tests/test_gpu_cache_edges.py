"""KV-cache operators at the ends of their ranges, against their definitions."""
import numpy as np
import pytest
import torch

import oracle
from cache_common import i32

pytestmark = pytest.mark.gpu


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
