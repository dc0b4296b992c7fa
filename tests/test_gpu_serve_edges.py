"""Where the rotary, 8-bit cache and modified-score operators can go wrong by
their numbers: each test names its case."""
import math

import pytest
import torch

import block_sparse_bidirectional_select_b200 as sp
import serve_ref as R
from test_gpu_serve_ops import check_cache_attn, check_scored, gen, i32, randn, random_cache, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [2, 40])            # a tile's keys in two slots; pairs of tiles
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("what", [300.0, 1e30, math.inf, math.nan])
def test_capped_scores_and_padding(H, bias, what):
    """What K and V hold at keys that no row sees changes no bit, whatever the size of the scores there."""
    g = gen(71)
    L = 700
    q, k, v = randn(g, H, L, 64), randn(g, 2, L, 64), randn(g, 2, L, 64)
    ranges = torch.zeros(L, 2, dtype=torch.int32)
    ranges[:300] = torch.tensor([0, 300], dtype=torch.int32)
    ranges[420:690] = torch.tensor([420, 690], dtype=torch.int32)
    ranges = ranges.cuda()
    slopes = slopes_of(H) if bias else None
    want = sp.scored_attn(q, k, v, softcap=30.0, slopes=slopes, ranges=ranges)
    for x in (k, v):
        x[:, 300:420] = what
        x[:, 690:] = what
    got = sp.scored_attn(q, k, v, softcap=30.0, slopes=slopes, ranges=ranges)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    sp.device_check()
