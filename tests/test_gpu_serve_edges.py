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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap", [4000.0, 250.0, 50.0])
def test_small_scores_beside_scores_near_the_cap(d, softcap):
    """A row that sees one key has its score as log-sum (one product, exact in
    fp32). Even rows stay below cap / 40, odd ones lie between 0.6 and 0.9 of
    the cap and are in the same warps. The wide form 1 - 2 / (1 + e), e = e^2u:
    MUFU's 2^-22 and the rounded argument leave e off by 2^-21 of itself,
    1 / (1 + e) <= 1 by 2^-21 / 4 and the reciprocal's 2^-23, its double at most 1:
    together 2^-21.4 of the cap. Large scores are right to 2^-20 of the cap,
    small ones to the polynomial's 1e-6 of themselves, or to 2^-21 of a cap of
    at most 64, whose warps take the wide form for all; the log-sum adds 9 * 2^-22
    (as in the test of scores that are small throughout)."""
    L = 64
    g = gen(72)
    small = (torch.rand(L, generator=g) * 2 - 1) * softcap / 40
    large = (torch.rand(L, generator=g) * 0.3 + 0.6) * softcap * (1 - 2 * (torch.arange(L) // 2 % 2))
    odd = torch.arange(L) % 2 == 1
    x = torch.where(odd, large, small).bfloat16().cuda()
    q = torch.zeros(2, L, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 3] = x
    k = torch.zeros(2, L, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 3] = 1.0
    want = softcap * torch.tanh(x.double() / softcap)
    tol = torch.where(odd.cuda(), 2.0 ** -20 * softcap, 1e-6 * want.abs()) + 9 * 2.0 ** -22
    if softcap <= 64:
        tol = tol + 2.0 ** -21 * softcap
    at = torch.arange(L, device="cuda")
    ranges = torch.stack([at, at + 1], 1).int().contiguous()
    cache = sp.cache_append(sp.cache_alloc(1, 2, 64, d), k[None, :, :1], k[None, :, :1], i32([0]))
    for zero in (None, torch.zeros(2, device="cuda")):
        _, lse = sp.scored_attn(q, k, k, scale=1.0, softcap=softcap, ranges=ranges, slopes=zero)
        assert ((lse.double() - want).abs() <= tol).all(), float(((lse.double() - want).abs() / tol).max())
        _, lse = sp.cache_attn(q[None], cache, i32([1]), scale=1.0, softcap=softcap, slopes=zero)
        assert ((lse.double() - want).abs() <= tol).all(), float(((lse.double() - want).abs() / tol).max())


@pytest.mark.parametrize("q_start", [10 ** 6, -10 ** 6, 2 ** 24 + 77, 2 ** 29, -2 ** 29])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_positions_far_from_the_keys(q_start, softcap):
    """The distances to all keys are large and their differences small: what a chunk of keys far from the queries is."""
    g = gen(73)
    slopes = torch.tensor([1.0, 2.0 ** -4, 2.0 ** -9, 0.0], device="cuda")
    for Lq, H in ((100, 4), (700, 4)):
        q, k, v = randn(g, H, Lq, 64), randn(g, 2, 900, 64), randn(g, 2, 900, 64)
        check_scored(q, k, v, softcap, slopes, q_start=q_start)
        lo = torch.randint(-20, 900, (Lq,), generator=g)
        ranges = torch.stack([lo, lo + torch.randint(-2, 400, (Lq,), generator=g)], 1).to(torch.int32).cuda()
        check_scored(q, k, v, softcap, slopes, ranges, q_start=q_start)
    c = random_cache(g, 3, 2, 1088, 128)
    for B in (1, 20, 70):
        check_cache_attn(randn(g, 3, 4, B, 128), c, [1088, 1, 700], softcap, slopes, [q_start, q_start, 0])
    long = random_cache(g, 1, 2, 32768, 128)      # its parts are joined
    check_cache_attn(randn(g, 1, 4, 3, 128), long, [32700], softcap, slopes, [q_start])


@pytest.mark.parametrize("H", [2, 40])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_a_visible_nan_reaches_its_rows_however_far(H, softcap):
    g = gen(74)
    L = 1000
    q, k, v = randn(g, H, L, 64), randn(g, 2, L, 64), randn(g, 2, L, 64)
    k[:, 20, 5] = math.nan
    steep = torch.full((H,), 10.0, device="cuda")
    ranges = torch.tensor([[0, L]] * 600 + [[21, L]] * 400, dtype=torch.int32, device="cuda")
    o, lse = sp.scored_attn(q, k, v, softcap=softcap, slopes=steep, ranges=ranges)
    assert torch.isnan(o[:, :600]).all() and torch.isnan(lse[:, :600]).all()
    assert not torch.isnan(o[:, 600:]).any() and not torch.isnan(lse[:, 600:]).any()
    c = random_cache(g, 1, 2, 1024, 64)
    c.k8.view(torch.uint8)[0, :, 20, 5] = 0x7F
    for B in (1, 40):
        o, lse = sp.cache_attn(randn(g, 1, 2, B, 64), c, i32([1000]), softcap=softcap, slopes=steep[:2])
        assert torch.isnan(o).all() and torch.isnan(lse).all()
    sp.device_check()


@pytest.mark.parametrize("shared,inter", [(False, False), (True, True)])
def test_rope_of_single_elements_next_to_a_quadrant(shared, inter):
    """Pairs with one element 0: the result is x cos t or x sin t, right to its
    own last bit also where that is nearly 0. The angle is off by position *
    2^-53 turns and the reference's by position * 2^-52 rad (together below
    position * 2^-50 rad), the sine by a few fp32 roundings of itself, the
    product by one, the result by half a bf16 step."""
    g = gen(75)
    L, d = 40000, 64
    x = (torch.rand(2, L, d, generator=g) + 0.5).to(torch.bfloat16).cuda()
    first = torch.arange(d, device="cuda") % 2 == 0 if inter else torch.arange(d, device="cuda") < d // 2
    x[0, :, ~first] = 0
    x[1, :, first] = 0
    pos = torch.arange(-L // 2, L - L // 2, dtype=torch.int32, device="cuda")[None].contiguous()
    for theta in (10000.0, 1e6):
        y = sp.rope_axes(x, pos, (32,), theta=theta, interleaved=inter, shared_ladder=shared)
        ref, amp = R.rope(x, pos, (32,), float(torch.tensor(theta)), inter, shared, False)
        tol = (R.U_BF16 + 2.0 ** -20) * ref.abs() + 2.0 ** -50 * pos[0].abs().double()[None, :, None] * amp + 2.0 ** -133
        err = (y.double() - ref).abs()
        assert (err <= tol).all(), f"{int((err > tol).sum())} elements, {float((err / tol).max()):.1f} of the bound"


@pytest.mark.parametrize("d,N,Hq,Hkv,B,C,bias", [(128, 1, 8, 2, 1, 16384, False), (64, 1, 2, 1, 1, 32768, False),
                                                 (128, 2, 4, 4, 16, 8192, True), (128, 1, 2, 2, 64, 16384, False),
                                                 (64, 3, 2, 1, 40, 8192, False), (128, 1, 4, 1, 70, 16384, False)])
def test_long_caches_whose_blocks_differ(d, N, Hq, Hkv, B, C, bias):
    """Block j of V fills the columns j mod 64 and no others, so a column holds a few blocks of the cache and a block
    that is left out, or that is given another's scale, shows there. That it does is checked with such a mistake in
    the reference."""
    g = gen(76 + B)
    c = random_cache(g, N, Hkv, C, d)
    blocks = C // 64
    at = torch.arange(blocks)
    own = (torch.arange(d)[None] % 64 == at[:, None] % 64).float()                  # [blocks, d]
    v = (torch.rand(N, Hkv, blocks, 64, d, generator=g) * 0.2 + 0.9) * own[:, None]
    scale = 2.0 ** torch.randint(-8, -5, (N, Hkv, blocks), generator=g).float()
    c.v_scale.copy_(scale)
    c.v8.copy_((v / scale[..., None, None]).reshape(N, Hkv, C, d).to(torch.float8_e4m3fn))
    c.k8.copy_((torch.randn(c.k8.shape, generator=g) * 20).to(torch.float8_e4m3fn))
    lengths = [C - 1 - 777 * n for n in range(N)]
    q, slopes = randn(g, N, Hq, B, d), slopes_of(Hq) * 1e-4 if bias else None
    o, lse = check_cache_attn(q, c, lengths, 0.0, slopes)
    k0, v0 = (R.dequant(x8, sc)[0, 0, :lengths[0]] for x8, sc in ((c.k8, c.k_scale), (c.v8, c.v_scale)))
    lo, pos = torch.zeros(B, dtype=torch.long, device="cuda"), torch.arange(B, device="cuda") + lengths[0] - B
    for j in (0, 1, blocks // 2, blocks - 2):
        for factor in (0.0, 2.0):
            wrong = v0.clone()
            wrong[64 * j:64 * j + 64] *= factor
            ref = R.attend(q[0, 0], k0, wrong, lo, lo + lengths[0], pos, sp.default_scale(d), 0.0,
                           None if slopes is None else float(slopes[0]))
            with pytest.raises(AssertionError, match="O off"):
                R.assert_attention(o[0, 0], lse[0, 0], ref)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_negative_slopes(softcap):
    """Far keys come nearer: the row maxima rise along the walk, and rows beside their keys are moved as with others."""
    g = gen(77)
    slopes = torch.tensor([-0.05, -0.5, 0.25, -2.0 ** -9], device="cuda")
    for Lq, Lk, start in ((700, 700, 0), (100, 1500, 700), (300, 400, 5000), (64, 900, -3000)):
        check_scored(randn(g, 4, Lq, 64), randn(g, 2, Lk, 64), randn(g, 2, Lk, 64), softcap, slopes, q_start=start)
    lo = torch.randint(0, 600, (700,), generator=g)
    ranges = torch.stack([lo, lo + torch.randint(0, 300, (700,), generator=g)], 1).to(torch.int32).cuda()
    check_scored(randn(g, 4, 700, 128), randn(g, 2, 700, 128), randn(g, 2, 700, 128), softcap, slopes, ranges)
    c = random_cache(g, 2, 2, 4096, 128)
    for B in (1, 24, 70):
        check_cache_attn(randn(g, 2, 4, B, 128), c, [4000, 130], softcap, slopes, None if B == 1 else [9000, -50])


@pytest.mark.parametrize("H,softcap", [(2, 0.0), (40, 0.0), (40, 30.0)])
def test_ranges_at_the_ends_of_their_type(H, softcap):
    """Bounds next to -2^31 and 2^31 - 1, as rows of a tile that other rows do see."""
    g = gen(78)
    L, lowest, most = 600, -2 ** 31, 2 ** 31 - 1
    q, k, v = randn(g, H, L, 64), randn(g, 2, L, 64), randn(g, 2, L, 64)
    rows = [[0, lowest], [300, lowest], [0, lowest + 1], [lowest, most], [most, most], [most, lowest], [250, -1], [lowest, 400]]
    ranges = torch.tensor([[0, L]] * L, dtype=torch.int32)
    for i in range(L):
        if i % 3:
            ranges[i] = torch.tensor(rows[(i // 3) % len(rows)], dtype=torch.int32)
    check_scored(q, k, v, softcap, None, ranges.cuda())
