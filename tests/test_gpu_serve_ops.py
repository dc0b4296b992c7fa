"""Rotary axes, the 8-bit cache and attention with modified scores on the GPU
against their plain fp64 forms."""
import itertools
import math

import pytest
import torch

import block_sparse_bidirectional_select_b200 as sp
import serve_ref as R

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def randn(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ rotary axes

ROPE = [
    # H, L, d, sections, interleaved, shared, inverse, far
    (1, 1, 64, (32,), False, False, False, 0),
    (3, 65, 64, (16, 16), True, False, False, 1 << 20),
    (5, 129, 128, (16, 24, 24), False, True, False, 100003),
    (2, 300, 128, (32,), False, False, True, 0),          # half of the head is turned
    (2, 37, 128, (7, 0, 20), True, True, False, 50),      # odd sections, one of them empty
    (2, 37, 128, (7, 6), False, False, False, 2 ** 31 - 400),
    (7, 33, 8, (1,), False, False, False, 9),
    (2, 5, 512, (64, 64), True, False, True, 77),
    (40, 1000, 128, (64,), False, False, False, 32768),
]


@pytest.mark.parametrize("H,L,d,sections,inter,shared,inv,far", ROPE)
def test_rope(H, L, d, sections, inter, shared, inv, far):
    g = gen(H * 1000 + L)
    x = randn(g, H, L, d)
    pos = (torch.randint(-300, 300, (len(sections), L), generator=g) + far).clamp(max=2 ** 31 - 1).to(torch.int32).cuda()
    y = sp.rope_axes(x, pos, sections, theta=10000.0, interleaved=inter, shared_ladder=shared, inverse=inv)
    ref, amp = R.rope(x, pos, sections, 10000.0, inter, shared, inv)
    # the angle: 2^-32 turns and 2^31 * 2^-53 turns at most (2^-19 rad); sine,
    # cosine, two products and a sum in fp32; one rounding to bf16
    tol = R.U_BF16 * ref.abs() + 2.0 ** -18 * amp
    assert ((y.double() - ref).abs() <= tol).all()
    assert torch.equal(y[..., 2 * sum(sections):], x[..., 2 * sum(sections):])


@pytest.mark.parametrize("inter", [False, True])
def test_rope_strided_views_in_place_and_unaligned(inter):
    g = gen(5)
    qkv = randn(g, 77, 12, 128)
    pos = i32(torch.randint(0, 9999, (2, 77), generator=g).tolist())
    x = qkv[:, 2:9].transpose(0, 1)
    want = sp.rope_axes(x.contiguous(), pos, (30, 34), interleaved=inter)
    assert torch.equal(sp.rope_axes(x, pos, (30, 34), interleaved=inter), want)
    # rows of 129 elements from an odd base: no 16-byte access possible
    odd = torch.zeros(7 * 77 * 129 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(7, 77, 129)[..., :128]
    odd.copy_(x)
    out = torch.full((7, 77, 136), 3.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(sp.rope_axes(odd, pos, (30, 34), interleaved=inter, out=out[..., 3:131]), want)
    assert (out[..., :3] == 3).all() and (out[..., 131:] == 3).all()
    before = qkv.clone()
    sp.rope_axes(x, pos, (30, 34), interleaved=inter, out=x)       # in place, inside the projection's output
    assert torch.equal(x, want)
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 9:], before[:, 9:])


def test_rope_inverse_is_the_gradient():
    """y = R x is linear with R^T = R^-1: <w, R x> has the gradient R^T w, checked against differences in fp64."""
    g = gen(6)
    x, w = randn(g, 2, 19, 64), randn(g, 2, 19, 64)
    pos = i32(torch.randint(0, 5000, (1, 19), generator=g).tolist())
    grad = sp.rope_axes(w, pos, (32,), inverse=True).double()
    base, _ = R.rope(x, pos, (32,), 10000.0, False, False, False)
    for h, l, e in ((0, 0, 0), (1, 7, 31), (1, 18, 63), (0, 11, 32)):
        xs = x.double().clone()
        xs[h, l, e] += 0.5
        moved, _ = R.rope(xs, pos, (32,), 10000.0, False, False, False)
        num = float(((moved - base) * w.double()).sum()) / 0.5
        amp = float(w[h, l].double().abs().max()) * 2
        assert abs(float(grad[h, l, e]) - num) <= R.U_BF16 * abs(num) + 2.0 ** -18 * amp + 1e-9


# ------------------------------------------------------------------ cache append

def random_cache(g, N, H, C, d, e_lo=-9, e_hi=-4):
    c = sp.cache_alloc(N, H, C, d)
    for x8, sc in ((c.k8, c.k_scale), (c.v8, c.v_scale)):
        x8.copy_((torch.randn(x8.shape, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
        sc.copy_(2.0 ** torch.randint(e_lo, e_hi, sc.shape, generator=g).float())
    return c


def check_append(c, k, v, starts, counts, **kw):
    before = sp.Cache8(*(t.cpu() for t in (c.k8, c.v8, c.k_scale, c.v_scale)))
    sp.cache_append(c, k, v, i32(starts), i32(counts) if kw.get("count", True) else None)
    sp.device_check()
    for x, x8, sc, b8, bs in ((k, c.k8, c.k_scale, before.k8, before.k_scale),
                              (v, c.v8, c.v_scale, before.v8, before.v_scale)):
        r8, rs = R.append(x.cpu(), b8, bs, starts, counts)
        assert torch.equal(sc.cpu(), rs)
        assert torch.equal(x8.cpu().view(torch.uint8), r8.view(torch.uint8))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,H,B,C,starts,counts", [
    (1, 1, 1, 64, [0], [1]),
    (1, 2, 1, 64, [63], [1]),
    (3, 2, 65, 256, [0, 63, 191], [65, 64, 65]),
    (4, 1, 130, 320, [1, 0, 190, 77], [130, 0, 130, 1]),
    (2, 3, 64, 192, [64, 100], [64, 37]),
])
def test_append(d, N, H, B, C, starts, counts):
    g = gen(N * 100 + B + d)
    c = random_cache(g, N, H, C, d)
    # values of mixed size, so that some blocks' scales grow and others keep the older one
    k = randn(g, N, H, B, d, scale=1.0) * i32([[8.0 ** ((n + h) % 3 - 1) for h in range(H)] for n in range(N)])[..., None, None]
    k = k.to(torch.bfloat16)
    v = randn(g, N, H, B, d, scale=0.01)
    check_append(c, k, v, starts, counts)


def test_append_strided_views_unaligned_and_default_count():
    g = gen(8)
    kv = randn(g, 2, 70, 6, 64)
    c = random_cache(g, 2, 3, 256, 64)
    check_append(c, kv[:, :, :3].transpose(1, 2), kv[:, :, 3:].transpose(1, 2), [5, 130], [70, 70], count=False)
    flat = torch.zeros(2 * 3 * 70 * 65 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 3, 70, 65)[..., :64]
    flat.copy_(kv[:, :, :3].transpose(1, 2))
    check_append(c, flat, flat, [5, 64], [70, 3])


def test_append_extremes():
    """Zeros, subnormals, the largest finite values, infinities and NaN."""
    g = gen(9)
    top = torch.finfo(torch.bfloat16).max
    c = random_cache(g, 1, 1, 192, 64)
    k = randn(g, 1, 1, 150, 64)
    k[0, 0, 3, 5], k[0, 0, 9, 1], k[0, 0, 20, 2] = math.inf, -math.inf, math.nan
    k[0, 0, 80, 0], k[0, 0, 81, 0] = top, -top
    v = torch.zeros_like(k)
    v[0, 0, 70, 3] = 1e-40
    v[0, 0, 140:] = math.inf
    check_append(c, k, v, [10], [150])
    c2 = random_cache(g, 1, 1, 64, 64, -117, -116)
    check_append(c2, k[:, :, :20] * 0 + top, v[:, :, :20] + 448.0, [30], [20])   # older values far below the new scale


def test_append_bad_places_are_reported_and_skipped():
    g = gen(10)
    c = random_cache(g, 3, 1, 128, 64)
    before = [t.clone() for t in (c.k8.view(torch.uint8), c.k_scale)]
    k = randn(g, 3, 1, 8, 64)
    for starts, counts in (([121, -1, 0], [8, 8, 9]), ([2 ** 31 - 1, -2 ** 31, 0], [8, 8, -1])):
        sp.cache_append(c, k, k, i32(starts), i32(counts))
        with pytest.raises(sp.SparsedError):
            sp.device_check()
    assert torch.equal(before[0], c.k8.view(torch.uint8)) and torch.equal(before[1], c.k_scale)


# ------------------------------------------------------------------ attention over the cache

def check_cache_attn(q, c, lengths, softcap=0.0, slopes=None, q_start=None, scale=None, what=""):
    N, Hq, B, d = q.shape
    Hkv = c.k8.shape[1]
    o, lse = sp.cache_attn(q, c, i32(lengths), scale=scale, softcap=softcap, slopes=slopes,
                           q_start=None if q_start is None else i32(q_start))
    sp.device_check()
    scale = sp.default_scale(d) if scale is None else scale
    k, v = R.dequant(c.k8, c.k_scale), R.dequant(c.v8, c.v_scale)
    for n, h in itertools.product(range(N), range(Hq)):
        L = lengths[n]
        at = torch.arange(B, device="cuda") + (L - B if q_start is None else q_start[n])
        lo = torch.zeros(B, dtype=torch.long, device="cuda")
        ref = R.attend(q[n, h], k[n, h * Hkv // Hq, :L], v[n, h * Hkv // Hq, :L], lo, lo + L, at, scale, softcap,
                       None if slopes is None else float(slopes[h]))
        R.assert_attention(o[n, h], lse[n, h], ref, f"{what} n={n} h={h}")
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,Hq,Hkv,B,C,lengths", [
    (1, 1, 1, 1, 64, [1]),
    (3, 2, 1, 1, 320, [0, 64, 320]),
    (4, 8, 2, 1, 1024, [63, 129, 1000, 1024]),
    (2, 4, 4, 32, 576, [33, 575]),
    (2, 6, 2, 61, 448, [100, 448]),          # 183 rows of a kv head: two row tiles, the last ragged
    (1, 2, 1, 64, 16384, [16001]),
    (1, 1, 1, 300, 192, [130]),
    (2, 2, 2, 48, 1024, [1000, 65]),         # 48 rows
    (3, 3, 1, 8, 704, [704, 8, 641]),        # 24 rows
    (5, 15, 1, 1, 2048, [2048, 1, 0, 2047, 64]),
    (40, 2, 2, 1, 128, [1 + (37 * n) % 128 for n in range(40)]),   # several items to a run
    (33, 1, 1, 20, 64, [20 + n for n in range(33)]),
    (300, 1, 1, 1, 128, [(n * 53) % 129 for n in range(300)]),     # many sequences, some of them empty
    (5, 4, 2, 70, 384, [0, 70, 384, 129, 200]),
])
def test_cache_attn(d, N, Hq, Hkv, B, C, lengths):
    g = gen(N + Hq * 10 + B)
    c = random_cache(g, N, Hkv, C, d)
    check_cache_attn(randn(g, N, Hq, B, d), c, lengths)


@pytest.mark.parametrize("N,Hq,Hkv,B,C,d,softcap,bias", [
    (28, 48, 16, 16, 512, 64, 20.0, False), (13, 48, 16, 16, 2240, 128, 0.0, False), (10, 48, 16, 16, 1152, 128, 0.0, True),
    (20, 32, 16, 18, 1216, 64, 0.0, False), (7, 64, 32, 32, 2432, 64, 0.0, False), (13, 64, 32, 32, 1216, 128, 0.0, False),
    (16, 64, 16, 1, 2048, 64, 20.0, False), (6, 32, 32, 16, 5824, 64, 0.0, False), (26, 32, 32, 1, 1216, 128, 0.0, False),
    (21, 8, 8, 64, 384, 128, 0.0, False)])
def test_cache_attn_many_short_parts(N, Hq, Hkv, B, C, d, softcap, bias):
    """Warps that hold no rows, and rows whose maximum rises while the other
    half's tiles lag: several calls, bit for bit the same."""
    g = gen(N * C + B)
    q = randn(g, N, Hq, B, d, scale=4.0)
    c = random_cache(g, N, Hkv, C, d)
    lengths = [C - 37 * n % (C // 2) for n in range(N)]
    slopes = slopes_of(Hq) if bias else None
    check_cache_attn(q, c, lengths, softcap, slopes)
    first = sp.cache_attn(q, c, i32(lengths), softcap=softcap, slopes=slopes)
    for _ in range(20):
        again = sp.cache_attn(q, c, i32(lengths), softcap=softcap, slopes=slopes)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    sp.device_check()


@pytest.mark.parametrize("softcap,bias,given", [(5.0, False, False), (50.0, False, False), (0.0, True, False),
                                                (30.0, True, True)])
def test_cache_attn_modified_scores(softcap, bias, given):
    g = gen(21)
    c = random_cache(g, 2, 2, 1088, 128)
    q = randn(g, 2, 8, 5, 128, scale=4.0)     # scores that reach the cap
    slopes = torch.tensor([2.0 ** -(h + 1) for h in range(8)], device="cuda") if bias else None
    check_cache_attn(q, c, [1088, 700], softcap, slopes, [3, 2000] if given else None)
    check_cache_attn(randn(g, 2, 8, 61, 128, scale=4.0), c, [1088, 700], softcap, slopes, [500, -90] if given else None)
    check_cache_attn(randn(g, 2, 8, 9, 128, scale=4.0), c, [70, 1001], softcap, None if slopes is None else slopes * 30)


def test_cache_attn_far_scales_and_large_queries():
    """Blocks whose scales differ by 2^30, an attention sink, queries of 1e4 and 1e-4."""
    g = gen(22)
    c = random_cache(g, 1, 1, 512, 128)
    c.v_scale[0, 0, 2] = 2.0 ** -38
    c.k_scale[0, 0, 3] = 2.0 ** -30
    c.v_scale[0, 0, 5] = 2.0 ** -117
    c.v8[0, 0, 5 * 64:6 * 64] = 0
    q = randn(g, 1, 2, 3, 128)
    q[0, 0] *= 1e4
    q[0, 1] *= 1e-4
    check_cache_attn(q, c, [512], scale=1e-3)
    # one key far above all others, whose weights are alike: the tail's sum is systematic
    c2 = sp.cache_alloc(1, 1, 32768, 64)
    k, v = torch.zeros(1, 1, 32768, 64), torch.ones(1, 1, 32768, 64)
    k[..., 0, 0] = 10.4
    v[..., 0, :] = -1.0
    sp.cache_append(c2, k.bfloat16().cuda(), v.bfloat16().cuda(), i32([0]))
    q = torch.zeros(1, 1, 1, 64)
    q[..., 0] = 8.0
    check_cache_attn(q.bfloat16().cuda(), c2, [32768])


def test_cache_attn_ignores_bytes_past_the_length():
    g = gen(23)
    c = random_cache(g, 2, 2, 384, 128)
    q = randn(g, 2, 4, 2, 128)
    want, wl = sp.cache_attn(q, c, i32([70, 257]))
    for n, L in enumerate((70, 257)):
        for x8, sc in ((c.k8, c.k_scale), (c.v8, c.v_scale)):
            x8.view(torch.uint8)[n, :, L:] = 0x7F                  # NaN
            sc[n, :, -(-L // 64):] = math.nan
    o, lse = sp.cache_attn(q, c, i32([70, 257]))
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_cache_attn_strided_queries_other_stream_and_graph():
    g = gen(24)
    c = random_cache(g, 3, 2, 640, 64)
    proj = randn(g, 3, 7, 6, 64)                                   # [N, B, heads, d]
    q = proj[:, :, 1:5].transpose(1, 2)
    lengths = i32([640, 0, 333])
    want, wl = sp.cache_attn(q.contiguous(), c, lengths)
    o, lse = sp.cache_attn(q, c, lengths)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = sp.cache_attn(q, c, lengths, stream=s)
    s.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    out, out_lse = torch.empty_like(want), torch.empty_like(wl)
    ws = torch.empty(sp.cache_attn_workspace_bytes(3, 4, 2, 7, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.cache_attn(q, c, lengths, out=out, lse=out_lse, workspace=ws)
    for new in ([1, 640, 65], [640, 0, 333]):                      # lengths are read at replay
        lengths.copy_(i32(new))
        ws.fill_(0xAB)
        graph.replay()
        w2, l2 = sp.cache_attn(q, c, lengths)
        assert torch.equal(out, w2) and torch.equal(out_lse, l2)


def test_cache_attn_far_into_a_long_cache():
    """Offsets past 2^32 bytes: the second sequence's last tokens lie beyond them."""
    C, d = 17_000_000 // 64 * 64, 128
    g = gen(25)
    c = sp.cache_alloc(2, 1, C, d)
    k, v = randn(g, 2, 1, 200, d), randn(g, 2, 1, 200, d)
    starts = [0, C - 200]
    sp.cache_append(c, k, v, i32(starts))
    sp.device_check()
    for x, x8, sc in ((k, c.k8, c.k_scale), (v, c.v8, c.v_scale)):
        lo = C - 256
        r8, rs = R.append(x[1:].cpu(), torch.zeros(1, 1, 256, d).to(torch.float8_e4m3fn), torch.full((1, 1, 4), 2.0 ** -117), [56], [200])
        assert torch.equal(x8[1:, :, lo + 56:].cpu().view(torch.uint8), r8[:, :, 56:].view(torch.uint8))
        assert torch.equal(sc[1:, :, -4:].cpu(), rs)
    q = randn(g, 2, 2, 3, d)
    slopes = torch.tensor([1.0, 0.5], device="cuda")
    o, lse = sp.cache_attn(q, c, i32([200, C]), slopes=slopes)
    sp.device_check()
    # a slope of 0.5 leaves nothing of keys over 4096 tokens away
    for n, (a, b) in enumerate(((0, 256), (C - 4096, C))):
        L = 200 if n == 0 else 4096
        kd, vd = (R.dequant(t8[n:n + 1, :, a:b], sc[n:n + 1, :, a // 64:b // 64])[0, 0, :L]
                  for t8, sc in ((c.k8, c.k_scale), (c.v8, c.v_scale)))
        at = torch.arange(L - 3, L, device="cuda")
        lo = torch.zeros(3, dtype=torch.long, device="cuda")
        for h in range(2):
            ref = R.attend(q[n, h], kd, vd, lo, lo + L, at, sp.default_scale(d), 0.0, float(slopes[h]))
            R.assert_attention(o[n, h], lse[n, h], ref, f"n={n} h={h}")


def test_cache_attn_two_calls_at_once_and_a_spoiled_row():
    """Calls on two streams with workspaces of their own, and a NaN or infinite query that spoils its own row only."""
    g = gen(26)
    c = random_cache(g, 4, 2, 4096, 128)
    lengths = i32([4096, 17, 0, 2500])
    qs = [randn(g, 4, 4, b, 128) for b in (1, 40)]
    want = [sp.cache_attn(q, c, lengths, softcap=20.0) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [None, None]
    for _ in range(5):
        for i, (q, s) in enumerate(zip(qs, streams)):
            with torch.cuda.stream(s):
                got[i] = sp.cache_attn(q, c, lengths, softcap=20.0)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    q = qs[1].clone()
    q[0, 1, 7, 3], q[3, 2, 0, 0] = math.nan, math.inf
    o, l = sp.cache_attn(q, c, lengths, softcap=20.0)
    for n, h, b in ((0, 1, 7), (3, 2, 0)):
        assert torch.isnan(o[n, h, b]).all() and torch.isnan(l[n, h, b])
        o[n, h, b], l[n, h, b] = want[1][0][n, h, b], want[1][1][n, h, b]
    assert torch.equal(o, want[1][0]) and torch.equal(l, want[1][1])


def test_zero_and_extreme_options():
    g = gen(27)
    c = random_cache(g, 1, 1, 192, 64)
    q = randn(g, 1, 2, 2, 64)
    check_cache_attn(q, c, [130], scale=0.0)
    check_cache_attn(q, c, [130], softcap=1e-30)
    check_cache_attn(q, c, [130], softcap=1e30)
    k, v = randn(g, 1, 130, 64), randn(g, 1, 130, 64)
    r = torch.tensor([[5, 100], [129, 130]], dtype=torch.int32, device="cuda")
    for kw in (dict(scale=0.0), dict(softcap=1e-30), dict(softcap=1e30), dict(scale=0.0, softcap=5.0, slopes=slopes_of(2))):
        check_scored(q[0], k, v, ranges=r, **kw)
    o, lse = sp.scored_attn(q[0], k[:, :0], v[:, :0])
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = sp.cache_attn(q, sp.cache_alloc(1, 1, 0, 64), i32([0]))
    assert (o == 0).all() and torch.isneginf(lse).all()


# ------------------------------------------------------------------ dense attention with modified scores

def check_scored(q, k, v, softcap=0.0, slopes=None, ranges=None, q_start=0, scale=None, what=""):
    Hq, Lq, d = q.shape
    Hkv, Lk = k.shape[:2]
    o, lse = sp.scored_attn(q, k, v, scale=scale, softcap=softcap, slopes=slopes, ranges=ranges, q_start=q_start)
    sp.device_check()
    scale = sp.default_scale(d) if scale is None else scale
    lo, hi = (torch.zeros(Lq, dtype=torch.long, device="cuda"), torch.full((Lq,), Lk, device="cuda")) \
        if ranges is None else (ranges[:, 0].long().clamp(min=0), ranges[:, 1].long().clamp(max=Lk))
    at = torch.arange(Lq, device="cuda") + q_start
    for h in range(Hq):
        ref = R.attend(q[h], k[h * Hkv // Hq], v[h * Hkv // Hq], lo, hi, at, scale, softcap,
                       None if slopes is None else float(slopes[h]))
        R.assert_attention(o[h], lse[h], ref, f"{what} h={h}")
    return o, lse


def slopes_of(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,Lq,Lk", [(1, 1, 1, 1), (2, 1, 1, 700), (4, 2, 129, 63), (3, 3, 300, 300),
                                          (6, 2, 257, 640), (1, 1, 1000, 1025)])
def test_scored_plain(d, Hq, Hkv, Lq, Lk):
    g = gen(Hq + Lq + d)
    check_scored(randn(g, Hq, Lq, d), randn(g, Hkv, Lk, d), randn(g, Hkv, Lk, d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap,bias,spread", [(50.0, False, 1.0), (5.0, False, 3.0), (0.0, True, 1.0),
                                                 (20.0, True, 4.0)])
def test_scored_modified(d, softcap, bias, spread):
    g = gen(31 + d)
    q, k, v = randn(g, 4, 390, d, scale=spread), randn(g, 2, 390, d), randn(g, 2, 390, d)
    check_scored(q, k, v, softcap, slopes_of(4) if bias else None)
    check_scored(q[:, :100], k, v, softcap, slopes_of(4) if bias else None, q_start=290)
    check_scored(q[:, :100], k, v, softcap, slopes_of(4) * 40 if bias else None, q_start=-1000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap", [4000.0, 250.0])
def test_capped_scores_far_below_the_cap(d, softcap):
    """A row that sees one key has its score as log-sum. With one product per
    score, exact in fp32, a score is off by the tanh polynomial's 5.7e-7 and at
    most six roundings of 2^-24 (coefficients, square, steps, log 2), together
    below 1e-6; the logarithm adds MUFU's 2^-22 times its argument's exponent
    (the cache's weights stand at 2^7) and the final sums another 2^-22."""
    L = 64
    x = torch.linspace(-100.0, 100.0, L, device="cuda").bfloat16()
    q = torch.zeros(2, L, d, dtype=torch.bfloat16, device="cuda")
    q[:, :, 3] = x
    k = torch.zeros(2, L, d, dtype=torch.bfloat16, device="cuda")
    k[:, :, 3] = 1.0
    want = softcap * torch.tanh(x.double() / softcap)
    tol = 1e-6 * want.abs() + 9 * 2.0 ** -22
    at = torch.arange(L, device="cuda")
    ranges = torch.stack([at, at + 1], 1).int().contiguous()
    _, lse = sp.scored_attn(q, k, k, scale=1.0, softcap=softcap, ranges=ranges)
    assert ((lse.double() - want).abs() <= tol).all(), float(((lse.double() - want).abs() / tol).max())
    cache = sp.cache_append(sp.cache_alloc(1, 2, 64, d), k[None, :, :1], k[None, :, :1], i32([0]))
    _, lse = sp.cache_attn(q[None], cache, i32([1]), scale=1.0, softcap=softcap)
    assert ((lse.double() - want).abs() <= tol).all(), float(((lse.double() - want).abs() / tol).max())


@pytest.mark.parametrize("softcap,bias", [(0.0, False), (30.0, False), (0.0, True)])
def test_scored_documents_and_prefixes(softcap, bias):
    g = gen(41)
    L, starts, prefix = 777, [0, 1, 130, 131, 500, 770], [0, 40, 5, 0, 100000]
    q, k, v = randn(g, 2, L, 64), randn(g, 2, L, 64), randn(g, 2, L, 64)
    slopes = slopes_of(2) if bias else None
    for p in (None, prefix):
        r = sp.document_ranges(i32(starts), L, None if p is None else i32(p))
        want = []
        for t in range(L):
            i = max([j for j in range(5) if starts[j] <= t])
            if t >= starts[-1]:
                want.append([0, 0])
            elif p is None:
                want.append([starts[i], starts[i + 1]])
            else:
                want.append([starts[i], min(starts[i + 1], max(starts[i] + p[i], t + 1))])
        assert r.tolist() == want
        check_scored(q, k, v, softcap, slopes, r)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap,bias,masked", [(0.0, False, False), (0.0, False, True), (9.0, False, True),
                                                 (0.0, True, True), (9.0, True, False), (40.0, False, False)])
def test_scored_more_query_tiles_than_sms(d, softcap, bias, masked):
    """Pairs of query tiles and turns claimed from the counter: 40 heads of 6 tiles, odd tails."""
    g = gen(45 + d)
    L = 700
    q, k, v = randn(g, 40, L, d, scale=2.0), randn(g, 8, L, d), randn(g, 8, L, d)
    ranges = None
    if masked:
        ranges = sp.document_ranges(i32([0, 3, 260, 300, 655]), L, i32([0, 50, 1000, 120]))   # 45 rows see nothing
        ranges[400:420] = 0
    check_scored(q, k, v, softcap, slopes_of(40) if bias else None, ranges)


def test_scored_padding_in_pairs_may_hold_anything():
    g = gen(46)
    L = 700
    q, k, v = randn(g, 40, L, 64), randn(g, 4, L, 64), randn(g, 4, L, 64)
    ranges = torch.zeros(L, 2, dtype=torch.int32)
    ranges[:300] = torch.tensor([0, 300], dtype=torch.int32)
    ranges[420:690] = torch.tensor([420, 690], dtype=torch.int32)
    ranges = ranges.cuda()
    want = sp.scored_attn(q, k, v, ranges=ranges)
    for x in (k, v):
        x[:, 300:420] = math.nan
        x[:, 690:] = math.inf
    got = sp.scored_attn(q, k, v, ranges=ranges)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    sp.device_check()


def test_scored_arbitrary_ranges_and_empty_rows():
    """Ranges in any order, beyond the keys, reversed and empty; whole tiles of empty rows."""
    g = gen(42)
    q, k, v = randn(g, 2, 600, 128), randn(g, 1, 900, 128), randn(g, 1, 900, 128)
    a = torch.randint(-50, 950, (600, 2), generator=g)
    a[100:420] = torch.tensor([5, 5])
    a[421] = torch.tensor([900, 2000])
    a[422] = torch.tensor([-2 ** 31, 2 ** 31 - 1])
    ranges = a.to(torch.int32).cuda()
    check_scored(q, k, v, 0.0, None, ranges)
    check_scored(q, k, v, 8.0, slopes_of(2), ranges, q_start=77)
    o, lse = sp.scored_attn(q, k, v, ranges=torch.zeros(600, 2, dtype=torch.int32, device="cuda"))
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_scored_keys_that_no_row_sees_may_hold_anything():
    g = gen(43)
    L = 700
    q, k, v = randn(g, 2, L, 64), randn(g, 2, L, 64), randn(g, 2, L, 64)
    ranges = torch.zeros(L, 2, dtype=torch.int32)
    ranges[:200] = torch.tensor([0, 200], dtype=torch.int32)
    ranges[250:650] = torch.tensor([250, 650], dtype=torch.int32)
    ranges = ranges.cuda()
    want = sp.scored_attn(q, k, v, ranges=ranges)
    k2, v2 = k.clone(), v.clone()
    for t, x in ((k2, math.nan), (v2, math.nan)):
        t[:, 200:250] = x
        t[:, 650:] = math.inf
    got = sp.scored_attn(q, k2, v2, ranges=ranges)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # a row with a NaN query spoils nothing but itself
    q2 = q.clone()
    q2[:, 10] = math.nan
    got = sp.scored_attn(q2, k, v, ranges=ranges)
    keep = [r for r in range(L) if r != 10]
    assert torch.equal(want[0][:, keep], got[0][:, keep]) and torch.isnan(got[0][:, 10]).all()


def test_scored_strided_views_streams_and_graph():
    g = gen(44)
    qkv = randn(g, 333, 9, 64)
    q, k, v = (qkv[:, a:b].transpose(0, 1) for a, b in ((0, 6), (6, 7), (7, 8)))
    want, wl = check_scored(q.contiguous(), k.contiguous(), v.contiguous(), 9.0, slopes_of(6))
    o, lse = sp.scored_attn(q, k, v, softcap=9.0, slopes=slopes_of(6))
    assert torch.equal(o, want) and torch.equal(lse, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = sp.scored_attn(q, k, v, softcap=9.0, slopes=slopes_of(6), stream=s)
    s.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, wl)
    slopes, out, out_lse = slopes_of(6), torch.empty_like(want), torch.empty_like(wl)
    ws = torch.empty(sp.scored_attn_workspace_bytes(6, 333), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp.scored_attn(q, k, v, softcap=9.0, slopes=slopes, out=out, lse=out_lse, workspace=ws)
    ws.fill_(0xAB)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(out_lse, wl)


# ------------------------------------------------------------------ together

def test_block_wise_generation_with_the_cache():
    """Two blocks of a batch: project, rotate, append, attend; the cache's attention equals dense attention over
    the same (dequantised) keys, and the prompt's pass equals the dense entry point."""
    g = gen(51)
    N, Hq, Hkv, B, d, C = 2, 4, 2, 48, 64, 256
    cache = sp.cache_alloc(N, Hkv, C, d)
    done = [0, 0]
    for step, counts in enumerate(([48, 30], [48, 48])):
        qkv = randn(g, N * B, Hq + 2 * Hkv, d)
        pos = i32([[done[n] + b for n in range(N) for b in range(B)]])
        x = sp.rope_axes(qkv[:, :Hq + Hkv].transpose(0, 1), pos, (d // 2,)).view(Hq + Hkv, N, B, d).transpose(0, 1)
        v = qkv[:, Hq + Hkv:].view(N, B, Hkv, d).transpose(1, 2)
        sp.cache_append(cache, x[:, Hq:], v, i32(done), i32(counts))
        done = [a + b for a, b in zip(done, counts)]
        o, lse = sp.cache_attn(x[:, :Hq], cache, i32(done), slopes=slopes_of(Hq), q_start=i32([a - B for a in done]))
        sp.device_check()
        kd, vd = R.dequant(cache.k8, cache.k_scale), R.dequant(cache.v8, cache.v_scale)
        for n in range(N):
            od, ld = sp.scored_attn(x[n, :Hq], kd[n, :, :done[n]].bfloat16(), vd[n, :, :done[n]].bfloat16(),
                                    slopes=slopes_of(Hq), q_start=done[n] - B)
            # the same numbers through two kernels: each within its bound of the definition
            assert (o[n].double() - od.double()).abs().max() <= 2 * (2 * R.U_BF16 + 2.0 ** -10) * vd[n].abs().max()
            assert (lse[n] - ld).abs().max() <= 1e-3
    q, k, v = randn(g, 3, 500, 64), randn(g, 3, 500, 64), randn(g, 3, 500, 64)
    (a, la), (b, lb) = sp.scored_attn(q, k, v), sp.dense_attn(q, k, v)
    assert (a.double() - b.double()).abs().max() <= 2 * (2 * R.U_BF16 + 2.0 ** -10) * v.double().abs().max()
    assert (la - lb).abs().max() <= 1e-4
