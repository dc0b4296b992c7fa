"""Plain fp64 forms of the rotary, 8-bit cache and modified-score operators, and
the error bounds of the kernels against them (derived from roundings, before
any run)."""
import math

import torch

BLOCK = 64
E_MIN, E_MAX = -117, 119
U_BF16, U_E4M3 = 2.0 ** -8, 2.0 ** -4  # half a step, relative


def rope(x, pos, sections, theta, interleaved, shared, inverse):
    """x [H, L, d], pos [A, L]: (y, |a| + |b| of every element's pair) in fp64."""
    J = sum(sections)
    y = x.double().clone()
    amp = x.double().abs()
    j = 0
    for a, n in enumerate(sections):
        for i in range(n):
            t = pos[a].double() * theta ** (-(j / J if shared else i / n))
            c, s = torch.cos(t), torch.sin(t) * (-1 if inverse else 1)
            ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, J + j)
            xa, xb = x[..., ia].double(), x[..., ib].double()
            y[..., ia], y[..., ib] = xa * c - xb * s, xb * c + xa * s
            amp[..., ia] = amp[..., ib] = xa.abs() + xb.abs()
            j += 1
    return y, amp


def exponent(amax: float) -> int:
    """Smallest e with amax <= 448 * 2^e, within the scales' range."""
    if amax == 0.0:
        return E_MIN
    e = math.floor(math.log2(amax)) - 9
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return min(max(e, E_MIN), E_MAX)


def append(x, x8, scale, starts, counts):
    """CPU reference of one of K, V: x [N, H, B, d] bf16 into copies of x8
    (float8_e4m3fn), scale. Values exact in fp64, rounded by torch's cast."""
    x8, scale = x8.clone(), scale.clone()
    for n, (p, m) in enumerate(zip(starts, counts)):
        if m == 0:
            continue
        for blk in range(p // BLOCK, (p + m - 1) // BLOCK + 1):
            a, b = max(p, blk * BLOCK), min(p + m, (blk + 1) * BLOCK)
            for h in range(x.shape[1]):
                new = x[n, h, a - p:b - p].double()
                fin = new[torch.isfinite(new)]
                e = exponent(float(fin.abs().max()) if fin.numel() else 0.0)
                if blk * BLOCK < p:
                    old = int(round(math.log2(float(scale[n, h, blk]))))
                    e = max(e, old)
                    if e > old:
                        held = x8[n, h, blk * BLOCK:a].double() * 2.0 ** (old - e)
                        x8[n, h, blk * BLOCK:a] = held.float().to(torch.float8_e4m3fn)
                scale[n, h, blk] = 2.0 ** e
                q = (new * 2.0 ** -e).clamp(-448.0, 448.0)
                x8[n, h, a:b] = q.float().to(torch.float8_e4m3fn)
    return x8, scale


def dequant(x8, scale):
    N, H, C, d = x8.shape
    return (x8.double().view(N, H, C // BLOCK, BLOCK, d) * scale.double()[..., None, None]).view(N, H, C, d)


def attend(q, k, v, lo, hi, at, scale, softcap=0.0, slope=None):
    """One head in fp64: q [R, d], k, v [Lk, d], rows see keys [lo, hi). Returns
    o, lse, sum_c p |v| (per element) and scale * max|q| * sum_e |k| (the largest
    term a score can hold, per row)."""
    q, k, v = q.double(), k.double(), v.double()
    R, Lk = q.shape[0], k.shape[0]
    x = scale * (q @ k.T)
    if softcap > 0:
        x = softcap * torch.tanh(x / softcap)
    key = torch.arange(Lk, device=q.device)
    if slope is not None:
        x = x - slope * (at[:, None] - key[None]).abs().double()
    seen = (key >= lo[:, None]) & (key < hi[:, None])
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.max(1, keepdim=True).values if Lk else torch.full((R, 1), -math.inf, dtype=torch.float64, device=q.device)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(1, keepdim=True)
    empty = l == 0
    p = p / torch.where(empty, torch.ones_like(l), l)
    v = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))  # keys no row sees take no part
    lse = torch.where(empty, torch.full_like(l, -math.inf), m + torch.log(l)).squeeze(1)
    k = torch.where(seen.any(0)[:, None], k, torch.zeros_like(k))
    top = k.abs().sum(1).max() if Lk else torch.zeros((), dtype=torch.float64, device=q.device)
    return p @ v, lse, p @ v.abs(), scale * q.abs().max(1).values * top


def assert_attention(o, lse, ref, what=""):
    """ref: (o, lse, sum p|v|, score amplitude T) in fp64.

    A score is off by at most 2^-16 T + 2^-16: fp32 sums of d <= 128 exact
    products (128 * 2^-24 T = 2^-17 T), a query held as two e4m3 terms or bf16
    (2^-10 below its largest value 224 or more, 2^-17.8 T), and the bounded
    errors of the capped score, bias, fp32 exp and log near 1 (2^-16 covers a
    capped score of 100: 100 * 2^-23 several times over, and MUFU's 2^-22). A
    weight then carries 2 * that twice (numerator and sum), and its rounding to
    16 bits, at most half a bf16 step 2^-8; the output one more 2^-8."""
    ro, rl, av, amp = ref
    ds = 2.0 ** -16 * amp + 2.0 ** -16
    o, lse = o.double(), lse.double()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(rl)), f"{what}: empty rows differ"
    tol = (U_BF16 + 4 * ds)[:, None] * av + U_BF16 * ro.abs() + 1e-30
    bad = ((o - ro).abs() - tol)
    assert not torch.isnan(bad).any(), f"{what}: NaN"
    assert bad.max() <= 0, f"{what}: O off by {(o - ro).abs().max():.3e}, {float(((o - ro).abs() / tol).max()):.2f} of the bound"
    fin = ~torch.isneginf(rl)
    if fin.any():
        ltol = (2 * ds + 2.0 ** -20 * rl.abs())[fin]
        err = (lse - rl).abs()[fin]
        assert (err <= ltol).all(), f"{what}: LSE off by {err.max():.3e}, {float((err / ltol).max()):.2f} of the bound"
