"""Workloads of the operators around block-wise generation: rotary positions
with several axes, the 8-bit block-scaled cache (append, attention) and dense
attention with modified scores.

Each case is one call as a generation or scoring program makes it. `run` is the
call in plain torch (fp32, fp64 for angles) or, with `own`, through the
package's entry points; `exact` is the definition in fp64.
"""
import math
import random

import torch

own = False

QUANT_BLOCK = 64          # tokens that share a scale
E4M3_MAX = 448.0
E_MIN, E_MAX = -117, 119  # range of a scale's exponent


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the q and k heads of one 64-token block during block-wise generation (latency)
        dict(name="rope_block", op="rope", H=40, Hv=8, L=64, d=128, sections="64", interleaved=False,
             shared=False, far=32768),
        # a clip's tokens: time, height and width share one ladder of frequencies; odd length
        dict(name="rope_video", op="rope", H=40, Hv=8, L=8190, d=128, sections="16,24,24", interleaved=False,
             shared=True, far=0),
        # images of a long context: height and width, adjacent pairs, a ladder for each axis
        dict(name="rope_image", op="rope", H=32, Hv=32, L=32768, d=128, sections="32,32", interleaved=True,
             shared=False, far=0),
        # one new token of each of 16 sequences into the cache (latency)
        dict(name="append_token", op="append", N=16, H=8, B=1, C=8192, d=128, ragged=False),
        # a finished 64-token block of each of 8 sequences, some of them shorter
        dict(name="append_block", op="append", N=8, H=8, B=64, C=32768, d=128, ragged=True),
        # two prompts into an empty cache
        dict(name="append_prompt", op="append", N=2, H=32, B=16384, C=16384, d=128, ragged=False),
        # single-token step of one sequence, 8 kv heads shared by 32 q heads (latency)
        dict(name="cache_token", op="cache", N=1, Hq=32, Hkv=8, B=1, C=8192, d=128, ragged=False, softcap=0.0,
             bias=False),
        # single-token steps of a batch with mixed lengths and capped scores
        dict(name="cache_batch", op="cache", N=32, Hq=32, Hkv=8, B=1, C=16384, d=128, ragged=True, softcap=30.0,
             bias=False),
        # denoising step of a 64-token block on a 32768-token prefix, distance bias
        dict(name="cache_block", op="cache", N=2, Hq=32, Hkv=32, B=64, C=32768, d=128, ragged=False, softcap=0.0,
             bias=True),
        # short packed documents (latency)
        dict(name="scored_packed", op="scored", Hq=8, Hkv=8, L=1000, d=64, softcap=0.0, bias=False, docs=5,
             prefix=-1),
        # one long sequence with capped scores
        dict(name="scored_softcap", op="scored", Hq=32, Hkv=32, L=8192, d=128, softcap=50.0, bias=False, docs=1,
             prefix=-1),
        # packed documents, each with a prompt seen by all its tokens and a causal rest, distance bias, odd length
        dict(name="scored_prefix", op="scored", Hq=32, Hkv=8, L=8190, d=128, softcap=0.0, bias=True, docs=3,
             prefix=700),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "cache", "scored"))
    d = rng.choice((64, 128))
    if op == "rope":
        H = rng.randint(1, 64)
        L = _log_int(rng, 1, min(32768, (1 << 27) // (H * d)))
        axes = rng.randint(1, 3)
        pairs = d // 2 if rng.random() < 0.7 else d // 4
        ends = [0] + sorted(rng.sample(range(1, pairs), axes - 1)) + [pairs]
        return dict(op="rope", H=H, Hv=rng.randint(0, 16), L=L, d=d,
                    sections=",".join(str(b - a) for a, b in zip(ends, ends[1:])),
                    interleaved=rng.random() < 0.5, shared=rng.random() < 0.5, far=rng.choice((0, 1000, 1000003)))
    if op == "append":
        N, H = _log_int(rng, 1, 64), _log_int(rng, 1, 32)
        B = _log_int(rng, 1, max(1, min(16384, (1 << 27) // (N * H * d))))
        room = (1 << 28) // (N * H * d) // QUANT_BLOCK
        C = QUANT_BLOCK * (-(-B // QUANT_BLOCK) + rng.randint(0, max(0, min(64, room))))
        return dict(op="append", N=N, H=H, B=B, C=C, d=d, ragged=rng.random() < 0.5)
    softcap = rng.choice((0.0, 0.0, 20.0, 50.0))
    bias = rng.random() < 0.4
    if op == "cache":
        Hkv = rng.choice((1, 2, 4, 8, 16, 32))
        group = rng.choice([g for g in (1, 2, 3, 4, 8) if g * Hkv <= 64])
        N = _log_int(rng, 1, 32)
        C = QUANT_BLOCK * _log_int(rng, 1, max(1, min(1024, (1 << 28) // (N * Hkv * d * QUANT_BLOCK))))
        B = min(rng.choice((1, 1, 1, 4, 16, 32, 61, 64)), C, max(1, (1 << 27) // (N * group * Hkv * C)))
        return dict(op="cache", N=N, Hq=group * Hkv, Hkv=Hkv, B=B, C=C, d=d, ragged=rng.random() < 0.6,
                    softcap=softcap, bias=bias)
    Hkv = rng.choice((1, 2, 4, 8, 32))
    group = rng.choice([g for g in (1, 2, 4) if g * Hkv <= 32])
    L = _log_int(rng, 1, min(16384, int(math.sqrt((1 << 31) / (group * Hkv)))))
    return dict(op="scored", Hq=group * Hkv, Hkv=Hkv, L=L, d=d, softcap=softcap, bias=bias,
                docs=rng.randint(1, min(8, L)), prefix=rng.choice((-1, -1, 0, 100, 1000)))


# ------------------------------------------------------------------ what a case fixes

def _sections(c):
    return [int(x) for x in c["sections"].split(",")]


def _doc_starts(c):
    """Boundaries of a case's documents: uneven, the first at 0, the last at L."""
    r = random.Random(c["L"] * 31 + c["docs"])
    cuts = sorted(r.sample(range(1, c["L"]), c["docs"] - 1)) if c["docs"] > 1 else []
    return [0] + cuts + [c["L"]]


def _ranges(c):
    """Visible keys [lo, hi) of every token: its document, all of it (prefix
    -1) or the document's first `prefix` tokens and those up to its own."""
    lo, hi = [], []
    starts = _doc_starts(c)
    for a, b in zip(starts, starts[1:]):
        lo += [a] * (b - a)
        hi += [b] * (b - a) if c["prefix"] < 0 else [min(b, max(a + c["prefix"], r + 1)) for r in range(a, b)]
    return lo, hi


def _lengths(c):
    r = random.Random(c["C"] * 31 + c["N"])
    if not c["ragged"]:
        return [c["C"]] * c["N"]
    return [r.randint(c["B"], c["C"]) for _ in range(c["N"])]


def _starts_counts(c):
    """Where each sequence's new tokens begin, and how many they are."""
    r = random.Random(c["C"] * 31 + c["N"])
    counts = [r.randint(1, c["B"]) if c["ragged"] else c["B"] for _ in range(c["N"])]
    return [r.randint(0, c["C"] - n) for n in counts], counts


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["H"] * c["L"] * c["d"]
        return {"bytes": 4 * n + 4 * c["L"] * len(_sections(c)), "flops": 3 * n}
    if c["op"] == "append":
        starts, counts = _starts_counts(c)
        blocks = sum((s + n - 1) // QUANT_BLOCK - s // QUANT_BLOCK + 1 for s, n in zip(starts, counts))
        # bf16 in, 8 bits out; the tokens already in a shared first block change only where its scale grows
        return {"bytes": 2 * c["H"] * (3 * sum(counts) * c["d"] + 4 * blocks), "flops": 2 * c["H"] * sum(counts) * c["d"]}
    if c["op"] == "cache":
        keys = sum(_lengths(c))
        rows = c["N"] * c["Hq"] * c["B"]
        blocks = sum(-(-n // QUANT_BLOCK) for n in _lengths(c))
        return {"bytes": c["Hkv"] * (2 * keys * c["d"] + 8 * blocks) + rows * (4 * c["d"] + 4),
                "flops": 4 * c["Hq"] * c["B"] * keys * c["d"]}
    lo, hi = _ranges(c)
    pairs = sum(max(0, h - l) for l, h in zip(lo, hi))
    return {"bytes": 4 * c["L"] * c["d"] * (c["Hq"] + c["Hkv"]) + 4 * c["Hq"] * c["L"], "flops": 4 * c["Hq"] * pairs * c["d"]}


# ------------------------------------------------------------------ inputs

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _slopes(H):
    """The geometric slopes of a linear distance bias, one for each head."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32, device="cuda")


def _codes(g, shape):
    """Cache content of about unit variance: e4m3 values and a power of two for each block of tokens."""
    N, H, C, d = shape
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(96.0)
    x = x.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    e = torch.randint(-8, -5, (N, H, C // QUANT_BLOCK), generator=g, device="cuda")
    return x, torch.exp2(e.float())


def _frequencies(c):
    """Angle per position of every pair, and the pair's axis."""
    sections, theta = _sections(c), 10000.0
    J, j, inv, axis = sum(sections), 0, [], []
    for a, n in enumerate(sections):
        for i in range(n):
            inv.append(theta ** (-(j / J if c["shared"] else i / n)))
            axis.append(a)
            j += 1
    return torch.tensor(inv, dtype=torch.float64, device="cuda"), torch.tensor(axis, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    s = dict(case=c)
    if c["op"] == "rope":
        # the projection's output: a token's q and k heads, then its v heads
        s["qkv"] = randn(c["L"], c["H"] + c["Hv"], c["d"])
        t = torch.arange(c["L"], device="cuda")
        side = max(1, int(math.sqrt(c["L"])) // 2)
        axes = {1: [t], 2: [t // side, t % side], 3: [t // (side * side), t // side % side, t % side]}
        off = int(torch.randint(0, c["far"] + 1, (1,), generator=g, device="cuda"))
        s["pos"] = torch.stack([p + off for p in axes[len(_sections(c))]]).to(torch.int32)
        s["inv"], s["axis"] = _frequencies(c)
    elif c["op"] == "append":
        # the projection's output: a token's k heads and v heads side by side
        s["kv"] = randn(c["N"], c["B"], 2 * c["H"], c["d"])
        starts, counts = _starts_counts(c)
        s["start"], s["count"] = _i32(starts), _i32(counts)
        s["k8"], s["ks"] = _codes(g, (c["N"], c["H"], c["C"], c["d"]))
        s["v8"], s["vs"] = _codes(g, (c["N"], c["H"], c["C"], c["d"]))
    elif c["op"] == "cache":
        s["q"] = randn(c["N"], c["Hq"], c["B"], c["d"])
        s["k8"], s["ks"] = _codes(g, (c["N"], c["Hkv"], c["C"], c["d"]))
        s["v8"], s["vs"] = _codes(g, (c["N"], c["Hkv"], c["C"], c["d"]))
        s["len"] = _i32(_lengths(c))
        s["slopes"] = _slopes(c["Hq"]) if c["bias"] else None
    else:
        s["q"] = randn(c["Hq"], c["L"], c["d"])
        s["k"], s["v"] = randn(c["Hkv"], c["L"], c["d"]), randn(c["Hkv"], c["L"], c["d"])
        s["ranges"] = _i32(list(zip(*_ranges(c)))) if c["docs"] > 1 or c["prefix"] >= 0 else None
        s["slopes"] = _slopes(c["Hq"]) if c["bias"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _rope(s):
    c, inv, axis = s["case"], s["inv"], s["axis"]
    angle = s["pos"].double()[axis].t() * inv                      # [L, J]
    cos, sin = angle.cos().float(), angle.sin().float()
    x = s["qkv"][:, :c["H"]].transpose(0, 1).float()               # [H, L, d]
    r = 2 * inv.numel()
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., r:]), dim=-1).to(torch.bfloat16)


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, within the scales' range."""
    m, x = torch.frexp(amax / E4M3_MAX)                            # amax/448 = m * 2^x, m in [0.5, 1)
    e = torch.where(m == 0.5, x - 1, x)
    return torch.where(amax == 0, torch.full_like(e, E_MIN), e).clamp(E_MIN, E_MAX)


def _append_plain(x, x8, scale, start, count):
    """x [N, H, B, d] into x8 [N, H, C, d] at each sequence's start."""
    N, H, B, d = x.shape
    C = x8.shape[2]
    nb = C // QUANT_BLOCK
    pos = start.long()[:, None] + torch.arange(B, device=x.device)             # [N, B]
    there = torch.arange(B, device=x.device) < count[:, None]
    blk = torch.where(there, pos // QUANT_BLOCK, torch.full_like(pos, nb))     # block nb: dropped
    x = x.float()
    amax = torch.zeros(N, H, nb + 1, device=x.device).scatter_reduce(
        2, blk[:, None, :].expand(N, H, B), x.abs().amax(-1), "amax")[..., :nb]
    j = torch.arange(nb, device=x.device)
    first = start.long()[:, None] // QUANT_BLOCK
    touched = (j >= first) & (j * QUANT_BLOCK < (start + count)[:, None])      # [N, nb]
    shared = (j == first) & (start[:, None] % QUANT_BLOCK > 0) & touched       # holds older tokens
    e_old = torch.frexp(scale)[1] - 1
    e_new = _exponent(amax)
    e = torch.where(shared[:, None], torch.maximum(e_old, e_new), torch.where(touched[:, None], e_new, e_old))
    scale.copy_(torch.exp2(e.float()))
    # the shared block's older tokens at its new scale
    n = torch.arange(N, device=x.device)
    rows = (first * QUANT_BLOCK + torch.arange(QUANT_BLOCK, device=x.device)).clamp(max=C - 1)   # [N, 64]
    older = (rows < start.long()[:, None])[:, None, :, None]
    held = x8[n[:, None], :, rows].transpose(1, 2).float()                     # [N, H, 64, d]
    step = torch.exp2((e_old - e).float()).gather(2, first[:, None].clamp(max=nb - 1).expand(N, H, 1))
    moved = torch.where(older, held * step[..., None], held).to(x8.dtype)
    x8[n[:, None], :, rows] = moved.transpose(1, 2)
    inv = torch.exp2(-e.float()).gather(2, blk.clamp(max=nb - 1)[:, None].expand(N, H, B))
    y = (x * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(x8.dtype)
    at = torch.where(there)
    x8[at[0], :, pos[at]] = y[at[0], :, at[1]]
    return x8, scale


def _modified(scores, softcap, slopes, distance):
    if softcap > 0:
        scores = softcap * torch.tanh(scores / softcap)
    if slopes is not None:
        scores = scores - slopes * distance
    return scores


def _attend(scores, v):
    """softmax(scores) v and its log-sum; a row of -inf gives 0 and -inf."""
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    return o, (m + torch.log(l)).squeeze(-1)


def _cache(s):
    c = s["case"]
    N, Hq, Hkv, B, C, d = (c[k] for k in ("N", "Hq", "Hkv", "B", "C", "d"))
    k = (s["k8"].float().view(N, Hkv, -1, QUANT_BLOCK, d) * s["ks"][..., None, None]).view(N, Hkv, C, d)
    v = (s["v8"].float().view(N, Hkv, -1, QUANT_BLOCK, d) * s["vs"][..., None, None]).view(N, Hkv, C, d)
    x = torch.matmul(s["q"].float().reshape(N, Hkv, -1, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    x = x.view(N, Hq, B, C)
    key = torch.arange(C, device=x.device)
    at = (s["len"][:, None] - B + torch.arange(B, device=x.device))[:, None, :, None]   # the cache's last B tokens
    x = _modified(x, c["softcap"], None if s["slopes"] is None else s["slopes"][:, None, None], (at - key).abs())
    x = x.masked_fill(key >= s["len"][:, None, None, None], -math.inf)
    o, lse = _attend(x.view(N, Hkv, -1, C), v)
    return o.view(N, Hq, B, d).to(torch.bfloat16), lse.view(N, Hq, B)


def _scored(s):
    c = s["case"]
    Hq, Hkv, L, d = (c[k] for k in ("Hq", "Hkv", "L", "d"))
    x = torch.matmul(s["q"].float().reshape(Hkv, -1, d), s["k"].float().transpose(1, 2)) * (1.0 / math.sqrt(d))
    x = x.view(Hq, L, L)
    key = torch.arange(L, device=x.device)
    x = _modified(x, c["softcap"], None if s["slopes"] is None else s["slopes"][:, None, None],
                  (key[:, None] - key).abs())
    if s["ranges"] is not None:
        x = x.masked_fill((key < s["ranges"][:, :1]) | (key >= s["ranges"][:, 1:]), -math.inf)
    o, lse = _attend(x.view(Hkv, -1, L), s["v"].float())
    return o.view(Hq, L, d).to(torch.bfloat16), lse.view(Hq, L)


def _append_views(s):
    """The k and v heads of the projection's output, [N, H, B, d] each."""
    kv = s["kv"].transpose(1, 2)
    return kv[:, :s["case"]["H"]], kv[:, s["case"]["H"]:]


def run(state):
    s, c = state, state["case"]
    if own:
        import block_sparse_bidirectional_select_b200 as sp
        if c["op"] == "rope":
            return sp.rope_axes(s["qkv"][:, :c["H"]].transpose(0, 1), s["pos"], _sections(c),
                                interleaved=c["interleaved"], shared_ladder=c["shared"])
        if c["op"] == "append":
            k, v = _append_views(s)
            sp.cache_append(sp.Cache8(s["k8"], s["v8"], s["ks"], s["vs"]), k, v, s["start"], s["count"])
            return s["k8"], s["ks"], s["v8"], s["vs"]
        if c["op"] == "cache":
            return sp.cache_attn(s["q"], sp.Cache8(s["k8"], s["v8"], s["ks"], s["vs"]), s["len"],
                                 softcap=c["softcap"], slopes=s["slopes"])
        return sp.scored_attn(s["q"], s["k"], s["v"], softcap=c["softcap"], slopes=s["slopes"], ranges=s["ranges"])
    if c["op"] == "rope":
        return _rope(s)
    if c["op"] == "append":
        k, v = _append_views(s)
        # e4m3 values and, beside them, the scales that multiply them
        return _append_plain(k, s["k8"], s["ks"], s["start"], s["count"]) + _append_plain(
            v, s["v8"], s["vs"], s["start"], s["count"])
    if c["op"] == "cache":
        return _cache(s)
    return _scored(s)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(s):
    c, inv, axis = s["case"], s["inv"], s["axis"]
    out = s["qkv"][:, :c["H"]].transpose(0, 1).double().contiguous()
    J = inv.numel()
    for j in range(J):
        a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, J + j)
        z = torch.polar(torch.ones(c["L"], dtype=torch.float64, device="cuda"), s["pos"][axis[j]].double() * inv[j])
        y = torch.complex(out[..., a], out[..., b]) * z
        out[..., a], out[..., b] = y.real, y.imag
    return out


def _exact_append(x, x8, scale, starts, counts):
    """Stored values before their rounding to e4m3, and the scales; one block of tokens at a time."""
    values, scales = x8.double(), scale.double().clone()
    for n, (p, m) in enumerate(zip(starts, counts)):
        for j in range(p // QUANT_BLOCK, (p + m - 1) // QUANT_BLOCK + 1):
            a, b = max(p, j * QUANT_BLOCK), min(p + m, (j + 1) * QUANT_BLOCK)
            new = x[n, :, a - p:b - p].double()
            e = torch.ceil(torch.log2(new.abs().amax((1, 2)) / E4M3_MAX)).clamp(E_MIN, E_MAX)
            if j * QUANT_BLOCK < p:
                was = torch.log2(scales[n, :, j])
                e = torch.maximum(e, was)
                values[n, :, j * QUANT_BLOCK:a] *= torch.exp2(was - e)[:, None, None]
            scales[n, :, j] = torch.exp2(e)
            values[n, :, a:b] = new * torch.exp2(-e)[:, None, None]
    return values, scales


def _exact_rows(q, k, v, lo, hi, at, scale, softcap, slope):
    """One head: softmax over the keys [lo, hi) of each row, with scores as defined."""
    x = scale * (q @ k.T)
    if softcap > 0:
        x = softcap * torch.tanh(x / softcap)
    key = torch.arange(k.shape[0], device=x.device)
    if slope is not None:
        x = x - slope * (at[:, None] - key[None, :]).abs()
    x = torch.where((key >= lo[:, None]) & (key < hi[:, None]), x, -math.inf)
    return torch.softmax(x, -1) @ v, torch.logsumexp(x, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        return _exact_rope(s)
    if c["op"] == "append":
        starts, counts = _starts_counts(c)
        if sum(n // QUANT_BLOCK + 2 for n in counts) > 4096:
            return None
        k, v = _append_views(s)
        return _exact_append(k, s["k8"], s["ks"], starts, counts) + _exact_append(v, s["v8"], s["vs"], starts, counts)
    if c["op"] == "cache":
        group = c["Hq"] // c["Hkv"]
        o = torch.empty(c["N"], c["Hq"], c["B"], c["d"], dtype=torch.float64, device="cuda")
        lse = torch.empty(c["N"], c["Hq"], c["B"], dtype=torch.float64, device="cuda")
        for n, length in enumerate(_lengths(c)):
            at = torch.arange(length - c["B"], length, device="cuda")
            lo, hi = torch.zeros_like(at), torch.full_like(at, length)
            for h in range(c["Hq"]):
                k, v = ((t8[n, h // group, :length].double()
                         * sc[n, h // group].double().repeat_interleave(QUANT_BLOCK)[:length, None])
                        for t8, sc in ((s["k8"], s["ks"]), (s["v8"], s["vs"])))
                o[n, h], lse[n, h] = _exact_rows(s["q"][n, h].double(), k, v, lo, hi, at, 1 / math.sqrt(c["d"]),
                                                 c["softcap"], None if s["slopes"] is None else s["slopes"][h].double())
        return o, lse
    lo, hi = (torch.tensor(t, device="cuda") for t in _ranges(c))
    at = torch.arange(c["L"], device="cuda")
    heads = [_exact_rows(s["q"][h].double(), s["k"][h * c["Hkv"] // c["Hq"]].double(),
                         s["v"][h * c["Hkv"] // c["Hq"]].double(), lo, hi, at, 1 / math.sqrt(c["d"]), c["softcap"],
                         None if s["slopes"] is None else s["slopes"][h].double()) for h in range(c["Hq"])]
    return torch.stack([o for o, _ in heads]), torch.stack([l for _, l in heads])
