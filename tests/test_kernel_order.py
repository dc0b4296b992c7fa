"""Orders that the kernels have to establish by themselves, checked without a
GPU: on the source, or on a model of which phases of an mbarrier a warp knows
to be complete when it waits for the next one."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_bidirectional_select_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel_body(text, name):
    """The text between the braces of a kernel's definition."""
    at = re.search(r"\b%s\s*\(const __grid_constant__|\b%s\s*\(" % (name, name), text).start()
    start = text.index(") {", at) + 2
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(f"{name}: unbalanced braces")


def returns_before_a_wait(body):
    """`return`s that can be reached without a grid_dep_wait: none stands before
    them in their own block or in one around it."""
    waited, bad = [False], []
    for m in re.finditer(r"[{}]|\bgrid_dep_wait\s*\(\)|\breturn\b", body):
        if m.group() == "{":
            waited.append(waited[-1])
        elif m.group() == "}":
            waited.pop()
        elif m.group() == "return":
            if not waited[-1]:
                bad.append(body[max(0, m.start() - 60):m.end()].strip())
        else:
            waited[-1] = True
    return bad


@pytest.mark.parametrize("file,kernel", [("cache_attn_kernel.cuh", "cache_merge_kernel"),
                                         ("losa_kernels.cuh", "losa_lists_kernel"),
                                         ("losa_kernels.cuh", "losa_merge_kernel")])
def test_programmatic_dependents_wait_before_they_return(file, kernel):
    """A kernel launched as a programmatic dependent may begin before the one
    ahead of it has ended; what follows on the stream is ordered behind the
    dependent only. So each of its threads waits for the kernel ahead before it
    returns, on every path."""
    body = kernel_body(source(file), kernel)
    assert "grid_dep_wait" in body
    assert returns_before_a_wait(body) == []


def test_the_return_scan_finds_an_early_return():
    assert returns_before_a_wait("{ if (x) return; grid_dep_wait(); }")
    assert returns_before_a_wait("{ if (x) { grid_dep_wait(); } return; }")
    assert not returns_before_a_wait("{ if (x) { grid_dep_wait(); return; } grid_dep_wait(); if (y) return; }")


# ------------------------------------------------------------------ phases of an mbarrier

class Waiter:
    """What one warp knows about operations that complete in order and arrive
    alternately on two barriers. A wait for operation n looks at one bit: it
    can only tell phase n from n - 2, so n - 2 has to be known complete."""

    def __init__(self):
        self.known = -1

    def wait(self, n):
        if n >= 0:
            assert n <= self.known or n - 2 <= self.known, f"the wait for {n} may pass at {n - 2}: known {self.known}"
            self.known = max(self.known, n)


def softmax_waits(parts, hw, next_copy, mended=True):
    """cache_attn_kernel, few rows: the waits on PV of a softmax warp of parity
    hw over a run's parts (numbers of tiles), rescaling O at each of its tiles.
    next_copy: count what it learns where the warps join for the next part's Q."""
    w, g0 = Waiter(), 0
    for i, cnt in enumerate(parts):
        skip = (g0 ^ hw) & 1
        for jj in range(skip, cnt, 2):
            g = g0 + jj
            if jj > skip:           # a rescale
                w.wait(g - 2)
                w.wait(g - 1)
            w.wait(g - 2)           # before P is stored
        g = g0 + cnt
        if next_copy and i + 1 < len(parts):
            w.known = max(w.known, g - 3)   # the join of the next part's copy: tile g - 1's owners waited for g - 3
        if mended:
            w.wait(g - 2)
        w.wait(g - 1)
        g0 = g


PARTS = [[n] for n in range(1, 9)] + [[a, b, c] for a in (1, 2, 3, 4) for b in (1, 2, 5) for c in (1, 3, 4)]


@pytest.mark.parametrize("hw", [0, 1])
def test_cache_attention_waits_tell_their_phase(hw):
    for parts in PARTS:
        softmax_waits(parts, hw, next_copy=False)
    with pytest.raises(AssertionError, match="may pass"):
        for parts in PARTS:
            softmax_waits(parts, hw, next_copy=True, mended=False)   # a run's last part has no join before its end


def test_cache_attention_epilogue_waits_for_the_tile_before_the_last():
    body = kernel_body(source("cache_attn_kernel.cuh"), "cache_attn_kernel")
    at = body.index("if (have) {")
    assert re.match(r"if \(have\) \{\s*if \(!pv_before\(g, g & 1\) \|\|\s*!ptx::mbar_wait_warp\(bar\(C::B_PVDONE "
                    r"\+ \(\(g - 1\) & 1\)\)", body[at:])


# ------------------------------------------------------------------ ring stages of the two-tile kernels

class RingWaiter:
    """What a warp knows about loads that complete in any order: those that it
    waited for, and those whose stage was loaded again before one of them (the
    producer loads in order, and a stage only when its last load was consumed)."""

    def __init__(self, stages):
        self.stages, self.waited, self.top = stages, set(), -1

    def wait(self, seq):
        p = seq - self.stages
        assert p < 0 or p in self.waited or p + self.stages <= self.top, f"the wait for load {seq} may pass at {p}"
        self.waited.add(seq)
        self.top = max(self.top, seq)


def ring_waits(stages, split, turns, slot, lands=True):
    """The loads that an issuer of scored_attn_kernel or attn_fwd_kernel waits
    for: K_j is load 2 j, V_j load 2 j + 1. turns: (tiles, whether slot 1 has a
    query tile). lands: after a turn without, the producer waits for its loads
    before it publishes the next one, of which the issuers learn after that."""
    w, seq = RingWaiter(stages), 0
    for tiles, has1 in turns:
        for j in range(tiles):
            if (j & 1) == slot if split else (slot == 0 or has1):
                w.wait(seq)
                w.wait(seq + 1)
            seq += 2
        if lands and not split and not has1:
            w.waited.update(range(seq))
            w.top = max(w.top, seq - 1)


TURNS = [[(n, b) for n in (1, 2, 3, 9)] + [(5, True), (7, False), (4, True)] for b in (False, True)]


def test_ring_waits_tell_their_phase(tmp_path):
    """With the ring sizes of the build, compiled from its headers."""
    from block_sparse_bidirectional_select_b200.build import CSRC as csrc, nvcc_path
    src, exe = tmp_path / "ring.cu", tmp_path / "ring"
    src.write_text('#include <cstdio>\n#include "scored_kernel.cuh"\nusing namespace sparsed;\n'
                   'int main() { std::printf("%d %d %d %d %d %d %d %d\\n", ScoredCfg<64>::NST, ScoredCfg<64>::NST_SPLIT, '
                   'ScoredCfg<128>::NST, ScoredCfg<128>::NST_SPLIT, AttnCfg<64, 64>::NST, AttnCfg<64, 128>::NST, '
                   'AttnCfg<128, 64>::NST, AttnCfg<128, 128>::NST); }\n')
    subprocess.run([nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-I", csrc, "-o",
                    str(exe), str(src)], check=True)
    sizes = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    for slot in (0, 1):
        for ring, ring_split in (sizes[:2], sizes[2:4]):
            ring_waits(ring_split, True, [(40, False)], slot)
        for ring in (sizes[0], sizes[2], *sizes[4:]):
            for turns in TURNS:
                ring_waits(ring, False, turns, slot)


def test_the_ring_model_finds_the_unsafe_forms():
    with pytest.raises(AssertionError, match="may pass"):
        ring_waits(5, True, [(8, False)], 0)
    with pytest.raises(AssertionError, match="may pass"):
        ring_waits(5, False, [(3, False), (3, True)], 1, lands=False)
    # the split form has its own ring, and the producers wait at the end of such a turn
    body = kernel_body(source("scored_kernel.cuh"), "scored_attn_kernel")
    assert "constexpr int NST = SPLIT ? S::NST_SPLIT : S::NST;" in body
    for text, given in ((body, "!split && !pr.has1"),
                        (kernel_body(source("attn_kernel.cuh"), "attn_fwd_kernel"), "!pr.has1")):
        assert re.search(r"ok = load_tile\(&tm_v, \w+\);\s*\}\s*if \(%s\)\s*for \(int u = seq > NST \? seq - NST : 0; ok && "
                         r"u < seq; \+\+u\) ok = wait\(C::B_FULL \+ u %% NST, u / NST\);\s*w = w_next;" % re.escape(given), text)
