"""Orders that the kernels have to establish by themselves, checked without a
GPU: on the source, or on a model of which phases of an mbarrier a warp knows
to be complete when it waits for the next one."""
import os
import re

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
