"""The rotary, 8-bit cache and modified-score calls as programs make them: on
streams, in captured graphs, with buffers of the caller's."""
import math

import pytest
import torch

import block_sparse_bidirectional_select_b200 as sp
import serve_ref as R
from test_gpu_serve_ops import check_cache_attn, check_scored, gen, i32, randn, random_cache, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,lengths", [(1, [1, 40, 64, 7]), (70, [128, 70, 100, 99])])
def test_short_sequences_are_ordered_before_what_follows(B, lengths):
    """Each item lies whole in one run, so nothing is joined: what follows the call in a captured graph reads its
    output at once."""
    g = gen(61 + B)
    c = random_cache(g, 4, 2, 128, 128)
    q, n = randn(g, 4, 4, B, 128), i32(lengths)
    want, wl = check_cache_attn(q, c, lengths)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    ws = torch.empty(sp.cache_attn_workspace_bytes(4, 4, 2, B, 128), dtype=torch.uint8, device="cuda")
    copies = [(torch.empty_like(want), torch.empty_like(wl)) for _ in range(10)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for co, cl in copies:
            out.fill_(3.0)
            lse.fill_(3.0)
            sp.cache_attn(q, c, n, out=out, lse=lse, workspace=ws)
            co.copy_(out)
            cl.copy_(lse)
    for _ in range(20):
        graph.replay()
        for co, cl in copies:
            assert torch.equal(co, want) and torch.equal(cl, wl)
    sp.device_check()


@pytest.mark.parametrize("d,Lq,Lk", [(128, 130, 5000), (128, 64, 20000), (64, 130, 5000)])
def test_scored_few_query_tiles_over_many_keys(d, Lq, Lk):
    """A query tile's keys in two slots with a ring of their own: the same bits on every call."""
    g = gen(62 + Lq)
    q, k, v = randn(g, 8, Lq, d), randn(g, 2, Lk, d), randn(g, 2, Lk, d)
    ranges = torch.stack([torch.arange(Lq) * 7, Lk - torch.arange(Lq) * 11], 1).to(torch.int32).cuda()
    for r in (None, ranges):
        first = check_scored(q, k, v, 0.0, slopes_of(8), r, q_start=Lk - Lq)
        for _ in range(20):
            again = sp.scored_attn(q, k, v, slopes=slopes_of(8), ranges=r, q_start=Lk - Lq)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    sp.device_check()


@pytest.mark.parametrize("d", [64, 128])
def test_scored_odd_query_tiles(d):
    """Heads of an odd number of query tiles, so that the last pair of each has one: more pairs than SMs."""
    g = gen(63 + d)
    q, k, v = randn(g, 90, 300, d), randn(g, 9, 900, d), randn(g, 9, 900, d)
    first = check_scored(q, k, v)
    for _ in range(10):
        again = sp.scored_attn(q, k, v)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    sp.device_check()


def test_calls_back_to_back_on_two_streams():
    """A call on the current stream and one with ``stream=``, at once and with buffers of the library's: the second
    one's do not come from memory that the first is still using. Nothing synchronises in between."""
    g = gen(64)
    c = random_cache(g, 4, 4, 16384, 128)
    n = i32([16384, 9000, 12345, 16000])
    q1, q2 = randn(g, 4, 16, 1, 128), randn(g, 4, 16, 1, 128)
    want1, want2 = sp.cache_attn(q1, c, n), sp.cache_attn(q2, c, n)
    sq1, sq2, k, v = (randn(g, h, 3000, 64) for h in (160, 160, 8, 8))
    swant1, swant2 = sp.scored_attn(sq1, k, v), sp.scored_attn(sq2, k, v)
    x, pos = randn(g, 16, 4000, 128), i32([list(range(4000))])
    rwant = sp.rope_axes(x, pos, (64,))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got1, got2 = sp.cache_attn(q1, c, n), sp.cache_attn(q2, c, n, stream=s)
        sgot1, sgot2 = sp.scored_attn(sq1, k, v), sp.scored_attn(sq2, k, v, stream=s)
        rgot = sp.rope_axes(x, pos, (64,), stream=s)
        torch.cuda.current_stream().wait_stream(s)
        for got, want in zip((*got1, *got2, *sgot1, *sgot2, rgot), (*want1, *want2, *swant1, *swant2, rwant)):
            assert torch.equal(got, want)
        del got1, got2, sgot1, sgot2, rgot, got, want
    sp.device_check()


def test_calls_with_a_stream_of_the_graph():
    """A captured call that is given the capturing stream, and one that forks to another."""
    g = gen(65)
    q, k, v = randn(g, 4, 300, 64), randn(g, 2, 300, 64), randn(g, 2, 300, 64)
    want = sp.scored_attn(q, k, v)
    s, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a = sp.scored_attn(q, k, v, stream=s)
        side.wait_stream(s)
        b = sp.scored_attn(q, k, v, stream=side)
        s.wait_stream(side)
    for _ in range(3):
        a[0].zero_(), b[0].zero_()
        graph.replay()
        assert torch.equal(a[0], want[0]) and torch.equal(b[0], want[0]) and torch.equal(b[1], want[1])
    sp.device_check()
