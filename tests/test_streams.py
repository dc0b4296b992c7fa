"""The argument ``stream`` of the binding, without a GPU: a call given a stream
makes it current before it allocates or launches anything."""
import contextlib
import inspect

import pytest
import torch

import block_sparse_bidirectional_select_b200 as sp


class FakeStream:
    device = torch.device("cuda", 0)
    cuda_stream = 0x1234


@pytest.fixture
def seen(monkeypatch):
    """What the call does: (what, the current stream), with tensors on the host in place of the device."""
    now, log = [None], []

    @contextlib.contextmanager
    def current(stream):
        now[0], was = stream, now[0]
        yield
        now[0] = was

    def spy(owner, name, fake=None):
        real = getattr(owner, name)

        def call(*a, **kw):
            log.append((name, now[0]))
            return (fake or real)(*a, **kw)
        monkeypatch.setattr(owner, name, call)

    monkeypatch.setattr(torch.cuda, "stream", current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    monkeypatch.setattr(sp, "_device_of", lambda first, **tensors: FakeStream.device)
    monkeypatch.setattr(sp, "_check_cache", lambda c: (*c.k8.shape, FakeStream.device))
    spy(sp, "_launch", lambda *a: None)
    for name in ("empty", "empty_like", "full", "zeros"):
        spy(torch, name)
    spy(torch.Tensor, "new_empty")
    return log


def serve_calls():
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    pos, one, starts = (torch.zeros(*s, dtype=torch.int32) for s in ((1, 8), (1,), (3,)))
    c = sp.Cache8(*(torch.zeros(1, 2, 64, 64, dtype=torch.float8_e4m3fn) for _ in range(2)),
                  *(torch.zeros(1, 2, 1) for _ in range(2)))
    return {
        "rope_axes": lambda **kw: sp.rope_axes(x, pos, (32,), **kw),
        "cache_append": lambda **kw: sp.cache_append(c, x[None], x[None], one, **kw),
        "cache_attn": lambda **kw: sp.cache_attn(x[None], c, one, **kw),
        "document_ranges": lambda **kw: sp.document_ranges(starts, 8, **kw),
        "scored_attn": lambda **kw: sp.scored_attn(x, x, x, **kw),
    }


@pytest.mark.parametrize("name", list(serve_calls()))
def test_a_given_stream_is_current_for_the_whole_call(seen, name):
    call = serve_calls()[name]
    del seen[:]
    stream = FakeStream()
    call(stream=stream)
    assert any(what == "_launch" for what, _ in seen)
    assert all(where is stream for _, where in seen), seen
    del seen[:]
    call()
    assert seen and all(where is None for _, where in seen), seen


def loop_calls():
    x = torch.zeros(2, 128, 64, dtype=torch.bfloat16)
    idx, count, ws = (torch.zeros(*s, dtype=torch.int32) for s in ((2, 1, 1), (2, 1), (64,)))
    state = sp.BlockState(x, idx[..., 0].float(), idx, 0.1, 64, 64, 1, ws)
    return {
        "dense_attn": lambda **kw: sp.dense_attn(x, x, x, **kw),
        "select_pattern": lambda **kw: sp.select_pattern(x, x, x, **kw),
        "block_sparse_attn": lambda **kw: sp.block_sparse_attn(x, x, x, idx, count, **kw),
        "drift_queries": lambda **kw: sp.drift_queries(x, 1, 1, **kw),
        "run_steps": lambda **kw: sp.run_steps(x, x, x, 2, **kw),
        "select_columns": lambda **kw: sp.select_columns(x, x, x, **kw),
        "column_sparse_attn": lambda **kw: sp.column_sparse_attn(x, x, x, idx[:, 0], **kw),
        "run_steps_columns": lambda **kw: sp.run_steps_columns(x, x, x, 2, **kw),
        "select_head_entropy": lambda **kw: sp.select_head_entropy(x, x, x, **kw),
        "select_with_head_k": lambda **kw: sp.select_with_head_k(2, 128, [1, 1], ws, **kw),
        "select_pattern_sharded": lambda **kw: sp.select_pattern_sharded(x, x, x, **kw),
        "losa_init": lambda **kw: sp.losa_init(x, x, x, x, x, splits=1, **kw),
        "losa_step": lambda **kw: sp.losa_step(x, x, x, x, x, x, state, 0.1, **kw),
        "run_steps_sharded": lambda **kw: sp.run_steps_sharded(x, x, x, 2, **kw),
    }


@pytest.mark.parametrize("name", list(loop_calls()))
def test_a_given_stream_is_current_for_the_older_calls_too(seen, monkeypatch, name):
    class Library:
        def __getattr__(self, entry):
            def run(*args):
                seen.append((entry, torch.cuda.current_stream()))
                return 0
            return run

    call = loop_calls()[name]
    base, stream = FakeStream(), FakeStream()
    stream.device = torch.device("cpu")   # where this test's tensors are
    inner = torch.cuda.current_stream
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: inner() or base)
    monkeypatch.setattr(sp._lib, "load", lambda *a: Library())
    monkeypatch.setattr(sp, "_check_qkv", lambda q, k, v: q.shape)
    monkeypatch.setattr(sp, "_check_prefix", lambda k, v, H, d, dev: k.shape[1])
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    del seen[:]
    call(stream=stream)
    work = [(what, where) for what, where in seen if not what.endswith(("_bytes", "_keep", "_splits", "entropy_budget"))]
    assert any(what.startswith("sparsed_") for what, _ in work)
    assert all(where is stream for _, where in work), work


def test_every_call_with_a_stream_goes_through_it():
    for name in set(sp.__all__) - {"device_check"}:   # which allocates nothing
        fn = getattr(sp, name)
        if inspect.isfunction(fn) and "stream" in inspect.signature(fn).parameters:
            assert hasattr(fn, "__wrapped__"), name


def test_results_and_arguments_are_recorded_on_the_other_stream(seen, monkeypatch):
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: FakeStream.device))
    stream, x = FakeStream(), torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    monkeypatch.setattr(torch.Tensor, "new_empty", lambda t, shape, dtype=None: torch.zeros(shape, dtype=dtype))
    monkeypatch.setattr(sp, "_contiguous_like", lambda t: torch.zeros(t.shape, dtype=t.dtype))
    o, lse = sp.scored_attn(x, x, x, stream=stream)
    assert recorded == [(x.data_ptr(), stream)] * 3 + [(o.data_ptr(), None), (lse.data_ptr(), None)]


def test_a_stream_of_another_device_is_refused(seen, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="the stream on"):
        sp.scored_attn(x, x, x, stream=FakeStream())
    with pytest.raises(TypeError):
        sp.document_ranges(torch.zeros(3, dtype=torch.int32), 8, None, FakeStream(), stream=FakeStream())
