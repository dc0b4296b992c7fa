"""What the binding of the operators around block-wise generation makes of its
arguments, without a GPU: the launch is replaced by a record of it."""
import ctypes
import random

import pytest
import torch

import block_sparse_bidirectional_select_b200 as sp


@pytest.fixture
def launched(monkeypatch):
    """The arguments of every launch, with tensors on the host in place of the device."""
    log = []
    dev = torch.device("cuda", 0)
    monkeypatch.setattr(sp, "_device_of", lambda first, **tensors: dev)
    monkeypatch.setattr(sp, "_check_cache", lambda c: (*c.k8.shape, dev))
    monkeypatch.setattr(sp, "_launch", lambda name, dev, args: log.append((name, args)))
    return log


def calls():
    x = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    c = sp.Cache8(*(torch.zeros(1, 2, 64, 64, dtype=torch.float8_e4m3fn) for _ in range(2)),
                  *(torch.zeros(1, 2, 1) for _ in range(2)))
    one = torch.zeros(1, dtype=torch.int32)
    return {"cache_attn": lambda **kw: sp.cache_attn(x[None], c, one, **kw),
            "scored_attn": lambda **kw: sp.scored_attn(x, x, x, **kw)}


@pytest.mark.parametrize("name", list(calls()))
def test_workspace_is_one_piece_of_memory(launched, name):
    """The size that reaches the library is that of the memory from the first element on."""
    call = calls()[name]
    for ws, room in ((torch.zeros(1 << 16, dtype=torch.uint8), 1 << 16), (torch.zeros(1 << 14), 1 << 16),
                     (torch.zeros(16, 1 << 10, dtype=torch.int16), 1 << 15)):
        call(workspace=ws)
        assert launched[-1][1][-2:] == (ws.data_ptr(), room)
    done = len(launched)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 16), torch.zeros(1 << 16, dtype=torch.uint8)[::2],
               torch.zeros(256, 256, dtype=torch.uint8).t()):
        with pytest.raises(ValueError, match="workspace"):
            call(workspace=ws)
    assert len(launched) == done


def rows(H, sh, L, sl, d):
    """Whether two of the rows of d elements at h * sh + l * sl share one, by looking at every element."""
    seen = set()
    for h in range(H):
        for l in range(L):
            for e in range(d):
                at = h * sh + l * sl + e
                if at in seen:
                    return True
                seen.add(at)
    return False


@pytest.mark.skipif(torch.cuda.is_available(), reason="accepted calls end where there is no device")
def test_rope_refuses_rows_of_the_output_that_overlap():
    lib, p = sp._lib.load(), ctypes.c_void_p(0x10000)
    one = (ctypes.c_int * 1)(4)
    rng = random.Random(5)
    cases = [(2, 0, 3, 8, 8), (2, 24, 3, 0, 8), (2, 24, 3, 8, 8), (2, 8, 3, 16, 8), (3, 16, 2, 24, 8), (1, 0, 5, 8, 8),
             (5, 8, 1, 0, 8), (1, 0, 1, 0, 8), (2, 20, 3, 8, 8), (3, 16, 2, 40, 8), (3, 17, 2, 40, 8)]
    cases += [(rng.randint(1, 6), rng.choice((0, 4, 8, 9, 16, 24, 25, 40, 48)), rng.randint(1, 6),
               rng.choice((0, 3, 8, 10, 16, 24, 32, 47, 56)), 8) for _ in range(400)]
    refused = 0
    for H, sh, L, sl, d in cases:
        rc = lib.sparsed_rope_axes(p, L * d, d, p, 1, ctypes.addressof(one), H, L, d, 1e4, 0, 0, 0, p, sh, sl, None)
        assert rc == (sp._lib.ERR_INVALID_ARG if rows(H, sh, L, sl, d) else sp._lib.ERR_NO_DEVICE), (H, sh, L, sl)
        refused += rc == sp._lib.ERR_INVALID_ARG
    assert 50 < refused < len(cases) - 50
