"""What the binding of the operators around block-wise generation makes of its
arguments, without a GPU: the launch is replaced by a record of it."""
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
