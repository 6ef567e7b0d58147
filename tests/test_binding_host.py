"""The binding's choice of the stream, without a GPU."""
import types

import pytest
import torch

from compress_kv_write_gb300 import kvq


@pytest.mark.parametrize("raw", [True, False])
def test_current_stream_of_the_device(monkeypatch, raw):
    """torch's raw handle where this torch has it, the Stream object's otherwise: the same stream."""
    if raw:
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 1000 + dev, raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: pytest.fail("not needed"))
    else:
        monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=1000 + dev))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert kvq._stream(None) == 1003
    assert kvq._on(3, None, lambda s: s) == 1003
    mine = types.SimpleNamespace(cuda_stream=77)
    assert kvq._stream(mine) == 77 and kvq._on(3, mine, lambda s: s) == 77
