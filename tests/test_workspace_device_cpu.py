"""A workspace on another device than the current one is refused before anything is launched (the library's kernels
would be given pointers that their device may not reach)."""

import pytest
import torch

from qlora_fine_tuning_nf4_b200 import ops


class _Buf:
    def __init__(self, device):
        self.device, self.index = torch.device("cuda", device), device

    def get_device(self):
        return self.index

    def numel(self):
        return 256


def _workspace(device):
    ws = object.__new__(ops.Workspace)
    ws.device, ws.buf, ws.captured, ws.apart, ws.kept = f"cuda:{device}", _Buf(device), False, False, []
    return ws


@pytest.mark.parametrize("nbytes", [0, 256, 1 << 20])
def test_workspace_of_another_device_is_refused(monkeypatch, nbytes):
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    monkeypatch.setattr(ops, "_capturing", lambda: False)
    with pytest.raises(ValueError, match="workspace is on cuda:1, not on the current device cuda:0"):
        _workspace(1).get(nbytes)


def test_workspace_of_the_current_device_is_taken(monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 1)
    monkeypatch.setattr(ops, "_capturing", lambda: False)
    ws = _workspace(1)
    assert ws.get(0) is ws.buf and ws.get(256) is ws.buf
