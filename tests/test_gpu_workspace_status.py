"""A recorded device error is reported by qlora_last_device_status after the workspace has grown: from the buffers that
captured graphs still use, and from a buffer that a larger call has replaced."""

import pytest
import torch

from qlora_fine_tuning_nf4_b200 import ops

pytestmark = pytest.mark.gpu

OTHER_BIT = 32  # a bit of the status word that no wait looks at


def test_error_of_a_graph_whose_buffer_has_been_outgrown():
    ws, word = ops.Workspace(), torch.full((1,), OTHER_BIT, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ws.get(1 << 12)[:1].copy_(word)  # what a call of the graph that runs into an error does
    ws.get(1 << 16)
    assert ops.qlora_last_device_status(ws) == 0
    for _ in range(2):
        g.replay()
        assert ops.qlora_last_device_status(ws) == 7  # QLORA_ERR_DEVICE
        assert ops.qlora_last_device_status(ws) == 0


def test_error_recorded_before_the_workspace_grows():
    ws = ops.Workspace()
    ws.buf[0] = OTHER_BIT
    ws.get(1 << 16)
    assert ops.qlora_last_device_status(ws) == 7 and ops.qlora_last_device_status(ws) == 0
    ws.buf[0] = 1  # QL_DEV_TIMEOUT
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ws.get(1 << 20)
        torch.ones(8, device="cuda")
    assert ops.qlora_last_device_status(ws) == 6 and ops.qlora_last_device_status(ws) == 0


def test_the_timeout_is_reported_first():
    ws = ops.Workspace()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ws.get(256)
        torch.ones(8, device="cuda")
    ws.buf[0] = 1
    ws.get(1 << 12)[0] = OTHER_BIT
    assert ops.qlora_last_device_status(ws) == 6 and ops.qlora_last_device_status(ws) == 0
