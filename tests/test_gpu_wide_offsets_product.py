"""The 8-bit product over rows of more than 2^31 elements, bit for bit: the last rows against a call on enough of them
that the library takes the same tiles and leaves the reduction whole (each output is then the same sums in the same
order, whichever tile it lies in)."""

import pytest
import torch

from qlora_fine_tuning_nf4_b200 import ops

pytestmark = pytest.mark.gpu


def test_last_rows_of_a_product_beyond_2_31_elements():
    K, N, tail = 4096, 64, 16384      # 64 row tiles: more than half of the CTA pairs of any device the kernels run on
    M = (1 << 31) // K + 1000
    g = torch.Generator(device="cuda").manual_seed(4)
    codes = torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    codes[-tail:] = (torch.randn(tail, K, device="cuda", generator=g) * 40).to(torch.float8_e4m3fn)
    scale = torch.rand(K // 128, M, device="cuda", generator=g) + 0.5
    W = ops.fp8_quantize(torch.randn(N, K, device="cuda", generator=g).bfloat16())
    ws = ops.Workspace()
    Y = ops.fp8_matmul(ops.FP8Rows(codes, scale), W, ws)
    y = ops.fp8_matmul(ops.FP8Rows(codes[-tail:].clone(), scale[:, -tail:].contiguous()), W, ws)
    assert torch.equal(Y[-tail:], y) and torch.all(Y[:-tail] == 0) and torch.count_nonzero(y) > y.numel() // 2
    assert ops.qlora_last_device_status(ws) == 0
