"""The 8-bit, residual-norm and rotary operators on tensors of more than 2^31 elements: the last rows give the same
bits as the same rows alone (the operators' own tests hold small cases to fp64)."""

import pytest
import torch

from qlora_fine_tuning_nf4_b200 import ops

pytestmark = pytest.mark.gpu

D = 4096
M = (1 << 31) // D + 1000   # rows of 4096: 2^31 elements and a little more
TAIL = 3


def _rows(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, D, device="cuda", generator=g).bfloat16()


def _big(seed):
    """Distinct last rows behind repeated ones (drawing 2^31 numbers would take most of the test)."""
    base = _rows(1024, seed)
    X = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, M, 1024):
        X[lo:lo + 1024] = base[:min(1024, M - lo)]
    X[-TAIL:] = _rows(TAIL, seed + 1)
    return X


def test_norm_quantise_product_and_rope():
    X, R = _big(1), _big(2)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    t = slice(M - TAIL, M)
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(X, R, w, 1e-5, quantize=True)
    h, y, r, y8 = ops.qlora_add_rmsnorm_fwd(X[t].clone(), R[t].clone(), w, 1e-5, quantize=True)
    assert torch.equal(H[t], h) and torch.equal(Y[t], y) and torch.equal(rstd[t], r)
    assert torch.equal(Y8.codes[t].view(torch.uint8), y8.codes.view(torch.uint8))
    assert torch.equal(Y8.scale[:, t], y8.scale)
    del Y
    dX = ops.qlora_add_rmsnorm_bwd(H, w, rstd, X, dH=R, dX=R)
    assert torch.equal(dX[t], ops.qlora_add_rmsnorm_bwd(h, w, r, X[t].clone(), dH=_rows(TAIL, 3)))
    del dX, R, H
    q = ops.fp8_quantize_rows(X)
    q1 = ops.fp8_quantize_rows(X[t].clone())
    assert torch.equal(q.codes[t].view(torch.uint8), q1.codes.view(torch.uint8)) and torch.equal(q.scale[:, t], q1.scale)
    W = ops.fp8_quantize(torch.randn(64, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
                         .bfloat16())
    ws = ops.Workspace()
    Z = ops.fp8_matmul(Y8, W, ws)
    z = ops.fp8_matmul(ops.FP8Rows(Y8.codes[-300:].clone(), Y8.scale[:, -300:].contiguous()), W, ws)
    # another split of the rows into tiles: the same products, added in the same order
    assert torch.allclose(Z[-300:].float(), z.float(), rtol=2.0 ** -7, atol=0.0)
    assert ops.qlora_last_device_status(ws) == 0
    plan = ops.rope_plan(128)
    pos = torch.arange(M, device="cuda") % 5000
    last = X[t].clone()
    ops.qlora_rope_fwd(X, 32, 128, plan, positions=pos, out=X)
    assert torch.equal(X[t], ops.qlora_rope_fwd(last, 32, 128, plan, positions=pos[t].clone()))


def test_a_weight_of_more_than_2_31_elements():
    """n_out * k_in above 2^31: the last output columns, and the reduction over the last weight rows."""
    n_out, k_in, M_ = (1 << 31) // 4096 + 512, 4096, 40
    codes = torch.zeros(n_out, k_in, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(256, k_in, device="cuda", generator=g).to(torch.float8_e4m3fn)
    codes[-256:] = tail
    scale = torch.ones(n_out // 128, k_in // 128, device="cuda")
    W, small = ops.FP8Weight(codes, scale), ops.FP8Weight(tail, torch.ones(2, k_in // 128, device="cuda"))
    ws = ops.Workspace()
    for m in (5, M_):
        x = ops.fp8_quantize_rows(_rows(m, 2))
        Y = ops.fp8_matmul(x, W, ws)
        assert torch.allclose(Y[:, -256:].float(), ops.fp8_matmul(x, small, ws).float(), rtol=2.0 ** -7, atol=1e-3)
        assert torch.all(Y[:, :-256] == 0)
        d = torch.zeros(m, n_out, dtype=torch.bfloat16, device="cuda")
        d[:, -256:] = _rows(m, 3)[:, :256]
        dq = ops.fp8_quantize_rows(d)
        dX = ops.fp8_matmul_t(dq, W, ws)
        ref = ops.fp8_matmul_t(ops.fp8_quantize_rows(d[:, -256:].contiguous()), small, ws)
        assert torch.allclose(dX.float(), ref.float(), rtol=2.0 ** -7, atol=1e-3)
        assert ops.qlora_last_device_status(ws) == 0
