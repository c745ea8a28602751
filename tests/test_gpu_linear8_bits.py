"""How many bits the low-rank operand of the e4m3 projection keeps between its products: s X A and s dY B^T are fp32
sums that Y, dX and dA go on from, held as two bf16 numbers that leave 2^-16 of each.

The base weight is small here, so that the low-rank terms are what the outputs consist of.  Bounds, with u = 2^-8 one
bf16 rounding of the result: Y is off by u |Y| + s (2^-16 |XA| + K 2^-24 |X||A|) |B| and the products' own sums
(test_gpu_fp8.py), dX and dA alike.  One bf16 rounding of the operand would add u |XA| instead of 2^-16 |XA|, which is
beyond the bound wherever the terms of an output cancel to a part of their magnitudes."""

import numpy as np
import pytest
import torch

from oracle import fp8
from qlora_fine_tuning_nf4_b200 import ops

from parity import gpu_f64
from test_gpu_fp8 import U16, _linear, _mma_slack

pytestmark = pytest.mark.gpu

PAIR = 2.0 ** -16  # what two bf16 numbers leave of a value: (2^-8)^2


# rows on both sides of the few-row product (64), the one-launch passes (64 backward, 256 forward), reductions in parts
@pytest.mark.parametrize("M,K,N,r,s", [
    (1, 64, 48, 16, 1.0), (3, 272, 144, 32, 0.5), (20, 128, 400, 64, 0.25), (33, 64, 64, 32, 1.7), (64, 272, 144, 16, 0.5),
    (65, 128, 144, 16, 0.5), (130, 272, 144, 32, 2.0), (130, 1680, 64, 64, 1.0), (256, 64, 272, 16, 1.0),
    (258, 64, 272, 64, 0.5), (300, 144, 528, 32, 1.0), (1030, 272, 384, 16, 1.7), (2050, 528, 400, 64, 1.0)])
def test_low_rank_operand_keeps_sixteen_bits(M, K, N, r, s):
    X, dY, W, A, B = _linear(M, K, N, r, s, M + N)
    W, B = W * 2.0 ** -10, B * 32
    ws, w = ops.Workspace(), ops.fp8_quantize(W.cuda())
    lin = ops.LoraLinear8(w, A.cuda(), B.cuda(), s)
    Y, XA = ops.qlora_linear8_fwd(lin, X.cuda(), ws)
    dX, dA, dB = ops.qlora_linear8_bwd(lin, X.cuda(), XA, dY.cuda(), ws)
    assert ops.qlora_last_device_status(ws) == 0
    x, dy, a, b = (t.double().numpy() for t in (X, dY, A, B))
    wv = fp8.dequantize_weight(*fp8.quantize_weight(W.double().numpy()))
    xq, dq = (fp8.dequantize_rows(*fp8.quantize_rows(v)) for v in (x, dy))
    ab = np.abs
    xa, g = x @ a, dy @ b.T
    sum_xa, sum_g = K * 2.0 ** -24 * (ab(x) @ ab(a)), N * 2.0 ** -24 * (ab(dy) @ ab(b).T)
    low = lambda v, sv, m: s * (PAIR * ab(v) + sv) @ ab(m) + 2 * r * 2.0 ** -22 * s * ab(v) @ ab(m)
    y = xq @ wv.T + s * xa @ b
    assert np.all(ab(gpu_f64(Y) - y) <= U16 * ab(y) + 1.01 * (_mma_slack(K) * (ab(xq) @ ab(wv).T) + low(xa, sum_xa, b)))
    ref = dq @ wv + s * g @ a.T
    assert np.all(ab(gpu_f64(dX) - ref) <= U16 * ab(ref) + 1.01 * (_mma_slack(N) * (ab(dq) @ ab(wv)) + low(g, sum_g, a.T)))
    ref = s * x.T @ g
    tol = s * ab(x).T @ (PAIR * ab(g) + sum_g) + 2 * M * 2.0 ** -23 * s * ab(x).T @ ab(g)
    assert np.all(ab(gpu_f64(dA) - ref) <= U16 * ab(ref) + 1.01 * tol)
    # dB is s XA^T dY of the XA that the caller hands in: one rounding of the result
    xs = gpu_f64(XA)
    ref = s * xs.T @ dy
    tol = (M + 2) * 2.0 ** -23 * s * ab(xs).T @ ab(dy)
    assert np.all(ab(gpu_f64(dB) - ref) <= U16 * ab(ref) + 1.01 * tol)


@pytest.mark.parametrize("M", [2, 40, 70, 300])
@pytest.mark.parametrize("r", [16, 64])
def test_low_rank_sum_beyond_bf16_is_infinite_not_nan(M, r):
    """A low-rank sum beyond the range is infinite (in both numbers of the pair it would be inf - inf), in its own row."""
    K, N = 144, 272
    X, dY, W, A, B = _linear(M, K, N, r, 1.0, 3)
    A, B, W = A.abs() + 0.5, B.abs() + 0.5, W * 2.0 ** -10
    lin, ws = ops.LoraLinear8(ops.fp8_quantize(W.cuda()), A.cuda(), B.cuda(), 1.0), ops.Workspace()
    good = ops.qlora_linear8_fwd(lin, X.cuda(), ws)
    gback = ops.qlora_linear8_bwd(lin, X.cuda(), good[1], dY.cuda(), ws)
    X2, dY2, m = X.clone(), dY.clone(), M // 2
    X2[m], dY2[m] = 3e38, 3e38
    Y, XA = ops.qlora_linear8_fwd(lin, X2.cuda(), ws)
    dX, dA, _ = ops.qlora_linear8_bwd(lin, X.abs().cuda(), good[1], dY2.cuda(), ws)
    assert ops.qlora_last_device_status(ws) == 0
    others = [i for i in range(M) if i != m]
    assert torch.all(XA[m] == float("inf")) and torch.all(Y[m] == float("inf"))
    assert torch.equal(Y[others], good[0][others]) and torch.equal(dX[others], gback[0][others])
    assert torch.all(dX[m] == float("inf")) and torch.all(dA == float("inf"))
