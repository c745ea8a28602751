"""qlora_add_rmsnorm_fwd / _bwd on finite rows whose squares leave binary32: beyond 2^64 and below 2^-75.

Bounds as in test_gpu_addnorm.py: the formula has no other rounding at these magnitudes, since rstd (1e-25 to 1e25
here) is a normal binary32 number and so is every product that the formula names."""

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from qlora_fine_tuning_nf4_b200 import ops

from parity import gpu_f64

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
# a row width of every kernel: a warp per row (two sizes), 128, 256 and 512 threads, wider than registers
WIDTHS = [136, 1000, 2056, 5000, 12808, 16392]


def _rows(d, size, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    # three rows of that size between two ordinary ones
    t = torch.tensor([1.0, size, size, size, 1.0])[:, None]
    return (n(5, d) * t).bfloat16(), (n(5, d) * t * 0.5).bfloat16(), (n(d) * 0.1 + 1.0).bfloat16(), n(5, d).bfloat16()


@pytest.mark.parametrize("size,eps", [(3e19, 1e-5), (1e25, 1e-5), (1e25, 0.0), (1e-20, 0.0), (1e-23, 0.0), (1e-25, 0.0)])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward(d, size, eps):
    X, R, w, _ = _rows(d, size, d)
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(X.cuda(), R.cuda(), w.cuda(), eps, quantize=True)
    h = (X.double() + R.double()).bfloat16()
    assert torch.equal(H.cpu(), h)
    y_ref, r_ref = oracle.rmsnorm_fwd(h.double().numpy(), w.double().numpy(), float(np.float32(eps)))
    assert np.all(np.abs(gpu_f64(rstd) - r_ref) <= U32 * (1 + 2.0 ** -10) * r_ref)
    assert np.all(np.abs(gpu_f64(Y) - y_ref) <= ((1 + U16) * (1 + U32) ** 4 - 1) * np.abs(y_ref))
    codes, scale = fp8.quantize_rows(gpu_f64(Y))
    assert np.array_equal(Y8.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(gpu_f64(Y8.scale), scale)


@pytest.mark.parametrize("size", [1e25, 3e19, 1e-20, 1e-25])
@pytest.mark.parametrize("d", WIDTHS)
def test_backward(d, size):
    H, _, w, dY = _rows(d, size, d + 1)
    h, wf, dy = (t.double().numpy() for t in (H, w, dY))
    _, r = oracle.rmsnorm_fwd(h, wf, 0.0)
    rstd = torch.tensor(r, dtype=torch.float32, device="cuda")
    dX = ops.qlora_add_rmsnorm_bwd(H.cuda(), w.cuda(), rstd, dY.cuda())
    ref = oracle.rmsnorm_bwd(h, wf, 0.0, dy)
    n = h * r[:, None]
    c = np.mean(np.abs(n * wf * dy), axis=1, keepdims=True)
    slack = r[:, None] * (8 * U32 * (np.abs(wf * dy) + np.abs(n) * c) + (d + 8) * U32 * np.abs(n) * c)
    assert np.all(np.abs(gpu_f64(dX) - ref) <= U16 * np.abs(ref) + (1 + U16) * slack)
