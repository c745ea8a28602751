"""GPU parity of qlora_add_rmsnorm_fwd / _bwd against fp64: every row width class (a warp per row, 128 to 512
threads, wider than registers), widths whose last block of 128 is short, one row and many, with and without the
residual and the 8-bit output, in place.

Bounds from the arithmetic: H is one bf16 rounding of an exact sum; rstd is one binary32 rounding of a binary64
value; Y = bf16(H * rstd * g) adds the roundings of rstd, g and two products (2^-24 each) to its own 2^-8; the
8-bit rows are the oracle's of the Y that the call wrote, bit for bit."""

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8
from qlora_fine_tuning_nf4_b200 import ops

from parity import gpu_f64

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8
SHAPES = [(1, 8), (5, 136), (7, 520), (33, 1024), (9, 2056), (300, 4096), (17, 5000), (3, 8192), (5, 12808),
          (2, 16384), (3, 16392), (2, 20104)]


def _inputs(M, d, gemma, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    X = (n(M, d) * 0.3).bfloat16()
    R = (n(M, d) * (0.5 + torch.rand(M, 1, generator=g))).bfloat16()
    w = (n(d) * 0.1 + (0.0 if gemma else 1.0)).bfloat16()
    return X, R, w, n(M, d).bfloat16(), n(M, d).bfloat16()


def _check_fwd(X, R, w, eps, gemma, H, Y, rstd, Y8):
    h = (X.double() + R.double()).bfloat16() if R is not None else X  # exact sum, one rounding
    assert torch.equal(H.cpu(), h)
    y_ref, r_ref = oracle.rmsnorm_fwd(h.double().numpy(), w.double().numpy(), np.float32(eps).astype(float), gemma)
    assert np.all(np.abs(gpu_f64(rstd) - r_ref) <= U32 * (1 + 2.0 ** -10) * r_ref)
    if Y is not None:
        bound = ((1 + U16) * (1 + U32) ** 4 - 1) * np.abs(y_ref)
        assert np.all(np.abs(gpu_f64(Y) - y_ref) <= bound)
    if Y8 is not None and Y is not None:
        codes, scale = fp8.quantize_rows(gpu_f64(Y))
        assert np.array_equal(Y8.codes.view(torch.uint8).cpu().numpy(), codes)
        assert np.array_equal(gpu_f64(Y8.scale), scale)


@pytest.mark.parametrize("gemma", [False, True])
@pytest.mark.parametrize("M,d", SHAPES)
def test_forward(M, d, gemma):
    eps = 1e-6 if gemma else 1e-5
    X, R, w, _, _ = _inputs(M, d, gemma, M + d)
    Xg, Rg, wg = X.cuda(), R.cuda(), w.cuda()
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(Xg, Rg, wg, eps, plus_one=gemma, quantize=True)
    _check_fwd(X, R, w, eps, gemma, H, Y, rstd, Y8)
    assert torch.equal(Xg.cpu(), X) and torch.equal(Rg.cpu(), R)
    # only the 8-bit rows
    H2, none, rstd2, Y82 = ops.qlora_add_rmsnorm_fwd(Xg, Rg, wg, eps, plus_one=gemma, quantize=True, want_y=False)
    assert none is None and torch.equal(H2, H) and torch.equal(rstd2, rstd)
    assert torch.equal(Y82.codes.view(torch.uint8), Y8.codes.view(torch.uint8)) and torch.equal(Y82.scale, Y8.scale)
    # only bf16, and no residual: the plain norm of X
    Hn, Yn, rn, q = ops.qlora_add_rmsnorm_fwd(Xg, None, wg, eps, plus_one=gemma)
    assert Hn is Xg and q is None
    _check_fwd(X, None, w, eps, gemma, Hn, Yn, rn, None)
    # in place on the residual stream, and on the sublayer's output
    for k in range(2):
        a, b = Xg.clone(), Rg.clone()
        Hi, Yi, _, _ = ops.qlora_add_rmsnorm_fwd(a, b, wg, eps, plus_one=gemma, H=(a, b)[k])
        assert Hi is (a, b)[k] and torch.equal(Hi, H) and torch.equal(Yi, Y) and torch.equal((b, a)[k], (Rg, Xg)[k])


@pytest.mark.parametrize("gemma", [False, True])
@pytest.mark.parametrize("M,d", SHAPES)
def test_backward(M, d, gemma):
    eps = 1e-6 if gemma else 1e-5
    H, _, w, dY, dH = _inputs(M, d, gemma, 3 * M + d)
    hg, wg, dyg, dhg = H.cuda(), w.cuda(), dY.cuda(), dH.cuda()
    _, _, rstd, _ = ops.qlora_add_rmsnorm_fwd(hg, None, wg, eps, plus_one=gemma)
    dX = ops.qlora_add_rmsnorm_bwd(hg, wg, rstd, dyg, dH=dhg, plus_one=gemma)
    alone = ops.qlora_add_rmsnorm_bwd(hg, wg, rstd, dyg, plus_one=gemma)
    h, wf, dy, dh = (t.double().numpy() for t in (H, w, dY, dH))
    e = float(np.float32(eps))
    base = oracle.rmsnorm_bwd(h, wf, e, dy, gemma)
    _, r = oracle.rmsnorm_fwd(h, wf, e, gemma)
    g, n = (1.0 + wf if gemma else wf), h * r[:, None]
    c = np.mean(np.abs(n * g * dy), axis=1, keepdims=True)
    # the sum of d products: at most d roundings of 2^-24 of the sum of their magnitudes; a handful per element
    terms = r[:, None] * (8 * U32 * (np.abs(g * dy) + np.abs(n) * c) + (d + 8) * U32 * np.abs(n) * c)
    for got, ref in ((dX, dh + base), (alone, base)):
        slack = terms + 8 * U32 * np.abs(dh)
        assert np.all(np.abs(gpu_f64(got) - ref) <= U16 * np.abs(ref) + (1 + U16) * slack)
    for k in range(2):  # in place on either incoming gradient
        a, b = dyg.clone(), dhg.clone()
        out = ops.qlora_add_rmsnorm_bwd(hg, wg, rstd, a, dH=b, plus_one=gemma, dX=(a, b)[k])
        assert torch.equal(out, dX) and torch.equal((b, a)[k], (dhg, dyg)[k])


def test_backward_by_differences():
    """Directional derivatives of the forward itself (fp64 differences of the formula at the same point)."""
    H, _, w, dY, dH = _inputs(4, 264, False, 9)
    hg, wg = H.cuda(), w.cuda()
    _, _, rstd, _ = ops.qlora_add_rmsnorm_fwd(hg, None, wg, 1e-5)
    dX = gpu_f64(ops.qlora_add_rmsnorm_bwd(hg, wg, rstd, dY.cuda(), dH=dH.cuda()))
    h, wf, dy, dh = (t.double().numpy() for t in (H, w, dY, dH))
    e = float(np.float32(1e-5))
    f = lambda x: np.sum(oracle.rmsnorm_fwd(x, wf, e)[0] * dy, axis=1) + np.sum(x * dh, axis=1)
    v = np.random.default_rng(1).standard_normal(h.shape)
    step = 1e-5
    num = (f(h + step * v) - f(h - step * v)) / (2 * step)
    # dX is off by 2^-8 of each element; the difference by about step^2
    assert np.all(np.abs(np.sum(dX * v, axis=1) - num) <= np.sum(2.0 ** -8 * np.abs(dX * v), axis=1) * 1.01 + 1e-6)


def test_special_values():
    """An infinite or NaN element spoils its own row only; a row of zeros stays zeros."""
    X, R, w, _, _ = _inputs(6, 520, False, 2)
    X[1, 3], X[2, 500], X[4] = float("inf"), float("nan"), 0.0
    R[4] = 0.0
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(X.cuda(), R.cuda(), w.cuda(), 1e-5, quantize=True)
    for m in (0, 3, 5):
        _check_fwd(X[m:m + 1], R[m:m + 1], w, 1e-5, False, H[m:m + 1], Y[m:m + 1], rstd[m:m + 1], None)
        codes, scale = fp8.quantize_rows(gpu_f64(Y[m:m + 1]))
        assert np.array_equal(Y8.codes[m:m + 1].view(torch.uint8).cpu().numpy(), codes)
    assert torch.isnan(Y[1, 3]) and torch.isnan(Y[2, 500])
    assert torch.equal(Y[4].float(), torch.zeros(520, device="cuda"))
    assert torch.equal(Y8.codes[4].float(), torch.zeros(520, device="cuda"))
    codes, scale = fp8.quantize_rows(gpu_f64(Y))
    back, ref = Y8.codes.double().cpu().numpy(), fp8.e4m3_values()[codes]
    assert np.array_equal(back, ref, equal_nan=True)
    assert np.array_equal(gpu_f64(Y8.scale), scale)


@pytest.mark.parametrize("d", [40, 1208, 4096, 16392])
def test_rstd_is_the_correctly_rounded_value(d):
    """The sum of squares in binary64 and eps as the binary32 number that the call takes: rstd is the nearest binary32
    number.  In any order, a sum of d exact positive squares is off by d 2^-53 relative at most, the mean, eps, root
    and division by 2^-53 each; both sides carry that, so rows nearer than 2 (d + 4) 2^-53 to a border are left out."""
    M = 4096
    X, R, w, _, _ = (t.cuda() for t in _inputs(M, d, False, d))
    H, _, rstd, _ = ops.qlora_add_rmsnorm_fwd(X, R, w, 1e-5)
    ref = 1.0 / torch.sqrt(H.double().square().mean(1) + float(np.float32(1e-5)))
    m = 2 * (d + 4) * 2.0 ** -53
    lo, hi = (ref * (1 - m)).float(), (ref * (1 + m)).float()
    assert torch.all((rstd == lo) | (rstd == hi))
    # 4096 rows, each within m of a border with probability 2 m / 2^-24 at most: 0.5 rows expected at the widest d, and
    # more than 8 with a probability below 1e-8
    assert int((lo != hi).sum()) <= 8


def test_zero_row_without_eps():
    """eps = 0 is allowed: a row of zeros has rstd = 1 / 0 = inf and Y = 0 * inf = NaN; other rows are untouched by it."""
    X, _, w, _, _ = _inputs(3, 264, False, 8)
    X[1] = 0.0
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(X.cuda(), None, w.cuda(), 0.0, quantize=True)
    assert torch.isinf(rstd[1]) and torch.isnan(Y[1]).all() and torch.isnan(Y8.codes[1].float()).all()
    for m in (0, 2):
        s = slice(m, m + 1)
        _check_fwd(X[s], None, w, 0.0, False, H[s].contiguous(), Y[s], rstd[s], None)
        codes, _ = fp8.quantize_rows(gpu_f64(Y[s]))
        assert np.array_equal(Y8.codes[s].view(torch.uint8).cpu().numpy(), codes)


def test_many_rows_same_as_one_by_one():
    """A row's result does not depend on the rows beside it (bit for bit)."""
    X, R, w, dY, dH = _inputs(37, 1000, True, 4)
    X, R, w, dY, dH = (t.cuda() for t in (X, R, w, dY, dH))
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(X, R, w, 1e-6, plus_one=True, quantize=True)
    dX = ops.qlora_add_rmsnorm_bwd(H, w, rstd, dY, dH=dH, plus_one=True)
    for m in (0, 17, 36):
        s = slice(m, m + 1)
        h, y, r, y8 = ops.qlora_add_rmsnorm_fwd(X[s], R[s], w, 1e-6, plus_one=True, quantize=True)
        assert torch.equal(h, H[s]) and torch.equal(y, Y[s]) and torch.equal(r, rstd[s])
        assert torch.equal(y8.codes.view(torch.uint8), Y8.codes[s].view(torch.uint8))
        assert torch.equal(y8.scale[:, 0], Y8.scale[:, m])
        assert torch.equal(ops.qlora_add_rmsnorm_bwd(h, w, r, dY[s], dH=dH[s], plus_one=True), dX[s])


def test_empty_batch():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(e, e, w, 1e-5, quantize=True)
    assert H.shape == Y.shape == (0, 64) and rstd.shape == (0,) and Y8.scale.shape == (1, 0)
    assert ops.qlora_add_rmsnorm_bwd(H, w, rstd, Y, dH=Y).shape == (0, 64)
