"""GPU parity of the 8-bit quantisers (bit for bit) and of fp8_matmul / fp8_matmul_t and the LoRA projection over an
e4m3 weight against fp64.

Bounds: products of e4m3 values are exact; one MMA adds 32 of them and its accumulator within 2^-22 of the sum of
their magnitudes, a block's scaled sum is one binary32 fma and its scale one binary32 product, and the result one
bf16 rounding.  With S = |x| |w|^T over the values, the error is below
2^-8 |ref| + (K / 32 * 2^-22 + ceil(K / 128) * 2^-24 + 2^-22) S."""

import numpy as np
import pytest
import torch

from oracle import fp8
from qlora_fine_tuning_nf4_b200 import ops

from parity import gpu_f64

pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _mma_slack(red):
    return red / 32 * 2.0 ** -22 + -(-red // 128) * 2.0 ** -24 + 2.0 ** -22


# ------------------------------------------------------------- quantisers --

@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (33, 136), (64, 256), (31, 2056), (100, 1000), (5, 9000)])
def test_quantize_rows_bit_exact(M, K):
    X = (torch.randn(M, K, generator=_gen(M + K)) * torch.exp(4 * torch.randn(M, 1, generator=_gen(1)))).bfloat16()
    X[0, :3] = torch.tensor([0.0, -0.0, 1e-40])
    q = ops.fp8_quantize_rows(X.cuda())
    codes, scale = fp8.quantize_rows(X.double().numpy())
    assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(gpu_f64(q.scale), scale)


def test_quantize_rows_every_bf16_value():
    """All finite bf16 values, each in a block whose amax it is and in one with 448 beside it, and special ones."""
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    n = v.numel()
    X = torch.zeros(n, 256, dtype=torch.bfloat16)
    X[:, 0], X[:, 128], X[:, 129] = v, v, 448.0
    X[:, 1] = v / 3
    q = ops.fp8_quantize_rows(X.cuda())
    codes, scale = fp8.quantize_rows(X.double().numpy())
    assert np.array_equal(gpu_f64(q.scale), scale)
    assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), codes)
    S = torch.zeros(4, 384, dtype=torch.bfloat16)
    S[0, 5], S[1, 130], S[2, 260], S[3, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    S[:, 7], S[:, 140] = 3.0, -5.0
    q = ops.fp8_quantize_rows(S.cuda())
    codes, scale = fp8.quantize_rows(S.double().numpy())
    assert np.array_equal(gpu_f64(q.scale), scale)
    assert np.array_equal(q.codes.double().cpu().numpy(), fp8.e4m3_values()[codes], equal_nan=True)


@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (144, 272), (1000 // 16 * 16, 640), (256, 4096)])
def test_quantize_weight_bit_exact(N, K):
    W = (torch.randn(N, K, generator=_gen(N + K)) * 0.02).bfloat16()
    W[: N // 2, : K // 2] *= 100
    q = ops.fp8_quantize(W.cuda())
    codes, scale = fp8.quantize_weight(W.double().numpy())
    assert np.array_equal(q.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(gpu_f64(q.scale), scale)


# ---------------------------------------------------------------- product --

def _operands(M, K, N, red, seed):
    """e4m3 rows and weight with scales that are no powers of two and spread over 2^20 from block to block."""
    g = _gen(seed)
    spread = lambda *s: torch.exp2(4 * torch.randn(*s, generator=g)).clamp(2.0 ** -10, 2.0 ** 10)
    x = (torch.randn(M, red, generator=g) * 40).to(torch.float8_e4m3fn)
    w = (torch.randn(N, K, generator=g) * 40).to(torch.float8_e4m3fn)
    sx, sw = spread(-(-red // 128), M), spread(-(-N // 128), -(-K // 128))
    return x, sx, w, sw


def _values(x, sx, w, sw):
    return (fp8.dequantize_rows(x.view(torch.uint8).numpy(), sx.double().numpy()),
            fp8.dequantize_weight(w.view(torch.uint8).numpy(), sw.double().numpy()))


MM_SHAPES = [(1, 64, 16), (1, 4096, 4096), (3, 16, 16), (16, 1024, 512), (17, 144, 272), (64, 512, 128), (128, 256, 384),
             (130, 1040, 528), (200, 2048, 144), (256, 128, 256), (257, 400, 2064), (520, 384, 1552), (1025, 272, 640),
             # 17 to 32 rows; parts of a long reduction, in both directions; tiles of 256 columns, in both directions
             (20, 528, 400), (32, 2048, 1040), (33, 2048, 528), (64, 1552, 2064), (5, 14336, 144), (64, 16, 4112), (70, 4096, 80), (130, 144, 2064), (300, 80, 6160), (33, 1552, 16),
             (2050, 272, 1296), (2050, 1296, 272), (1300, 144, 2064), (4000, 80, 656)]


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("M,K,N", MM_SHAPES)
def test_matmul(M, K, N, bwd):
    red, cols = (N, K) if bwd else (K, N)
    x, sx, w, sw = _operands(M, K, N, red, M + K + N)
    xv, wv = _values(x, sx, w, sw)
    op = wv if bwd else wv.T
    ref, mag = xv @ op, np.abs(xv) @ np.abs(op)
    ws = ops.Workspace()
    f = ops.fp8_matmul_t if bwd else ops.fp8_matmul
    out = torch.full((M + 1, cols), 3.0, dtype=torch.bfloat16, device="cuda")
    f(ops.FP8Rows(x.cuda(), sx.cuda()), ops.FP8Weight(w.cuda(), sw.cuda()), ws, out[:M])
    assert ops.qlora_last_device_status(ws) == 0
    assert np.all(np.abs(gpu_f64(out[:M]) - ref) <= U16 * np.abs(ref) + 1.01 * _mma_slack(red) * mag)
    assert torch.all(out[M] == 3.0)  # the row behind the last one is left as it was


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("M,K,N", [(700, 640, 1296), (130, 1680, 1680), (2100, 1200, 1300 // 16 * 16)])
def test_matmul_few_ctas(M, K, N, bwd):
    """Every CTA walks many tiles (rings and accumulators wrap), with the same result: tiles of 128 columns, parts of
    a reduction, tiles of 256 columns."""
    red = N if bwd else K
    x, sx, w, sw = _operands(M, K, N, red, 5)
    xg, wg = ops.FP8Rows(x.cuda(), sx.cuda()), ops.FP8Weight(w.cuda(), sw.cuda())
    f = ops.fp8_matmul_t if bwd else ops.fp8_matmul
    ws = ops.Workspace()
    full = f(xg, wg, ws)
    for cap in (2, 6):
        ops.qlora_test_set_grid_cap(cap)
        assert torch.equal(f(xg, wg, ws), full)
    assert ops.qlora_last_device_status(ws) == 0
    xv, wv = _values(x, sx, w, sw)
    op = wv if bwd else wv.T
    ref = xv @ op
    assert np.all(np.abs(gpu_f64(full) - ref) <= U16 * np.abs(ref) + 1.01 * _mma_slack(red) * (np.abs(xv) @ np.abs(op)))


@pytest.mark.parametrize("M", [1, 30, 40, 300])
@pytest.mark.parametrize("bwd", [False, True])
def test_matmul_row_with_nan_spoils_itself_only(M, bwd):
    K, N = 400, 272
    red = N if bwd else K
    x, sx, w, sw = _operands(M, K, N, red, 6)
    f = ops.fp8_matmul_t if bwd else ops.fp8_matmul
    ws, wg = ops.Workspace(), ops.FP8Weight(w.cuda(), sw.cuda())
    good = f(ops.FP8Rows(x.cuda(), sx.cuda()), wg, ws)
    bad = x.clone()
    bad.view(torch.uint8)[M // 2, red - 1] = 0x7F
    out = f(ops.FP8Rows(bad.cuda(), sx.cuda()), wg, ws)
    others = [m for m in range(M) if m != M // 2]
    assert torch.isnan(out[M // 2]).all() and torch.equal(out[others], good[others])
    inf = sx.clone()
    inf[0, M // 2] = float("inf")
    out = f(ops.FP8Rows(x.cuda(), inf.cuda()), wg, ws)
    assert not torch.isfinite(out[M // 2]).any() and torch.equal(out[others], good[others])


@pytest.mark.parametrize("M", [1, 25, 60, 600, 3000])
def test_matmul_repeats_bit_for_bit(M):
    x, sx, w, sw = _operands(M, 1600, 1040, 1600, 7)
    xg, wg, ws = ops.FP8Rows(x.cuda(), sx.cuda()), ops.FP8Weight(w.cuda(), sw.cuda()), ops.Workspace()
    first = ops.fp8_matmul(xg, wg, ws)
    for _ in range(5):
        assert torch.equal(ops.fp8_matmul(xg, wg, ws), first)


# ------------------------------------------------------------- projection --

def _linear(M, K, N, r, s, seed):
    g = _gen(seed)
    X, dY = torch.randn(M, K, generator=g).bfloat16(), torch.randn(M, N, generator=g).bfloat16()
    W = (torch.randn(N, K, generator=g) * 0.02).bfloat16()
    A = ((torch.rand(K, r, generator=g) * 2 - 1) / K ** 0.5).bfloat16()
    B = (torch.randn(r, N, generator=g) * 0.02).bfloat16()
    return X, dY, W, A, B


LIN_SHAPES = [(1, 64, 16, 16, 1.0), (1, 1024, 528, 64, 0.25), (64, 4096, 1024, 64, 0.25), (130, 400, 272, 16, 2.0),
              (300, 512, 1040, 32, 0.5), (1030, 272, 384, 16, 1.0), (257, 1040, 2064, 64, 1.7),
              (20, 512, 400, 32, 0.5), (33, 1680, 144, 16, 1.0), (90, 144, 1680, 64, 0.25), (2050, 1296, 1296, 32, 0.5),
              # the few-row passes' ends: 64 and 65 rows, one block of columns and more than a cluster's, each rank
              (64, 272, 144, 32, 1.7), (65, 272, 144, 16, 0.5), (16, 4112, 2064, 64, 0.25), (48, 144, 6160, 16, 1.0),
              (17, 128, 2064, 32, 1.0), (2, 16, 16, 64, 3.0),
              # the forward's one-launch pass and the general one, around their border
              (256, 400, 144, 32, 0.5), (250, 2064, 144, 64, 1.0), (258, 400, 144, 64, 0.5)]


@pytest.mark.parametrize("cap", [2, 10])
@pytest.mark.parametrize("M,K,N,r,s", [(700, 640, 1296, 32, 0.5), (130, 1680, 1680, 16, 1.0), (2100, 1200, 1296, 64, 2.0)])
def test_linear8_few_ctas(M, K, N, r, s, cap):
    """The LoRA block between other tiles' blocks: every CTA pair walks many tiles or parts."""
    ops.qlora_test_set_grid_cap(cap)
    _check_linear8(M, K, N, r, s)


@pytest.mark.parametrize("M,K,N,r,s", LIN_SHAPES)
def test_linear8(M, K, N, r, s):
    _check_linear8(M, K, N, r, s)


def _check_linear8(M, K, N, r, s):
    X, dY, W, A, B = _linear(M, K, N, r, s, M + N)
    ws = ops.Workspace()
    w = ops.fp8_quantize(W.cuda())
    lin = ops.LoraLinear8(w, A.cuda(), B.cuda(), s)
    Xg, dYg = X.cuda(), dY.cuda()
    Y, XA = ops.qlora_linear8_fwd(lin, Xg, ws)
    dX, dA, dB = ops.qlora_linear8_bwd(lin, Xg, XA, dYg, ws)
    assert ops.qlora_last_device_status(ws) == 0
    x, dy, a, b = (t.double().numpy() for t in (X, dY, A, B))
    wv = fp8.dequantize_weight(*fp8.quantize_weight(W.double().numpy()))
    xq, dq = (fp8.dequantize_rows(*fp8.quantize_rows(v)) for v in (x, dy))
    ab = np.abs
    xa, g = x @ a, dy @ b.T
    # fp32 sums of bf16 products: n roundings of 2^-24 at most, over the sum of magnitudes
    sum_xa, sum_g = K * 2.0 ** -24 * (ab(x) @ ab(a)), N * 2.0 ** -24 * (ab(dy) @ ab(b).T)
    assert np.all(ab(gpu_f64(XA) - xa) <= U16 * ab(xa) + 1.01 * sum_xa)
    # the low-rank operand is rounded to bf16 once (s XA, s G); r products of it
    low = lambda v, sv, m: s * (U16 * ab(v) + 1.01 * sv) @ ab(m) + r * 2.0 ** -22 * s * ab(v) @ ab(m)
    y = xq @ wv.T + s * xa @ b
    assert np.all(ab(gpu_f64(Y) - y) <= U16 * ab(y) + 1.01 * (_mma_slack(K) * (ab(xq) @ ab(wv).T) + low(xa, sum_xa, b)))
    ref = dq @ wv + s * g @ a.T
    assert np.all(ab(gpu_f64(dX) - ref) <= U16 * ab(ref) + 1.01 * (_mma_slack(N) * (ab(dq) @ ab(wv)) + low(g, sum_g, a.T)))
    ref = s * x.T @ g
    tol = s * ab(x).T @ (U16 * ab(g) + 1.01 * sum_g) + M * 2.0 ** -23 * s * ab(x).T @ ab(g)
    assert np.all(ab(gpu_f64(dA) - ref) <= U16 * ab(ref) + 1.01 * tol)
    ref = s * xa.T @ dy  # from the saved XA, rounded once
    tol = s * (U16 * ab(xa) + 1.01 * sum_xa).T @ ab(dy) + (M + 2) * 2.0 ** -23 * s * ab(xa).T @ ab(dy)
    assert np.all(ab(gpu_f64(dB) - ref) <= U16 * ab(ref) + 1.01 * tol)
    # X already in 8 bits: the same result bit for bit
    Y2, XA2 = ops.qlora_linear8_fwd(lin, Xg, ws, X8=ops.fp8_quantize_rows(Xg))
    assert torch.equal(Y2, Y) and torch.equal(XA2, XA)


def test_linear8_gradients_by_differences():
    """The adapter's gradients against differences of the forward (linear in A and in B separately)."""
    M, K, N, r, s = 48, 256, 144, 16, 0.5
    X, dY, W, A, B = _linear(M, K, N, r, s, 1)
    ws = ops.Workspace()
    lin = ops.LoraLinear8(ops.fp8_quantize(W.cuda()), A.cuda(), B.cuda(), s)
    _, XA = ops.qlora_linear8_fwd(lin, X.cuda(), ws)
    _, dA, dB = ops.qlora_linear8_bwd(lin, X.cuda(), XA, dY.cuda(), ws)
    x, dy, a, b = (t.double().numpy() for t in (X, dY, A, B))
    f = lambda a_, b_: np.sum(s * (x @ a_) @ b_ * dy)
    rng = np.random.default_rng(0)
    va, vb = rng.standard_normal(a.shape), rng.standard_normal(b.shape)
    for got, v, num in ((dA, va, f(a + va, b) / 2 - f(a - va, b) / 2), (dB, vb, f(a, b + vb) / 2 - f(a, b - vb) / 2)):
        d = gpu_f64(got)
        # each element carries its own rounding and one of its low-rank operand (over the sum's magnitudes)
        xs = np.abs(x).T @ np.abs(dy @ b.T) if got is dA else np.abs(x @ a).T @ np.abs(dy)
        assert abs(np.sum(d * v) - num) <= np.sum((U16 * np.abs(d) + 1.02 * U16 * s * xs) * np.abs(v))


def test_linear8_empty_batch():
    _, _, W, A, B = _linear(1, 64, 32, 16, 1.0, 1)
    lin = ops.LoraLinear8(ops.fp8_quantize(W.cuda()), A.cuda(), B.cuda(), 1.0)
    ws = ops.Workspace()
    e = lambda n: torch.empty(0, n, dtype=torch.bfloat16, device="cuda")
    Y, XA = ops.qlora_linear8_fwd(lin, e(64), ws)
    nan = lambda t: torch.full_like(t, float("nan"))
    dX, dA, dB = ops.qlora_linear8_bwd(lin, e(64), XA, Y, ws, dA=nan(lin.A), dB=nan(lin.B))
    assert Y.shape == (0, 32) and dX.shape == (0, 64)
    assert torch.all(dA == 0) and torch.all(dB == 0)
    assert ops.fp8_matmul(ops.fp8_quantize_rows(e(64)), lin.w, ws).shape == (0, 32)
