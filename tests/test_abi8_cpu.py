"""CPU checks of the 8-bit, residual-norm and rotary entry points: what they reject on the host before any CUDA call
(fake device addresses), what the binding rejects before calling the library, and the workspace sizes."""

import ctypes

import pytest
import torch

from qlora_fine_tuning_nf4_b200 import build, ops

BIG = 1 << 40
MAX = 1 << 23


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.lib()


def _w(codes=16, scale=16, n=512, k=256):
    return ops.QloraFP8(codes, scale, n, k)


def _lin(A=16, B=16, r=16, s=1.0, **kw):
    return ops.QloraLoraLinear8(_w(**kw), A, B, r, s)


def _rows(codes=16, scale=16):
    return ops.QloraFP8Rows(codes, scale)


def test_quantisers(lib):
    q = lib.fp8_quantize_rows
    assert q(16, 0, 64, 16, 16, None) == 0                 # no rows
    assert q(None, 4, 64, 16, 16, None) == 1
    assert q(16, -1, 64, 16, 16, None) == 1
    assert q(16, 4, 0, 16, 16, None) == 1
    assert q(16, 4, 68, 16, 16, None) == 2                 # K % 8
    assert q(16, MAX + 1, 64, 16, 16, None) == 2
    assert q(16, MAX, MAX, 16, 16, None) == 2              # more tiles than a grid holds
    assert q(24, 4, 64, 16, 16, None) == 3
    assert q(16, 4, 64, 16, 8, None) == 3
    w = lib.fp8_quantize
    assert w(16, 16, 0, 16, 16, None) == 1
    assert w(16, 24, 64, 16, 16, None) == 2                # n_out % 16
    assert w(16, 16, 72, 16, 16, None) == 2                # k_in % 16
    assert w(16, MAX, MAX, 16, 16, None) == 2              # more blocks than 32-bit integers count
    assert w(16, 16, 64, 16, None, None) == 1
    assert w(16, 16, 64, 8, 16, None) == 3


@pytest.mark.parametrize("name", ["fp8_matmul", "fp8_matmul_t"])
def test_matmul(lib, name):
    f = getattr(lib, name)
    x, w = _rows(), _w()
    call = lambda x=x, w=w, M=8, out=16, ws=16, nb=BIG: f(ctypes.byref(x) if x else None,
                                                          ctypes.byref(w) if w else None, M, out, ws, nb, None)
    assert call(M=0) == 0
    assert call(M=-1) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(out=None) == 1 and call(ws=None) == 1
    assert call(x=_rows(scale=None)) == 1 and call(x=_rows(codes=None)) == 1
    assert call(w=_w(codes=None)) == 1 and call(w=_w(n=0)) == 1 and call(w=_w(k=-16)) == 1
    assert call(w=_w(n=520)) == 2 and call(w=_w(k=264)) == 2    # multiples of 8, not of 16
    assert call(M=MAX + 1) == 2 and call(w=_w(n=MAX + 16)) == 2
    assert call(w=_w(n=MAX, k=MAX)) == 2
    assert call(x=_rows(codes=24)) == 3 and call(x=_rows(scale=8)) == 3 and call(out=24) == 3 and call(ws=24) == 3
    assert call(w=_w(scale=8)) == 3
    assert call(nb=255) == 4
    # a long reduction over few tiles is split: its partials are part of the workspace
    need = ops.fp8_matmul_workspace_bytes(100, 4096, 128)
    assert need > 256 + 2 * 256 * 128 * 4 - 1
    assert call(w=_w(n=128, k=4096), M=100, nb=need - 1) == 4


def test_workspace_queries(lib):
    assert ops.fp8_matmul_workspace_bytes(0, 64, 64) == 256
    assert ops.fp8_matmul_workspace_bytes(8192, 4096, 4096) == 256  # enough tiles: nothing is split
    assert ops.qlora_linear8_workspace_bytes(0, 64, 64) == 256
    assert ops.qlora_linear8_workspace_bytes(16, 512, 1024, 8) == 256  # unsupported rank
    sizes = [ops.qlora_linear8_workspace_bytes(8192, 4096, n, 16) for n in (512, 4096, 14336)]
    assert sizes == sorted(sizes) and sizes[0] > 8192 * 4096
    # no staged weight: far less than the NF4 projection's
    assert ops.qlora_linear8_workspace_bytes(64, 4096, 14336, 16) < 14336 * 4096


def test_linear8(lib):
    c = _lin()
    call = lambda c=c, X=16, X8=None, M=8, Y=16, XA=16, ws=16, nb=BIG: lib.qlora_linear8_fwd(
        ctypes.byref(c) if c else None, X, ctypes.byref(X8) if X8 else None, M, Y, XA, ws, nb, None)
    assert call(M=0) == 0
    assert call(c=None) == 1 and call(X=None) == 1 and call(Y=None) == 1 and call(XA=None) == 1 and call(ws=None) == 1
    assert call(c=_lin(A=None)) == 1 and call(c=_lin(codes=None)) == 1 and call(M=-1) == 1
    assert call(X8=_rows(codes=None)) == 1
    assert call(c=_lin(r=8)) == 2 and call(c=_lin(r=48)) == 2 and call(c=_lin(k=264)) == 2 and call(c=_lin(n=520)) == 2
    assert call(M=MAX + 1) == 2
    assert call(X=24) == 3 and call(c=_lin(B=24)) == 3 and call(X8=_rows(scale=24)) == 3
    assert call(nb=ops.qlora_linear8_workspace_bytes(8, 256, 512, 16) - 1) == 4
    b = lambda c=c, X=16, XA=16, dY=16, M=8, dX=16, dA=16, dB=16, ws=16, nb=BIG: lib.qlora_linear8_bwd(
        ctypes.byref(c), X, XA, dY, M, dX, dA, dB, ws, nb, None)
    assert b(M=0, dA=None) == 1 and b(M=0, dB=24) == 3  # M = 0 clears dA and dB
    for name in ("X", "XA", "dY", "dX", "dA", "dB", "ws"):
        assert b(**{name: None}) == 1 and b(**{name: 24}) == 3
    assert b(nb=256) == 4 and b(M=-1) == 1 and b(c=_lin(r=20)) == 2


def test_add_rmsnorm(lib):
    y8 = _rows()
    f = lambda X=16, R=16, w=16, M=4, d=64, eps=1e-5, H=16, Y=16, Y8=None, rstd=16: lib.qlora_add_rmsnorm_fwd(
        X, R, w, M, d, eps, 0, H, Y, ctypes.byref(Y8) if Y8 else None, rstd, None)
    assert f(M=0) == 0 and f(M=-1) == 1 and f(d=0) == 1 and f(eps=-1.0) == 1 and f(eps=float("nan")) == 1
    assert f(d=68) == 2 and f(d=MAX + 8) == 2 and f(M=MAX + 1) == 2
    for name in ("X", "w", "rstd"):
        assert f(**{name: None}) == 1 and f(**{name: 24}) == 3
    assert f(R=None) == 1 and f(H=None) == 1            # together or not at all
    assert f(R=24) == 3 and f(H=24) == 3 and f(Y=24) == 3
    assert f(Y=None) == 1                                # neither output
    assert f(Y8=_rows(scale=None)) == 1 and f(Y8=_rows(codes=24)) == 3
    b = lambda H=16, w=16, rstd=16, dY=16, dH=16, M=4, d=64, dX=16: lib.qlora_add_rmsnorm_bwd(
        H, w, rstd, dY, dH, M, d, 0, dX, None)
    assert b(M=0) == 0 and b(M=-1) == 1 and b(d=68) == 2 and b(M=MAX + 1) == 2 and b(dH=24) == 3
    for name in ("H", "w", "rstd", "dY", "dX"):
        assert b(**{name: None}) == 1 and b(**{name: 24}) == 3


@pytest.mark.parametrize("name", ["qlora_rope_fwd", "qlora_rope_bwd"])
def test_rope(lib, name):
    f = lambda X=16, M=4, ldx=256, heads=2, D=128, turns=16, rot=128, factor=1.0, pos=None, seq=0, out=1024, ldo=256: \
        getattr(lib, name)(X, M, ldx, heads, D, turns, rot, 0, factor, pos, seq, out, ldo, None)
    assert f(M=0) == 0
    assert f(M=-1) == 1 and f(heads=0) == 1 and f(D=0) == 1 and f(rot=0) == 1 and f(rot=130) == 1 and f(seq=-1) == 1
    assert f(ldx=248) == 1 and f(ldo=248) == 1           # rows shorter than the heads
    assert f(factor=float("inf")) == 1 and f(factor=float("nan")) == 1
    assert f(X=None) == 1 and f(turns=None) == 1 and f(out=None) == 1
    assert f(out=16, ldo=264) == 1                       # in place with another row stride
    assert f(D=100, rot=64) == 2 and f(rot=63) == 2 and f(D=520, rot=64, ldx=1040, ldo=1040) == 2
    assert f(ldx=260) == 2 and f(ldo=260) == 2 and f(M=MAX + 1) == 2
    assert f(X=24) == 3 and f(out=24) == 3 and f(turns=24) == 3 and f(pos=12) == 3


def test_binding_rejects_before_any_library_call():
    bf = torch.bfloat16
    X, w = torch.zeros(8, 256, dtype=bf), torch.ones(256, dtype=bf)
    W = ops.FP8Weight(torch.zeros(512, 256, dtype=torch.float8_e4m3fn), torch.ones(4, 2))
    rows = ops.FP8Rows(torch.zeros(8, 256, dtype=torch.float8_e4m3fn), torch.ones(2, 8))
    lin = ops.LoraLinear8(W, torch.zeros(256, 16, dtype=bf), torch.zeros(16, 512, dtype=bf), 1.0)
    plan = ops.rope_plan(64, device="cpu")
    for call in (lambda: ops.fp8_quantize_rows(X), lambda: ops.fp8_quantize(X), lambda: ops.fp8_matmul(rows, W, None),
                 lambda: ops.fp8_matmul_t(rows, W, None), lambda: ops.qlora_linear8_fwd(lin, X, None),
                 lambda: ops.qlora_linear8_bwd(lin, X, X, X, None),
                 lambda: ops.qlora_add_rmsnorm_fwd(X, X, w, 1e-5),
                 lambda: ops.qlora_add_rmsnorm_bwd(X, w, torch.ones(8), X),
                 lambda: ops.qlora_rope_fwd(X, 4, 64, plan), lambda: ops.qlora_rope_bwd(X, 4, 64, plan)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        ops.fp8_matmul(X, W, None)
    with pytest.raises(TypeError):
        ops.fp8_matmul(rows, X, None)
    with pytest.raises(ValueError, match="2-D"):
        ops.fp8_matmul(ops.FP8Rows(torch.zeros(8, dtype=torch.float8_e4m3fn), torch.ones(1)), W, None)
    with pytest.raises(ValueError, match="H is X"):
        ops.qlora_add_rmsnorm_fwd(X, None, w, 1e-5, H=torch.zeros_like(X))
    with pytest.raises(ValueError, match="shape"):
        ops.qlora_rope_fwd(X, 3, 64, plan)
