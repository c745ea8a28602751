"""The operators in a row, as a decoder layer's attention input uses them: the residual stream takes a sublayer's
output and is normed (bf16 and 8-bit rows), the fused projection over an e4m3 weight reads the 8-bit rows, the q and k
columns of its output are rotated in place; and the backward of all of it, down to the gradient of the residual stream.

Each step is held to fp64 with the values that went into it (the bounds of the operators' own tests, loosened to the
larger of their terms), then the whole run is captured in a graph, run on another stream, and run twice at once."""

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8, rope as oracle_rope
from qlora_fine_tuning_nf4_b200 import ops

from parity import gpu_f64

pytestmark = pytest.mark.gpu

D_MODEL, HEADS, KV, HD = 512, 4, 2, 64          # q 256 + k 128 + v 128 columns
N = (HEADS + 2 * KV) * HD


class Layer:
    def __init__(self, seed=0, r=16):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)
        self.w = (1 + 0.1 * n(D_MODEL)).bfloat16().cuda()
        self.W = (n(N, D_MODEL) * 0.02).bfloat16()
        self.lin = ops.LoraLinear8(ops.fp8_quantize(self.W.cuda()), (n(D_MODEL, r) * 0.05).bfloat16().cuda(),
                                   (n(r, N) * 0.02).bfloat16().cuda(), 0.5)
        self.plan = ops.rope_plan(HD)

    def forward(self, x, res, ws, seq):
        H, Y, rstd, Y8 = ops.qlora_add_rmsnorm_fwd(x, res, self.w, 1e-5, quantize=True)
        QKV, XA = ops.qlora_linear8_fwd(self.lin, Y, ws, X8=Y8)
        raw = QKV.clone()
        qk = QKV[:, :(HEADS + KV) * HD]
        ops.qlora_rope_fwd(qk, HEADS + KV, HD, self.plan, seq_len=seq, out=qk)
        return dict(H=H, Y=Y, rstd=rstd, Y8=Y8, raw=raw, QKV=QKV, XA=XA)

    def backward(self, f, dQKV, dH, ws, seq):
        d = dQKV.clone()
        qk = d[:, :(HEADS + KV) * HD]
        ops.qlora_rope_bwd(qk, HEADS + KV, HD, self.plan, seq_len=seq, out=qk)
        dY, dA, dB = ops.qlora_linear8_bwd(self.lin, f["Y"], f["XA"], d, ws)
        return dict(d=d, dY=dY, dA=dA, dB=dB, dX=ops.qlora_add_rmsnorm_bwd(f["H"], self.w, f["rstd"], dY, dH=dH))


def _data(M, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    return n(M, D_MODEL), n(M, D_MODEL), n(M, N), n(M, D_MODEL)


def _near(got, ref, slack):
    assert np.all(np.abs(gpu_f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + slack)


@pytest.mark.parametrize("M", [1, 24, 200, 1500])
def test_chain(M):
    L, ws = Layer(), ops.Workspace()
    x, res, dQKV, dH = _data(M, M)
    f = L.forward(x, res, ws, 100)
    b = L.backward(f, dQKV, dH, ws, 100)
    assert ops.qlora_last_device_status(ws) == 0
    # norm
    assert torch.equal(f["H"], (x.double() + res.double()).bfloat16())
    w = gpu_f64(L.w)
    y, _ = oracle.rmsnorm_fwd(gpu_f64(f["H"]), w, float(np.float32(1e-5)))
    _near(f["Y"], y, 2.0 ** -20 * np.abs(y))
    # projection, from the rows the norm wrote
    wv = fp8.dequantize_weight(*fp8.quantize_weight(L.W.double().numpy()))
    yq = fp8.dequantize_rows(*fp8.quantize_rows(gpu_f64(f["Y"])))
    yy, A, B, s = gpu_f64(f["Y"]), gpu_f64(L.lin.A), gpu_f64(L.lin.B), 0.5
    low = lambda p, q: s * 2.0 ** -8 * 1.1 * np.abs(p) @ np.abs(q)  # the low-rank operand's own rounding
    ref = yq @ wv.T + s * yy @ A @ B
    _near(f["raw"], ref, 2.0 ** -16 * np.abs(yq) @ np.abs(wv).T + low(yy @ A, B))
    # rotation of q and k, v as it was
    nqk = (HEADS + KV) * HD
    freq = ops.rope_frequencies(HD)[0]
    pos = np.arange(M) % 100
    raw = gpu_f64(f["raw"])
    ref = oracle_rope.rope(raw[:, :nqk], pos, HEADS + KV, HD, freq, HD)
    _near(f["QKV"][:, :nqk], ref, 2.0 ** -19 * np.max(np.abs(raw)))
    assert torch.equal(f["QKV"][:, nqk:], f["raw"][:, nqk:])
    # backward
    d = gpu_f64(b["d"])
    ref = oracle_rope.rope(gpu_f64(dQKV)[:, :nqk], pos, HEADS + KV, HD, freq, HD, transpose=True)
    _near(b["d"][:, :nqk], ref, 2.0 ** -19 * np.max(np.abs(gpu_f64(dQKV))))
    dq, G = fp8.dequantize_rows(*fp8.quantize_rows(d)), d @ B.T
    _near(b["dY"], dq @ wv + s * G @ A.T, 2.0 ** -16 * np.abs(dq) @ np.abs(wv) + low(G, A.T))
    _near(b["dA"], s * yy.T @ G, s * np.abs(yy).T @ np.abs(G) * (2.0 ** -8 * 1.1 + M * 2.0 ** -23))
    xa = gpu_f64(f["XA"])
    _near(b["dB"], s * xa.T @ d, s * np.abs(xa).T @ np.abs(d) * (M + 2) * 2.0 ** -23)
    h, g = gpu_f64(f["H"]), gpu_f64(b["dY"])
    ref = gpu_f64(dH) + oracle.rmsnorm_bwd(h, w, float(np.float32(1e-5)), g)
    _near(b["dX"], ref, 2.0 ** -12 * (np.max(np.abs(g)) + np.max(np.abs(h))))


def _run(L, data, ws, seq=64):
    f = L.forward(data[0], data[1], ws, seq)
    b = L.backward(f, data[2], data[3], ws, seq)
    return [f["H"], f["QKV"], f["XA"], f["rstd"], b["dX"], b["dA"], b["dB"]]


@pytest.mark.parametrize("r", [16, 64])
@pytest.mark.parametrize("M", [3, 24, 400, 2100])
def test_captured_graph_replays_the_same_bits(M, r):
    """Two graphs, of different sizes, share one workspace that grows between their captures; each replay, in any
    order, gives the eager run's bits, with the inputs of the moment."""
    L, ws = Layer(r=r), ops.Workspace()
    sizes = (M, 3 * M + 1)
    data = [_data(m, 10 + m) for m in sizes]
    graphs, outs = [], []
    for d in data:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _run(L, d, ops.Workspace())  # warm-up with a workspace of its own: the shared one grows in the capture
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = _run(L, d, ws)
        graphs.append(g)
        outs.append(o)
    for seed in (1, 2):
        for d, m in zip(data, sizes):
            for t, n in zip(d, _data(m, seed + m)):
                t.copy_(n)
        refs = [_run(L, d, ops.Workspace()) for d in data]
        torch.cuda.synchronize()
        for i in (0, 1, 0):
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[i], refs[i]):
                assert torch.equal(a, b)


def test_other_streams_and_two_at_once():
    """On a side stream, and on two streams at once with a workspace each, the result is the default stream's."""
    L = Layer()
    data = [_data(700, 5), _data(90, 6)]
    refs = [_run(L, d, ops.Workspace()) for d in data]
    streams = [torch.cuda.Stream() for _ in data]
    spaces = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            spaces.append(ops.Workspace())
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(_run(L, data[i], spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            for a, b in zip(o, refs[i]):
                assert torch.equal(a, b)
        assert ops.qlora_last_device_status(spaces[i]) == 0


def test_training_step_gradients_by_differences():
    """The adapter's gradients of the whole run against central differences of an fp64 run (quantisation as an
    identity in the derivative: the low-rank branch reads the bf16 rows, so the loss is smooth in A and B)."""
    M, L, ws = 32, Layer(3), ops.Workspace()
    x, res, dQKV, dH = _data(M, 7)
    f = L.forward(x, res, ws, 0)
    b = L.backward(f, dQKV, dH, ws, 0)
    y, A, B, s = gpu_f64(f["Y"]), gpu_f64(L.lin.A), gpu_f64(L.lin.B), 0.5
    freq, nqk, pos = ops.rope_frequencies(HD)[0], (HEADS + KV) * HD, np.arange(M)

    def loss(A_, B_):
        q = s * y @ A_ @ B_
        q[:, :nqk] = oracle_rope.rope(q[:, :nqk], pos, HEADS + KV, HD, freq, HD)
        return np.sum(q * gpu_f64(dQKV))

    rng = np.random.default_rng(0)
    G = gpu_f64(b["d"]) @ B.T
    for got, ref, mag in ((b["dA"], 0, np.abs(y).T @ np.abs(G)), (b["dB"], 1, np.abs(y @ A).T @ np.abs(gpu_f64(b["d"])))):
        v = rng.standard_normal(tuple(got.shape))
        num = (loss(A + v, B) - loss(A - v, B)) / 2 if ref == 0 else (loss(A, B + v) - loss(A, B - v)) / 2
        # roundings of the rotated gradient, the low-rank operand and the result, each 2^-8 over the sums' magnitudes
        tol = np.sum((2.0 ** -8 * np.abs(gpu_f64(got)) + 2.1 * 2.0 ** -8 * s * mag) * np.abs(v))
        assert abs(np.sum(gpu_f64(got) * v) - num) <= tol
