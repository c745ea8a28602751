"""A workspace that grows while its stream is being captured: the new buffer is zero from then on, for calls outside
the graph and for graphs captured later, whichever of them runs first, and no replay clears its status word."""

import pytest
import torch

from qlora_fine_tuning_nf4_b200 import ops

pytestmark = pytest.mark.gpu

M, K, N = 200, 256, 144
OTHER_BIT = 32  # a bit of the status word that no wait looks at


def _operands(seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    lin = ops.LoraLinear8(ops.fp8_quantize((n(N, K) * 0.02).bfloat16().cuda()), (n(K, 16) * 0.05).bfloat16().cuda(),
                          (n(16, N) * 0.02).bfloat16().cuda(), 0.5)
    return lin, n(M, K).bfloat16().cuda(), n(M, N).bfloat16().cuda()


def _step(lin, X, dY, ws):
    Y, XA = ops.qlora_linear8_fwd(lin, X, ws)
    return (Y, XA, *ops.qlora_linear8_bwd(lin, X, XA, dY, ws))


def _graph(f, pool=None):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, pool=pool):
        out = f()
    return g, out


def _soiled_pool(nbytes):
    """A graph memory pool whose free block of nbytes holds ones in every bit."""
    pool = torch.cuda.graph_pool_handle()
    g, t = _graph(lambda: torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda"), pool)
    g.replay()
    torch.cuda.synchronize()
    del t  # the block goes back to the pool, with its contents
    return pool, g


def test_grown_buffer_is_zero_before_any_replay():
    n = 1 << 20
    pool, keep = _soiled_pool(n)
    ws = ops.Workspace()
    g, _ = _graph(lambda: (ws.get(n), torch.ones(8, device="cuda"))[1], pool)
    assert ws.buf.numel() >= n and torch.count_nonzero(ws.buf).item() == 0


def test_made_in_a_capture():
    pool, keep = _soiled_pool(256)
    made = []
    g, _ = _graph(lambda: (made.append(ops.Workspace()), torch.ones(8, device="cuda"))[1], pool)
    assert torch.count_nonzero(made[0].buf).item() == 0


def test_no_replay_clears_the_status_word():
    ws = ops.Workspace()
    g, _ = _graph(lambda: (ws.get(1 << 16), torch.ones(8, device="cuda"))[1])
    ws.buf[0] = OTHER_BIT
    for _ in range(2):
        g.replay()
    assert ops.qlora_last_device_status(ws) == 7 and ops.qlora_last_device_status(ws) == 0


def test_calls_before_the_first_replay_and_the_second_graph_first():
    """Grown in a capture, then used by a call, then by a second graph that is replayed before the first."""
    lin, X, dY = _operands()
    ref = [t.clone() for t in _step(lin, X, dY, ops.Workspace())]
    ws = ops.Workspace()
    pool, keep = _soiled_pool(ops.qlora_linear8_workspace_bytes(M, K, N, 16))
    g1, o1 = _graph(lambda: _step(lin, X, dY, ws), pool)
    for a, b in zip(_step(lin, X, dY, ws), ref):  # a call, before any replay
        assert torch.equal(a, b)
    assert ops.qlora_last_device_status(ws) == 0
    g2, o2 = _graph(lambda: _step(lin, X, dY, ws))
    for g, out in ((g2, o2), (g1, o1), (g2, o2)):
        for t in out:
            t.fill_(float("nan"))
        g.replay()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    assert ops.qlora_last_device_status(ws) == 0


def test_bf16_and_nf4_calls_grow_in_a_capture_too():
    """The same workspace class serves the other bases."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g)
    lin = ops.LoraLinear16((n(N, K) * 0.02).bfloat16().cuda(), (n(K, 16) * 0.05).bfloat16().cuda(),
                           (n(16, N) * 0.02).bfloat16().cuda(), 0.5)
    X = n(M, K).bfloat16().cuda()
    ref = ops.qlora_linear16_fwd(lin, X, ops.Workspace())
    ws = ops.Workspace()
    pool, keep = _soiled_pool(ops.qlora_linear16_workspace_bytes(M, K, N, 16))
    graph, out = _graph(lambda: ops.qlora_linear16_fwd(lin, X, ws), pool)
    eager = ops.qlora_linear16_fwd(lin, X, ws)
    graph.replay()
    for a, b, c in zip(ref, eager, out):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert ops.qlora_last_device_status(ws) == 0
