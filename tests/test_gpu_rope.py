"""GPU parity of qlora_rope_fwd / _bwd against fp64: both pairings, every vector width (rotated parts that divide
by 16, 8, 4 and 2), part of the head, far and negative positions, sliced rows, in place.

Bound: the angle is exact to 2^-32 turns and a binary32 rounding of half a turn (2^-25 of pi), cosine and sine to
two units in the last place: together below 2^-21 absolute, times |a| + |b|; four fp32 roundings; one bf16
rounding (2^-8)."""

import numpy as np
import pytest
import torch

from oracle import rope as oracle_rope
from qlora_fine_tuning_nf4_b200 import ops

from parity import gpu_f64

pytestmark = pytest.mark.gpu

SHAPES = [  # M, heads, D, rot
    (1, 40, 128, 128), (7, 3, 128, 64), (130, 5, 64, 64), (33, 2, 96, 48), (5, 9, 80, 40), (6, 1, 256, 256),
    (9, 4, 40, 20), (11, 3, 24, 6), (4, 7, 8, 2), (3, 2, 512, 512), (2, 1, 512, 34), (515, 64, 32, 32)]


def _bound(X, ref, heads, D, rot, inter, factor=1.0):
    M = X.shape[0]
    x = np.abs(X).reshape(M, heads, D)
    s = np.zeros_like(x)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    s[:, :, a] = s[:, :, b] = x[:, :, a] + x[:, :, b]
    return 2.0 ** -8 * np.abs(ref) + 1.01 * factor * (2.0 ** -21 + 2.0 ** -22) * s.reshape(M, heads * D)


def _data(M, cols, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(M, cols, generator=g).bfloat16()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("M,heads,D,rot", SHAPES)
def test_parity(M, heads, D, rot, inter):
    X = _data(M, heads * D, M + rot)
    pos = torch.randint(0, 1 << 20, (M,), generator=torch.Generator().manual_seed(M))
    plan = ops.rope_plan(rot)
    freq, _ = ops.rope_frequencies(rot)
    Xg, pg = X.cuda(), pos.cuda()
    for f, t in ((ops.qlora_rope_fwd, False), (ops.qlora_rope_bwd, True)):
        ref = oracle_rope.rope(X.double().numpy(), pos.numpy(), heads, D, freq, rot, inter, transpose=t)
        out = f(Xg, heads, D, plan, positions=pg, interleaved=inter)
        assert np.all(np.abs(gpu_f64(out) - ref) <= _bound(X.double().numpy(), ref, heads, D, rot, inter))
        same = Xg.clone()
        assert f(same, heads, D, plan, positions=pg, interleaved=inter, out=same) is same
        assert torch.equal(same, out)
    assert torch.equal(Xg.cpu(), X)


@pytest.mark.parametrize("inter", [False, True])
def test_slices_of_wider_rows(inter):
    """The q | k columns of rows of 6 x 64: rotated in place, the v columns left as they were; out in a slice too."""
    full = _data(50, 6 * 64 + 8, 1).cuda()
    keep = full.clone()
    plan, freq = ops.rope_plan(64), ops.rope_frequencies(64)[0]
    pos = torch.arange(50, device="cuda") * 1000
    qk = full[:, :4 * 64]
    ref = oracle_rope.rope(gpu_f64(qk), pos.cpu().numpy(), 4, 64, freq, 64, inter)
    plain = ops.qlora_rope_fwd(qk, 4, 64, plan, positions=pos, interleaved=inter)
    assert np.all(np.abs(gpu_f64(plain) - ref) <= _bound(gpu_f64(qk), ref, 4, 64, 64, inter))
    wide = torch.full((50, 4 * 64 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.qlora_rope_fwd(qk, 4, 64, plan, positions=pos, interleaved=inter, out=wide[:, 8:8 + 256])
    assert torch.equal(wide[:, 8:264], plain)
    assert torch.all(wide[:, :8] == 7.0) and torch.all(wide[:, 264:] == 7.0)
    ops.qlora_rope_fwd(qk, 4, 64, plan, positions=pos, interleaved=inter, out=qk)
    assert torch.equal(full[:, :256], plain) and torch.equal(full[:, 256:], keep[:, 256:])
    # other columns of the same rows
    ops.qlora_rope_fwd(keep[:, :128], 2, 64, plan, positions=pos, interleaved=inter, out=keep[:, 256:384])
    assert torch.equal(keep[:, 256:384], plain[:, :128])


def test_positions():
    """None counts rows (modulo seq_len); far and negative positions are exact; position 0 changes nothing."""
    X = _data(10, 2 * 128, 3)
    Xg = X.cuda()
    plan, freq = ops.rope_plan(128), ops.rope_frequencies(128)[0]
    a = lambda p: torch.tensor(p, device="cuda")
    assert torch.equal(ops.qlora_rope_fwd(Xg, 2, 128, plan),
                       ops.qlora_rope_fwd(Xg, 2, 128, plan, positions=a(list(range(10)))))
    assert torch.equal(ops.qlora_rope_fwd(Xg, 2, 128, plan, seq_len=4),
                       ops.qlora_rope_fwd(Xg, 2, 128, plan, positions=a([i % 4 for i in range(10)])))
    assert torch.equal(ops.qlora_rope_fwd(Xg, 2, 128, plan, positions=a([0] * 10)), Xg)
    far = [2 ** 31 - 1, 2 ** 24 + 1, 10 ** 7, -1, -12345, 123456789, 1, 2, 3, 4]
    out = ops.qlora_rope_fwd(Xg, 2, 128, plan, positions=a(far))
    # the reference's own angle: position * frequency in binary64 is off by 2^-53 of 2^31 radians
    ref = oracle_rope.rope(X.double().numpy(), np.array(far), 2, 128, freq, 128)
    bound = _bound(X.double().numpy(), ref, 2, 128, 128, False)
    assert np.all(np.abs(gpu_f64(out) - ref) <= bound + 2.0 ** -21)
    # a rotation by p and its transpose give X back, to two roundings of a pair's length
    back = ops.qlora_rope_bwd(out, 2, 128, plan, positions=a(far))
    pair = np.hypot(*np.split(gpu_f64(Xg).reshape(10, 2, 128), 2, axis=2))
    err = np.abs(gpu_f64(back) - gpu_f64(Xg)).reshape(10, 2, 128)
    assert np.all(err <= np.concatenate([pair, pair], 2) * (2.0 ** -8 * 2.5 + 2.0 ** -18))


def test_scaled_frequencies_and_factor():
    X = _data(20, 3 * 64, 4)
    pos = torch.arange(20) * 5000
    s = {"type": "yarn", "factor": 16.0, "original_max_position": 4096}
    plan, (freq, factor) = ops.rope_plan(64, 10000.0, s), ops.rope_frequencies(64, 10000.0, s)
    assert factor > 1.2
    for f, t in ((ops.qlora_rope_fwd, False), (ops.qlora_rope_bwd, True)):
        ref = oracle_rope.rope(X.double().numpy(), pos.numpy(), 3, 64, freq, 64, factor=factor, transpose=t)
        out = f(X.cuda(), 3, 64, plan, positions=pos.cuda())
        assert np.all(np.abs(gpu_f64(out) - ref) <= _bound(X.double().numpy(), ref, 3, 64, 64, False, factor))


def test_gradient_by_differences():
    """<rope(x + h v) - rope(x - h v), dy> / 2h = <v, rope_bwd(dy)>: the map is linear."""
    X, dY, V = (_data(6, 2 * 32, s) for s in (1, 2, 3))
    plan, freq = ops.rope_plan(24), ops.rope_frequencies(24)[0]
    pos = torch.arange(6, device="cuda") * 37
    dX = gpu_f64(ops.qlora_rope_bwd(dY.cuda(), 2, 32, plan, positions=pos, interleaved=True))
    f = lambda x: np.sum(oracle_rope.rope(x, pos.cpu().numpy(), 2, 32, freq, 24, True) * dY.double().numpy())
    x, v = X.double().numpy(), V.double().numpy()
    num = (f(x + 0.5 * v) - f(x - 0.5 * v)) / 1.0
    assert abs(np.sum(dX * v) - num) <= np.sum(np.abs(dX * v)) * 2.0 ** -8 + 1e-6


def test_empty_batch_and_overlap_refused():
    plan = ops.rope_plan(64)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert ops.qlora_rope_fwd(e, 2, 64, plan).shape == (0, 128)
    buf = torch.zeros(8, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        ops.qlora_rope_fwd(buf[:, :128], 2, 64, plan, out=buf[:, 64:192])
    with pytest.raises(ValueError, match="overlaps"):
        ops.qlora_rope_fwd(buf[:4, :128], 2, 64, plan, out=buf[1:5, :128])
    with pytest.raises(ValueError, match="overlaps"):
        flat = buf.view(-1)[:8 * 128].view(8, 128)
        ops.qlora_rope_fwd(buf[:, :128], 2, 64, plan, out=flat)
