"""Pins of the 8-bit and rotary oracles (oracle/fp8.py, oracle/rope.py) to things other than themselves."""

import math

import numpy as np
import pytest
import torch

from oracle import fp8, rope
from qlora_fine_tuning_nf4_b200 import ops


def test_e4m3_values_match_torch():
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp8.e4m3_values(), ref, equal_nan=True)


def test_encode_matches_torch_on_all_bf16_values():
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v) & (v.abs() <= 448)]
    ref = v.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.e4m3_encode(v.double().numpy()), ref)
    assert fp8.e4m3_encode(np.array([np.nan]))[0] == 0x7F
    # ties go to the even mantissa: halfway between 1 (0x38) and 1.125 (0x39), and 1.125 and 1.25 (0x3a)
    assert list(fp8.e4m3_encode(np.array([1.0625, 1.1875, -1.0625]))) == [0x38, 0x3A, 0xB8]


def test_scale_is_the_smallest_power_of_two():
    for amax in (0.0, 1e-45, 448.0, 448.1, 1.75, 1.7500001, 3e38, 2.0 ** -126 * 448, 2.0 ** -126 * 449):
        s = float(fp8.scale_of(np.array(amax)))
        assert math.frexp(s)[0] == 0.5 and s >= 2.0 ** -126
        assert amax / s <= 448.0
        assert s == 2.0 ** -126 or amax / (s / 2) > 448.0
    assert np.isinf(fp8.scale_of(np.array(np.inf)))


def test_quantize_error_and_special_values():
    rng = np.random.default_rng(0)
    X = rng.standard_normal((5, 300)) * rng.uniform(1e-3, 1e3, (5, 1))
    codes, scale = fp8.quantize_rows(X)
    back = fp8.dequantize_rows(codes, scale)
    assert scale.shape == (3, 5)
    # half a step of 2^-3 relative, or half a subnormal step of 2^-9
    assert np.all(np.abs(back - X) <= np.maximum(2.0 ** -4 * np.abs(X), 2.0 ** -10 * np.repeat(scale.T, 128, 1)[:, :300]))
    X[1, 7] = np.nan
    X[2, 200] = -np.inf
    back = fp8.dequantize_rows(*fp8.quantize_rows(X))
    assert np.isnan(back[1, 7]) and np.isnan(back[1]).sum() == 1
    assert np.isnan(back[2, 128:256]).all() and np.isfinite(back[2, :128]).all() and np.isfinite(back[2, 256:]).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_the_rotation_matrix_and_its_transpose(interleaved):
    rng = np.random.default_rng(1)
    D, rot, heads, M = 24, 16, 3, 5
    freq, factor = ops.rope_frequencies(rot)
    assert factor == 1.0 and freq[0] == 1.0
    pos = rng.integers(0, 5000, M)
    X, dY = rng.standard_normal((M, heads * D)), rng.standard_normal((M, heads * D))
    Y = rope.rope(X, pos, heads, D, freq, rot, interleaved)
    dX = rope.rope(dY, pos, heads, D, freq, rot, interleaved, transpose=True)
    for m in range(M):
        R = rope.rope_matrix(pos[m], D, freq, rot, interleaved)
        assert np.allclose(Y[m].reshape(heads, D), X[m].reshape(heads, D) @ R.T, atol=1e-12)
        assert np.allclose(dX[m].reshape(heads, D), dY[m].reshape(heads, D) @ R, atol=1e-12)
    assert np.isclose(np.sum(Y * dY), np.sum(X * dX))  # the gradient of a linear map is its adjoint


def test_rope_frequencies():
    f0, _ = ops.rope_frequencies(128, 10000.0)
    assert np.allclose(f0, 10000.0 ** (-np.arange(0, 128, 2) / 128), rtol=1e-15)
    lin, a = ops.rope_frequencies(128, 10000.0, {"type": "linear", "factor": 4.0})
    assert np.allclose(np.array(lin) * 4, f0) and a == 1.0
    ntk, _ = ops.rope_frequencies(128, 10000.0, {"type": "ntk", "factor": 4.0})
    assert ntk[0] == 1.0 and np.isclose(ntk[-1] * 4, f0[-1])
    args = {"type": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
            "original_max_position": 8192}
    l3, a = ops.rope_frequencies(128, 500000.0, args)
    base, _ = ops.rope_frequencies(128, 500000.0)
    turns = 8192 * np.array(base) / (2 * np.pi)
    assert a == 1.0
    assert np.allclose(np.array(l3)[turns > 4], np.array(base)[turns > 4])
    assert np.allclose(np.array(l3)[turns < 1] * 8, np.array(base)[turns < 1])
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all(np.array(l3)[mid] < np.array(base)[mid]) and np.all(np.array(l3)[mid] * 8 > np.array(base)[mid])
    yarn, a = ops.rope_frequencies(128, 10000.0, {"type": "yarn", "factor": 16.0, "original_max_position": 4096})
    turns = 4096 * np.array(f0) / (2 * np.pi)
    assert np.isclose(a, 0.1 * np.log(16.0) + 1.0)
    r = np.array(yarn) / f0
    assert np.all(np.diff(r) <= 1e-12)  # from kept (1) to stretched (1 / 16), one way
    first_below = lambda t: int(np.argmax(turns < t))
    assert np.allclose(r[:first_below(32.0)], 1.0) and np.allclose(r[first_below(1.0) + 1:], 1 / 16)
    # a plan's 64-bit fractions stand for these frequencies
    plan = ops.rope_plan(128, 10000.0, {"type": "linear", "factor": 4.0}, device="cpu")
    turns = np.array([t % 2 ** 64 for t in plan.turns.tolist()], dtype=np.float64) / 2.0 ** 64
    assert np.allclose(turns * 2 * np.pi, lin, rtol=1e-15)
    # a frequency of more than one turn per position keeps its fraction
    fast = ops.rope_plan(4, 1e-4, device="cpu").turns.tolist()[1] % 2 ** 64 / 2.0 ** 64
    assert abs(fast - (100.0 / (2 * np.pi)) % 1.0) < 1e-12


@pytest.mark.parametrize("kw", [dict(rot=7), dict(rot=0), dict(rot=8, base=-1.0),
                                dict(rot=8, scaling={"type": "spiral"}), dict(rot=8, scaling={"type": "linear"}),
                                dict(rot=8, scaling={"type": "linear", "factor": 0.0}),
                                dict(rot=8, scaling={"type": "linear", "factor": 2.0, "theta": 3}),
                                dict(rot=2, scaling={"type": "ntk", "factor": 2.0}),
                                dict(rot=8, scaling={"type": "llama3", "factor": 2.0, "low_freq_factor": 4.0,
                                                     "high_freq_factor": 1.0, "original_max_position": 10})])
def test_rope_frequencies_refusals(kw):
    with pytest.raises(ValueError):
        ops.rope_frequencies(**kw)
