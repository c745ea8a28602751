"""The 8-bit formats and the block-scaled product, in fp64 numpy (oracle; test infrastructure only).

e4m3: 1 sign, 4 exponent (bias 7) and 3 mantissa bits, no infinities, 0x7f / 0xff NaN, largest value 448,
subnormals in steps of 2^-9.  A block (128 columns of a row, or 128 x 128 of a weight) has the scale s, the smallest
power of two at least 2^-126 with amax / s <= 448; codes are e4m3(v / s), to nearest, ties to even.  A NaN takes no
part in amax; an infinity makes s infinite and the block's codes 0 or NaN."""

import numpy as np

BLOCK = 128


def e4m3_values():
    """The 256 values of the codes 0..255."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = (-1.0 if c & 0x80 else 1.0), (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        else:
            out[c] = sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return out


_VALUES = e4m3_values()
_POS = _VALUES[:127]                       # 0 .. 448, ascending
_MID = (_POS[1:] + _POS[:-1]) / 2          # exact: the grid has 4 significant bits


def e4m3_encode(v):
    """fp64 -> codes: nearest, ties to the even mantissa; beyond 448 saturates, NaN is 0x7f."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    lo = np.searchsorted(_MID, a, side="left")   # midpoints strictly below a
    hi = np.searchsorted(_MID, a, side="right")
    code = np.where((lo != hi) & (lo % 2 == 1), hi, lo)  # on a midpoint the even one of lo, lo + 1
    code = np.where(np.signbit(v), code | 0x80, code)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def scale_of(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448 (infinite for an infinite amax)."""
    amax = np.asarray(amax, dtype=np.float64)
    s = np.full(amax.shape, 2.0 ** -126)
    fin = np.where(np.isfinite(amax), amax, 1.0)
    while np.any(fin > 448.0 * s):
        s = np.where(fin > 448.0 * s, 2.0 * s, s)
    return np.where(np.isfinite(amax), s, np.inf)


def _codes(t, s):
    with np.errstate(invalid="ignore"):
        return e4m3_encode(np.where(np.isinf(s), np.where(np.isfinite(t), 0.0 * t, np.nan), t / s))


def quantize_rows(X):
    """[M, K] -> (codes uint8 [M, K], scale [ceil(K / 128), M])."""
    X = np.asarray(X, dtype=np.float64)
    M, K = X.shape
    codes, scales = np.empty((M, K), np.uint8), []
    for c in range(0, K, BLOCK):
        t = X[:, c:c + BLOCK]
        s = scale_of(np.max(np.where(np.isnan(t), 0.0, np.abs(t)), axis=1, initial=0.0))
        codes[:, c:c + BLOCK] = _codes(t, s[:, None])
        scales.append(s)
    return codes, np.array(scales).reshape(-1, M)


def quantize_weight(W):
    """[N, K] -> (codes uint8 [N, K], scale [ceil(N / 128), ceil(K / 128)])."""
    W = np.asarray(W, dtype=np.float64)
    N, K = W.shape
    codes, scale = np.empty((N, K), np.uint8), np.empty((-(-N // BLOCK), -(-K // BLOCK)))
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            b = np.s_[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            s = scale_of(np.max(np.where(np.isnan(W[b]), 0.0, np.abs(W[b]))))
            scale[i, j] = s
            codes[b] = _codes(W[b], s)
    return codes, scale


def dequantize_rows(codes, scale):
    with np.errstate(invalid="ignore"):
        return _VALUES[codes] * np.repeat(np.asarray(scale, np.float64).T, BLOCK, axis=1)[:, :codes.shape[1]]


def dequantize_weight(codes, scale):
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), BLOCK, axis=0), BLOCK, axis=1)
    with np.errstate(invalid="ignore"):
        return _VALUES[codes] * s[:codes.shape[0], :codes.shape[1]]
