"""Rotary positions in fp64 numpy (oracle; test infrastructure only).

Pair i of a head turns by position * freq[i] radians; the pairs are (2i, 2i + 1) (interleaved) or (i, i + rot / 2).
The derivative is the transposed rotation."""

import numpy as np


def rope(X, positions, heads, head_dim, freq, rot, interleaved=False, factor=1.0, transpose=False):
    """X [M, heads * head_dim] -> rotated copy."""
    X = np.asarray(X, dtype=np.float64)
    M = X.shape[0]
    x = X.reshape(M, heads, head_dim)
    out = x.copy()
    t = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)[None, :]
    c, s = factor * np.cos(t)[:, None, :], factor * np.sin(t)[:, None, :] * (-1.0 if transpose else 1.0)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
    out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return out.reshape(M, heads * head_dim)


def rope_matrix(position, head_dim, freq, rot, interleaved=False):
    """The head's rotation written out as a matrix (y = R x)."""
    R = np.eye(head_dim)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        t = position * freq[i]
        R[a, a], R[a, b], R[b, a], R[b, b] = np.cos(t), -np.sin(t), np.sin(t), np.cos(t)
    return R
