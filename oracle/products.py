"""The experts' products in plain fp64 numpy (include/moe_step.h states the formulas).  Inputs are the values that
the stored bits stand for; nothing is rounded to a stored type."""
from __future__ import annotations

import numpy as np


def spans(offsets, n: int):
    """(first row, end) of each expert: offsets cut to an ascending range within [0, n]."""
    o = np.asarray(offsets, np.int64)
    for e in range(len(o) - 1):
        a = min(max(o[e], 0), n)
        yield int(a), int(max(a, min(o[e + 1], n)))


def scaled(codes, scale, rows: int) -> np.ndarray:
    """Values of 8-bit codes [R][C] with a scale per `rows` rows and 128 columns."""
    R, C = codes.shape
    return np.asarray(codes, np.float64) * np.asarray(scale, np.float64)[np.arange(R) // rows][:, np.arange(C) // 128]


def expert_matmul(x, w, offsets, n: int, row_slot=None, transposed: bool = False) -> np.ndarray:
    """[n][N]; NaN for rows that no expert has.  A row_slot outside x is a row of zeros."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    out = np.full((n, w.shape[2] if transposed else w.shape[1]), np.nan)
    for e, (a, b) in enumerate(spans(offsets, n)):
        rows = x[a:b]
        if row_slot is not None:
            s = np.asarray(row_slot[a:b], np.int64)
            ok = (s >= 0) & (s < len(x))
            rows = np.zeros((b - a, x.shape[1]))
            rows[ok] = x[s[ok]]
        out[a:b] = rows @ (w[e] if transposed else w[e].T)
    return out


def expert_matmul_backward(dout, x, offsets) -> np.ndarray:
    dout, x = np.asarray(dout, np.float64), np.asarray(x, np.float64)
    return np.stack([dout[a:b].T @ x[a:b] for a, b in spans(offsets, len(x))])


def sigmoid(g):
    g = np.asarray(g, np.float64)
    z = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + z), z / (1 + z))


def swiglu(gu) -> np.ndarray:
    I = gu.shape[1] // 2
    g, u = np.asarray(gu[:, :I], np.float64), np.asarray(gu[:, I:], np.float64)
    return g * sigmoid(g) * u


def swiglu_backward(gu, dh) -> np.ndarray:
    I = gu.shape[1] // 2
    g, u, d = np.asarray(gu[:, :I], np.float64), np.asarray(gu[:, I:], np.float64), np.asarray(dh, np.float64)
    s = sigmoid(g)
    return np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], 1)


def block_scales(w) -> np.ndarray:
    """[ceil(N / 128)][ceil(D / 128)]: max|w| / 448 over each 128 x 128 block, at least the smallest normal fp32, 1
    where all are 0."""
    N, D = w.shape
    out = np.ones((-(-N // 128), -(-D // 128)))
    for a in range(out.shape[0]):
        for b in range(out.shape[1]):
            m = np.abs(np.asarray(w[a * 128:a * 128 + 128, b * 128:b * 128 + 128], np.float64)).max()
            if m > 0:
                out[a, b] = max(m / 448, 2.0 ** -126)
    return out
