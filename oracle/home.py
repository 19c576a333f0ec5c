"""The home rank's operators in plain fp64 numpy: choice of experts, rows sorted by expert and
merged back, the residual norm, and their gradients (include/moe_step.h states the formulas).
Inputs are the values that the stored bits stand for; nothing is rounded to a stored type except
where a function says so."""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1
BIAS_ON_SCORE = 16  # or-ed to either


def _sigmoid(z):
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))


def _parts(l, m):
    """exp(l - m) with NaN and -inf as 0, equal shares where the largest is +inf."""
    with np.errstate(invalid="ignore", over="ignore"):
        fine = l > -np.inf
        p = np.where(np.isposinf(m), (l == np.inf) * 1.0, np.exp(np.where(fine, l, 0.0) - np.where(np.isfinite(m), m, 0.0)))
    return np.where(fine, p, 0.0)


def gate_scores(logits, score: int) -> np.ndarray:
    """[T][E]: the sigmoid of each logit or the softmax of each token's; 0 for NaN and -inf."""
    l = np.asarray(logits, np.float64)
    if score == SIGMOID:
        return np.where(l > -np.inf, _sigmoid(l), 0.0)
    m = np.max(np.where(np.isnan(l), -np.inf, l), axis=1, keepdims=True)
    p = _parts(l, m)
    z = p.sum(1, keepdims=True)
    return np.where(z > 0, p / np.where(z > 0, z, 1), 0.0)


def choose(logits: np.ndarray, K: int, bias=None, score: int = SOFTMAX, gate=None) -> np.ndarray:
    """[T][K] int32: the K largest ranks, ties to the lowest expert, -1 for positions that no expert
    with a logit and a rank above -inf is left for.  A rank is the logit, with a bias fp32 logit +
    fp32 bias, or with BIAS_ON_SCORE in `score` fp32 gate score + fp32 bias (the scores given as `gate`,
    or gate_scores)."""
    with np.errstate(invalid="ignore", over="ignore"):
        l = logits.astype(np.float32)
        rank = l
        if bias is not None and score & BIAS_ON_SCORE:
            rank = (gate_scores(logits, score & ~BIAS_ON_SCORE) if gate is None else gate).astype(np.float32)
        if bias is not None:
            rank = rank + np.asarray(bias, np.float32)
    ok = (l > -np.inf) & (rank > -np.inf)  # false for NaN
    key = np.where(ok, rank.astype(np.float64), -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :K]
    return np.where(np.take_along_axis(ok, order, 1), order, -1).astype(np.int32)


def shares(logits, expert, score: int, renorm: bool) -> np.ndarray:
    """The chosen positions' weights before the scale factor, [T][K]."""
    score &= ~BIAS_ON_SCORE
    l = np.asarray(logits, np.float64)
    there = expert >= 0
    lc = np.take_along_axis(l, np.where(there, expert, 0).astype(np.int64), 1)
    if score == SIGMOID and not renorm:
        return np.where(there, _sigmoid(lc), 0.0)
    if score == SIGMOID:
        lc = np.minimum(lc, 0) - np.log1p(np.exp(-np.abs(lc)))
    lc = np.where(there, lc, -np.inf)
    over = lc if renorm else l
    m = np.max(np.where(np.isnan(over), -np.inf, over), axis=1, keepdims=True)
    z = _parts(over, m).sum(1, keepdims=True)
    return np.where(z > 0, _parts(lc, m) / np.where(z > 0, z, 1), 0.0)


def route(logits, K: int, bias=None, score: int = SOFTMAX, renorm: bool = True, scale: float = 1.0):
    expert = choose(np.asarray(logits), K, bias, score)
    return expert, scale * shares(logits, expert, score, renorm)


def route_backward(logits, expert, dw, score: int = SOFTMAX, renorm: bool = True, scale: float = 1.0) -> np.ndarray:
    l = np.asarray(logits, np.float64)
    score &= ~BIAS_ON_SCORE
    T, E = l.shape
    expert = np.where((expert >= 0) & (expert < E), expert, -1)
    there = expert >= 0
    p = shares(l, expert, score, renorm)
    v = np.where(there, scale * np.asarray(dw, np.float64), 0.0)
    lc = np.take_along_axis(l, np.where(there, expert, 0).astype(np.int64), 1)
    vp = (v * p).sum(1, keepdims=True)
    d = np.zeros((T, E))
    if score == SOFTMAX and not renorm:
        m = np.max(np.where(np.isnan(l), -np.inf, l), axis=1, keepdims=True)
        e = _parts(l, m)
        z = e.sum(1, keepdims=True)
        d -= np.where(z > 0, e / np.where(z > 0, z, 1), 0.0) * vp
        g = p * v
    else:
        g = p * (v - vp) if renorm else p * v
        if score == SIGMOID:
            g = g * _sigmoid(-lc)
    rows, js = np.nonzero(there)
    np.add.at(d, (rows, expert[rows, js]), g[rows, js])
    return d


def sort_index(expert: np.ndarray, E_loc: int, expert_base: int = 0):
    """perm, pos, counts, offsets, row_slot, nonlocal (whether a pair's expert is neither -1 nor local)."""
    T, K = expert.shape
    flat = expert.reshape(-1).astype(np.int64)
    e = flat - expert_base
    ok = (flat != -1) & (e >= 0) & (e < E_loc)
    pairs = np.flatnonzero(ok)
    pairs = pairs[np.argsort(e[pairs], kind="stable")]
    n, total = flat.size, pairs.size
    perm = np.full(n, -1, np.int32)
    perm[:total] = pairs
    pos = np.full(n, -1, np.int32)
    pos[pairs] = np.arange(total)
    counts = np.bincount(e[ok], minlength=E_loc).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    row_slot = np.where(perm >= 0, perm // K, -1).astype(np.int32)
    return perm, pos, counts, offsets, row_slot, bool(((flat != -1) & ~ok).any())


def merge_rows(rows, pos, w=None) -> np.ndarray:
    """pos [T][K] with -1 for none; w [T][K] or None."""
    T, K = pos.shape
    out = np.zeros((T, rows.shape[1]))
    for j in range(K):
        t = np.flatnonzero((pos[:, j] >= 0) & (pos[:, j] < rows.shape[0]))
        out[t] += rows[pos[t, j]].astype(np.float64) * (1.0 if w is None else np.asarray(w, np.float64)[t, j][:, None])
    return out


def merge_rows_backward(dout, rows, pos, w=None):
    """drows (zero where no position names the row), dw."""
    T, K = pos.shape
    drows, dw = np.zeros(rows.shape), np.zeros((T, K))
    for j in range(K):
        t = np.flatnonzero((pos[:, j] >= 0) & (pos[:, j] < rows.shape[0]))
        g = dout[t].astype(np.float64)
        drows[pos[t, j]] = g * (1.0 if w is None else np.asarray(w, np.float64)[t, j][:, None])
        dw[t, j] = (g * rows[pos[t, j]].astype(np.float64)).sum(1)
    return drows, dw


def residual_norm(x, residual, gamma, eps: float):
    """y, h, r in fp64 (y before any rounding to 8 bits)."""
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * np.asarray(gamma, np.float64), h, r


def group_scales(y: np.ndarray, group: int) -> np.ndarray:
    """[T][groups]: max|y| / 448 over each group of columns (the whole row for 0), at least the
    smallest normal fp32, 1 where all are 0."""
    T, H = y.shape
    g = group or H
    out = [np.abs(y[:, a:a + g]).max(1) for a in range(0, H, g)]
    amax = np.stack(out, 1)
    return np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -126), 1.0)


def residual_norm_backward(dout, h, gamma, rstd, dres=None):
    """dh, dgamma for given h and rstd."""
    dout, h, r = (np.asarray(a, np.float64) for a in (dout, h, rstd))
    xhat = h * r[:, None]
    g = dout * np.asarray(gamma, np.float64)
    dh = r[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    return dh + (0 if dres is None else np.asarray(dres, np.float64)), (dout * xhat).sum(0)
