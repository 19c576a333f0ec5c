"""The home rank's operators on the GPU against the fp64 oracle (oracle/home.py).

Tolerances, with u = 2^-24 (half a step of fp32, relative) and v = half a step of the stored type
(fp32 u, bf16 2^-8, e4m3 2^-4 and 2^-10 scale below its normal numbers):
  * a sum of terms s_i through chains and trees of at most d additions is off by at most d u sum|s_i|;
    a lane's chain of a row of H elements is at most 8 ceil(H / 512) long, the tree over lanes and
    waves at most 10 deep, so d = 8 ceil(H / 512) + 10;
  * a product, quotient, root or conversion adds u, expf and log1pf 2 u and u times the size of the
    exponent that they are taken at.
Every bound below counts those for its formula and adds v |result| for the stored result."""
import math

import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M
from gpu_helpers import sync_err
from oracle import home as O
from oracle.moe_oracle import decode_e4m3

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
I32 = torch.int32


def depth(H):
    return 8 * math.ceil(H / 512) + 10


def gpu(a, dtype=None, pad=0):
    """A numpy array on the GPU in `dtype`; with pad, as a view of rows that are pad elements further apart."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    t = t.to(dtype) if dtype is not None else t
    if pad:
        full = torch.full((t.shape[0], t.shape[1] + pad), 7, dtype=t.dtype)
        full[:, :t.shape[1]] = t
        return full.cuda()[:, :t.shape[1]]
    return t.cuda()


def like(shape, dtype, pad=0, fill=0):
    kind = torch.uint8 if dtype == FP8 else dtype
    full = torch.full((shape[0], shape[1] + pad), fill, dtype=kind, device="cuda")
    return full.view(dtype)[:, :shape[1]]


def val(t):
    """Stored values as fp64."""
    t = t.detach().cpu()
    return decode_e4m3(t.view(torch.uint8).numpy()) if t.dtype == FP8 else t.double().numpy()


def errword():
    return torch.zeros(1, dtype=I32, device="cuda")


def within(got, ref, tol, what=""):
    off = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and off.max(initial=-1.0) <= 0, f"{what}: over its bound by {off.max():.3g}"


# ------------------------------------------------------------------------------------------ route
def hard_logits(rng, T, E, dtype):
    """Normal rows, and by turns: ties, all -inf, NaN and -inf among numbers, the type's lowest value
    as a mask, nothing but it, very large ones, signed zeros, one or two +inf."""
    l = rng.standard_normal((T, E)) * 2
    low = torch.finfo(dtype).min
    for t in range(T):
        kind = t % 9
        if kind == 1:
            l[t] = np.round(l[t])
        elif kind == 2:
            l[t] = -np.inf
        elif kind == 3:
            l[t, rng.random(E) < 0.7] = np.nan
            l[t, rng.random(E) < 0.3] = -np.inf
        elif kind == 4:
            l[t, rng.random(E) < 0.9] = low
        elif kind == 5:
            l[t] = low
        elif kind == 6:
            l[t] *= 40
        elif kind == 7:
            l[t] = rng.choice([0.0, -0.0, -1.0], E)
        elif kind == 8:
            l[t, rng.integers(0, E, 2)] = np.inf
    return l


ROUTES = [(8, 2), (16, 16), (5, 5), (32, 3), (60, 4), (64, 6), (100, 8), (128, 4), (256, 8), (384, 8), (512, 32), (1, 1),
          (130, 20)]


@pytest.mark.parametrize("E,K", ROUTES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route(E, K, dtype):
    rng = np.random.default_rng(E * 100 + K)
    for case, (T, pad, score, renorm, scale) in enumerate([(1, 0, 0, True, 1.0), (77, 0, 0, False, 2.5), (50, 3, 1, True, 2.5),
                                                           (33, 8, 1, False, 1.0), (19, 0, 0, True, 0.5)]):
        logits = gpu(hard_logits(rng, T, E, dtype), dtype, pad)
        bias = None
        if case >= 2:
            b = rng.standard_normal(E).astype(np.float32)
            b[rng.random(E) < 0.2] = -np.inf
            bias = gpu(b)
        expert, w = like((T, K), I32, fill=-7), like((T, K), F32, fill=-7)
        M.moe_route(logits, expert, w, bias=bias, score=score, renorm=renorm, scale=scale)
        l = val(logits)
        re, rw = O.route(l, K, None if bias is None else bias.cpu().numpy(), score, renorm, scale)
        assert np.array_equal(expert.cpu().numpy(), re), f"case {case}"
        # exponents are taken at l - m, m the largest logit in finite rows; 2 u each for exp, log1p, the
        # quotients and the products, the sum over E of d <= 32 + 10
        with np.errstate(invalid="ignore", over="ignore"):
            lc = np.take_along_axis(l, np.maximum(re, 0).astype(np.int64), 1)
            top = np.nanmax(np.where(np.isfinite(l) & (np.abs(l) < 1e30), l, -np.inf), axis=1, keepdims=True)
            size = np.where(np.isfinite(lc) & np.isfinite(top), np.minimum(np.abs(lc) + np.abs(top), 1e3), 0)
        within(val(w), rw, rw * (60 + 4 * size) * U + 1e-37, f"case {case}")


@pytest.mark.parametrize("E,K", ROUTES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_backward(E, K, dtype):
    rng = np.random.default_rng(E * 100 + K + 1)
    for case, (T, pad, score, renorm, scale) in enumerate([(1, 0, 0, True, 1.0), (77, 0, 0, False, 2.5), (50, 3, 1, True, 2.5),
                                                           (33, 8, 1, False, 1.0)]):
        logits = gpu(hard_logits(rng, T, E, dtype), dtype, pad)
        l = val(logits)
        expert = O.choose(l, K)
        wild = case == 1
        if wild and K > 1:  # the same expert twice, and one that does not exist
            expert[3, 1] = expert[3, 0]
            expert[4, 0] = E + 5
            expert[5, 1] = -2
        dw = rng.standard_normal((T, K)).astype(np.float32)
        dl, err = like((T, E), dtype, pad, fill=3), errword()
        M.moe_route_backward(logits, gpu(expert), gpu(dw), dl, err, score=score, renorm=renorm, scale=scale)
        assert sync_err(err) == (M.ERR_EXPERT_NONLOCAL if wild and K > 1 else 0)
        ref = O.route_backward(l, expert, dw, score, renorm, scale)
        e = np.where((expert >= 0) & (expert < E), expert, -1)
        p = O.shares(l, e, score, renorm)
        v = scale * np.abs(dw)
        # every term is a product of shares (off by (60 + 4 size) u, as above) and of v; at most K meet
        with np.errstate(invalid="ignore", over="ignore"):
            top = np.nanmax(np.where(np.isfinite(l) & (np.abs(l) < 1e30), np.abs(l), 0), axis=1, keepdims=True)
        mag = (p * v).max(1, keepdims=True) + (p * v).sum(1, keepdims=True)
        tol = 2 * mag * (80 + 8 * np.minimum(top, 1e3) + K) * U + HALF[dtype] * np.abs(ref) + 1e-37
        within(val(dl), ref, tol, f"case {case}")


def test_route_differences():
    """The gradient against differences of moe_route itself: fp32 shares off by 100 u, over a step of
    2^-7, is 100 2^-24 2^8 = 1.6e-3 a term, two terms and K = 4; the formula's own error is below 1e-4."""
    T, E, K, step = 6, 12, 4, 2.0 ** -7
    rng = np.random.default_rng(9)
    l = rng.permutation(T * E).reshape(T, E) / 16.0 - 2  # gaps of 1/16 or more: no step changes the choice
    l = l - l.mean(1, keepdims=True)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    for score in (M.MOE_SOFTMAX, M.MOE_SIGMOID):
        for renorm in (True, False):
            def f(a):
                lg = gpu(a, F32)
                e, w = like((T, K), I32), like((T, K), F32)
                M.moe_route(lg, e, w, score=score, renorm=renorm)
                return (val(w) * dw).sum(1), e
            _, e = f(l)
            dl, err = like((T, E), F32), errword()
            M.moe_route_backward(gpu(l, F32), e, gpu(dw), dl, err, score=score, renorm=renorm)
            got = val(dl)
            for c in range(E):
                hi, lo = l.copy(), l.copy()
                hi[:, c] += step
                lo[:, c] -= step
                fh, eh = f(hi)
                fl, el = f(lo)
                assert torch.equal(eh, e) and torch.equal(el, e)
                assert np.abs((fh - fl) / (2 * step) - got[:, c]).max() <= 1.4e-2


# ------------------------------------------------------------------------------------------- sort
def choices(rng, T, K, E, kind="some"):
    if kind == "one":
        return np.full((T, K), E // 2, np.int32)
    e = rng.integers(0, E, (T, K)).astype(np.int32)
    if kind == "skewed":
        e = np.minimum(e, rng.integers(0, E, (T, K)) // 4).astype(np.int32)
    e[rng.random(T) < 0.1] = -1
    return e


SORTS = [(1, 1, 1, 8, "some"), (1, 8, 256, 64, "some"), (3, 2, 5, 2056, "one"), (64, 4, 128, 2880, "some"),
         (257, 4, 8, 512, "skewed"), (511, 8, 60, 136, "some"), (513, 8, 60, 136, "skewed"), (1025, 1, 7, 72, "one"),
         (2000, 6, 256, 264, "skewed"), (70001, 2, 33, 8, "some"), (9000, 32, 200, 16, "skewed"), (700, 16, 8, 40, "one"), (2048, 1, 64, 24, "some"), (2049, 1, 64, 24, "skewed"),
         (1024, 4, 128, 4104, "some"), (128, 32, 256, 72, "skewed"), (300000, 1, 256, 8, "skewed")]


@pytest.mark.parametrize("T,K,E,H,kind", SORTS)
@pytest.mark.parametrize("dtype,group", [(F32, 0), (BF16, 0), (FP8, 0), (FP8, 32), (FP8, 128)])
def test_sort_rows(T, K, E, H, kind, dtype, group):
    rng = np.random.default_rng(T + K)
    n, base, pad = T * K, 3, 8 * (T % 3)
    expert = choices(rng, T, K, E, kind)
    expert = np.where(expert >= 0, expert + base, -1).astype(np.int32)
    x = gpu(rng.standard_normal((T, H)).astype(np.float32), dtype if dtype != FP8 else F32, 0)
    if dtype == FP8:
        full = torch.zeros(T, H + pad, dtype=torch.uint8, device="cuda")
        full[:, :H] = x.to(FP8).view(torch.uint8)
        x = full.view(FP8)[:, :H]
    elif pad:
        full = torch.zeros(T, H + pad, dtype=dtype, device="cuda")
        full[:, :H] = x
        x = full[:, :H]
    groups = -(-H // group) if group else 1
    scale = gpu(rng.uniform(0.01, 0.1, (T, groups)).astype(np.float32)) if dtype == FP8 else None
    out = F32 if dtype == F32 else BF16
    xs = torch.full((n, H + 16), 5, dtype=out, device="cuda")[:, :H]
    perm, pos, slot = (torch.full((n,), -9, dtype=I32, device="cuda") for _ in range(3))
    counts, offsets = torch.full((E,), -9, dtype=I32, device="cuda"), torch.full((E + 1,), -9, dtype=I32, device="cuda")
    ws, err = torch.full((1 << 18,), 77, dtype=torch.uint8, device="cuda"), errword()
    M.moe_sort_rows(gpu(expert), E, x, xs, perm, pos, counts, offsets, err, ws, expert_base=base, row_slot=slot,
                    x_scale=scale, group=group)
    rperm, rpos, rcounts, roffsets, rslot, bad = O.sort_index(expert, E, base)
    assert sync_err(err) == 0 and not bad
    for got, ref, what in ((perm, rperm, "perm"), (pos, rpos, "pos"), (counts, rcounts, "counts"),
                           (offsets, roffsets, "offsets"), (slot, rslot, "row_slot")):
        assert np.array_equal(got.cpu().numpy(), ref), what
    total = int(roffsets[E])
    at = torch.from_numpy(rslot[:total].astype(np.int64)).cuda()
    if dtype == FP8:
        cols = torch.arange(H, device="cuda") // (group or H)
        ref = val(x.view(torch.uint8)[at].view(FP8)) * val(scale[at][:, cols])
        within(val(xs[:total]), ref, np.abs(ref) * (HALF[BF16] + 2 * U))
    else:
        assert torch.equal(xs[:total], x[at])
    assert (xs[total:] == 5).all(), "rows past the last were written"


def test_sort_rows_foreign_experts_and_index_only():
    rng = np.random.default_rng(12)
    for T, K in ((40, 4), (5000, 4)):
        expert = rng.integers(-1, 40, (T, K)).astype(np.int32)
        expert[0, 0], expert[1, 1] = -5, 2 ** 31 - 1
        pos = torch.full((T * K,), -9, dtype=I32, device="cuda")
        counts, offsets = torch.empty(8, dtype=I32, device="cuda"), torch.empty(9, dtype=I32, device="cuda")
        err = errword()
        M.moe_sort_rows(gpu(expert), 8, None, None, None, pos, counts, offsets, err,
                        torch.empty(1 << 18, dtype=torch.uint8, device="cuda"), expert_base=16)
        _, rpos, rcounts, roffsets, _, bad = O.sort_index(expert, 8, 16)
        assert bad and sync_err(err) == M.ERR_EXPERT_NONLOCAL
        assert np.array_equal(pos.cpu().numpy(), rpos) and np.array_equal(offsets.cpu().numpy(), roffsets)
        assert np.array_equal(counts.cpu().numpy(), rcounts)
        # nothing local at all
        M.moe_sort_rows(gpu(np.full((T, K), -1, np.int32)), 8, None, None, None, pos, counts, offsets, err,
                        torch.empty(1 << 18, dtype=torch.uint8, device="cuda"))
        assert (pos == -1).all() and not offsets.any() and not counts.any()


def test_no_tokens():
    err, ws = errword(), torch.empty(1 << 18, dtype=torch.uint8, device="cuda")
    counts, offsets = torch.full((4,), 9, dtype=I32, device="cuda"), torch.full((5,), 9, dtype=I32, device="cuda")
    none = torch.empty(0, dtype=I32, device="cuda")
    x, e = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda")
    w = torch.empty(0, 2, device="cuda")
    M.moe_sort_rows(e, 4, x, x, none, none, counts, offsets, err, ws)
    assert not counts.any() and not offsets.any()
    M.moe_route(torch.empty(0, 4, device="cuda"), e, w)
    M.moe_route_backward(torch.empty(0, 4, device="cuda"), e, w, torch.empty(0, 4, device="cuda"), err)
    M.moe_merge_rows(x, e, w, x, err)
    M.moe_merge_rows_backward(x, x, e, w, x, w, err)
    g = torch.ones(64, dtype=BF16, device="cuda")
    M.moe_residual_norm(x, x, g, 1e-5, x)
    dg = torch.full((64,), 9.0, device="cuda")
    M.moe_residual_norm_backward(x, x, g, torch.empty(0, device="cuda"), x, dg, torch.empty(2048 * 64, dtype=torch.uint8, device="cuda"))
    assert not dg.any() and sync_err(err) == 0


# ------------------------------------------------------------------------------------------ merge
MERGES = [(1, 1, 8), (1, 8, 2880), (3, 32, 64), (64, 4, 2880), (301, 4, 4096), (130, 8, 7168), (2000, 2, 136), (500, 6, 2056),
          (70, 3, 16384 + 8), (5, 5, 65536)]


def merge_case(rng, T, K, H, dtype, pad):
    n = T * K + 3
    pos = rng.permutation(n)[:T * K].reshape(T, K).astype(np.int32)
    pos[rng.random((T, K)) < 0.15] = -1
    pos[rng.random(T) < 0.1] = -1
    rows = rng.standard_normal((n, H)).astype(np.float32)
    named = np.zeros(n, bool)
    named[pos[pos >= 0]] = True
    rows[~named] = np.nan  # nothing may read these
    w = rng.standard_normal((T, K)).astype(np.float32)
    w[pos < 0] = np.nan  # nor these
    return pos, gpu(rows, dtype, pad), w


@pytest.mark.parametrize("T,K,H", MERGES)
@pytest.mark.parametrize("rt,ot", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_merge_rows(T, K, H, rt, ot):
    rng = np.random.default_rng(T * K + H)
    pos, rows, w = merge_case(rng, T, K, H, rt, 8 * (T % 2))
    r = val(rows)
    for weights in (w, None):
        out, err = like((T, H), ot, 24, fill=9), errword()
        M.moe_merge_rows(rows, gpu(pos), None if weights is None else gpu(weights), out, err)
        ref = O.merge_rows(r, pos, weights)
        size = O.merge_rows(np.abs(r), pos, None if weights is None else np.abs(weights))
        assert sync_err(err) == 0
        within(val(out), ref, (K + 1) * U * size + HALF[ot] * np.abs(ref))


@pytest.mark.parametrize("T,K,H", MERGES)
@pytest.mark.parametrize("dt,rt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
def test_merge_rows_backward(T, K, H, dt, rt):
    rng = np.random.default_rng(T * K + H + 1)
    pos, rows, w = merge_case(rng, T, K, H, rt, 8 * (T % 2))
    dout = gpu(rng.standard_normal((T, H)).astype(np.float32), dt, 16)
    r, g = np.nan_to_num(val(rows)), val(dout)
    n = rows.shape[0]
    for weights in (w, None):
        drows, dw, err = like((n, H), rt, 8, fill=9), like((T, K), F32, fill=9), errword()
        M.moe_merge_rows_backward(dout, rows, gpu(pos), None if weights is None else gpu(weights), drows, dw, err)
        assert sync_err(err) == 0
        rd, rw = O.merge_rows_backward(g, r, pos, weights)
        size = O.merge_rows_backward(np.abs(g), np.abs(r), pos)[1]
        within(val(dw), rw, (depth(H) + 1) * U * size, "dw")
        named = np.zeros(n, bool)
        named[pos[pos >= 0]] = True
        within(val(drows)[named], rd[named], (HALF[rt] + U) * np.abs(rd[named]), "drows")
        assert (val(drows)[~named] == 9).all(), "a row that nothing names was written"
        # each output alone gives the same bits
        one, two = like((n, H), rt, 8, fill=9), like((T, K), F32, fill=9)
        M.moe_merge_rows_backward(dout, None, gpu(pos), None if weights is None else gpu(weights), one, None, err)
        M.moe_merge_rows_backward(dout, rows, gpu(pos), None if weights is None else gpu(weights), None, two, err)
        assert torch.equal(one, drows) and torch.equal(two, dw)


def test_merge_rows_refuses_rows_out_of_range():
    rng = np.random.default_rng(3)
    T, K, H, n = 40, 4, 64, 100
    pos = rng.integers(-1, n, (T, K)).astype(np.int32)
    wild = pos.copy()
    wild[3, 1], wild[7, 0], wild[9, 3] = n, -2, 2 ** 31 - 1
    clean = np.where((wild >= 0) & (wild < n), wild, -1)
    rows, w, dout = (gpu(rng.standard_normal(s).astype(np.float32)) for s in ((n, H), (T, K), (T, H)))
    for p, want in ((clean, 0), (wild, M.ERR_ROW_RANGE)):
        out, dw, err, err2 = like((T, H), F32), like((T, K), F32), errword(), errword()
        M.moe_merge_rows(rows, gpu(p), w, out, err)
        M.moe_merge_rows_backward(dout, rows, gpu(p), w, None, dw, err2)
        assert sync_err(err) == want == sync_err(err2)
        if want == 0:
            keep = out.clone(), dw.clone()
    assert torch.equal(out, keep[0]) and torch.equal(dw, keep[1])
    empty = torch.empty(0, H, device="cuda")  # no rows at all
    err = errword()
    M.moe_merge_rows(empty, gpu(np.full((T, K), -1, np.int32)), w, out, err)
    assert sync_err(err) == 0 and not out.any()


# ------------------------------------------------------------------------------------------- norm
NORMS = [(1, 8), (3, 72), (64, 2880), (131, 4096), (40, 2056), (33, 7168), (9, 16384), (700, 520), (17, 12296), (2, 2048)]
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]


def rows_for_norm(rng, T, H):
    x, res = rng.standard_normal((T, H)).astype(np.float32), 3 * rng.standard_normal((T, H)).astype(np.float32)
    for t in range(T):
        if t % 7 == 3:
            x[t] = res[t] = 0
        elif t % 7 == 4:
            x[t] *= 1e-3
            res[t] *= 1e-3
        elif t % 7 == 5:
            x[t], res[t] = x[t] * 1e4, res[t] * 1e4
        elif t % 7 == 6:  # all but a few columns are zero: whole groups of zeros
            x[t, 8:] = res[t, 8:] = 0
    return x, res


def check_norm(out, out_scale, group, y, tol_rel):
    """out against y, off by tol_rel before it is stored."""
    if out.dtype != FP8:
        return within(val(out), y, np.abs(y) * (HALF[out.dtype] + tol_rel) + 1e-37)
    s = O.group_scales(y, group)
    within(val(out_scale), s, s * (tol_rel + 2 * U), "out_scale")
    cols = np.arange(y.shape[1]) // (group or y.shape[1])
    used = val(out_scale)[:, cols]
    within(val(out) * used, y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * used) * (1 + 1e-5) + np.abs(y) * (tol_rel + 4 * U))
    # nothing coarser than the type: the largest of a group of more than rounding noise is at least half range
    peak = np.stack([np.abs(val(out)[:, a:a + (group or y.shape[1])]).max(1) for a in range(0, y.shape[1], group or y.shape[1])], 1)
    big = s > 1e-30
    assert ((peak == 448) | ~big | (np.stack([np.abs(y[:, a:a + (group or y.shape[1])]).max(1) for a in range(0, y.shape[1], group or y.shape[1])], 1) == 0)).all()


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("ot,group", [(F32, 0), (BF16, 0), (FP8, 0), (FP8, 32), (FP8, 64), (FP8, 128)])
def test_residual_norm(T, H, xt, rt, ot, group):
    rng = np.random.default_rng(T + H)
    xn, rn = rows_for_norm(rng, T, H)
    pad = 8 * (T % 3)
    x, res = gpu(xn, xt, pad), gpu(rn, rt, 2 * pad)
    gamma = gpu((1 + 0.2 * rng.standard_normal(H)).astype(np.float32), [F32, BF16][T % 2])
    groups = -(-H // group) if group else 1
    for residual in (res, None):
        out, scale = like((T, H), ot, pad, 1), torch.zeros(T, groups, device="cuda") if ot == FP8 else None
        ro, rstd = like((T, H), rt, pad, 1), torch.zeros(T, device="cuda")
        M.moe_residual_norm(x, residual, gamma, 1e-5, out, residual_out=ro, rstd=rstd, out_scale=scale, group=group)
        y, h, r = O.residual_norm(val(x), None if residual is None else val(residual), val(gamma), 1e-5)
        torch.cuda.synchronize()
        # h: u of |x| + |residual|, at most 1e-7 relative of the row's root mean square in the sum; r half
        # of the sum's d u and 4 more roundings
        rel = (depth(H) / 2 + 10) * U
        within(val(rstd), r, r * rel, "rstd")
        within(val(ro), h, np.abs(h) * (HALF[rt] + U) + U * (np.abs(val(x)) + 0), "residual_out")
        # columns where x and residual nearly cancel carry h's own rounding
        slack = U * (np.abs(val(x)) + (0 if residual is None else np.abs(val(residual)))) * r[:, None] * np.abs(val(gamma))
        if ot == FP8:
            check_norm(out, scale, group, y, rel + 4 * U)
        else:
            within(val(out), y, np.abs(y) * (HALF[ot] + rel + 4 * U) + slack + 1e-37)


def test_residual_norm_in_place_and_listed_rows():
    rng = np.random.default_rng(8)
    T, H = 50, 2880
    x, res, gamma = (gpu(rng.standard_normal(s).astype(np.float32), BF16) for s in ((T, H), (T, H), (H,)))
    out, ro = like((T, H), BF16), like((T, H), BF16)
    M.moe_residual_norm(x, res, gamma, 1e-5, out, residual_out=ro)
    a, b = x.clone(), res.clone()
    M.moe_residual_norm(a, b, gamma, 1e-5, a, residual_out=b)
    assert torch.equal(a, out) and torch.equal(b, ro)
    for count in (0, 1, 20, T, T + 9, -4):
        listed = torch.from_numpy(rng.permutation(T).astype(np.int32)).cuda()
        o, r2, rs, err = like((T, H), FP8, fill=3), like((T, H), BF16, fill=4), torch.full((T,), 5.0, device="cuda"), errword()
        sc = torch.full((T, 90), 6.0, device="cuda")
        M.moe_residual_norm(x, res, gamma, 1e-5, o, residual_out=r2, rstd=rs, out_scale=sc, group=32, row_list=listed,
                            row_count=torch.tensor([count], dtype=I32, device="cuda"), err=err)
        assert sync_err(err) == 0
        there = torch.zeros(T, dtype=torch.bool, device="cuda")
        there[listed[:max(0, min(T, count))].long()] = True
        assert torch.equal(r2[there], ro[there]) and (r2[~there] == 4).all()
        assert (o.view(torch.uint8)[~there] == 3).all() and (rs[~there] == 5).all() and (sc[~there] == 6).all()
        full, fs = like((T, H), FP8), torch.zeros(T, 90, device="cuda")
        M.moe_residual_norm(x, res, gamma, 1e-5, full, out_scale=fs, group=32)
        assert torch.equal(o.view(torch.uint8)[there], full.view(torch.uint8)[there]) and torch.equal(sc[there], fs[there])
    listed = torch.tensor([3, T, -1, 5] + [0] * (T - 4), dtype=I32, device="cuda")
    o, err = like((T, H), BF16, fill=4), errword()
    M.moe_residual_norm(x, res, gamma, 1e-5, o, row_list=listed, row_count=torch.tensor([4], dtype=I32, device="cuda"), err=err)
    assert sync_err(err) == M.ERR_ROW_RANGE and torch.equal(o[3], out[3]) and torch.equal(o[5], out[5]) and (o[4] == 4).all()


def test_residual_norm_not_finite_and_tiny():
    H = 256
    x = torch.ones(6, H, device="cuda")
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 1e-30
    x[4] = 0
    x[4, 40] = 1e-38
    gamma = torch.ones(H, device="cuda")
    gamma[100] = 1e-44  # a denormal
    out, sc = like((6, H), FP8), torch.zeros(6, H // 32, device="cuda")
    M.moe_residual_norm(x, None, gamma, 0.0, out, out_scale=sc, group=32)
    f32 = like((6, H), F32)
    M.moe_residual_norm(x, None, gamma, 1e-12, f32)
    o, s = val(out), val(sc)
    assert np.isnan(o[1]).all() and np.isnan(val(f32[1])).all() and np.isnan(o[2, 7])
    assert np.isfinite(o[0]).all() and (s[0] == np.float32(1 / 448)).all() and np.isfinite(val(f32)[[0, 3, 4, 5]]).all()


@pytest.mark.parametrize("T,H", NORMS + [(1500, 264), (513, 1032), (2049, 8), (1027, 1536)])
@pytest.mark.parametrize("dt,ht", TYPES)
def test_residual_norm_backward(T, H, dt, ht):
    rng = np.random.default_rng(T + H + 5)
    pad = 8 * (T % 3)
    dout = gpu(rng.standard_normal((T, H)).astype(np.float32), dt, pad)
    h = gpu((3 * rng.standard_normal((T, H))).astype(np.float32), ht, pad)
    dres = gpu(rng.standard_normal((T, H)).astype(np.float32), ht, 2 * pad)
    gamma = gpu((1 + 0.2 * rng.standard_normal(H)).astype(np.float32), [F32, BF16][T % 2])
    hv, g, gm = val(h), val(dout), val(gamma)
    rstd = gpu((1 / np.sqrt((hv * hv).mean(1) + 1e-5)).astype(np.float32))
    r = val(rstd)
    ws = torch.full((2048 * H,), 0xff, dtype=torch.uint8, device="cuda")
    for d in (dres, None):
        dx, dr, dgamma = like((T, H), dt, pad), like((T, H), ht, pad), torch.empty(H, device="cuda")
        M.moe_residual_norm_backward(dout, h, gamma, rstd, dx, dgamma, ws, dres=d, dresidual=dr)
        ref, rgamma = O.residual_norm_backward(g, hv, gm, r, None if d is None else val(d))
        xh, gg = hv * r[:, None], g * gm
        mean, size = (gg * xh).mean(1, keepdims=True), np.abs(gg * xh).mean(1, keepdims=True)
        tol = r[:, None] * (6 * U * np.abs(gg) + np.abs(xh) * (6 * U * np.abs(mean) + (depth(H) + 4) * U * size))
        tol = tol + (0 if d is None else U * np.abs(val(d))) + U * np.abs(ref)
        torch.cuda.synchronize()
        within(val(dx), ref, tol + HALF[dt] * np.abs(ref), "dx")
        within(val(dr), ref, tol + HALF[ht] * np.abs(ref), "dresidual")
        # dgamma: runs of at most ceil(T / 256) tokens, then the partial sums in 16 runs of 32 at most
        within(val(dgamma), rgamma, (math.ceil(T / 256) + 60) * U * np.abs(g * xh).sum(0), "dgamma")
        one = torch.empty(H, device="cuda")
        M.moe_residual_norm_backward(dout, h, gamma, rstd, None, one, ws, dres=d)
        a, b = dout.clone(), h.clone()
        M.moe_residual_norm_backward(a, b, gamma, rstd, a, None, None, dres=d, dresidual=b)  # over its own inputs
        assert torch.equal(one, dgamma) and torch.equal(a, dx) and torch.equal(b, dr)


def test_norm_differences():
    """dx and dgamma against differences of moe_residual_norm in fp32: y off by 40 u of its size (about 3)
    in sums over H = 64 of |dout| about 1, over a step of 2^-5: 64 * 3 * 40 * 2^-24 * 2^4 = 7e-3 at most;
    the formula's own error is a third derivative of order 1 times 2^-10 / 6."""
    T, H, step = 4, 64, 2.0 ** -5
    rng = np.random.default_rng(2)
    x, res, gm, dout = (rng.standard_normal(s) for s in ((T, H), (T, H), H, (T, H)))
    gm, dout = np.float32(gm).astype(np.float64), np.float32(dout).astype(np.float64)

    def f(a, b):
        out = like((T, H), F32)
        M.moe_residual_norm(gpu(a, F32), gpu(res, F32), gpu(b, F32), 1e-3, out)
        return val(out) * dout

    h, rstd = like((T, H), F32), torch.empty(T, device="cuda")
    M.moe_residual_norm(gpu(x, F32), gpu(res, F32), gpu(gm, F32), 1e-3, like((T, H), F32), residual_out=h, rstd=rstd)
    dx, dgamma = like((T, H), F32), torch.empty(H, device="cuda")
    M.moe_residual_norm_backward(gpu(dout, F32), h, gpu(gm, F32), rstd, dx, dgamma,
                                 torch.empty(2048 * H, dtype=torch.uint8, device="cuda"))
    for c in range(0, H, 7):
        hi, lo = x.copy(), x.copy()
        hi[:, c] += step
        lo[:, c] -= step
        assert np.abs((f(hi, gm) - f(lo, gm)).sum(1) / (2 * step) - val(dx)[:, c]).max() <= 1e-2
        hi, lo = gm.copy(), gm.copy()
        hi[c] += step
        lo[c] -= step
        assert abs((f(x, hi) - f(x, lo)).sum() / (2 * step) - val(dgamma)[c]) <= 1e-2
