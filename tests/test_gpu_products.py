"""The experts' products on the GPU against the fp64 oracle (oracle/products.py).

Most inputs are small whole numbers: every product and every partial sum of them is below 2^24 in size and so
exact in fp32 in any order, which makes the fp32 outputs equal to the oracle's and the bf16 ones its rounding to
nearest even.  Tolerances of the others, with u = 2^-24 (half a step of fp32, relative) and v = half a step of the
stored type (fp32 u, bf16 2^-8):
  * a sum of D terms s_i in any order takes at most D additions on the way of a term, each off by at most one
    step 2 u (whatever the matrix instruction rounds to inside): 2 u D sum|s_i|;
  * scales: one rounding of their product, one of its product with a block's sum: 2 u more;
  * the stored result v |result|."""
import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M
from gpu_helpers import sync_err
from oracle import products as O
from oracle.moe_oracle import decode_e4m3

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, FP8, I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32
HALF = {F32: U, BF16: 2.0 ** -8}
NAN = float("nan")

# rows of each expert: single rows, empty experts, tiles' sizes and their neighbours, many experts with few rows
ROWS = [[1], [0, 5, 0], [33, 0, 64, 7], [130, 1, 0, 255, 256, 257], [600, 0, 31, 513], [64] * 8, "many"]
SIZES = [(8, 16), (24, 48), (264, 144), (520, 208), (256, 64), (72, 1040), (128, 384)]


def rows_of(which, rng):
    return list(rng.integers(0, 4, 256)) if which == "many" else which


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: I32}[t.element_size()])


def wide(a, dtype, pad, poison=NAN):
    """A numpy array on the GPU in `dtype`, as a view whose rows are pad elements further apart; what lies between
    them is `poison`."""
    t = torch.from_numpy(np.ascontiguousarray(a)).float()
    full = torch.full((*t.shape[:-1], t.shape[-1] + pad), poison, dtype=F32)
    full[..., :t.shape[-1]] = t
    return full.to(dtype).cuda()[..., :t.shape[-1]]


def offsets_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def whole(rng, *shape, most=4):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def rounded(ref, dtype):
    return torch.from_numpy(ref).to(F32).to(dtype)  # exact in fp32, then to nearest even


def same_bits(got, ref, dtype, what):
    want = rounded(ref, dtype)
    got = got.cpu()
    off = (got != want).nonzero()
    assert off.numel() == 0, f"{what}: {off.shape[0]} differ, first {off[0].tolist()}: {got[tuple(off[0])]} for {want[tuple(off[0])]}"


@pytest.mark.parametrize("rows", range(len(ROWS)))
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16->f32", "fp8", "fp8->f32"])
@pytest.mark.parametrize("transposed", [False, True])
def test_matmul_of_whole_numbers(rows, kind, transposed):
    if kind.startswith("fp8") and transposed:
        pytest.skip("8-bit weights have one orientation")
    dtype = {"f": F32, "b": BF16}[kind[0]] if not kind.startswith("fp8") else FP8
    odt = F32 if kind.endswith("f32") else BF16
    rng = np.random.default_rng(rows * 10 + transposed)
    for case, (N, D) in enumerate(SIZES):
        sizes = rows_of(ROWS[rows], rng)
        E, total = len(sizes), int(sum(sizes))
        n, pad = total + (case % 3), 16 * (case % 2)
        print("matmul", kind, transposed, rows, N, D, flush=True)
        offsets = offsets_of(sizes)
        gather = case % 2 == 0
        x_rows = n // 3 + 2 if gather else n
        x, w = whole(rng, x_rows, D), whole(rng, E, *((D, N) if transposed else (N, D)))
        slot = rng.integers(0, x_rows, n).astype(np.int32) if gather else None
        xv, wv, xs, ws = x, w, None, None
        if dtype == FP8:
            kb, nb = -(-D // 128), -(-N // 128)
            xs, ws = 2.0 ** rng.integers(-2, 3, (x_rows, kb)), 2.0 ** rng.integers(-2, 3, (E, nb, kb))
            xv = O.scaled(x, xs, 1)
            wv = np.stack([O.scaled(w[e], ws[e], 128) for e in range(E)])
        if not gather:
            x = x.copy()
            x[total:] = np.nan  # rows behind the last expert's are not read
        ref = O.expert_matmul(xv, wv, offsets, n, slot, transposed)
        out = torch.full((n, N + pad), -7, dtype=odt, device="cuda")[:, :N]
        err = torch.zeros(1, dtype=I32, device="cuda")
        M.moe_expert_matmul(wide(x, dtype, pad), wide(w, dtype, pad), cuda(offsets), out, err,
                            row_slot=None if slot is None else cuda(slot),
                            x_scale=None if xs is None else cuda(xs, F32), w_scale=None if ws is None else cuda(ws, F32),
                            transposed=transposed)
        assert sync_err(err) == 0
        ref[total:] = -7
        same_bits(out, ref, odt, f"N {N} D {D}")


@pytest.mark.parametrize("rows", range(len(ROWS)))
@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16->f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradient_of_whole_numbers(rows, kind, accumulate):
    dtype = F32 if kind == "f32" else BF16
    odt = F32 if kind.endswith("f32") else BF16
    rng = np.random.default_rng(rows * 10 + 5 + accumulate)
    for case, (N, D) in enumerate(SIZES):
        sizes = rows_of(ROWS[rows], rng)
        E, total = len(sizes), int(sum(sizes))
        n, pad = total + (case % 3), 16 * (case % 2)
        print("wgrad", kind, accumulate, rows, N, D, flush=True)
        offsets = offsets_of(sizes)
        dout, x = whole(rng, n, N), whole(rng, n, D)
        ref = O.expert_matmul_backward(dout, x, offsets)
        dout[total:], x[total:] = np.nan, np.inf
        before = whole(rng, E, N, D, most=100)
        dw = wide(before, odt, pad, poison=-7)
        M.moe_expert_matmul_backward(wide(dout, dtype, pad), wide(x, dtype, pad), cuda(offsets), dw, accumulate)
        if accumulate:
            ref = ref + before
        same_bits(dw, ref, odt, f"N {N} D {D}")
        if pad:
            behind = torch.as_strided(dw, (E * N, pad), (D + pad, 1), D)
            assert bool((behind == -7).all())


@pytest.mark.parametrize("kind", ["f32", "bf16", "bf16->f32", "fp8", "fp8->f32"])
@pytest.mark.parametrize("sizes", [[40, 0, 21, 3], [300, 150]])
def test_matmul_of_normal_numbers(kind, sizes):
    dtype = {"f": F32, "b": BF16}[kind[0]] if not kind.startswith("fp8") else FP8
    odt = F32 if kind.endswith("f32") else BF16
    rng = np.random.default_rng(len(kind))
    E, n, N, D, offsets = len(sizes), sum(sizes), 328, 720, offsets_of(sizes)
    x, w = rng.standard_normal((n, D)), rng.standard_normal((E, N, D)) * 0.05
    xs = ws = None
    if dtype == FP8:
        xs, ws = rng.uniform(0.01, 0.1, (n, 6)).astype(np.float32), rng.uniform(0.01, 0.1, (E, 3, 6)).astype(np.float32)
        xt, wt = wide(x * 40, dtype, 0), wide(w * 800, dtype, 0)
        decode = lambda t: decode_e4m3(t.view(torch.uint8).cpu().numpy())  # noqa: E731
        xv = O.scaled(decode(xt), xs, 1)
        wv = np.stack([O.scaled(c, s, 128) for c, s in zip(decode(wt), ws)])
    else:
        xt, wt = wide(x, dtype, 0), wide(w, dtype, 0)
        xv, wv = xt.double().cpu().numpy(), wt.double().cpu().numpy()
    out = torch.empty(n, N, dtype=odt, device="cuda")
    M.moe_expert_matmul(xt, wt, cuda(offsets), out, x_scale=None if xs is None else cuda(xs),
                        w_scale=None if ws is None else cuda(ws))
    ref, size = O.expert_matmul(xv, wv, offsets, n), O.expert_matmul(np.abs(xv), np.abs(wv), offsets, n)
    off = np.abs(out.double().cpu().numpy() - ref) - (2 * U * (D + 3) * size + HALF[odt] * np.abs(ref))
    assert off.max() <= 0
    if dtype == FP8:
        return
    dout = wide(rng.standard_normal((n, N)), dtype, 0)
    dv = dout.double().cpu().numpy()
    dx, dw = torch.empty(n, D, dtype=odt, device="cuda"), torch.empty(E, N, D, dtype=odt, device="cuda")
    M.moe_expert_matmul(dout, wt, cuda(offsets), dx, transposed=True)
    ref, size = O.expert_matmul(dv, wv, offsets, n, transposed=True), O.expert_matmul(np.abs(dv), np.abs(wv), offsets, n, transposed=True)
    assert (np.abs(dx.double().cpu().numpy() - ref) - (2 * U * N * size + HALF[odt] * np.abs(ref))).max() <= 0
    M.moe_expert_matmul_backward(dout, xt, cuda(offsets), dw)
    ref, size = O.expert_matmul_backward(dv, xv, offsets), O.expert_matmul_backward(np.abs(dv), np.abs(xv), offsets)
    assert (np.abs(dw.double().cpu().numpy() - ref) - (2 * U * max(sizes) * size + HALF[odt] * np.abs(ref))).max() <= 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("rows", [20, 90, 300])
def test_what_is_not_finite_stays_in_its_row(kind, rows):
    dtype = dict(f32=F32, bf16=BF16, fp8=FP8)[kind]
    odt = F32
    rng = np.random.default_rng(rows)
    sizes = [rows, rows // 2, rows + 3]
    E, n, N, D = 3, sum(sizes), 136, 176
    offsets = offsets_of(sizes)
    x, w = whole(rng, n, D), whole(rng, E, N, D)
    bad = [1, rows - 1, rows, n - 1]
    x[bad, [0, D - 1, 7, 100]] = np.nan
    w[1, 5, 3] = np.nan
    if dtype != FP8:
        x[bad[2], 7] = np.inf
    ones = dict(x_scale=torch.ones(n, 2, device="cuda"), w_scale=torch.ones(E, 2, 2, device="cuda")) if dtype == FP8 else {}
    out = torch.empty(n, N, dtype=odt, device="cuda")
    M.moe_expert_matmul(wide(x, dtype, 16), wide(w, dtype, 16), cuda(offsets), out, **ones)
    with np.errstate(invalid="ignore"):
        ref = O.expert_matmul(x, w, offsets, n)
    got = out.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    assert np.isnan(ref).sum() < 5 * N + rows
    if dtype == FP8:
        return
    dout = whole(rng, n, N)
    dout[n - 1, 9] = np.inf
    dw = torch.empty(E, N, D, dtype=odt, device="cuda")
    M.moe_expert_matmul_backward(wide(dout, dtype, 16), wide(x, dtype, 16), cuda(offsets), dw)
    with np.errstate(invalid="ignore"):
        ref = O.expert_matmul_backward(dout, x, offsets)
    got = dw.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("rows", [9, 200])
def test_slots_out_of_range(kind, rows):
    dtype = dict(f32=F32, bf16=BF16, fp8=FP8)[kind]
    rng = np.random.default_rng(rows)
    x_rows, n, N, D = 50, 2 * rows, 40, 80
    offsets = offsets_of([rows, rows])
    x, w = whole(rng, x_rows, D), whole(rng, 2, N, D)
    slot = rng.integers(0, x_rows, n).astype(np.int32)
    slot[[2, rows + 1, n - 1]] = [-1, x_rows, 2 ** 31 - 1]
    ones = dict(x_scale=torch.full((x_rows, 1), 2.0, device="cuda"), w_scale=torch.ones(2, 1, 1, device="cuda")) if dtype == FP8 else {}
    out, err = torch.empty(n, N, dtype=F32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    M.moe_expert_matmul(wide(x, dtype, 0), wide(w, dtype, 0), cuda(offsets), out, err, row_slot=cuda(slot), **ones)
    assert sync_err(err) == M.ERR_SLOT_RANGE
    same_bits(out, O.expert_matmul(x * (2 if dtype == FP8 else 1), w, offsets, n, slot), F32, kind)


def test_offsets_that_are_not_ascending_are_cut():
    rng = np.random.default_rng(0)
    for offsets in ([0, 40, 20, 90], [-5, 30, 1000, 70], [50, 50, 50, 10], [0, 0, 0, 0]):
        n, N, D = 70, 64, 64
        x, w, dout = whole(rng, n, D), whole(rng, 3, N, D), whole(rng, n, N)
        offs = np.array(offsets, np.int32)
        for dtype in (F32, BF16):
            out, dw = torch.full((n, N), 5.0, device="cuda"), torch.empty(3, N, D, device="cuda")
            M.moe_expert_matmul(wide(x, dtype, 0), wide(w, dtype, 0), cuda(offs), out)
            # where spans overlap, each element of a row is that of one of its experts
            got, owners = out.cpu().numpy(), [[] for _ in range(n)]
            for e, (a, b) in enumerate(O.spans(offs, n)):
                for r in range(a, b):
                    owners[r].append(e)
            for r in range(n):
                each = np.stack([w[e] @ x[r] for e in owners[r]]) if owners[r] else np.full((1, N), 5.0)
                assert (got[r] == each).any(0).all()
            M.moe_expert_matmul_backward(wide(dout, dtype, 0), wide(x, dtype, 0), cuda(offs), dw)
            same_bits(dw, O.expert_matmul_backward(dout, x, offs), F32, str(offsets))


def test_strided_weights_and_matrices():
    """The up half of gate/up weights, and gradients written into halves."""
    rng = np.random.default_rng(3)
    sizes, N, D = [30, 5, 140], 48, 96
    n, offsets = sum(sizes), offsets_of(sizes)
    x, both, dout = whole(rng, n, D), whole(rng, 3, 2 * N, D), whole(rng, n, N)
    w = cuda(both, BF16)[:, N:]
    out = torch.empty(n, N, device="cuda")
    M.moe_expert_matmul(cuda(x, BF16), w, cuda(offsets), out)
    same_bits(out, O.expert_matmul(x, both[:, N:], offsets, n), F32, "half")
    dx = torch.empty(n, D, device="cuda")
    M.moe_expert_matmul(cuda(dout, BF16), w, cuda(offsets), dx, transposed=True)
    same_bits(dx, O.expert_matmul(dout, both[:, N:], offsets, n, transposed=True), F32, "half transposed")
    dw = torch.zeros(3, 2 * N, D, device="cuda")
    M.moe_expert_matmul_backward(cuda(dout, BF16), cuda(x, BF16), cuda(offsets), dw[:, N:])
    same_bits(dw[:, N:], O.expert_matmul_backward(dout, x, offsets), F32, "half gradient")
    assert not dw[:, :N].any()


def test_no_rows():
    w, offsets = torch.ones(2, 8, 16, device="cuda"), torch.zeros(3, dtype=I32, device="cuda")
    M.moe_expert_matmul(torch.empty(0, 16, device="cuda"), w, offsets, torch.empty(0, 8, device="cuda"))
    dw = torch.full((2, 8, 16), 3.0, device="cuda")
    M.moe_expert_matmul_backward(torch.empty(0, 8, device="cuda"), torch.empty(0, 16, device="cuda"), offsets, dw, True)
    assert bool((dw == 3).all())
    M.moe_expert_matmul_backward(torch.empty(0, 8, device="cuda"), torch.empty(0, 16, device="cuda"), offsets, dw)
    assert not dw.any()
    count = torch.zeros(1, dtype=I32, device="cuda")
    h = torch.full((5, 8), 2.0, device="cuda")
    M.moe_swiglu(torch.ones(5, 16, device="cuda"), h, count=count)
    count.fill_(-3)
    M.moe_swiglu(torch.ones(5, 16, device="cuda"), h, count=count)
    assert bool((h == 2).all())


def hard_gates(rng, n, I):
    gu = rng.standard_normal((n, 2 * I)) * 2
    gu[0] = 0
    if n > 2:
        gu[1, :I] *= 20
        gu[2, :I] = rng.choice([-88.0, -104.0, 100.0, 1e-30, -1e-30], I)
    return gu


@pytest.mark.parametrize("I", [8, 40, 128, 136, 1032, 2880, 4104, 32768])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("out", [(F32, 0), (BF16, 0), (FP8, 0), (FP8, 32), (FP8, 64), (FP8, 128)])
def test_swiglu(I, dtype, out):
    """s takes 4 u (its exponential 3, a quotient), its product with g and u two more roundings; a scale two more.
    s itself is 0 where it lies below the normal fp32 numbers (g below -87.3): it is off by up to 2^-126 there and h
    by |g u| times as much, and h's own subnormal values by 2^-126."""
    odt, group = out
    rng = np.random.default_rng(I)
    n, there = 9, 7
    gu = wide(hard_gates(rng, n, I), dtype, 8)
    val = gu.double().cpu().numpy()
    ref = O.swiglu(val)
    count = torch.tensor([there], dtype=I32, device="cuda")
    groups = -(-I // group) if group else 1
    scale = torch.full((n, groups), 5.0, device="cuda") if odt == FP8 else None
    kind = torch.uint8 if odt == FP8 else odt
    h = torch.full((n, I + 8), 3, dtype=kind, device="cuda").view(odt)[:, :I]
    M.moe_swiglu(gu, h, scale, group, count=count)
    room = 8 * U * np.abs(ref) + 2.0 ** -126 * (1 + np.abs(val[:, :I] * val[:, I:]))
    if odt != FP8:
        got = h.double().cpu().numpy()
        assert (np.abs(got - ref) - room - HALF[odt] * np.abs(ref))[:there].max() <= 0
        assert (got[there:] == 3).all()
        return
    got = decode_e4m3(h.view(torch.uint8).cpu().numpy())
    sc = scale.cpu().numpy().astype(np.float64)
    assert (sc[there:] == 5).all() and bool((h.view(torch.uint8)[there:] == 3).all())
    g = group or I
    amax = np.stack([np.abs(ref[:, a:a + g]).max(1) for a in range(0, I, g)], 1)
    rs = np.where(amax > 0, np.maximum(amax / 448, 2.0 ** -126), 1.0)
    tiny = amax < 2.0 ** -100
    assert (np.abs(sc - rs) <= 12 * U * rs + 2.0 ** -120)[:there][~tiny[:there]].all()
    cols = np.arange(I) // g
    each, wide_ = sc[:, cols], np.broadcast_to(rs[:, cols], ref.shape)
    off = np.abs(got * each - ref) - room - 20 * U * np.abs(ref) - np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * wide_) * (1 + 32 * U)
    assert off[:there][~tiny[:, cols][:there]].max(initial=-1) <= 0
    top = np.abs(got).reshape(n, I)[:there]
    assert (top <= 448).all()


@pytest.mark.parametrize("I", [8, 40, 1032, 2880, 32768])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("inplace", [False, True])
def test_swiglu_backward(I, dtype, inplace):
    """dg = dh u s (1 + g (1 - s)): s 4 u, 1 - s 4 u of s and its own rounding, g (1 - s) and the sum two more, three
    products: 16 u of |dh u s| (1 + |g|) in all; du and h 8 u of themselves."""
    rng = np.random.default_rng(I + 1)
    n, there = 9, 7
    gu = wide(hard_gates(rng, n, I), dtype, 8)
    dh = wide(rng.standard_normal((n, I)), dtype, 16)
    val, dv = gu.double().cpu().numpy(), dh.double().cpu().numpy()
    g, u = val[:, :I], val[:, I:]
    ref, s = O.swiglu_backward(val, dv), O.sigmoid(g)
    count = torch.tensor([there], dtype=I32, device="cuda")
    dgu = gu if inplace else torch.full((n, 2 * I + 8), 3, dtype=dtype, device="cuda")[:, :2 * I]
    before = dgu[there:].clone()
    h = torch.full((n, I), 3, dtype=dtype, device="cuda")
    M.moe_swiglu_backward(gu, dh, dgu, h=h, count=count)
    got, gh = dgu.double().cpu().numpy(), h.double().cpu().numpy()
    v = HALF[dtype]
    floor = 2.0 ** -120 * (1 + np.abs(dv)) * (1 + np.abs(u)) * (1 + np.abs(g))
    room = np.concatenate([16 * U * np.abs(dv * u * s) * (1 + np.abs(g)) + floor, 8 * U * np.abs(ref[:, I:]) + floor], 1)
    assert (np.abs(got - ref) - room - v * np.abs(ref))[:there].max() <= 0
    rh = O.swiglu(val)
    assert (np.abs(gh - rh) - 8 * U * np.abs(rh) - floor - v * np.abs(rh))[:there].max() <= 0
    assert torch.equal(bits(dgu[there:]), bits(before)) and (gh[there:] == 3).all()


def test_swiglu_of_what_is_not_finite():
    I = 32
    gu = torch.ones(4, 2 * I, device="cuda")
    gu[0, 3], gu[1, 4], gu[2, I + 5], gu[3, 6] = NAN, float("inf"), float("inf"), -float("inf")
    h = torch.empty(4, I, device="cuda")
    M.moe_swiglu(gu, h)
    ordinary = h[0, 0].item()
    assert torch.isnan(h[0, 3]) and h[1, 4] == float("inf") and h[2, 5] == float("inf") and torch.isnan(h[3, 6])
    assert int((h == ordinary).sum()) == 4 * I - 4
    codes, scale = torch.empty(4, I, dtype=torch.uint8, device="cuda"), torch.empty(4, 1, device="cuda")
    for group in (0, 32):
        M.moe_swiglu(gu, codes, scale, group)
        c = decode_e4m3(codes.cpu().numpy())
        assert np.isnan(c[0, 3]) and np.isfinite(np.delete(c[0], 3)).all() and np.isnan(c[1]).all() and np.isnan(c[2]).all()


@pytest.mark.parametrize("E,N,D", [(1, 8, 8), (3, 128, 256), (2, 200, 136), (5, 264, 72)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_weights(E, N, D, dtype, transposed):
    """A scale takes one rounding, a code two: 2^-4 of the value and 2^-10 of the scale below the normal codes."""
    rng = np.random.default_rng(N)
    w = rng.standard_normal((E, N, D)) * 0.02
    w[0, 0] = 0
    if N > 128:
        w[-1, 128:] = 0
    t = wide(w, dtype, 16)
    v = t.double().cpu().numpy()
    if transposed:
        v = v.transpose(0, 2, 1)
    R, C = v.shape[1:]
    codes = torch.full((E, R, C + 16), 9, dtype=torch.uint8, device="cuda")
    scale = torch.empty(E, -(-R // 128), -(-C // 128), device="cuda")
    M.moe_quantize_weights(t, codes[:, :, :C], scale, transposed)
    rs = np.stack([O.block_scales(m) for m in v])
    assert (np.abs(scale.cpu().numpy() - rs) <= 2 * U * rs).all()
    assert bool((codes[:, :, C:] == 9).all())
    got = decode_e4m3(codes[:, :, :C].cpu().numpy())
    for e in range(E):
        back = O.scaled(got[e], scale[e].cpu().numpy(), 128)
        each = O.scaled(np.ones((R, C)), rs[e], 128)
        assert (np.abs(back - v[e]) <= np.maximum(2.0 ** -4 * np.abs(v[e]), 2.0 ** -10 * each) * (1 + 16 * U)).all()
    first = codes.clone()
    M.moe_quantize_weights(t, codes[:, :, :C].view(FP8), scale, transposed)
    assert torch.equal(first, codes)
