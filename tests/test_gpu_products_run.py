"""The experts' products at larger sizes and run together: every shape of workgroup, offsets past 32 bits, large
gradients, the whole layer against fp64 with its gradients, in 8 bits, captured, on other streams.

The references are fp64, a matrix product per expert.  Whole numbers of at most 4 in size make fp32 sums exact (up to
16 * 65536 < 2^24), as do the powers of two of the scales."""
import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M
from gpu_helpers import decode_tensor

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, FP8, I32, F64 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float64


def whole(gen, *shape, most=4):
    return torch.randint(-most, most + 1, shape, generator=gen, device="cuda").float()


def seeded(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets_of(sizes):
    return torch.tensor([0, *np.cumsum(sizes)], dtype=I32, device="cuda")


def each(sizes):
    at = np.concatenate([[0], np.cumsum(sizes)])
    return [(e, int(a), int(b)) for e, (a, b) in enumerate(zip(at, at[1:]))]


def same(got, ref, what):
    off = (got != ref.float().to(got.dtype)).nonzero()
    assert off.shape[0] == 0, f"{what}: {off.shape[0]} differ, first {off[0].tolist()}"


# With few rows: 32 columns and k in four parts, 128, 192 or 256 columns to a workgroup, two workgroups to a CU; an
# expert among them with several tiles of rows.  With more: each height of a tile, more than eight tiles of an expert,
# experts by the hundred; one to five steps along k.
FEW = [([3], 4096, 4096), ([1, 0, 2], 1032, 80), ([40] * 7 + [130], 4096, 208), ([32] * 8, 5760, 2880),
       ([64, 0, 65, 63] * 2, 8192, 144), ([17] * 30 + [300, 0], 4096, 272), ([2] * 100, 136, 64)]
MANY = [([70, 129, 200, 256, 300], 4104, 208), ([2300, 1, 0, 513], 520, 1040), ([100] * 130, 264, 64),
        ([8, 500, 1200], 264, 128), ([640, 65] * 3, 4096, 144), ([5000], 272, 320)]


@pytest.mark.parametrize("case", range(len(FEW) + len(MANY)))
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_every_shape_of_workgroup(case, kind):
    sizes, N, D = (FEW + MANY)[case]
    dtype = {"f32": F32, "bf16": BF16, "fp8": FP8}[kind]
    g, n, E, offsets = seeded(case), sum(sizes), len(sizes), offsets_of(sizes)
    print("products", kind, sizes[:4], E, N, D, flush=True)
    tokens = max(n // 2, 1)
    x, w = whole(g, tokens, D), whole(g, E, N, D)
    slot = torch.randint(0, tokens, (n,), generator=g, device="cuda", dtype=I32)
    xs = ws = None
    xv, wv = x, w
    if kind == "fp8":
        kb, nb = -(-D // 128), -(-N // 128)
        xs = 2.0 ** torch.randint(-1, 2, (tokens, kb), generator=g, device="cuda").float()
        ws = 2.0 ** torch.randint(-1, 2, (E, nb, kb), generator=g, device="cuda").float()
        xv = x * xs.repeat_interleave(128, 1)[:, :D]
        wv = w * ws.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :D]
    out = torch.full((n, N), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=I32, device="cuda")
    M.moe_expert_matmul(x.to(dtype), w.to(dtype), offsets, out, err, row_slot=slot, x_scale=xs, w_scale=ws)
    ref = torch.cat([xv[slot[a:b].long()].double() @ wv[e].double().t() for e, a, b in each(sizes)])
    same(out, ref, "forward")
    assert not int(err.item())
    if kind == "fp8":
        return
    dout, xr = whole(g, n, N), whole(g, n, D)
    dx = torch.full((n, D), float("nan"), device="cuda")
    M.moe_expert_matmul(dout.to(dtype), w.to(dtype), offsets, dx, transposed=True)
    same(dx, torch.cat([dout[a:b].double() @ w[e].double() for e, a, b in each(sizes)]), "rows' gradient")
    dw = torch.full((E, N, D), float("nan"), device="cuda")
    M.moe_expert_matmul_backward(dout.to(dtype), xr.to(dtype), offsets, dw)
    for e, a, b in each(sizes):
        same(dw[e], dout[a:b].double().t() @ xr[a:b].double(), f"weights' gradient of {e}")


@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("accumulate", [False, True])
def test_large_gradients(odt, accumulate):
    """More than 96 MiB of them."""
    sizes, N, D = [300, 0, 1, 64, 700, 90, 33], 4104, 2064 if odt == F32 else 4112
    g, n, E = seeded(3), sum(sizes), len(sizes)
    assert E * N * D * odt.itemsize > 96 << 20
    print("large gradients", odt, accumulate, flush=True)
    dout, x, dw = whole(g, n, N), whole(g, n, D), whole(g, E, N, D, most=100).to(odt)
    before = dw.clone()
    M.moe_expert_matmul_backward(dout.to(BF16), x.to(BF16), offsets_of(sizes), dw, accumulate)
    for e, a, b in each(sizes):
        ref = dout[a:b].double().t() @ x[a:b].double()
        same(dw[e], ref + before[e].double() if accumulate else ref, f"of {e}")


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("sizes", [[20, 0, 12], [200, 90, 0]])
def test_offsets_past_32_bits(kind, sizes):
    """Rows of the largest pitch, matrices more than 2^32 bytes apart."""
    dtype = {"f32": F32, "bf16": BF16, "fp8": FP8}[kind]
    es, E, N, D, n = dtype.itemsize, len(sizes), 264, 400, sum(sizes)
    g, pitch, offsets = seeded(9), (16 << 20) // dtype.itemsize, offsets_of(sizes)
    print("far apart", kind, sizes, flush=True)
    stride = (N - 1) * pitch + D + 16
    assert (E - 1) * stride * es > 1 << 32 and 310 * (16 << 20) > 1 << 32
    def far(rows, cols, dt):
        p = (16 << 20) // dt.itemsize
        t = torch.empty(rows * p, dtype=dt, device="cuda")
        return t, torch.as_strided(t, (rows, cols), (p, 1))
    x0, w0 = whole(g, 310, D), whole(g, E, N, D)
    _, x = far(310, D, dtype)
    x.copy_(x0.to(dtype))
    ws = torch.empty((E - 1) * stride + N * pitch, dtype=dtype, device="cuda")
    w = torch.as_strided(ws, (E, N, D), (stride, pitch, 1))
    w.copy_(w0.to(dtype))
    slot = 309 - torch.arange(n, dtype=I32, device="cuda")
    one = dict(x_scale=torch.ones(310, 4, device="cuda"), w_scale=torch.ones(E, 3, 4, device="cuda")) if kind == "fp8" else {}
    _, out = far(n, N, F32)
    err = torch.zeros(1, dtype=I32, device="cuda")
    M.moe_expert_matmul(x, w, offsets, out, err, row_slot=slot, **one)
    ref = torch.cat([x0[slot[a:b].long()].double() @ w0[e].double().t() for e, a, b in each(sizes)])
    same(out, ref, "forward")
    if kind == "fp8":
        return
    _, dout = far(n, N, dtype)
    d0 = whole(g, n, N)
    dout.copy_(d0.to(dtype))
    dx = torch.empty(n, D, device="cuda")
    M.moe_expert_matmul(dout, w, offsets, dx, transposed=True)
    same(dx, torch.cat([d0[a:b].double() @ w0[e].double() for e, a, b in each(sizes)]), "rows' gradient")
    M.moe_expert_matmul_backward(dout, x[:n], offsets, w)  # the gradient lies where the weights did
    for e, a, b in each(sizes):
        same(w[e], d0[a:b].double().t() @ x0[a:b].double(), f"weights' gradient of {e}")


def _layer(T, E, K, H, I, dtype, seed, skew=0.0):
    g = seeded(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    i = dict(x=rand(T, H).to(dtype), w_gu=(rand(E, 2 * I, H) * H ** -0.5).to(dtype),
             w_d=(rand(E, H, I) * I ** -0.5).to(dtype), dout=rand(T, H).to(dtype),
             logits=(rand(T, E) - skew * torch.arange(E, device="cuda")).clamp(-4, 4))
    o = {k: torch.empty_like(i[v]) for k, v in dict(out="x", dx="x", dlogits="logits", dw_gu="w_gu", dw_d="w_d").items()}
    code = M.MOE_F32 if dtype == F32 else M.MOE_BF16
    layer = M.ExpertTrainLayer(E, H, I, K, code, T)

    def step(stream=None):
        layer.run(i["x"], i["logits"], i["w_gu"], i["w_d"], o["out"], train=True, stream=stream)
        layer.backward(i["dout"], o["dx"], o["dlogits"], o["dw_gu"], o["dw_d"], stream=stream)

    return layer, i, o, step


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,K,H,I", [(1, 4, 2, 64, 32), (37, 6, 3, 72, 40), (700, 3, 2, 136, 264), (260, 40, 4, 64, 48)])
def test_layer_and_gradients(dtype, T, E, K, H, I):
    """Against fp64 autograd with the layer's choice of experts.  The tolerances follow the errors through the
    formulas, to first order in u = 2^-24 and v (half a step of the stored type), doubled for the rest: a sum of D
    terms is off by 2 u D sum|terms|, a stored value by v |value|; |silu'| <= 1.1, |silu''| <= 0.5, |silu(z)| <=
    |z|; silu, its derivative and their products are off by less than 32 u of the products' size; a weight of the
    gate, for |logits| <= 4, by at most 64 u of itself (differences of logits up to 8 are off by 8 u, exp by as much
    and its own 2 u, the sum of K and the quotient by K + 2 more, twice over)."""
    v = U if dtype == F32 else 2.0 ** -8
    layer, i, o, step = _layer(T, E, K, H, I, dtype, T + E)
    print("layer", dtype, T, E, K, H, I, flush=True)
    layer.run(i["x"], i["logits"], i["w_gu"], i["w_d"], o["out"])  # without train: gathers its rows
    first = o["out"].clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(first, o["out"]) and not int(layer.err.item())
    expert = layer.expert.long().cpu()
    a = {k: t.double().cpu() for k, t in i.items()}
    x, wgu, wd, l = (a[k].requires_grad_() for k in ("x", "w_gu", "w_d", "logits"))
    gate = torch.softmax(l.gather(1, expert), 1)
    out = torch.zeros(T, H, dtype=F64)
    e_out, e_dx, s_dx = (torch.zeros(T, H, dtype=F64) for _ in range(3))
    e_dgate, s_dgate = torch.zeros(T, K, dtype=F64), torch.zeros(T, K, dtype=F64)
    e_gu, e_d = torch.zeros_like(wgu), torch.zeros_like(wd)
    dout, w_ = a["dout"], gate.detach()
    for e in range(E):
        t, k = (expert == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        gu = x[t] @ wgu[e].t()
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        y = h @ wd[e].t()
        out = out.index_add(0, t, gate[t, k][:, None] * y)
        with torch.no_grad():
            n, Wg, Wd, X = t.numel(), wgu[e].abs(), wd[e].abs(), x[t].abs()
            G, Up, Hh, Y = gu[:, :I].abs(), gu[:, I:].abs(), h.abs(), y.abs()
            d_gu = 2 * U * H * (X @ Wg.t()) + v * gu.abs()
            dg, du = d_gu[:, :I], d_gu[:, I:]
            d_h = 1.1 * dg * Up + G * du + 32 * U * G * Up + v * Hh
            d_y = d_h @ Wd.t() + 2 * U * I * (Hh @ Wd.t()) + v * Y
            gk = w_[t, k][:, None]
            e_out.index_add_(0, t, gk * (d_y + (64 + 2 * K) * U * Y))
            # backward
            dy = (gk * dout[t])
            e_dy = (64 * U + 2 * U + v) * dy.abs()
            e_dgate[t, k] = (dout[t].abs() * (d_y + 2 * U * H * Y)).sum(1)
            s_dgate[t, k] = (dout[t].abs() * Y).sum(1)
            dh, s = dy @ wd[e], torch.sigmoid(gu[:, :I])
            e_dh = e_dy @ Wd + 2 * U * H * (dy.abs() @ Wd) + v * dh.abs()
            D = dh.abs()
            d1 = dh * gu[:, I:] * s * (1 + gu[:, :I] * (1 - s))
            d2 = dh * gu[:, :I] * s
            e_1 = 1.1 * e_dh * Up + D * (1.1 * du + 0.5 * Up * dg + 32 * U * Up * (1 + G)) + v * d1.abs()
            e_2 = e_dh * G + D * (1.1 * dg + 32 * U * G) + v * d2.abs()
            dgu, e_dgu = torch.cat([d1, d2], 1).abs(), torch.cat([e_1, e_2], 1)
            e_gu[e] = e_dgu.t() @ X + 2 * U * n * (dgu.t() @ X)
            e_d[e] = e_dy.t() @ Hh + dy.abs().t() @ d_h + 2 * U * n * (dy.abs().t() @ Hh)
            dxs = torch.cat([d1, d2], 1) @ wgu[e]
            e_dx.index_add_(0, t, e_dgu @ Wg + 4 * U * I * (dgu @ Wg) + v * dxs.abs())
            s_dx.index_add_(0, t, dxs.abs())
    out.backward(dout)
    mean, size = (w_ * e_dgate).sum(1, keepdim=True), (w_ * s_dgate).sum(1, keepdim=True)
    e_l = torch.zeros(T, E, dtype=F64).scatter_(1, expert, w_ * (e_dgate + mean) + w_ * 200 * U * (s_dgate + size))

    def check(name, ref, off, half=v):
        ref = ref.detach()
        far = (o[name].double().cpu() - ref).abs() - (2 * off + half * ref.abs())
        assert float(far.max()) <= 0, (name, float(far.max()), float((2 * off).max()))

    check("out", out, e_out)
    check("dx", x.grad, e_dx + 2 * U * K * s_dx)
    check("dw_gu", wgu.grad, e_gu)
    check("dw_d", wd.grad, e_d)
    check("dlogits", l.grad, e_l, U)


def test_gradients_against_differences():
    """fp32: the derivative of <out, dout> along a direction of each input, from the layer's own outputs at x +- s d.
    With s = 2^-6 the differences' third-order term is below 2^-12 of the terms' size times |d|^3 here, and the
    outputs' rounding, 2^-20 of the sum of absolute terms over 2 s, is below that."""
    layer, i, o, step = _layer(24, 4, 4, 64, 32, F32, 11)  # all experts are chosen: a step changes no choice
    step()
    g = seeded(12)
    grads = {k: o[v].clone() for k, v in dict(x="dx", logits="dlogits", w_gu="dw_gu", w_d="dw_d").items()}
    s = 2.0 ** -6
    for name, grad in grads.items():
        d = torch.randn(i[name].shape, generator=g, device="cuda")
        d /= d.norm()
        at = i[name].clone()
        value = []
        for sign in (s, -s):
            i[name].copy_(at + sign * d)
            layer.run(i["x"], i["logits"], i["w_gu"], i["w_d"], o["out"], train=True)
            value.append((o["out"].double() * i["dout"].double()).sum())
        i[name].copy_(at)
        terms = float((o["out"].double() * i["dout"].double()).abs().sum())
        got, want = float((value[0] - value[1]) / (2 * s)), float((grad.double() * d.double()).sum())
        assert abs(got - want) <= 2.0 ** -12 * terms + 2.0 ** -20 * terms / s, (name, got, want)


def test_layer_in_8_bits():
    """Through moe_residual_norm's 8-bit rows and moe_quantize_weights; each stage against fp64 from the stage before
    it as stored.  A code is off by half a step, 2^-4 of its value, or 2^-10 of its scale where that is larger."""
    T, E, K, H, I = 150, 5, 2, 272, 160
    g = seeded(4)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    hidden, w_gu, w_d = rand(T, H).to(BF16), (rand(E, 2 * I, H) * 0.06).to(BF16), (rand(E, H, I) * 0.08).to(BF16)
    x, xs = torch.empty(T, H, dtype=FP8, device="cuda"), torch.empty(T, 3, device="cuda")
    M.moe_residual_norm(hidden, None, torch.ones(H, dtype=BF16, device="cuda"), 1e-5, x, out_scale=xs, group=128)
    q = [torch.empty(w.shape, dtype=FP8, device="cuda") for w in (w_gu, w_d)]
    sc = [torch.empty(E, 3, 3, device="cuda"), torch.empty(E, 3, 2, device="cuda")]
    for w, c, s in zip((w_gu, w_d), q, sc):
        M.moe_quantize_weights(w, c, s)
    layer = M.ExpertTrainLayer(E, H, I, K, M.MOE_FP8_E4M3, T)
    out = torch.empty(T, H, dtype=BF16, device="cuda")
    layer.run(x, rand(T, E), q[0], q[1], out, x_scale=xs, s_gu=sc[0], s_d=sc[1])
    torch.cuda.synchronize()
    assert not int(layer.err.item())

    def plain(codes, scale, rows):
        v = codes.view(FP8).double().cpu()
        s = scale.double().cpu()
        return v * s.repeat_interleave(rows, -2)[..., :v.shape[-2], :].repeat_interleave(128, -1)[..., :v.shape[-1]]

    wv = [plain(c, s, 128) for c, s in zip(q, sc)]
    xv, hv = plain(x, xs, 1), plain(layer.h, layer.h_scale, 1)
    pos, expert, at = layer.pos.cpu().long().view(T, K), layer.expert.cpu().long(), layer.offsets.cpu().tolist()
    gu, y = layer.gu.double().cpu(), layer.y.double().cpu()
    token = torch.empty(T * K, dtype=torch.long)
    token[pos.flatten()] = torch.arange(T).repeat_interleave(K)
    bf = 2.0 ** -8
    for e in range(E):
        a, b = at[e], at[e + 1]
        assert bool((expert.flatten()[torch.argsort(pos.flatten())][a:b] == e).all())
        r = xv[token[a:b]]
        ref, size = r @ wv[0][e].t(), r.abs() @ wv[0][e].abs().t()
        assert float(((gu[a:b] - ref).abs() - 2 * U * (H + 3) * size - bf * ref.abs()).max()) <= 0
        ref, size = hv[a:b] @ wv[1][e].t(), hv[a:b].abs() @ wv[1][e].abs().t()
        assert float(((y[a:b] - ref).abs() - 2 * U * (I + 3) * size - bf * ref.abs()).max()) <= 0
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    step = layer.h_scale.double().cpu().repeat_interleave(128, 1)[:, :I]
    room = 2.0 ** -4 * h.abs() * (1 + 64 * U) + 2.0 ** -10 * step + 64 * U * (gu[:, :I] * gu[:, I:]).abs()
    assert float(((hv - h).abs() - room).max()) <= 0
    wgt = layer.w.double().cpu()
    ref, size = (wgt[:, :, None] * y[pos]).sum(1), (wgt[:, :, None] * y[pos]).abs().sum(1)
    assert float(((out.double().cpu() - ref).abs() - 2 * U * (K + 1) * size - bf * ref.abs()).max()) <= 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", [(30, 24), (1200, 6)])
def test_captured_step(dtype, T, E):
    """Forward and backward captured once; each replay against the eager step, with other inputs."""
    print("captured", dtype, T, E, flush=True)
    layer, i, o, step = _layer(T, E, 3, 136, 72, dtype, 1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6, 7):
        g = seeded(seed)
        for k in ("x", "logits", "dout"):
            i[k].copy_(torch.randn(i[k].shape, generator=g, device="cuda"))
        for t in o.values():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in o.items()}
        for t in o.values():
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        for k in o:
            assert not bool(got[k].isnan().any()) and torch.equal(got[k], o[k]), (seed, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_two_streams(dtype):
    """Steps on two streams at once, each with its own layer, give the bits of the steps one after another."""
    sets = [_layer(T, E, 2, 264, 136, dtype, T) for T, E in ((900, 4), (60, 30))]
    alone = []
    for _, _, o, step in sets:
        step()
        torch.cuda.synchronize()
        alone.append({k: t.clone() for k, t in o.items()})
        for t in o.values():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        for s, (_, _, _, step) in zip(streams, sets):
            step(stream=s)
    torch.cuda.synchronize()
    for (_, _, o, _), ref in zip(sets, alone):
        for k in ref:
            assert torch.equal(o[k], ref[k]), k


def test_no_tokens_and_rows_behind_the_last():
    """A layer of no tokens writes zero gradients and nothing else; rows behind offsets' last keep what they hold."""
    layer, i, o, step = _layer(0, 3, 2, 64, 32, BF16, 2)
    step()
    assert not bool(o["dw_gu"].any()) and not bool(o["dw_d"].any())
    g = seeded(8)
    for dtype in (F32, BF16):
        for sizes, n in (([5, 2], 40), ([300, 70], 600)):
            x, w = whole(g, n, 64).to(dtype), whole(g, 2, 72, 64).to(dtype)
            out = torch.full((n, 72), -7.0, device="cuda")
            M.moe_expert_matmul(x, w, offsets_of(sizes), out)
            assert bool((out[sum(sizes):] == -7).all())
            h = torch.full((n, 32), -7.0, dtype=dtype, device="cuda")
            M.moe_swiglu(x, h, count=offsets_of(sizes)[2:])
            assert bool((h[sum(sizes):] == -7).all())


@pytest.mark.parametrize("rows", [3, 40, 200, 700])
@pytest.mark.parametrize("D", [16, 80, 128])
def test_sums_of_8_bit_products_are_fp32(rows, D):
    """Codes +-(8 .. 15) 2^(e - 3), e from -3 to 1, are multiples of 2^-6 below 4: products are multiples of 2^-12 and
    128 of them stay below 2^11, so that fp32 sums in any order are exact, however far the products lie apart."""
    print("8-bit sums", rows, D, flush=True)
    g, E, N = seeded(rows + D), 3, 264

    def codes(*shape):
        m = torch.randint(8, 16, shape, generator=g, device="cuda") * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1)
        return m * 2.0 ** (torch.randint(-3, 2, shape, generator=g, device="cuda") - 3)

    sizes = [rows, 0, rows // 2 + 1]
    x, w = codes(sum(sizes), D), codes(E, N, D)
    assert torch.equal(x.to(FP8).float(), x) and torch.equal(w.to(FP8).float(), w)
    out = torch.full((sum(sizes), N), float("nan"), device="cuda")
    M.moe_expert_matmul(x.to(FP8), w.to(FP8), offsets_of(sizes), out, x_scale=torch.ones(sum(sizes), 1, device="cuda"),
                        w_scale=torch.ones(E, 3, 1, device="cuda"))
    same(out, torch.cat([x[a:b].double() @ w[e].double().t() for e, a, b in each(sizes)]), "sums")


@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("E,n", [(64, 4000), (2, 3), (8, 900)])
def test_rows_of_many_experts_at_once(kind, E, n):
    """offsets 0, n, 0, n, ..: every other expert has all rows, more tiles than any disjoint spans make.  The experts'
    weights are the same, so that it does not matter whose product a row gets."""
    dtype = {"f32": F32, "bf16": BF16, "fp8": FP8}[kind]
    print("shared rows", kind, E, n, flush=True)
    g, N, D = seeded(E), 264, 144
    offsets = torch.tensor([0, n] * (E // 2) + [0], dtype=I32, device="cuda")
    x, one = whole(g, n, D), whole(g, 1, N, D)
    w = one.expand(E, N, D).contiguous().to(dtype)
    out = torch.full((n, N), float("nan"), device="cuda")
    scales = dict(x_scale=torch.ones(n, 2, device="cuda"), w_scale=torch.ones(E, 3, 2, device="cuda")) if kind == "fp8" else {}
    M.moe_expert_matmul(x.to(dtype), w, offsets, out, **scales)
    same(out, x.double() @ one[0].double().t(), "forward")
    if kind == "fp8":
        return
    dx, d = torch.full((n, D), float("nan"), device="cuda"), whole(g, n, N)
    M.moe_expert_matmul(d.to(dtype), w, offsets, dx, transposed=True)
    same(dx, d.double() @ one[0].double(), "rows' gradient")
