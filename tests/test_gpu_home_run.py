"""The home rank's operators as they are used together: a whole layer, a layer with gradients, the
rows that a step released going on to the next layer's pool, a captured layer, two streams at once."""
import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M
import oracle as MO
import workloads as W
from gpu_helpers import TOL, decode_tensor, dev, row_rel_err, sync_err
from oracle import home as O
from workloads.device import batch_tensors, to_numpy_bits, weight_tensors
from workloads.gen import make_layer_weights

pytestmark = pytest.mark.gpu

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def expert_rows(wts, xb, offsets):
    """The experts' rows for the sorted rows xb (fp64)."""
    return MO.expert_ffn(xb, offsets, wts)


@pytest.mark.parametrize("act,wt,T,E,K,H,I", [("f32", "f32", 33, 8, 2, 64, 128), ("bf16", "bf16", 61, 16, 4, 320, 192),
                                             ("bf16", "fp8", 900, 8, 2, 256, 128)])
def test_expert_layer(act, wt, T, E, K, H, I):
    print("expert layer", act, wt, T, flush=True)
    rng = np.random.default_rng(T)
    wts = make_layer_weights(rng, E, H, I, 0.05, wt)
    w = weight_tensors(wts)
    code = dict(f32=M.MOE_F32, bf16=M.MOE_BF16, fp8=M.MOE_FP8_E4M3)
    tdt = F32 if act == "f32" else BF16
    layer = M.ExpertLayer(E, H, I, K, code[act], code[wt], T + 5)
    layer.load_weights(w["wg"], w["wu"], w["wd"], w.get("s_gate"), w.get("s_up"), w.get("s_down"))
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda().to(tdt)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    logits[3] = float("-inf")  # a padding token
    out = torch.empty(T, H, dtype=tdt, device="cuda")
    layer.run(x, logits, out)
    expert, weight = O.route(logits.cpu().numpy(), K)
    perm, pos, counts, offsets, slot, _ = O.sort_index(expert, E)
    total = offsets[E]
    assert sync_err(layer.err) == 0
    assert np.array_equal(layer.expert.cpu().numpy(), expert) and np.array_equal(layer.offsets.cpu().numpy(), offsets)
    xv = decode_tensor(x)
    y = np.zeros((T * K, H))
    y[:total] = expert_rows(wts, xv[slot[:total]], offsets)
    ref = O.merge_rows(y, pos.reshape(T, K), weight)
    assert not ref[3].any()
    assert row_rel_err(decode_tensor(out), ref) <= TOL["fp8" if wt == "fp8" else act]
    # on another stream, and with fewer tokens from a wider buffer
    s = torch.cuda.Stream()
    wide = torch.zeros(7, H + 64, dtype=tdt, device="cuda")
    wide[:, :H] = x[:7]
    few, again = torch.empty(7, H, dtype=tdt, device="cuda"), torch.empty_like(out)
    s.wait_stream(torch.cuda.current_stream())
    layer.run(x, logits, again, stream=s)
    s.synchronize()
    assert torch.equal(again, out)
    layer.run(wide[:, :H], logits[:7], few)
    assert row_rel_err(decode_tensor(few), ref[:7]) <= TOL["fp8" if wt == "fp8" else act]
    layer.run(x[:0], logits[:0], out[:0])
    torch.cuda.synchronize()
    assert not layer.offsets.any()
    for bad in (torch.empty(H, T, dtype=tdt, device="cuda").t(), x[:5], x[:, :H - 8], x.double()):
        with pytest.raises(M.MoeError, match="logits"):
            layer.run(bad, logits, out)
    with pytest.raises(M.MoeError, match="layer on"):
        layer.run(x.cpu(), logits, out)
    with pytest.raises(M.MoeError, match="tokens"):
        layer.run(torch.empty(T + 6, H, dtype=tdt, device="cuda"), logits, out)


def test_layer_with_gradients():
    """norm -> gate -> route -> sort -> an elementwise expert -> merge in fp32, and back to x, the
    norm's weight and the gate, against autograd of the same layer in fp64.  Each operator is held to
    its own bounds elsewhere; here 1e-4 of the largest gradient stands for the chain's roundings:
    about ten operators of at most 100 x 2^-24 each, times a condition of 10."""
    rng = np.random.default_rng(11)
    T, E, K, H = 53, 12, 3, 128
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x, res, gate, gain, dout, dnext = f(T, H), f(T, H), f(E, H) / H ** 0.5, 1 + 0.2 * f(E, H), f(T, H), f(T, H)
    gamma = 1 + 0.1 * f(H)
    xd, rd, gd, md = (a.double().requires_grad_() for a in (x, res, gate, gamma))
    hd = xd + rd
    yd = hd * (hd.square().mean(1, keepdim=True) + 1e-5).rsqrt() * md
    ld = yd @ gd.t()
    chosen = torch.topk(ld, K, 1).indices
    wd = torch.softmax(ld.gather(1, chosen), 1)
    rows = torch.tanh(yd[:, None] * gain.double()[chosen])
    ((rows * wd[:, :, None]).sum(1) * dout.double()).sum().add((hd * dnext.double()).sum()).backward()

    x, res, gate, gain, gamma, dout, dnext = (a.cuda() for a in (x, res, gate, gain, gamma, dout, dnext))
    e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    n, err, ws = T * K, torch.zeros(1, dtype=I32, device="cuda"), torch.empty(1 << 18, dtype=torch.uint8, device="cuda")
    y, h, rstd = e(T, H), e(T, H), e(T)
    M.moe_residual_norm(x, res, gamma, 1e-5, y, residual_out=h, rstd=rstd)
    logits = y @ gate.t()
    expert, w = e(T, K, dtype=I32), e(T, K)
    M.moe_route(logits, expert, w)
    assert torch.equal(expert.cpu(), chosen.int())
    xs, pos, counts, offsets, slot = e(n, H), e(n, dtype=I32), e(E, dtype=I32), e(E + 1, dtype=I32), e(n, dtype=I32)
    perm = e(n, dtype=I32)
    M.moe_sort_rows(expert, E, y, xs, perm, pos, counts, offsets, err, ws, row_slot=slot)
    which = expert.view(-1)[perm.long()].long()
    rows = torch.tanh(xs * gain[which])
    out = e(T, H)
    M.moe_merge_rows(rows, pos, w, out, err)
    drows, dw = e(n, H), e(T, K)
    M.moe_merge_rows_backward(dout, rows, pos, w, drows, dw, err)
    dxs = drows * (1 - rows * rows) * gain[which]
    dy = e(T, H)
    M.moe_merge_rows(dxs, pos, None, dy, err)
    dlogits = e(T, E)
    M.moe_route_backward(logits, expert, dw, dlogits, err)
    dy = dy + dlogits @ gate
    dx, dgamma = e(T, H), e(H)
    M.moe_residual_norm_backward(dy, h, gamma, rstd, dx, dgamma, torch.empty(2048 * H, dtype=torch.uint8, device="cuda"), dres=dnext)
    assert sync_err(err) == 0
    for got, ref in ((dx, xd.grad), (dx, rd.grad), (dgamma, md.grad), (dlogits.t() @ y, gd.grad)):
        assert (got.cpu().double() - ref).abs().max() <= 1e-4 * ref.abs().max()


def test_released_rows_go_on_through_the_norm():
    """A step's released rows, listed on the device, added to the residual and normed into the next
    layer's pool in 8 bits; the pool's rows then sorted as bf16 rows."""
    rng = np.random.default_rng(2)
    b, wts = W.c0_tiny()
    d, w = batch_tensors(b), weight_tensors(wts)
    st = M.ExpertStep(b.E_loc, b.H, wts.I, b.K, M.MOE_F32, M.MOE_F32, b.n, b.T)
    st.load_weights(w["wg"], w["wu"], w["wd"])
    half = torch.arange(b.n, device="cuda")[d["tok"][:b.n] % 3 != 1]  # a third of the tokens stays incomplete
    m = half.numel()
    st.run(d["slot"][half], d["expert"][half], b.expert_base, d["pool"], d["tok"][half], d["kslot"][half], d["w"][half],
           d["gen"][half])
    T, H = b.T, b.H
    res = dev(rng.standard_normal((T, H)).astype(np.float32))
    gamma = dev((1 + 0.1 * rng.standard_normal(H)).astype(np.float32))
    before = res.clone()
    pool, scale = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(T, 2, device="cuda")
    M.moe_residual_norm(st.out, res, gamma, 1e-5, pool, residual_out=res, out_scale=scale, group=32,
                        row_list=st.rel_list[:T], row_count=st.rel_count, err=st.err)
    assert sync_err(st.err) == 0 and m > 0
    released = st.rel_list[:int(st.rel_count.item())].long()
    waiting = torch.ones(T, dtype=torch.bool, device="cuda")
    waiting[released] = False
    assert 0 < released.numel() < T
    assert torch.equal(res[waiting], before[waiting]) and not pool[waiting].any()
    assert torch.equal(res[released], before[released] + st.out[released])
    y, _, _ = O.residual_norm(st.out[released].cpu().numpy(), before[released].cpu().numpy(), gamma.cpu().numpy(), 1e-5)
    got = MO.decode_e4m3(pool[released].cpu().numpy()) * scale[released].cpu().numpy().repeat(32, axis=1)
    # half a step of e4m3: 2^-4 of the value, 2^-10 scales below 2^-6; fp32 roundings are far below 1e-3 of it
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * O.group_scales(y, 32).repeat(32, axis=1)) * (1 + 1e-3)
    assert (np.abs(got - y) <= tol).all()
    expert = torch.full((T, 2), -1, dtype=I32, device="cuda")
    expert[released] = torch.randint(0, 4, (released.numel(), 2), device="cuda", dtype=I32)
    xs = torch.zeros(2 * T, H, dtype=BF16, device="cuda")
    perm, pos = (torch.empty(2 * T, dtype=I32, device="cuda") for _ in range(2))
    counts, offsets = torch.empty(4, dtype=I32, device="cuda"), torch.empty(5, dtype=I32, device="cuda")
    M.moe_sort_rows(expert, 4, pool, xs, perm, pos, counts, offsets, st.err, torch.empty(1 << 18, dtype=torch.uint8, device="cuda"),
                    x_scale=scale, group=32)
    total = int(offsets[4].item())
    assert total == 2 * released.numel()
    rows = (pool.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(32, 1)).to(BF16)
    assert torch.equal(xs[:total], rows[perm[:total].long() // 2])


def _one_of_everything(T, K, E, H, seed):
    """Buffers and the calls of a training pass on them, all outputs among the buffers."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, dtype=BF16: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    z = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    n = T * K
    inputs = dict(x=r(T, H), res=r(T, H), gamma=r(H), logits=r(T, E, dtype=F32), dout=r(T, H))
    out = dict(y=z(T, H, dtype=BF16), h=z(T, H, dtype=BF16), rstd=z(T), expert=z(T, K, dtype=I32), w=z(T, K), xs=z(n, H, dtype=BF16),
               perm=z(n, dtype=I32), pos=z(n, dtype=I32), counts=z(E, dtype=I32), offsets=z(E + 1, dtype=I32),
               merged=z(T, H, dtype=BF16), drows=z(n, H, dtype=BF16), dw=z(T, K), dlogits=z(T, E), dy=z(T, H, dtype=BF16),
               dx=z(T, H, dtype=BF16), dgamma=z(H), err=z(1, dtype=I32))
    ws, ws2 = z(1 << 18, dtype=torch.uint8), z(2048 * H, dtype=torch.uint8)

    def calls(stream=None):
        i, o = inputs, out
        M.moe_residual_norm(i["x"], i["res"], i["gamma"], 1e-5, o["y"], residual_out=o["h"], rstd=o["rstd"], stream=stream)
        M.moe_route(i["logits"], o["expert"], o["w"], stream=stream)
        M.moe_sort_rows(o["expert"], E, o["y"], o["xs"], o["perm"], o["pos"], o["counts"], o["offsets"], o["err"], ws, stream=stream)
        M.moe_merge_rows(o["xs"], o["pos"], o["w"], o["merged"], o["err"], stream=stream)
        M.moe_merge_rows_backward(i["dout"], o["xs"], o["pos"], o["w"], o["drows"], o["dw"], o["err"], stream=stream)
        M.moe_merge_rows(o["drows"], o["pos"], None, o["dy"], o["err"], stream=stream)
        M.moe_route_backward(i["logits"], o["expert"], o["dw"], o["dlogits"], o["err"], stream=stream)
        M.moe_residual_norm_backward(o["dy"], o["h"], i["gamma"], o["rstd"], o["dx"], o["dgamma"], ws2, stream=stream)

    def refill(seed):
        g.manual_seed(seed)
        for t in inputs.values():
            t.copy_(torch.randn(*t.shape, generator=g, device="cuda"))

    return inputs, out, calls, refill


@pytest.mark.parametrize("T", [19, 3001])
def test_captured_pass(T):
    print("captured pass", T, flush=True)
    inputs, out, calls, refill = _one_of_everything(T, 4, 40, 264, 1)
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (5, 6, 7):
        refill(seed)
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in out.items()}
        for t in out.values():
            t.zero_()
        calls()
        torch.cuda.synchronize()
        assert not int(out["err"].item())
        for k in out:
            assert torch.equal(got[k], out[k]), (seed, k)


def test_two_streams_and_many_calls():
    """Passes on two streams at once, each with its own buffers, give the bits of the passes one after
    another; so does a pass on a stream that is not the current one."""
    sets = [_one_of_everything(T, 4, 40, 264, T) for T in (2500, 777)]
    alone = []
    for _, out, calls, _ in sets:
        calls()
        torch.cuda.synchronize()
        alone.append({k: t.clone() for k, t in out.items()})
        for t in out.values():
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for s, (_, _, calls, _) in zip(streams, sets):
            calls(stream=s)
    torch.cuda.synchronize()
    for (_, out, _, _), ref in zip(sets, alone):
        for k in ref:
            assert torch.equal(out[k], ref[k]), k


def test_tensors_may_go_while_another_stream_works():
    """A call on a side stream keeps its tensors: what the allocator hands out meanwhile is other memory."""
    T, H = 4096, 4096
    s = torch.cuda.Stream()
    x = torch.randn(T, H, device="cuda").to(BF16)
    gamma = torch.ones(H, dtype=BF16, device="cuda")
    ref = torch.empty_like(x)
    M.moe_residual_norm(x, None, gamma, 1e-5, ref)
    out = torch.empty_like(x)
    torch.cuda.synchronize()
    for _ in range(6):
        y = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        M.moe_residual_norm(y, None, gamma, 1e-5, out, stream=s)
        del y
        torch.full_like(x, 3.0)  # would take y's memory
        s.synchronize()
        assert torch.equal(out, ref)


def test_offsets_past_32_bits():
    """Rows far apart in one large buffer: element offsets beyond 2^31 and byte offsets beyond 2^32."""
    T, H, pitch = 5, 64, 1 << 29
    big = torch.zeros((T - 1) * pitch + H, dtype=BF16, device="cuda")
    x = big.as_strided((T, H), (pitch, 1))
    x.copy_(torch.randn(T, H, device="cuda"))
    near = x.clone()
    gamma = torch.ones(H, dtype=BF16, device="cuda")
    a, b = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, H, dtype=BF16, device="cuda")
    M.moe_residual_norm(x, None, gamma, 1e-5, a)
    M.moe_residual_norm(near, None, gamma, 1e-5, b)
    assert torch.equal(a, b)
    M.moe_residual_norm(near, None, gamma, 1e-5, x, residual_out=None)
    assert torch.equal(x, a)
    x.copy_(near)
    pos = torch.tensor([[4, 0], [3, -1], [1, 2]], dtype=I32, device="cuda")
    err = torch.zeros(1, dtype=I32, device="cuda")
    o1, o2 = (torch.empty(3, H, dtype=F32, device="cuda") for _ in range(2))
    M.moe_merge_rows(x, pos, None, o1, err)
    M.moe_merge_rows(near, pos, None, o2, err)
    assert torch.equal(o1, o2) and sync_err(err) == 0
    xs = torch.empty(T, H, dtype=BF16, device="cuda")
    p = [torch.empty(T, dtype=I32, device="cuda") for _ in range(2)]
    M.moe_sort_rows(torch.tensor([[2], [0], [1], [-1], [0]], dtype=I32, device="cuda"), 3, x, xs, p[0], p[1],
                    torch.empty(3, dtype=I32, device="cuda"), torch.empty(4, dtype=I32, device="cuda"), err,
                    torch.empty(1 << 18, dtype=torch.uint8, device="cuda"))
    assert torch.equal(xs[:4], near[[1, 4, 2, 0]])
    logits = torch.zeros((T - 1) * pitch + 16, dtype=BF16, device="cuda").as_strided((T, 16), (pitch, 1))
    logits.copy_(torch.randn(T, 16, device="cuda"))
    e1, e2, w1, w2 = *(torch.empty(T, 3, dtype=I32, device="cuda") for _ in range(2)), *(torch.empty(T, 3, device="cuda") for _ in range(2))
    M.moe_route(logits, e1, w1)
    M.moe_route(logits.clone(), e2, w2)
    assert torch.equal(e1, e2) and torch.equal(w1, w2)


# Calls that move 96 MiB of rows or more read them non-temporally, from 220 MiB on they write so too.
LARGE = [(5000, 4, 2880), (9600, 4, 2880)]


@pytest.mark.parametrize("T,K,H", LARGE)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_calls_give_the_bits_of_small_ones(T, K, H, dtype):
    T = T // 2 if dtype == F32 else T
    print("large calls", T, K, H, dtype, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    e = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    n, E, err = T * K, 64, e(1, dt=I32)
    expert = torch.randint(-1, E, (T, K), generator=g, device="cuda", dtype=I32)
    x, xs, perm, pos = r(T, H), e(n, H, dt=dtype), e(n, dt=I32), e(n, dt=I32)
    counts, offsets, slot, ws = e(E, dt=I32), e(E + 1, dt=I32), e(n, dt=I32), e(1 << 18, dt=torch.uint8)
    M.moe_sort_rows(expert, E, x, xs, perm, pos, counts, offsets, err, ws, row_slot=slot)
    total = int(offsets[E])
    assert total == int((expert >= 0).sum()) and torch.equal(xs[:total], x[slot[:total].long()]) and not xs[total:].any()
    w, out, part = torch.rand(T, K, generator=g, device="cuda"), e(T, H, dt=dtype), e(300, H, dt=dtype)
    M.moe_merge_rows(xs, pos, w, out, err)
    dout, drows, dw, dw2 = r(T, H), e(n, H, dt=dtype), e(T, K), e(300, K)
    M.moe_merge_rows_backward(dout, xs, pos, w, drows, dw, err)
    small = e(n, H, dt=dtype)
    for a in range(0, T, 300):
        b = min(T, a + 300)
        p = pos[a * K:b * K]
        M.moe_merge_rows(xs, p, w[a:b], part[:b - a], err)
        M.moe_merge_rows_backward(dout[a:b], xs, p, w[a:b], small, dw2[:b - a], err)
        assert torch.equal(part[:b - a], out[a:b]) and torch.equal(dw2[:b - a], dw[a:b])
    assert torch.equal(small, drows) and sync_err(err) == 0


@pytest.mark.parametrize("T", [3500, 9000, 14000])
@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, torch.float8_e4m3fn), (F32, F32)])
def test_large_norms_give_the_bits_of_small_ones(T, dtype, out_dtype):
    H, group = 4096, 128
    T = T // 2 if dtype == F32 else T
    print("large norms", T, dtype, out_dtype, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    z = lambda *s, dt=dtype: torch.zeros(*s, dtype=torch.uint8 if dt.itemsize == 1 else dt, device="cuda").view(dt)  # noqa: E731
    x, res, gamma = r(T, H), r(T, H), r(H)
    fp8 = out_dtype.itemsize == 1
    out, ro, rstd, sc = z(T, H, dt=out_dtype), z(T, H), z(T, dt=F32), z(T, H // group, dt=F32) if fp8 else None
    M.moe_residual_norm(x, res, gamma, 1e-5, out, residual_out=ro, rstd=rstd, out_scale=sc, group=group)
    dout, dx, dgamma, ws = r(T, H), z(T, H), z(H, dt=F32), z(2048 * H, dt=torch.uint8)
    M.moe_residual_norm_backward(dout, ro, gamma, rstd, dx, dgamma, ws, dres=res)
    for a in range(0, T, 500):
        b = min(T, a + 500)
        o2, ro2, rs2, sc2 = z(b - a, H, dt=out_dtype), z(b - a, H), z(b - a, dt=F32), z(b - a, H // group, dt=F32) if fp8 else None
        M.moe_residual_norm(x[a:b], res[a:b], gamma, 1e-5, o2, residual_out=ro2, rstd=rs2, out_scale=sc2, group=group)
        dx2 = z(b - a, H)
        M.moe_residual_norm_backward(dout[a:b], ro[a:b], gamma, rstd[a:b], dx2, None, None, dres=res[a:b])
        assert torch.equal(o2.view(torch.uint8) if fp8 else o2, out[a:b].view(torch.uint8) if fp8 else out[a:b])
        assert torch.equal(ro2, ro[a:b]) and torch.equal(rs2, rstd[a:b]) and torch.equal(dx2, dx[a:b])
        assert not fp8 or torch.equal(sc2, sc[a:b])
    ref, size = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for a in range(0, T, 1000):
        t = dout[a:a + 1000].double() * ro[a:a + 1000].double() * rstd[a:a + 1000].double()[:, None]
        ref += t.sum(0)
        size += t.abs().sum(0)
    # runs of ceil(T / 512) tokens, then 512 partial sums in runs of 8 and a tree; 3 roundings a term
    assert ((dgamma.double() - ref).abs() <= (-(-T // 512) + 20) * 2.0 ** -24 * size).all()


def test_the_largest_number_of_tokens():
    """T K = 2^24 pairs in every operator, rows of 8 columns."""
    T, H = 1 << 24, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    e = lambda *s, dt=F32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    err, ws = e(1, dt=I32), e(1 << 18, dt=torch.uint8)
    logits = torch.randn(T, 2, generator=g, device="cuda")
    expert, w = e(T, 1, dt=I32), e(T, 1)
    M.moe_route(logits, expert, w, renorm=False)
    assert torch.equal(expert[:, 0].long(), (logits[:, 1] > logits[:, 0]).long())
    dl = e(T, 2)
    M.moe_route_backward(logits, expert, w, dl, err, renorm=False)
    assert (dl.sum(1).abs() <= 2.0 ** -20).all()  # the two gradients of a softmax of two cancel
    del dl, logits
    wide = torch.randint(0, 256, (T, 1), generator=g, device="cuda", dtype=I32)
    x, xs = torch.randn(T, H, generator=g, device="cuda").to(BF16), e(T, H, dt=BF16)
    perm, pos, counts, offsets = e(T, dt=I32), e(T, dt=I32), e(256, dt=I32), e(257, dt=I32)
    M.moe_sort_rows(wide, 256, x, xs, perm, pos, counts, offsets, err, ws)
    order = torch.sort(wide[:, 0], stable=True).indices
    assert torch.equal(perm.long(), order) and torch.equal(xs, x[order])
    assert torch.equal(counts.long(), torch.bincount(wide[:, 0].long(), minlength=256))
    out, dw = e(T, H, dt=BF16), e(T, 1)
    M.moe_merge_rows(xs, pos, None, out, err)
    assert torch.equal(out, x)
    M.moe_merge_rows_backward(x, xs, pos, None, out, dw, err)
    assert torch.equal(out, xs)
    gamma, rstd, dgamma = torch.ones(H, device="cuda"), e(T), e(H)
    M.moe_residual_norm(x, None, gamma, 1e-5, out, rstd=rstd)
    few = e(1000, H, dt=BF16)
    M.moe_residual_norm(x[-1000:], None, gamma, 1e-5, few)
    assert torch.equal(out[-1000:], few)
    M.moe_residual_norm_backward(out, x, gamma, rstd, xs, dgamma, e(2048 * H, dt=torch.uint8))
    ref = (out.double() * x.double() * rstd.double()[:, None]).sum(0)
    # terms of one sign in chains of 2^15: off by 2^15 2^-24 at most, and 30 additions and roundings more
    assert ((dgamma.double() - ref).abs() <= (2 ** 15 + 30) * 2.0 ** -24 * ref.abs()).all()
    assert sync_err(err) == 0
