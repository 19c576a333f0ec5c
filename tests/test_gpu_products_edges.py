"""The experts' products where calls have gone wrong or could: rows of several passes in place, first runs on other
streams.  References are fp64."""
import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M
from oracle import products as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, FP8, I32 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.int32
HALF = {F32: U, BF16: 2.0 ** -8}


def bits(t):
    return t.view(I32 if t.element_size() == 4 else torch.int16)


@pytest.mark.parametrize("I", [4104, 5632, 5760, 11008, 20488])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu_gradient_of_long_rows_in_place(I, dtype):
    """Rows of several passes whose threads are no whole number of waves.  In place and not, the bits are the same;
    against fp64, dg = dh u s (1 + g (1 - s)) is off by 16 u of |dh u s| (1 + |g|) (s 4 u, 1 - s 4 u of s and its own
    rounding, g (1 - s) and the sum two more, three products), du and h by 8 u of themselves, and a stored value by
    half a step."""
    print("swiglu gradient", I, dtype, flush=True)
    g, n, there = torch.Generator(device="cuda").manual_seed(I), 600, 597
    gu = (torch.randn(n, 2 * I + 8, generator=g, device="cuda") * 2).to(dtype)[:, :2 * I]
    dh = torch.randn(n, I, generator=g, device="cuda").to(dtype)
    count = torch.tensor([there], dtype=I32, device="cuda")
    dgu = torch.full((n, 2 * I), 3, dtype=dtype, device="cuda")
    h, again, ahead = (torch.full((n, I), 3, dtype=dtype, device="cuda") for _ in range(3))
    M.moe_swiglu(gu, ahead, count=count)
    M.moe_swiglu_backward(gu, dh, dgu, h=h, count=count)
    rows = [0, 1, 255, 256, 511, there - 1]
    val, dv = gu[rows].double().cpu().numpy(), dh[rows].double().cpu().numpy()
    behind = gu[there:].clone()
    M.moe_swiglu_backward(gu, dh, gu, h=again, count=count)
    assert torch.equal(bits(gu[:there]), bits(dgu[:there])) and torch.equal(bits(gu[there:]), bits(behind))
    assert torch.equal(bits(h), bits(again)) and torch.equal(bits(h), bits(ahead))
    assert bool((dgu[there:] == 3).all()) and bool((h[there:] == 3).all())
    a, u = val[:, :I], val[:, I:]
    ref, rh, v = O.swiglu_backward(val, dv), O.swiglu(val), HALF[dtype]
    room = np.concatenate([16 * U * np.abs(dv * u * O.sigmoid(a)) * (1 + np.abs(a)), 8 * U * np.abs(ref[:, I:])], 1)
    assert (np.abs(dgu[rows].double().cpu().numpy() - ref) - room - v * np.abs(ref) - 2.0 ** -120).max() <= 0
    assert (np.abs(h[rows].double().cpu().numpy() - rh) - 8 * U * np.abs(rh) - v * np.abs(rh) - 2.0 ** -120).max() <= 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_first_training_run_on_another_stream(dtype):
    """The buffers that a first training run makes come from the current stream's memory, where work that was given
    before is still to write what has been freed since; its results are those of a layer that has run before."""
    print("first run elsewhere", dtype, flush=True)
    T, E, K, H, I = 3000, 5, 2, 264, 520
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x, dout, logits = rand(T, H).to(dtype), rand(T, H).to(dtype), rand(T, E)
    w_gu, w_d = (rand(E, 2 * I, H) * H ** -0.5).to(dtype), (rand(E, H, I) * I ** -0.5).to(dtype)
    code = M.MOE_F32 if dtype == F32 else M.MOE_BF16

    def step(layer, outs, stream=None, before=None):
        for part in range(2):
            if before:
                before(part)
            if part == 0:
                layer.run(x, logits, w_gu, w_d, outs[0], train=True, stream=stream)
            else:
                layer.backward(dout, *outs[1:], stream=stream)

    outs = [[torch.empty_like(t) for t in (x, x, logits, w_gu, w_d)] for _ in range(2)]
    first = M.ExpertTrainLayer(E, H, I, K, code, T)
    step(first, outs[0])
    step(first, outs[0])
    one, side = M.ExpertTrainLayer(E, H, I, K, code, T), torch.cuda.Stream()
    a, b = rand(8192, 8192), rand(8192, 8192)
    product = torch.empty_like(a)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    made = []

    def pending(part):
        for _ in range(6):
            torch.mm(a, b, out=product)  # some milliseconds each
        freed = [torch.empty(T * K, c, dtype=dtype, device="cuda") for c in ((H,) if part == 0 else (H, I, H))]
        for t in freed:
            t.fill_(float("nan"))
        made.append({t.data_ptr() for t in freed})

    step(one, outs[1], stream=side, before=pending)
    torch.cuda.synchronize()
    assert one.xs.data_ptr() in made[0] and one._back[0].data_ptr() in made[1]  # or this tests nothing
    for got, ref in zip(outs[1], outs[0]):
        assert torch.equal(bits(got), bits(ref))


def product8(x, w, odt):
    """x [n][D] and w [N][D], values that 8-bit codes hold, as one expert's product with scales of one."""
    (n, D), N = x.shape, w.shape[0]
    offsets, out = torch.tensor([0, n], dtype=I32, device="cuda"), torch.full((n, N), float("nan"), dtype=odt, device="cuda")
    M.moe_expert_matmul(x.to(FP8), w[None].to(FP8), offsets, out, x_scale=torch.ones(n, -(-D // 128), device="cuda"),
                        w_scale=torch.ones(1, -(-N // 128), -(-D // 128), device="cuda"))
    return out


@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("rows", [16, 300])
def test_8_bit_products_far_below_the_largest(rows, odt):
    """2^16 - 2^16 + 2^(16 - d) in one block: exact in bf16 outputs while the products lie within 13 bits, wherever
    they are, and in fp32 ones within 23, that type's own."""
    print("8-bit products", rows, odt, flush=True)
    for i, j, k in ((0, 1, 2), (0, 2, 1), (3, 9, 4), (0, 64, 127), (5, 100, 50), (126, 127, 0), (40, 47, 41)):
        for d in range(0, (13 if odt == BF16 else 23) + 1):
            x, w = torch.zeros(rows, 128, device="cuda"), torch.zeros(128, 128, device="cuda")
            small = min(d, 17)  # codes go down to 2^-9
            x[:, i], x[:, j], x[:, k] = 256.0, -256.0, 2.0 ** (8 - small)
            w[:, i], w[:, j], w[:, k] = 256.0, 256.0, 2.0 ** (8 - (d - small))
            assert bool((product8(x, w, odt) == 2.0 ** (16 - d)).all()), (i, j, k, d)


@pytest.mark.parametrize("large", [1, 30, 300])
@pytest.mark.parametrize("rows,D", [(40, 2880), (400, 1040)])
def test_8_bit_products_with_a_large_column(rows, D, large):
    """bf16 outputs: of eight products seven are cut by less than 2^-13 of the largest, so that an element is off by
    less than 7 2^-13 of the sum of its terms' sizes; the sums in fp32 of at most D of them 2 u (D + 3) of it, the
    result half a step.  fp32 outputs: the last two."""
    print("large column", rows, D, large, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + large)
    x, w = torch.randn(rows, D, generator=g, device="cuda") * 100 / large, torch.randn(264, D, generator=g, device="cuda") * 100
    x[:, ::128] *= large
    x, w = (t.clamp(-448, 448).to(FP8).double() for t in (x, w))
    ref, size = x @ w.t(), x.abs() @ w.abs().t()
    for odt in (BF16, F32):
        off = (product8(x.float(), w.float(), odt).double() - ref).abs() - HALF[odt] * ref.abs() - 2 * U * (D + 3) * size
        assert float((off - (7 * 2.0 ** -13 * size if odt == BF16 else 0)).max()) <= 0, odt


@pytest.mark.parametrize("rows", [30, 200])
def test_rows_gradient_through_weights_quantised_the_other_way(rows):
    """moe_quantize_weights(transposed) gives the weights of the 8-bit product in the other direction.  Against fp64 of
    the values that the codes stand for: a sum of N terms is off by 2 u (N + 3) of the sum of their sizes; and those
    values against the weights: a code is off by half a step, 2^-4 of its value or 2^-10 of its scale."""
    print("transposed codes", rows, flush=True)
    E, N, D = 3, 272, 200
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = (torch.randn(E, N, D, generator=g, device="cuda") * 0.05).to(BF16)
    codes, scale = torch.empty(E, D, N, dtype=FP8, device="cuda"), torch.empty(E, 2, 3, device="cuda")
    M.moe_quantize_weights(w, codes, scale, transposed=True)
    sizes = [rows, 0, rows // 3]
    n = sum(sizes)
    d8 = (torch.randn(n, N, generator=g, device="cuda") * 60).clamp(-448, 448).to(FP8)
    ds = torch.rand(n, 3, generator=g, device="cuda") + 0.5
    offsets = torch.tensor([0, *np.cumsum(sizes)], dtype=I32, device="cuda")
    dx = torch.empty(n, D, device="cuda")
    M.moe_expert_matmul(d8, codes, offsets, dx, x_scale=ds, w_scale=scale)
    each = scale.double().repeat_interleave(128, 1)[:, :D].repeat_interleave(128, 2)[:, :, :N]
    wv = codes.double() * each
    w0 = w.double().transpose(1, 2)
    assert float(((wv - w0).abs() - torch.maximum(2.0 ** -4 * w0.abs(), 2.0 ** -10 * each) * (1 + 16 * U)).max()) <= 0
    dv = d8.double() * ds.double().repeat_interleave(128, 1)[:, :N]
    at = 0
    for e, s in enumerate(sizes):
        r = dv[at:at + s]
        off = (dx[at:at + s].double() - r @ wv[e].t()).abs() - (2 * U * (N + 3) * (r.abs() @ wv[e].abs().t()) + U * (r @ wv[e].t()).abs())
        assert off.numel() == 0 or float(off.max()) <= 0, e
        at += s
