"""Refusals of the experts' products: the C entry points' host checks (they return before anything is enqueued, so
made-up addresses do), the binding's checks of its tensors, and the layer's."""
import ctypes as C
import os

import pytest
import torch

import asynchronous_moe_expert_amd as M
from asynchronous_moe_expert_amd import _native as N

NULL, SIZE, DTYPE, ALIGN, SHAPE = -1, -2, -3, -4, -5
P = 4096  # an aligned address that no refused call touches
F32, BF16, FP8 = M.MOE_F32, M.MOE_BF16, M.MOE_FP8_E4M3
BIG = (1 << 24) + 1


@pytest.fixture(scope="module")
def lib():
    from asynchronous_moe_expert_amd import build

    if not (os.path.exists(M.LIB_PATH) and os.path.exists(build.MARSHAL)):
        build.build()
    return M.load()


MATMUL = dict(n=4, E_loc=2, N=64, D=32, offsets=P, x=P, dtype=BF16, x_rows=9, x_pitch=32, row_slot=P, w=P,
              w_transposed=0, w_pitch=32, w_stride=64 * 32, out=P, out_dtype=BF16, out_pitch=64, err=P)
IN8 = dict(dtype=FP8, x_scale=P, w_scale=P)
MATMUL_B = dict(n=4, E_loc=2, N=64, D=32, offsets=P, dout=P, dout_pitch=64, x=P, x_pitch=32, dtype=BF16,
                accumulate=0, dw=P, dw_dtype=F32, dw_pitch=32, dw_stride=64 * 32)
SWIGLU = dict(n=4, I=32, gu=P, dtype=BF16, gu_pitch=64, count=P, h=P, h_dtype=FP8, h_pitch=32, h_scale=P, group=32)
SWIGLU_B = dict(n=4, I=32, gu=P, dtype=BF16, gu_pitch=64, dh=P, dh_pitch=32, count=P, dgu=P, dgu_pitch=64, h=P,
                h_pitch=32)
QUANTIZE = dict(E_loc=2, N=64, D=32, w=P, dtype=BF16, w_pitch=32, w_stride=64 * 32, transposed=0, codes=P,
                codes_pitch=32, codes_stride=64 * 32, scale=P)

SIZES = [(dict(n=-1), SIZE), (dict(n=BIG), SIZE), (dict(E_loc=0), SIZE), (dict(E_loc=257), SIZE), (dict(N=0), SIZE),
         (dict(D=0), SIZE), (dict(N=(1 << 16) + 8), SIZE), (dict(D=(1 << 16) + 8), SIZE), (dict(N=60), SHAPE),
         (dict(D=28), SHAPE)]
REFUSED = [
    ("moe_expert_matmul", N.ExpertMatmulArgs, MATMUL, SIZES + [
        (dict(w_transposed=2), SIZE), (dict(dtype=7), DTYPE), (dict(out_dtype=FP8), DTYPE),
        (dict(dtype=F32, out_dtype=BF16), DTYPE), (dict(IN8, w_transposed=1), DTYPE), (dict(IN8, D=24), SHAPE),
        (dict(x_rows=-1), SIZE), (dict(x_rows=BIG), SIZE), (dict(x_pitch=31), SIZE), (dict(out_pitch=63), SIZE),
        (dict(w_pitch=24), SIZE), (dict(w_stride=63 * 32 + 24), SIZE), (dict(w_transposed=1), SIZE),
        (dict(w_pitch=(1 << 23) + 8, w_stride=1 << 30), SIZE), (dict(w_stride=(1 << 36) + 8), SIZE),
        (dict(x_pitch=(1 << 23) + 8), SIZE), (dict(x_rows=1 << 24, x_pitch=1 << 16), SIZE),
        (dict(offsets=0), NULL), (dict(x=0), NULL), (dict(w=0), NULL), (dict(out=0), NULL), (dict(err=0), NULL),
        (dict(IN8, x_scale=0), NULL), (dict(IN8, w_scale=0), NULL), (dict(x=P + 8), ALIGN), (dict(w=P + 2), ALIGN),
        (dict(out=P + 8), ALIGN), (dict(x_pitch=36), ALIGN), (dict(w_pitch=36, w_stride=64 * 36), ALIGN),
        (dict(w_stride=64 * 32 + 4), ALIGN), (dict(out_pitch=68), ALIGN), (dict(IN8, x_pitch=40), ALIGN)]),
    ("moe_expert_matmul_backward", N.ExpertMatmulBackwardArgs, MATMUL_B, SIZES + [
        (dict(accumulate=2), SIZE), (dict(dtype=FP8), DTYPE), (dict(dw_dtype=FP8), DTYPE),
        (dict(dtype=F32, dw_dtype=BF16), DTYPE), (dict(dout_pitch=63), SIZE), (dict(x_pitch=31), SIZE),
        (dict(dw_pitch=31), SIZE), (dict(dw_stride=63 * 32 + 24), SIZE), (dict(dout_pitch=(1 << 23) + 8), SIZE),
        (dict(n=1 << 24, x_pitch=1 << 16), SIZE), (dict(offsets=0), NULL), (dict(dw=0), NULL), (dict(dout=0), NULL),
        (dict(x=0), NULL), (dict(dw=0, n=0), NULL), (dict(dout=P + 8), ALIGN), (dict(x=P + 4), ALIGN),
        (dict(dw=P + 4), ALIGN), (dict(dout_pitch=68), ALIGN), (dict(x_pitch=36), ALIGN), (dict(dw_stride=2050), ALIGN)]),
    ("moe_swiglu", N.SwigluArgs, SWIGLU, [
        (dict(n=-1), SIZE), (dict(n=BIG), SIZE), (dict(I=0), SIZE), (dict(I=32776), SIZE), (dict(I=28), SHAPE),
        (dict(dtype=FP8), DTYPE), (dict(h_dtype=9), DTYPE), (dict(gu_pitch=63), SIZE), (dict(h_pitch=31), SIZE),
        (dict(group=16), SIZE), (dict(gu=0), NULL), (dict(h=0), NULL), (dict(h_scale=0), NULL),
        (dict(gu=P + 8), ALIGN), (dict(gu_pitch=68), ALIGN), (dict(h=P + 4), ALIGN), (dict(h_pitch=36), ALIGN)]),
    ("moe_swiglu_backward", N.SwigluBackwardArgs, SWIGLU_B, [
        (dict(n=-1), SIZE), (dict(n=BIG), SIZE), (dict(I=32776), SIZE), (dict(I=28), SHAPE), (dict(dtype=FP8), DTYPE),
        (dict(gu_pitch=63), SIZE), (dict(dgu_pitch=63), SIZE), (dict(dh_pitch=31), SIZE), (dict(h_pitch=31), SIZE),
        (dict(gu=0), NULL), (dict(dh=0), NULL), (dict(dgu=0), NULL), (dict(gu=P + 8), ALIGN), (dict(dh=P + 8), ALIGN),
        (dict(dgu_pitch=68), ALIGN), (dict(h=P + 8), ALIGN)]),
    ("moe_quantize_weights", N.QuantizeWeightsArgs, QUANTIZE, SIZES[2:] + [
        (dict(transposed=2), SIZE), (dict(dtype=FP8), DTYPE), (dict(w_pitch=31), SIZE), (dict(codes_pitch=24), SIZE),
        (dict(transposed=1), SIZE), (dict(w_stride=63 * 32 + 24), SIZE), (dict(codes_stride=63 * 32 + 24), SIZE),
        (dict(w=0), NULL), (dict(codes=0), NULL), (dict(scale=0), NULL), (dict(w=P + 8), ALIGN),
        (dict(w_pitch=36, w_stride=64 * 36), ALIGN), (dict(codes=P + 4), ALIGN), (dict(codes_stride=2052), ALIGN)]),
]


@pytest.mark.parametrize("name,struct,good,cases", REFUSED, ids=[r[0] for r in REFUSED])
def test_host_refusals(lib, name, struct, good, cases):
    call = getattr(lib, name)
    assert call(None, None) == NULL
    for change, status in cases:
        assert call(C.byref(struct(**dict(good, **change))), None) == status, (name, change)


def test_no_rows_ask_for_no_addresses(lib):
    """n = 0 is not refused for what it does not read (the weights' gradient writes its zeros, so it needs dw)."""
    none = dict(x=0, out=0, w=0, offsets=0, err=0)
    assert lib.moe_expert_matmul(C.byref(N.ExpertMatmulArgs(**dict(MATMUL, n=0, **none))), None) == 0
    assert lib.moe_swiglu(C.byref(N.SwigluArgs(**dict(SWIGLU, n=0, gu=0, h=0, h_scale=0))), None) == 0
    assert lib.moe_swiglu_backward(C.byref(N.SwigluBackwardArgs(**dict(SWIGLU_B, n=0, gu=0, dh=0, dgu=0))), None) == 0


@pytest.mark.parametrize("which", range(12, 17))
def test_layouts_are_compared(lib, which):
    assert lib.moe_struct_size(which) == C.sizeof(N._STRUCTS[which])


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_what_the_kernels_cannot_address(lib):
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    x, w, o, out = _t(8, 32), _t(2, 64, 32), _t(3, dtype=i32), _t(8, 64)
    err, slot = _t(1, dtype=i32), _t(8, dtype=i32)
    x8, w8 = _t(8, 32, dtype=u8), _t(2, 64, 32, dtype=u8)
    xs, ws = _t(8, 1, dtype=f32), _t(2, 1, 1, dtype=f32)
    gu, h, dh = _t(8, 64), _t(8, 32), _t(8, 32)
    bad = [
        (lambda: M.moe_expert_matmul(x, w, o, out), "on a GPU"),
        (lambda: M.moe_expert_matmul(x.half(), w, o, out), "dtype"),
        (lambda: M.moe_expert_matmul(x.float(), w, o, out), "dtype"),
        (lambda: M.moe_expert_matmul(x, w[0], o, out), "dimensions"),
        (lambda: M.moe_expert_matmul(x[0], w, o, out), "dimensions"),
        (lambda: M.moe_expert_matmul(x, w, o.long(), out), "dtype"),
        (lambda: M.moe_expert_matmul(x, w, o[:2], out), "expected .1, 64, 32"),
        (lambda: M.moe_expert_matmul(x, w, o, out[:, :56]), "shape"),
        (lambda: M.moe_expert_matmul(x, w, o, out[:7]), "8 rows for 7"),
        (lambda: M.moe_expert_matmul(x, w.transpose(1, 2), o, _t(8, 32)), "contiguous|shape"),
        (lambda: M.moe_expert_matmul(x, w, o, out, transposed=True), "shape"),
        (lambda: M.moe_expert_matmul(x, w, o, out, row_slot=slot), "err"),
        (lambda: M.moe_expert_matmul(x8, w8, o, out), "scale"),
        (lambda: M.moe_expert_matmul(x8, w8, o, out, x_scale=xs[:7], w_scale=ws), "at least 8|shape"),
        (lambda: M.moe_expert_matmul(x8, w8, o, out, x_scale=xs, w_scale=ws[:1]), "at least 2|shape"),
        (lambda: M.moe_expert_matmul_backward(out, x, o, _t(2, 64, 24)), "shape"),
        (lambda: M.moe_expert_matmul_backward(out, x.float(), o, w), "dtype"),
        (lambda: M.moe_expert_matmul_backward(out, x[:7], o, w), "shape"),
        (lambda: M.moe_expert_matmul_backward(out, x, o, w), "on a GPU"),
        (lambda: M.moe_swiglu(gu, h), "on a GPU"),
        (lambda: M.moe_swiglu(gu, h[:, :24]), "shape"),
        (lambda: M.moe_swiglu(gu, x8), "h_scale"),
        (lambda: M.moe_swiglu(gu, x8, xs, 48), "group"),
        (lambda: M.moe_swiglu(gu, x8, xs[:7], 32), "at least 8|shape"),
        (lambda: M.moe_swiglu_backward(gu, dh.float(), gu), "dtype"),
        (lambda: M.moe_swiglu_backward(gu, dh, _t(8, 56)), "shape"),
        (lambda: M.moe_swiglu_backward(gu, dh, gu), "on a GPU"),
        (lambda: M.moe_quantize_weights(w, w8, ws), "on a GPU"),
        (lambda: M.moe_quantize_weights(w, w8, ws, transposed=True), "shape"),
        (lambda: M.moe_quantize_weights(w, w8[:, :, :24], ws), "shape"),
        (lambda: M.moe_quantize_weights(w8, w8, ws), "dtype"),
        (lambda: M.moe_quantize_weights(w, w8, ws[:1]), "at least 2|shape"),
    ]
    for call, text in bad:
        with pytest.raises(M.MoeError, match=text):
            call()


def test_layer_refusals(lib):
    def layer(E=4, H=64, I=32, K=2, dtype=BF16, T=8):
        return M.ExpertTrainLayer(E, H, I, K, dtype, T, device="cpu")

    for kw in (dict(E=0), dict(E=257), dict(K=0), dict(K=5), dict(E=64, K=33), dict(H=60), dict(I=4), dict(dtype=9),
               dict(dtype=FP8, H=72), dict(dtype=FP8, I=40), dict(T=-1), dict(T=1 << 24)):
        with pytest.raises(M.MoeError, match="ExpertTrainLayer"):
            layer(**kw)
    a = layer()
    x, l, gu, d, o = _t(8, 64), _t(8, 4, dtype=torch.float32), _t(4, 64, 64), _t(4, 64, 32), _t(8, 64)
    for args in ((_t(9, 64), _t(9, 4), gu, d, _t(9, 64)), (x, l, gu, d, o[:7]), (x, l[:, :3], gu, d, o),
                 (x, l, gu[:3], d, o), (x, l, gu, d[:, :, :24], o), (x.float(), l, gu, d, o), (x, l, gu.float(), d, o)):
        with pytest.raises(M.MoeError, match="ExpertTrainLayer"):
            a.run(*args)
    with pytest.raises(M.MoeError, match="after run"):
        a.backward(o, o, l, gu, d)
    with pytest.raises(M.MoeError, match="on a GPU"):
        a.run(x, l, gu, d, o, train=True)
    with pytest.raises(M.MoeError, match="after run"):  # that run did not come to its end
        a.backward(o, o, l, gu, d)
    b = layer(dtype=FP8)
    u8 = lambda t: t.to(torch.uint8)
    for kw in (dict(), dict(train=True, x_scale=l, s_gu=l, s_d=l)):
        with pytest.raises(M.MoeError, match="forward only"):
            b.run(u8(x), l, u8(gu), u8(d), o, **kw)
