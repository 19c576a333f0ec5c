"""Refusals of the home rank's operators: the C entry points' host checks (they return before
anything is enqueued, so made-up addresses do) and the binding's checks of its tensors."""
import ctypes as C
import os

import pytest
import torch

import asynchronous_moe_expert_amd as M
from asynchronous_moe_expert_amd import _native as N

NULL, SIZE, DTYPE, ALIGN, SHAPE, WORKSPACE = -1, -2, -3, -4, -5, -6
P = 4096  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    from asynchronous_moe_expert_amd import build

    if not (os.path.exists(M.LIB_PATH) and os.path.exists(build.MARSHAL)):
        build.build()
    return M.load()


ROUTE = dict(T=4, E=16, K=2, logits=P, dtype=M.MOE_F32, pitch=16, score=0, renorm=1, scale=1.0, expert=P, w=P)
ROUTE_B = dict(T=4, E=16, K=2, logits=P, dtype=M.MOE_F32, pitch=16, score=0, renorm=1, scale=1.0, expert=P, dw=P,
               dlogits=P, dlogits_pitch=16, err=P)
SORT = dict(T=4, K=2, H=64, expert_base=0, E_loc=8, expert=P, x=P, x_dtype=M.MOE_BF16, x_pitch=64, xs=P, xs_pitch=64,
            perm=P, pos=P, counts=P, offsets=P, row_slot=P, err=P, workspace=P, workspace_bytes=1 << 20)
MERGE = dict(T=4, K=2, H=64, rows=P, row_dtype=M.MOE_BF16, row_pitch=64, n_rows=8, pos=P, w=P, out=P,
             out_dtype=M.MOE_BF16, out_pitch=64, err=P)
MERGE_B = dict(T=4, K=2, H=64, dout=P, dout_dtype=M.MOE_BF16, dout_pitch=64, rows=P, row_dtype=M.MOE_BF16,
               row_pitch=64, n_rows=8, pos=P, w=P, drows=P, drows_pitch=64, dw=P, err=P)
NORM = dict(T=4, H=64, x=P, x_dtype=M.MOE_BF16, x_pitch=64, residual=P, res_dtype=M.MOE_BF16, res_pitch=64, gamma=P,
            gamma_dtype=M.MOE_F32, eps=1e-5, out=P, out_dtype=M.MOE_FP8_E4M3, out_pitch=64, out_scale=P, group=32,
            residual_out=P, res_out_pitch=64)
NORM_B = dict(T=4, H=64, dout=P, dtype=M.MOE_BF16, dout_pitch=64, h=P, h_dtype=M.MOE_BF16, h_pitch=64, gamma=P,
              gamma_dtype=M.MOE_BF16, rstd=P, dres=P, dres_pitch=64, dx=P, dx_pitch=64, dresidual=P,
              dresidual_pitch=64, dgamma=P, workspace=P, workspace_bytes=1 << 20)

BIG = (1 << 24) + 1
REFUSED = [
    ("moe_route", N.RouteArgs, ROUTE, [
        (dict(T=-1), SIZE), (dict(T=BIG), SIZE), (dict(T=1 << 23, K=4), SIZE), (dict(E=0), SIZE),
        (dict(E=513, pitch=513), SIZE), (dict(K=0), SIZE), (dict(K=17), SIZE), (dict(E=64, pitch=64, K=33), SIZE),
        (dict(pitch=15), SIZE), (dict(dtype=M.MOE_FP8_E4M3), DTYPE), (dict(score=2), SIZE), (dict(renorm=2), SIZE),
        (dict(logits=0), NULL), (dict(expert=0), NULL), (dict(w=0), NULL), (dict(logits=P + 2), ALIGN)]),
    ("moe_route_backward", N.RouteBackwardArgs, ROUTE_B, [
        (dict(K=33), SIZE), (dict(dtype=7), DTYPE), (dict(dlogits_pitch=15), SIZE), (dict(err=0), NULL),
        (dict(dw=0), NULL), (dict(dlogits=0), NULL), (dict(dlogits=P + 1), ALIGN)]),
    ("moe_sort_rows", N.SortRowsArgs, SORT, [
        (dict(T=-1), SIZE), (dict(K=0), SIZE), (dict(K=33), SIZE), (dict(T=BIG), SIZE), (dict(T=1 << 23, K=3), SIZE),
        (dict(E_loc=0), SIZE), (dict(E_loc=257), SIZE), (dict(H=0), SIZE), (dict(H=(1 << 16) + 8), SIZE),
        (dict(H=60), SHAPE), (dict(x_dtype=9), DTYPE), (dict(x_pitch=56), SIZE), (dict(xs_pitch=8), SIZE),
        (dict(x_pitch=68), ALIGN), (dict(x=P + 8), ALIGN), (dict(xs=P + 2), ALIGN), (dict(expert=0), NULL),
        (dict(pos=0), NULL), (dict(counts=0), NULL), (dict(offsets=0), NULL), (dict(err=0), NULL), (dict(x=0), NULL),
        (dict(x_dtype=M.MOE_FP8_E4M3), NULL), (dict(x_dtype=M.MOE_FP8_E4M3, x_scale=P, group=48), SIZE),
        (dict(x_dtype=M.MOE_FP8_E4M3, x_scale=P, x_pitch=68), ALIGN)]),
    ("moe_merge_rows", N.MergeRowsArgs, MERGE, [
        (dict(K=33), SIZE), (dict(n_rows=-1), SIZE), (dict(H=12), SHAPE), (dict(row_dtype=M.MOE_FP8_E4M3), DTYPE),
        (dict(out_dtype=5), DTYPE), (dict(row_pitch=63), SIZE), (dict(out_pitch=72 + 4), ALIGN), (dict(rows=0), NULL),
        (dict(pos=0), NULL), (dict(out=0), NULL), (dict(err=0), NULL), (dict(out=P + 4), ALIGN)]),
    ("moe_merge_rows_backward", N.MergeRowsBackwardArgs, MERGE_B, [
        (dict(T=BIG), SIZE), (dict(H=4), SHAPE), (dict(dout_dtype=M.MOE_FP8_E4M3), DTYPE), (dict(dw=0, drows=0), NULL),
        (dict(rows=0), NULL), (dict(dout=0), NULL), (dict(pos=0), NULL), (dict(err=0), NULL),
        (dict(drows_pitch=60), SIZE), (dict(drows=P + 8), ALIGN), (dict(dout_pitch=68), ALIGN)]),
    ("moe_residual_norm", N.ResidualNormArgs, NORM, [
        (dict(T=-1), SIZE), (dict(T=BIG), SIZE), (dict(H=0), SIZE), (dict(H=16392), SIZE), (dict(H=60), SHAPE),
        (dict(eps=-1.0), SIZE), (dict(eps=float("nan")), SIZE), (dict(x_dtype=M.MOE_F32), DTYPE),
        (dict(gamma_dtype=M.MOE_FP8_E4M3), DTYPE), (dict(out_dtype=4), DTYPE), (dict(group=16), SIZE),
        (dict(out_scale=0), NULL), (dict(x=0), NULL), (dict(gamma=0), NULL), (dict(out=0), NULL),
        (dict(row_list=P), NULL), (dict(row_count=P), NULL), (dict(row_list=P, row_count=P), NULL),
        (dict(res_pitch=60), SIZE), (dict(res_out_pitch=60), SIZE), (dict(residual=P + 8), ALIGN),
        (dict(gamma=P + 4), ALIGN), (dict(out=P + 4), ALIGN), (dict(x_pitch=68), ALIGN)]),
    ("moe_residual_norm_backward", N.ResidualNormBackwardArgs, NORM_B, [
        (dict(T=BIG), SIZE), (dict(H=16392), SIZE), (dict(H=4), SHAPE), (dict(dtype=M.MOE_F32), DTYPE),
        (dict(gamma_dtype=2), DTYPE), (dict(dx=0, dresidual=0, dgamma=0), NULL), (dict(dout=0), NULL),
        (dict(h=0), NULL), (dict(rstd=0), NULL), (dict(gamma=0), NULL), (dict(dres_pitch=60), SIZE),
        (dict(dx=P + 8), ALIGN), (dict(workspace=0), WORKSPACE), (dict(workspace_bytes=512 * 64 * 4 - 1), WORKSPACE),
        (dict(workspace=P + 8), ALIGN)]),
]


@pytest.mark.parametrize("name,struct,good,cases", REFUSED, ids=[r[0] for r in REFUSED])
def test_host_refusals(lib, name, struct, good, cases):
    call = getattr(lib, name)
    assert call(None, None) == NULL
    for change, status in cases:
        assert call(C.byref(struct(**dict(good, **change))), None) == status, (name, change)


def test_workspace_refusals_of_long_queues(lib):
    need = M.moe_sort_rows_workspace_size(1 << 20)
    assert 0 < need <= 1 << 18
    for change in (dict(workspace=0), dict(workspace_bytes=need - 1)):
        a = N.SortRowsArgs(**dict(SORT, T=1 << 19, K=2, **change))
        assert lib.moe_sort_rows(C.byref(a), None) == WORKSPACE
    a = N.SortRowsArgs(**dict(SORT, T=1 << 19, K=2, workspace=P + 4))
    assert lib.moe_sort_rows(C.byref(a), None) == ALIGN
    a = N.SortRowsArgs(**dict(SORT, T=2049, K=1, workspace=0))
    assert lib.moe_sort_rows(C.byref(a), None) == WORKSPACE
    assert M.moe_sort_rows_workspace_size(0) == M.moe_sort_rows_workspace_size(2048) == 0 and M.moe_sort_rows_workspace_size(1 << 24) <= 1 << 18
    assert M.moe_residual_norm_backward_workspace_size(2880) == 2048 * 2880


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_what_the_kernels_cannot_address(lib):
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    err = _t(1, dtype=i32)
    e, w, l = _t(4, 2, dtype=i32), _t(4, 2, dtype=f32), _t(4, 16, dtype=f32)
    bad = [
        (lambda: M.moe_route(l, e, w), "on a GPU"),
        (lambda: M.moe_route(l.double(), e, w), "dtype"),
        (lambda: M.moe_route(l[0], e, w), "dimensions"),
        (lambda: M.moe_route(l, e.long(), w), "dtype"),
        (lambda: M.moe_route(l, e[:3], w), "shape"),
        (lambda: M.moe_route(l, _t(2, 4, dtype=i32).t(), w), "contiguous"),
        (lambda: M.moe_route(_t(16, 4, dtype=f32).t(), e, w), "contiguous"),
        (lambda: M.moe_route(l[:1].expand(4, 16), e, w), "overlap"),
        (lambda: M.moe_route(l, e, w, bias=_t(15, dtype=f32)), "at least 16"),
        (lambda: M.moe_route(l, e, w, score=2), "score"),
        (lambda: M.moe_route_backward(l, e, w, _t(4, 16), err), "dtype"),
        (lambda: M.moe_route_backward(l, e, w, _t(4, 15, dtype=f32), err), "shape"),
        (lambda: M.moe_merge_rows(_t(8, 64), e, w, _t(4, 72), err), "shape"),
        (lambda: M.moe_merge_rows(_t(8, 64), _t(7, dtype=i32), w, _t(4, 64), err), "whole number"),
        (lambda: M.moe_merge_rows(_t(8, 64), e, w[:3].contiguous(), _t(4, 64), err), "w"),
        (lambda: M.moe_merge_rows(_t(8, 64, dtype=torch.float16), e, w, _t(4, 64), err), "dtype"),
        (lambda: M.moe_merge_rows_backward(_t(4, 64), None, e, w, None, None, err), "must be given"),
        (lambda: M.moe_merge_rows_backward(_t(4, 64), None, e, w, _t(8, 64), w, err), "must be given"),
        (lambda: M.moe_merge_rows_backward(_t(4, 64), _t(8, 64), e, w, _t(8, 64, dtype=f32), w, err), "dtype"),
        (lambda: M.moe_residual_norm(_t(4, 64), _t(4, 64), _t(64), 1e-5, _t(4, 64, dtype=torch.uint8)), "out_scale"),
        (lambda: M.moe_residual_norm(_t(4, 64), _t(3, 64), _t(64), 1e-5, _t(4, 64)), "shape"),
        (lambda: M.moe_residual_norm(_t(4, 64), None, _t(56), 1e-5, _t(4, 64)), "at least 64"),
        (lambda: M.moe_residual_norm(_t(4, 64), None, _t(64), 1e-5, _t(4, 64, dtype=torch.uint8),
                                     out_scale=w, group=40), "group"),
        (lambda: M.moe_residual_norm(_t(4, 64), None, _t(64), 1e-5, _t(4, 64), row_list=e[0], row_count=err), "at least 4"),
        (lambda: M.moe_residual_norm_backward(_t(4, 64), _t(4, 64), _t(64), _t(4, dtype=f32), _t(4, 64, dtype=f32),
                                              None, None), "dtype"),
        (lambda: M.moe_residual_norm_backward(_t(4, 64), _t(4, 64), _t(64), _t(3, dtype=f32), _t(4, 64), None, None),
         "at least 4"),
    ]
    n = 8

    def sort(expert=e, x=_t(4, 64), xs=_t(n, 64), pos=_t(n, dtype=i32), counts=_t(8, dtype=i32), E=8, **kw):
        M.moe_sort_rows(expert, E, x, xs, None, pos, counts, _t(9, dtype=i32), err, _t(1 << 18, dtype=torch.uint8), **kw)

    bad += [(lambda: sort(), "on a GPU"), (lambda: sort(x=None), "x: required"), (lambda: sort(xs=_t(n - 1, 64)), "shape"),
            (lambda: sort(pos=_t(n - 1, dtype=i32)), "at least 8"), (lambda: sort(E=12), "at least 12"),
            (lambda: sort(x=_t(4, 64, dtype=torch.uint8)), "x_scale"), (lambda: sort(xs=_t(n, 64, dtype=f32)), "dtype"),
            (lambda: sort(x=_t(4, 64, dtype=torch.uint8), x_scale=_t(4, 1, dtype=f32), group=32), "at least 8"),
            (lambda: sort(expert_base=1 << 40), "limits"), (lambda: sort(expert=_t(8, dtype=i32)), "dimensions")]
    for call, text in bad:
        with pytest.raises(M.MoeError, match=text):
            call()
