"""The home rank's operators at the edges of their documentation: calls and values that the other
files' cases do not reach."""
import numpy as np
import pytest
import torch

import asynchronous_moe_expert_amd as M
import workloads as W
from oracle import home as O
from test_gpu_home import HALF, I32, ROUTES, U, errword, gpu, hard_logits, like, val, within
from workloads.device import weight_tensors

pytestmark = pytest.mark.gpu

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("group", [32, 0])
@pytest.mark.parametrize("size", [1.0, 1e14])
def test_a_group_with_an_infinite_value_stands_for_nan(group, size):
    """gamma[40] infinite while r is ordinary (rows of size 1) and while it is small (1e14): every code of the
    groups that hold the column is NaN, the others' are those of a finite gamma."""
    T, H = 3, 256
    rng = np.random.default_rng(3)
    x = (size * torch.from_numpy(rng.uniform(0.5, 2, (T, H)).astype(np.float32))).cuda()
    gamma = torch.ones(H, device="cuda")
    outs = []
    for g in (1.0, float("inf")):
        gamma[40] = g
        out = torch.zeros(T, H, dtype=torch.uint8, device="cuda")
        scale = torch.zeros(T, H // group if group else 1, device="cuda")
        M.moe_residual_norm(x, None, gamma, 1e-5, out, out_scale=scale, group=group)
        outs.append(out.view(FP8).float().cpu() * scale.repeat_interleave(H // scale.shape[1], 1).cpu())
    finite, got = outs
    hit = torch.zeros(H, dtype=torch.bool)
    hit[32:64] = True
    if group == 0:
        hit[:] = True
    assert got[:, hit].isnan().all()
    assert finite.isfinite().all() and torch.equal(got[:, ~hit], finite[:, ~hit])


@pytest.mark.parametrize("out", [F32, FP8])
def test_rows_whose_squares_leave_fp32(out):
    """r is 0 for a row with an infinite h, or whose sum of squares passes fp32's range: y is 0 where h is finite
    and NaN where it is not; a NaN makes the whole row NaN.  The row beside them is as without them."""
    H = 256
    x = torch.ones(5, H, device="cuda")
    x[1, 7] = float("inf")
    x[2] = 1e25
    x[3, 9] = float("nan")
    gamma = torch.ones(H, device="cuda")
    got, rstd = torch.zeros(5, H, dtype=F32 if out == F32 else torch.uint8, device="cuda"), torch.full((5,), 9.0, device="cuda")
    scale = torch.zeros(5, H // 32, device="cuda") if out == FP8 else None
    M.moe_residual_norm(x, None, gamma, 0.0, got, rstd=rstd, out_scale=scale, group=32)
    y = got if out == F32 else got.view(FP8).float() * scale.repeat_interleave(32, 1)
    y, finite = y.cpu(), torch.ones(H, dtype=torch.bool)
    finite[7] = False
    assert rstd.cpu()[:3].tolist() == [1, 0, 0] and rstd[3].isnan()
    assert (y[1][finite] == 0).all() and y[1, 7].isnan() and (y[2] == 0).all() and y[3].isnan().all()
    # 448 codes times 1 / 448: two roundings
    assert (y[[0, 4]] - 1).abs().max() <= 2 * U


# --------------------------------------------------------------------------- the bias of the scores
def route(logits, K, **how):
    expert, w = like((logits.shape[0], K), I32, fill=-7), like((logits.shape[0], K), F32, fill=-7)
    M.moe_route(logits, expert, w, **how)
    return expert.cpu().numpy(), w


def scores_of(logits, score):
    """Every expert's gate score as moe_route rounds it: weights without renorm, 32 experts at a time, the others
    taken out of the choice by a bias of the logits; NaN where an expert cannot be chosen."""
    T, E = logits.shape
    s = np.full((T, E), np.nan, np.float32)
    for a in range(0, E, 32):
        K = min(32, E - a)
        bias = torch.full((E,), float("-inf"), device="cuda")
        bias[a:a + K] = 0
        expert, w = route(logits, K, bias=bias, score=score, renorm=False)
        t, k = np.nonzero(expert >= 0)
        s[t, expert[t, k]] = w.cpu().numpy()[t, k]
    return s


@pytest.mark.parametrize("E,K", ROUTES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", [M.MOE_SOFTMAX, M.MOE_SIGMOID])
def test_route_with_a_bias_of_the_scores(E, K, dtype, score):
    """The choice is that of fp32 score + fp32 bias, exactly, for the scores that the call itself gives as
    weights; those are off by 4 u (sigmoid: exp 2, sum and quotient 1 each) or as the weights' bounds are."""
    rng = np.random.default_rng(E * 100 + K + 7)
    for T, pad, renorm in ((1, 0, True), (77, 3, False), (50, 8, True)):
        logits = gpu(hard_logits(rng, T, E, dtype), dtype, pad)
        l = val(logits)
        s = scores_of(logits, score)
        ok = l > -np.inf
        assert np.array_equal(ok, ~np.isnan(s))
        exact = O.gate_scores(l, score)
        if score == M.MOE_SIGMOID:
            tol = 4 * U * exact
        else:
            with np.errstate(invalid="ignore", over="ignore"):
                top = np.nanmax(np.where(np.isfinite(l) & (np.abs(l) < 1e30), l, -np.inf), axis=1, keepdims=True)
                size = np.where(np.isfinite(l) & np.isfinite(top), np.minimum(np.abs(l) + np.abs(top), 1e3), 0)
            tol = exact * (60 + 4 * size) * U
        within(np.where(ok, s, 0), np.where(ok, exact, 0), tol + 1e-37)
        bias = np.round(rng.standard_normal(E) * 0.2, 2).astype(np.float32)  # some of them equal
        bias[rng.random(E) < 0.1] = -np.inf
        bias[rng.random(E) < 0.05] = np.nan
        bias[rng.random(E) < 0.05] = np.inf
        how = dict(score=score | M.MOE_BIAS_ON_SCORE, renorm=renorm, scale=2.5)
        expert, w = route(logits, K, bias=gpu(bias), **how)
        want = O.choose(l, K, bias, score | O.BIAS_ON_SCORE, gate=s)
        assert np.array_equal(expert, want)
        # the weights know nothing of the bias
        share = 2.5 * O.shares(l, want, score, renorm)
        with np.errstate(invalid="ignore", over="ignore"):
            lc = np.take_along_axis(l, np.maximum(want, 0).astype(np.int64), 1)
            top = np.nanmax(np.where(np.isfinite(l) & (np.abs(l) < 1e30), l, -np.inf), axis=1, keepdims=True)
            size = np.where(np.isfinite(lc) & np.isfinite(top), np.minimum(np.abs(lc) + np.abs(top), 1e3), 0)
        within(val(w), share, share * (60 + 4 * size) * U + 1e-37)
        # without a bias the flag changes nothing, nor does it in the gradient
        assert all(np.array_equal(a, b) for a, b in zip(
            (np.asarray(v) if isinstance(v, np.ndarray) else val(v) for v in route(logits, K, **how)),
            (np.asarray(v) if isinstance(v, np.ndarray) else val(v) for v in route(logits, K, score=score, renorm=renorm, scale=2.5))))
        dw, err = gpu(rng.standard_normal((T, K)).astype(np.float32)), errword()
        got = [like((T, E), dtype, fill=3) for _ in range(2)]
        for d, sc in zip(got, (score, how["score"])):
            M.moe_route_backward(logits, gpu(expert), dw, d, err, score=sc, renorm=renorm, scale=2.5)
        assert torch.equal(got[0], got[1])


def test_the_two_biases_by_hand():
    logits, bias = torch.tensor([[4.0, 1.0, -30.0]], device="cuda"), torch.tensor([0.0, 0.5, 0.9], device="cuda")
    for score, want in ((M.MOE_SIGMOID, [[0, 1, 2]]), (M.MOE_SIGMOID | M.MOE_BIAS_ON_SCORE, [[1, 0, 2]]),
                        (M.MOE_SOFTMAX, [[0, 1, 2]]), (M.MOE_SOFTMAX | M.MOE_BIAS_ON_SCORE, [[0, 2, 1]])):
        assert route(logits, 3, bias=bias, score=score)[0].tolist() == want


@pytest.mark.parametrize("on_score", [True, False])
def test_expert_layer_with_a_balancing_bias(on_score):
    rng = np.random.default_rng(5)
    T, E, K, H, I = 40, 8, 2, 64, 128
    wts = W.gen.make_layer_weights(rng, E, H, I, 0.05, "f32")
    w = weight_tensors(wts)
    layer = M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, T, score=M.MOE_SIGMOID, scale=2.5, bias_on_score=on_score)
    layer.load_weights(w["wg"], w["wu"], w["wd"])
    logits, bias = rng.permutation(T * E).reshape(T, E) / 64.0 - 2, rng.permutation(E) / 8.0  # no near ties
    logits, bias = logits.astype(np.float32), bias.astype(np.float32)
    x, out = gpu(rng.standard_normal((T, H)).astype(np.float32)), like((T, H), F32)
    layer.run(x, gpu(logits), out, bias=gpu(bias))
    want = O.choose(logits, K, bias, O.SIGMOID | (O.BIAS_ON_SCORE if on_score else 0))
    assert np.array_equal(layer.expert.cpu().numpy(), want)
    assert not np.array_equal(want, O.choose(logits, K, bias, O.SIGMOID | (0 if on_score else O.BIAS_ON_SCORE)))


# ----------------------------------------------------------------------------------- other streams
@pytest.mark.parametrize("raw", [True, False])
def test_a_layer_and_its_input_may_go_while_another_stream_works(raw):
    """x, the weights and the layer are dropped as soon as run() returns, behind work that keeps the side
    stream busy; what the allocator hands out meanwhile is other memory."""
    rng = np.random.default_rng(6)
    T, E, K, H, I = 64, 8, 2, 256, 256
    w = weight_tensors(W.gen.make_layer_weights(rng, E, H, I, 0.05, "f32"))
    x0, logits = gpu(rng.standard_normal((T, H)).astype(np.float32)), gpu(rng.standard_normal((T, E)).astype(np.float32))
    outs = []
    s = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for other in (False, True):
        layer = M.ExpertLayer(E, H, I, K, M.MOE_F32, M.MOE_F32, T)
        wg, wu, wd = (w[k].clone() for k in ("wg", "wu", "wd"))
        x, out = x0.clone(), torch.zeros(T, H, device="cuda")
        torch.cuda.synchronize()
        handle = None
        if other:
            with torch.cuda.stream(s):
                for _ in range(20):
                    busy @ busy
            handle = s.cuda_stream if raw else s
        layer.load_weights(wg, wu, wd, stream=handle)
        layer.run(x, logits, out, stream=handle)
        sizes = [t.numel() * t.element_size() for t in (x, wg, wu, wd, layer.w_gu, layer.w_d, layer.workspace, layer.y)]
        del layer, x, wg, wu, wd
        taken = [torch.full((n,), 0xee, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        del taken
        outs.append(out)
    assert outs[0].abs().max() > 0 and torch.equal(outs[0], outs[1])
