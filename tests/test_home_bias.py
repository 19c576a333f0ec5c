"""The two biases of the choice of experts: of the logits, and of the gate's scores (the balancing
bias), where the oracle's rule is held to values worked out by hand."""
import ctypes as C
import os

import numpy as np
import pytest

import asynchronous_moe_expert_amd as M
from asynchronous_moe_expert_amd import _native as N
from oracle import home as O

LOGITS = np.array([[4.0, 1.0, -30.0]], np.float32)


def test_the_two_biases_choose_differently():
    b = np.array([0.0, 0.5, 0.0])  # sigmoids 0.982, 0.731, 0.000 and the sums 0.982, 1.231, 0.000
    assert O.choose(LOGITS, 2, b, O.SIGMOID).tolist() == [[0, 1]]
    assert O.choose(LOGITS, 2, b, O.SIGMOID | O.BIAS_ON_SCORE).tolist() == [[1, 0]]
    b = np.array([0.0, 0.0, 0.9])  # softmax 0.953, 0.047, 0.000 and the sums 0.953, 0.047, 0.900
    assert O.choose(LOGITS, 3, b, O.SOFTMAX).tolist() == [[0, 1, 2]]
    assert O.choose(LOGITS, 3, b, O.SOFTMAX | O.BIAS_ON_SCORE).tolist() == [[0, 2, 1]]


def test_weights_come_from_the_scores_alone():
    s = 1 / (1 + np.exp([-4.0, -1.0]))
    e, w = O.route(LOGITS, 2, np.array([0.0, 0.5, 0.0]), O.SIGMOID | O.BIAS_ON_SCORE, False, 2.5)
    assert e.tolist() == [[1, 0]] and np.allclose(w, 2.5 * s[None, ::-1], atol=1e-15)
    _, w = O.route(LOGITS, 2, np.array([0.0, 0.5, 0.0]), O.SIGMOID | O.BIAS_ON_SCORE)
    assert np.allclose(w, s[None, ::-1] / s.sum(), atol=1e-15)


def test_what_is_never_chosen_and_equal_ranks():
    inf, nan = np.inf, np.nan
    l = np.array([[20, 30, nan, -inf, 0, 18]], np.float32)  # fp32 sigmoids of 18 and above are 1
    b = np.array([0, 0, 9, 9, -inf, 0], np.float32)
    for score in (O.SIGMOID, O.SOFTMAX):
        e = O.choose(l, 6, b, score | O.BIAS_ON_SCORE)[0].tolist()
        assert e[3:] == [-1, -1, -1] and sorted(e[:3]) == [0, 1, 5]
    assert O.choose(l, 3, b, O.SIGMOID | O.BIAS_ON_SCORE).tolist() == [[0, 1, 5]]


def test_the_flag_is_checked_on_the_host():
    from asynchronous_moe_expert_amd import build

    if not (os.path.exists(M.LIB_PATH) and os.path.exists(build.MARSHAL)):
        build.build()
    lib = M.load()
    good = dict(T=0, E=16, K=2, dtype=M.MOE_F32, pitch=16, renorm=1, scale=1.0)  # no tokens: nothing is enqueued
    for score, status in ((16, 0), (17, 0), (2, -2), (18, -2), (32, -2), (-1, -2)):
        assert lib.moe_route(C.byref(N.RouteArgs(score=score, **good)), None) == status
        assert lib.moe_route_backward(C.byref(N.RouteBackwardArgs(score=score, dlogits_pitch=16, err=4096, **good)), None) == status
    import torch

    t = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d)  # noqa: E731
    for score, text in ((17, "on a GPU"), (18, "score must be"), (-1, "score must be")):
        with pytest.raises(M.MoeError, match=text):
            M.moe_route(t(4, 16), t(4, 2, d=torch.int32), t(4, 2), score=score)


def test_expert_layer_adds_its_bias_to_the_scores():
    from asynchronous_moe_expert_amd.step import ExpertLayer

    make = lambda **k: ExpertLayer(8, 64, 64, 2, M.MOE_F32, M.MOE_F32, 4, device="cpu", **k).how["score"]  # noqa: E731
    assert make(score=M.MOE_SIGMOID) == M.MOE_SIGMOID | M.MOE_BIAS_ON_SCORE
    assert make(score=M.MOE_SIGMOID, bias_on_score=False) == M.MOE_SIGMOID
