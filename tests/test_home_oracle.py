"""The fp64 oracle of the home rank's operators against hand-computed values and, for the
gradients, against central differences.

The differences' step is 1e-5: their own error is about |f'''| 1e-10 / 6 from the formula and
2^-53 |f| / 1e-5 = 1e-11 |f| from the subtraction, so 1e-7 covers both for values of order 1."""
import numpy as np
import pytest

from oracle import home as O

STEP, TOL = 1e-5, 1e-7


def differences(f, x):
    """The gradient of the scalar f at x, entry by entry."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        at = x[i]
        x[i] = at + STEP
        hi = f(x)
        x[i] = at - STEP
        lo = f(x)
        x[i] = at
        g[i] = (hi - lo) / (2 * STEP)
    return g


def test_choice_by_hand():
    inf, nan = np.inf, np.nan
    logits = np.array([[1, 3, 3, 2], [nan, -inf, 0, nan], [-inf, nan, -inf, nan], [-0.0, 0.0, -1, -2],
                       [0, inf, 5, inf]], np.float32)
    assert O.choose(logits, 3).tolist() == [[1, 2, 3], [2, -1, -1], [-1, -1, -1], [0, 1, 2], [1, 3, 2]]
    assert O.choose(logits[:1], 2, bias=np.array([10, 0, -inf, 0])).tolist() == [[0, 1]]
    e, w = O.route(logits, 3)
    assert np.allclose(w[0], np.exp([0, 0, -1]) / (2 + np.exp(-1)), atol=1e-15)
    assert w[1].tolist() == [1, 0, 0] and w[2].tolist() == [0, 0, 0] and w[4].tolist() == [0.5, 0.5, 0]
    _, w = O.route(logits[:1], 2, renorm=False, scale=2.0)
    assert np.allclose(w[0], 2 * np.exp([3, 3]) / np.exp([1, 3, 3, 2]).sum(), atol=1e-15)
    _, w = O.route(np.array([[0.0, -200.0, -201.0]]), 3, score=O.SIGMOID)
    assert np.allclose(w[0], [1, 2 * np.exp(-200), 2 * np.exp(-201)], rtol=1e-12)
    _, w = O.route(np.array([[-1000.0, -1001.0]]), 2, score=O.SIGMOID)  # both sigmoids are 0 in fp64
    assert np.allclose(w[0], np.array([1, np.exp(-1)]) / (1 + np.exp(-1)), rtol=1e-12)


@pytest.mark.parametrize("score", [O.SOFTMAX, O.SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient(score, renorm):
    rng = np.random.default_rng(3)
    l, dw = rng.standard_normal((5, 7)), rng.standard_normal((5, 3))
    expert = O.choose(l, 3)
    expert[1, 2] = -1
    f = lambda x: (dw * 1.7 * O.shares(x, expert, score, renorm)).sum()  # noqa: E731
    got = O.route_backward(l, expert, dw, score, renorm, 1.7)
    assert np.abs(got - differences(f, l.copy())).max() <= TOL


def test_sort_by_hand():
    expert = np.array([[4, 3], [-1, 4], [9, 3]])
    perm, pos, counts, offsets, slot, bad = O.sort_index(expert, 2, expert_base=3)
    assert perm.tolist() == [1, 5, 0, 3, -1, -1] and pos.tolist() == [2, 0, -1, 3, -1, 1]
    assert counts.tolist() == [2, 2] and offsets.tolist() == [0, 2, 4] and slot.tolist() == [0, 2, 0, 1, -1, -1]
    assert bad and not O.sort_index(expert[:2], 2, expert_base=3)[5]


def test_merge_and_its_gradients():
    rng = np.random.default_rng(4)
    rows, w, dout = rng.standard_normal((9, 4)), rng.standard_normal((3, 3)), rng.standard_normal((3, 4))
    pos = np.array([[4, -1, 0], [-1, -1, -1], [8, 2, 3]])
    out = O.merge_rows(rows, pos, w)
    assert np.allclose(out[0], w[0, 0] * rows[4] + w[0, 2] * rows[0], atol=1e-15) and not out[1].any()
    drows, dw = O.merge_rows_backward(dout, rows, pos, w)
    assert np.abs(drows - differences(lambda r: (dout * O.merge_rows(r, pos, w)).sum(), rows.copy())).max() <= TOL
    assert np.abs(dw - differences(lambda a: (dout * O.merge_rows(rows, pos, a)).sum(), w.copy())).max() <= TOL


def test_gradient_of_sorted_rows_is_a_merge():
    rng = np.random.default_rng(5)
    expert = np.array([[1, 0, 2], [2, -1, 1]])
    perm, pos, *_ = O.sort_index(expert, 3)
    x, dxs = rng.standard_normal((2, 4)), rng.standard_normal((6, 4))
    f = lambda v: (dxs[:5] * v[perm[:5] // 3]).sum()  # noqa: E731
    assert np.abs(O.merge_rows(dxs, pos.reshape(2, 3)) - differences(f, x.copy())).max() <= TOL


def test_norm_and_its_gradients():
    rng = np.random.default_rng(6)
    x, res, gamma, dout, dres = (rng.standard_normal(s) for s in ((3, 8), (3, 8), 8, (3, 8), (3, 8)))
    y, h, r = O.residual_norm(x, res, gamma, 1e-3)
    assert np.allclose(r, 1 / np.sqrt(((x + res) ** 2).mean(1) + 1e-3), atol=1e-15)
    dh, dgamma = O.residual_norm_backward(dout, h, gamma, r, dres)
    f = lambda a, b, g: (dout * O.residual_norm(a, b, g, 1e-3)[0]).sum() + (dres * (a + b)).sum()  # noqa: E731
    assert np.abs(dh - differences(lambda a: f(a, res, gamma), x.copy())).max() <= TOL
    assert np.abs(dh - differences(lambda a: f(x, a, gamma), res.copy())).max() <= TOL
    assert np.abs(dgamma - differences(lambda a: f(x, res, a), gamma.copy())).max() <= TOL


def test_group_scales_by_hand():
    y = np.array([[448.0, -896.0, 0, 0, 1e-50, 0]])
    assert O.group_scales(y, 0).tolist() == [[2.0]]
    assert O.group_scales(y, 2).tolist() == [[2.0, 1.0, 2.0 ** -126]]
    assert O.group_scales(y, 4).shape == (1, 2)  # the last group is shorter
