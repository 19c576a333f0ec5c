"""The products' oracle against loops over its formulas' indexes and central differences."""
import numpy as np
import pytest

from oracle import products as O


def test_products_by_index():
    rng = np.random.default_rng(0)
    n, E, N, D, T = 9, 4, 5, 6, 4
    offsets = np.array([0, 3, 3, 8, 8])  # an empty expert in the middle and at the end, row 8 has none
    x, w, slot = rng.standard_normal((T, D)), rng.standard_normal((E, N, D)), rng.integers(-1, T + 1, n)
    out = O.expert_matmul(x, w, offsets, n, slot)
    xs = np.array([x[s] if 0 <= s < T else np.zeros(D) for s in slot])
    for r in range(n):
        e = [k for k in range(E) if offsets[k] <= r < offsets[k + 1]]
        for j in range(N):
            want = sum(w[e[0], j, d] * xs[r, d] for d in range(D)) if e else np.nan
            assert np.isclose(out[r, j], want, rtol=1e-12, atol=1e-12, equal_nan=True)
    assert np.allclose(O.expert_matmul(xs, w, offsets, n), out, equal_nan=True)
    dout = rng.standard_normal((n, N))
    dw = O.expert_matmul_backward(dout, xs, offsets)
    dxs = O.expert_matmul(dout, w, offsets, n, transposed=True)
    assert not dw[1].any() and not dw[3].any()
    step = 1e-6

    def loss(x_, w_):
        return np.nansum(O.expert_matmul(x_, w_, offsets, n) * dout)

    for e, j, d in [(0, 1, 2), (2, 4, 5), (2, 0, 0), (1, 3, 3)]:
        up, down = w.copy(), w.copy()
        up[e, j, d] += step
        down[e, j, d] -= step
        assert abs((loss(xs, up) - loss(xs, down)) / (2 * step) - dw[e, j, d]) < 1e-7
    for r, d in [(0, 0), (5, 3), (7, 5)]:
        up, down = xs.copy(), xs.copy()
        up[r, d] += step
        down[r, d] -= step
        assert abs((loss(up, w) - loss(down, w)) / (2 * step) - dxs[r, d]) < 1e-7
    assert np.isnan(dxs[8]).all()


@pytest.mark.parametrize("offsets,want", [([0, 4, 2, 9], [(0, 4), (4, 4), (2, 6)]), ([-3, 2, 100, 5], [(0, 2), (2, 6), (6, 6)])])
def test_offsets_are_cut(offsets, want):
    assert list(O.spans(offsets, 6)) == want


def test_swiglu_by_difference():
    rng = np.random.default_rng(1)
    gu, dh = rng.standard_normal((4, 10)) * 3, rng.standard_normal((4, 5))
    gu[0, 0], gu[1, 1] = 0.0, -60.0
    d, step = O.swiglu_backward(gu, dh), 1e-6
    for r in range(4):
        for c in range(10):
            up, down = gu.copy(), gu.copy()
            up[r, c] += step
            down[r, c] -= step
            assert abs(((O.swiglu(up) - O.swiglu(down)) * dh).sum() / (2 * step) - d[r, c]) < 1e-7
    assert np.isclose(O.swiglu(np.array([[np.log(3.0), 2.0]]))[0, 0], np.log(3) * 0.75 * 2)


def test_scales():
    w = np.zeros((130, 260))
    w[5, 130], w[129, 259] = -896.0, 1e-44
    s = O.block_scales(w)
    assert s.shape == (2, 3) and s[0, 1] == 2 and s[0, 0] == 1 and s[1, 2] == 2.0 ** -126
    v = O.scaled(np.ones((130, 260)), s, 128)
    assert v[127, 128] == 2 and v[128, 127] == 1 and v[129, 256] == 2.0 ** -126
