"""The float64 definitions of the grouped products and of 4-bit weights: gradients against
central differences, codes against a search over every code."""
import numpy as np
import pytest

from oracle import grouped as G


def _case(seed, counts, n, k, T=None):
    rng = np.random.default_rng(seed)
    rows = sum(counts) + 2  # two rows behind the last segment
    offsets = np.concatenate([[0], np.cumsum(counts)])
    a_rows = None if T is None else rng.integers(0, T, rows)
    a = rng.standard_normal((rows if T is None else T, k))
    return rng, rows, offsets, a_rows, a, rng.standard_normal((len(counts), n, k))


@pytest.mark.parametrize("T", [None, 3])
def test_gradients_against_differences(T):
    rng, rows, offsets, a_rows, a, w = _case(1, [2, 0, 3, 1], 3, 4, T)
    dy = rng.standard_normal((rows, 3))
    live = slice(0, int(offsets[-1]))

    def loss(a, w):
        out, _ = G.product(a, offsets, w, rows, a_rows)
        assert np.isnan(out[offsets[-1]:]).all()
        return (dy[live] * out[live]).sum()

    drows, _ = G.data_gradient(dy, offsets, w)
    da = np.zeros(a.shape)
    for p in range(int(offsets[-1])):
        da[p if a_rows is None else a_rows[p]] += drows[p]
    dw, _ = G.weight_gradient(dy, a, offsets, w.shape[0], None, a_rows)
    h = 1e-6
    for grad, x, f in ((da, a, lambda v: loss(v, w)), (dw, w, lambda v: loss(a, v))):
        for i in np.ndindex(*x.shape):
            up, down = x.copy(), x.copy()
            up[i] += h
            down[i] -= h
            assert abs((f(up) - f(down)) / (2 * h) - grad[i]) < 1e-7
    assert not dw[1].any()
    add = rng.standard_normal(w.shape)
    np.testing.assert_allclose(G.weight_gradient(dy, a, offsets, w.shape[0], add, a_rows)[0], dw + add, atol=1e-12)


def test_segments_stay_inside():
    assert G.segments([-5, 3, 2, 99, 7], 4, 10) == [(0, 3), (3, 3), (2, 10), (10, 10)]
    assert G.segments(None, 1, 7) == [(0, 7)]


def test_pack4_takes_the_nearest_value():
    rng = np.random.default_rng(3)
    w = rng.standard_normal((40, 64)) * 2.0 ** rng.integers(-20, 20, (40, 1))
    code, scale, v = G.pack4(w)
    b, s = w.reshape(40, 2, 32), 2.0 ** (scale.astype(float) - 127)
    every = np.concatenate([G.GRID, -G.GRID]) * s[..., None]
    best = np.abs(b[..., None] - every[:, :, None, :]).min(-1)
    np.testing.assert_allclose(np.abs(b - v.reshape(40, 2, 32)), best, rtol=0, atol=0)
    top = np.abs(b).max(-1) / s
    assert ((top >= 4) & (top < 8)).all()
    np.testing.assert_array_equal(G.values4(code, scale), v)
    got = G.bytes4(code)
    np.testing.assert_array_equal(got & 15, code[:, 0::2])
    np.testing.assert_array_equal(got >> 4, code[:, 1::2])


def test_pack4_error_by_size():
    """|w - value| by the size of w in steps: a quarter of a step up to 2, half up to 4, one up to
    6, below two beyond; below a quarter of the block's largest in all."""
    rng = np.random.default_rng(8)
    w = rng.uniform(-1, 1, (500, 64)) * 2.0 ** rng.uniform(-8, 8, (500, 1))
    _, scale, v = G.pack4(w)
    step = np.repeat(2.0 ** (scale.astype(float) - 127), 32, 1)
    m, err = np.abs(w) / step, np.abs(w - v) / step
    for lo, hi, most in ((0, 2, 0.25), (2, 4, 0.5), (4, 6, 1.0), (6, 8, 2.0)):
        here = (m >= lo) & (m <= hi)
        assert here.any() and (err[here] <= most).all()
    amax = np.repeat(np.abs(w.reshape(500, 2, 32)).max(-1), 32, 1)
    assert (np.abs(w - v) < amax / 4).all()


def test_pack4_ties_and_ends():
    row = np.zeros((1, 32))
    row[0, :9] = [4.0, 0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5.0, 6.5]
    code, scale, v = G.pack4(row)
    assert scale[0, 0] == 127
    np.testing.assert_array_equal(v[0, :9], [4.0, 0.0, -1.0, 1.0, 2.0, 2.0, -4.0, 4.0, 6.0])
    for x in (0.0, 2.0 ** -149, 2.0 ** -126):
        _, scale, v = G.pack4(np.full((1, 32), x))
        assert scale[0, 0] == 1 and (v == np.where(x < 2.0 ** -128, 0.0, x)).all()
    for bad in (np.inf, -np.inf, np.nan):
        row[0, 5] = bad
        code, scale, v = G.pack4(row)
        assert scale[0, 0] == 255 and not code.any() and np.isnan(v).all()
