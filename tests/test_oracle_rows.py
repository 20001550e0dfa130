"""The float64 definitions of the row operators against differences and closed forms."""
import numpy as np
import pytest

from oracle import rows as R


def _slots(rng, T, K, N):
    """Slot positions as a counting sort leaves them, some tokens without real slots."""
    n = rng.integers(0, K + 1, T)
    expert = np.where(np.arange(K) < n[:, None], rng.permuted(np.tile(np.arange(N), (T, 1)), axis=1)[:, :K], N)
    order = np.argsort(expert.reshape(-1), kind="stable")
    pos = np.empty(T * K, int)
    pos[order] = np.arange(T * K)
    return np.where(expert < N, pos.reshape(T, K), -1)


def _central(f, a, eps=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + eps
        hi = f()
        a[i] = keep - eps
        lo = f()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("null", ["zero", "copy", "constant"])
def test_combine_gradient_matches_differences(null):
    rng = np.random.default_rng(3)
    T, K, N, d = 5, 3, 4, 8
    sp, w = _slots(rng, T, K, N), rng.random((T, K))
    rows, dy = rng.standard_normal((T * K, d)), rng.standard_normal((T, d))
    src = {"zero": None, "copy": rng.standard_normal((T, d)), "constant": rng.standard_normal(d)}[null]

    def loss():
        return float((R.combine(rows, sp, w, None, src)[0] * dy).sum())

    drows, dw, dnull, _, _ = R.combine_backward(dy, rows, sp, w, src)
    np.testing.assert_allclose(drows, _central(loss, rows), atol=1e-7)
    np.testing.assert_allclose(dw, _central(loss, w), atol=1e-7)
    if src is not None:
        np.testing.assert_allclose(dnull, _central(loss, src), atol=1e-7)


def test_gather_gradient_matches_differences():
    rng = np.random.default_rng(4)
    T, K, N, d = 4, 3, 5, 8
    sp = _slots(rng, T, K, N)
    x, dp = rng.standard_normal((T, d)), rng.standard_normal((T * K, d))
    tok = {int(sp[t, k]): t for t in range(T) for k in range(K) if sp[t, k] >= 0}

    def loss():
        return float(sum((x[t] * dp[p]).sum() for p, t in tok.items()))

    np.testing.assert_allclose(R.permute_backward(dp, sp, None)[0], _central(loss, x), atol=1e-7)


def test_swiglu_gradient_matches_differences():
    rng = np.random.default_rng(5)
    g, u, dh = (rng.standard_normal((3, 8)) * 2 for _ in range(3))
    w = rng.random(3)

    def loss():
        return float((w[:, None] * dh * R.swiglu(g, u)).sum())

    dg, du, h, dw = R.swiglu_backward(g, u, dh, w)
    np.testing.assert_allclose(dg, _central(loss, g), atol=1e-7)
    np.testing.assert_allclose(du, _central(loss, u), atol=1e-7)
    np.testing.assert_allclose(dw, _central(loss, w), atol=1e-7)
    np.testing.assert_array_equal(h, R.swiglu(g, u))


def test_act8_definition():
    x = np.zeros((4, 40))
    x[0, :4] = [1.0, -0.5, 127 / 64, 2.0 ** -7]  # amax 1.984: steps of 2^-6
    x[1, 0] = 255 / 128  # 127.5 steps of 2^-6: rounds to 128, clamped
    x[2, 33] = 5.0       # the short second block only
    x[3, 0], x[3, 35] = np.inf, np.nan
    q, s, v = R.act8(x)
    assert q[0, :4].tolist() == [64, -32, 127, 0] and s[0].tolist() == [127 - 6, 1]  # a half step ties to even 0
    assert q[1, 0] == 127 and v[1, 0] == 127 / 64
    assert s[2].tolist() == [1, 127 + 2 - 6] and v[2, 33] == 5.0 and q[2, 33] == 80
    assert s[3].tolist() == [255, 255] and np.isnan(v[3]).all() and (q[3] == 0).all()


def test_act8_error_bound():
    rng = np.random.default_rng(6)
    x = rng.standard_normal((64, 72)) * np.exp(8 * rng.standard_normal((64, 1)))
    _, s, v = R.act8(x)
    step = np.ldexp(1.0, s.astype(int) - 127).repeat(32, 1)[:, :72]
    clamped = np.abs(x) > 127.5 * step
    assert (np.abs(x - v) <= np.where(clamped, step, step / 2)).all()
