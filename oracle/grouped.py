"""Float64 definitions of the grouped expert products with their gradients, and of 4-bit
weights. NumPy only; imports nothing of the library.

Formulas: the experts' contractions of the paper review of arXiv:2601.15370, section 3
("implementation": a grouped product over the expert-sorted rows), SwiGLU from the primer's
section 2; 4-bit weights are OCP microscaling's e2m1 in blocks of 32.
"""
import numpy as np

BLOCK = 32
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def segments(offsets, groups, rows):
    """[(start, end)] of the groups, clamped into [0, rows]."""
    if offsets is None:
        return [(0, rows)]
    out = []
    for e in range(groups):
        a = min(max(int(offsets[e]), 0), rows)
        out.append((a, min(max(int(offsets[e + 1]), a), rows)))
    return out


def _source(a, a_rows, lo, hi):
    return a[lo:hi] if a_rows is None else a[np.clip(a_rows[lo:hi], 0, a.shape[0] - 1)]


def product(a, offsets, w, rows, a_rows=None):
    """out [rows][n] (NaN in rows of no segment) and, per element, the sum of its terms'
    magnitudes."""
    out = np.full((rows, w.shape[1]), np.nan)
    mag = np.zeros(out.shape)
    for e, (lo, hi) in enumerate(segments(offsets, w.shape[0], rows)):
        x = _source(a, a_rows, lo, hi)
        out[lo:hi] = x @ w[e].T
        mag[lo:hi] = np.abs(x) @ np.abs(w[e]).T
    return out, mag


def data_gradient(dy, offsets, w):
    """Gradient of <dy, product(...)> for the rows that go into it, and its terms' magnitudes."""
    return product(dy, offsets, w.transpose(0, 2, 1), dy.shape[0])


def weight_gradient(dy, a, offsets, groups, add=None, a_rows=None):
    """Gradient of <dy, product(...)> for the weights, added to `add`, and its terms'
    magnitudes."""
    out = np.zeros((groups, dy.shape[1], a.shape[1])) if add is None else add.astype(np.float64).copy()
    mag = np.abs(out)
    for e, (lo, hi) in enumerate(segments(offsets, groups, dy.shape[0])):
        x = _source(a, a_rows, lo, hi)
        out[e] += dy[lo:hi].T @ x
        mag[e] += np.abs(dy[lo:hi]).T @ np.abs(x)
    return out, mag


def swiglu(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def pack4(w):
    """(codes [rows][cols] 0..15, scale bytes [rows][cols / 32], values) of w [rows][cols]."""
    rows, cols = w.shape
    b = w.reshape(rows, cols // BLOCK, BLOCK).astype(np.float64)
    amax = np.abs(b).max(axis=2)
    finite = np.isfinite(amax)
    safe = np.where(finite & (amax > 0), amax, 1.0)
    e = np.where(amax > 0, np.maximum(np.frexp(safe)[1] - 1 - 2, -126), -126)
    m = np.abs(np.where(finite[..., None], b, 0.0)) * 2.0 ** -e.astype(np.float64)[..., None]
    # distance to every grid value; of two equally near the one with the even index
    dist = np.abs(m[..., None] - GRID)
    best = dist.min(axis=-1, keepdims=True)
    near = dist == best
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[np.argmax(near[..., order], axis=-1)]
    code = np.where(finite[..., None], code | (np.signbit(b) << 3), 0)
    scale = np.where(finite, e + 127, 255)
    return (code.reshape(rows, cols).astype(np.uint8), scale.astype(np.uint8),
            values4(code.reshape(rows, cols), scale))


def values4(codes, scales):
    """float64 values that codes [..., cols] (one a column) and scale bytes stand for."""
    mag = GRID[codes & 7]
    v = np.where(codes & 8, -mag, mag)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, axis=-1)


def bytes4(codes):
    """Codes, one a column, as the bytes that hold them (even columns in the low half)."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
