"""Float64 definitions of the row operators around the experts: the weighted way back
from expert order with its gradient, the gradient of the gather, 8-bit activation
checkpoints and the SwiGLU on them. NumPy only; imports nothing of the library.

Formulas: paper review of arXiv:2601.15370, section 3, core formula
y_t = E_shared(x_t) + sum_k g_k E_{i_k}(x_t) with null slots that output zero, the
token (copy) or a vector (constant); SwiGLU from the primer's section 2.
"""
import numpy as np

BLOCK = 32


def _slot_row(rows, slot_pos, null_src, t, k):
    p = slot_pos[t, k]
    if 0 <= p < rows.shape[0]:
        return rows[p]
    if p == -1 and null_src is not None:
        return null_src[t] if null_src.ndim == 2 else null_src
    return None


def combine(rows, slot_pos, topk_w, shared, null_src):
    """y and, per element, the sum of its terms' magnitudes."""
    T, K = slot_pos.shape
    d = rows.shape[1]
    y = np.zeros((T, d)) if shared is None else shared.astype(np.float64).copy()
    mag = np.abs(y)
    for t in range(T):
        for k in range(K):
            r = _slot_row(rows, slot_pos, null_src, t, k)
            if r is not None:
                y[t] += topk_w[t, k] * r
                mag[t] += np.abs(topk_w[t, k] * r)
    return y, mag


def combine_backward(dy, rows, slot_pos, topk_w, null_src):
    """Gradients of <dy, combine(...)>: rows, topk_w, null_src (None without one); and the
    magnitude sums of the weights' and the null source's gradients."""
    T, K = slot_pos.shape
    drows, dw, mag = np.zeros(rows.shape), np.zeros((T, K)), np.zeros((T, K))
    dnull = None if null_src is None else np.zeros(null_src.shape)
    dnull_mag = None if null_src is None else np.zeros(null_src.shape)
    for t in range(T):
        for k in range(K):
            p = slot_pos[t, k]
            r = _slot_row(rows, slot_pos, null_src, t, k)
            if r is None:
                continue
            dw[t, k] = np.dot(dy[t], r)
            mag[t, k] = np.dot(np.abs(dy[t]), np.abs(r))
            if p >= 0:
                drows[p] += topk_w[t, k] * dy[t]
            elif null_src.ndim == 2:
                dnull[t] += topk_w[t, k] * dy[t]
                dnull_mag[t] += np.abs(topk_w[t, k] * dy[t])
            else:
                dnull += topk_w[t, k] * dy[t]
                dnull_mag += np.abs(topk_w[t, k] * dy[t])
    return drows, dw, dnull, mag, dnull_mag


def permute_backward(drows, slot_pos, add):
    """Gradient of x_perm[p] = x[token of p], on top of add; and the magnitude sums."""
    return combine(drows, slot_pos, np.ones(slot_pos.shape), add, None)


def act8(x):
    """(codes, scale bytes, values) of the 8-bit checkpoint of x [rows][cols], block by
    block from the definition."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    q, s, v = np.zeros((rows, cols), np.int8), np.zeros((rows, nb), np.uint8), np.zeros((rows, cols))
    for r in range(rows):
        for b in range(nb):
            sl = slice(b * BLOCK, min(cols, (b + 1) * BLOCK))
            blk = x[r, sl]
            if not np.isfinite(blk).all():
                s[r, b], v[r, sl] = 255, np.nan
                continue
            amax = np.abs(blk).max()
            k = int(np.frexp(amax)[1]) - 1 if amax > 0 else -1000  # floor(log2 amax)
            e = max(k - 6, -126)
            code = np.clip(np.rint(np.ldexp(blk, -e)), -127, 127)
            q[r, sl], s[r, b], v[r, sl] = code.astype(np.int8), e + 127, np.ldexp(code, e)
    return q, s, v


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_backward(z, u, dh, w=None):
    """dg, du, h and dw = <dh, h> per row, of h = silu(z) u, with dh scaled by w in dg, du."""
    s = sigmoid(z)
    h = z * s * u
    d = dh if w is None else dh * w[:, None]
    return d * u * (s * (1.0 + z * (1.0 - s))), d * z * s, h, (dh * h).sum(1)
