"""Row operators at the ends of what their documentation allows: the widest rows, more
work than one pass of the largest grid, slots and rows outside the outputs, and blocks
that are not finite. Tolerances as in tests/test_gpu_rows.py."""
import numpy as np
import pytest
import torch

import token_choice_routing_amd as tcr
from oracle import rows as R
from tests.gpu_util import say
from tests.test_gpu_rows import U, _swiglu_tol, _within, host

pytestmark = pytest.mark.gpu


# Widths whose count of scale bytes, cols / 32 rounded up, needs more than 32 bits on the
# way (cols + 31): 16 columns per lane and step, and 8 with a last block of 24.
WIDE = [2 ** 31 - 16, 2 ** 31 - 8]


def _wide(cols, seed):
    """[2][cols] half zeros with a few blocks of values, their (row, first column, width),
    and the values as float64."""
    x = torch.zeros((2, cols), dtype=torch.float16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    last = (cols - 1) // 32 * 32
    at = [(r, c, min(32, cols - c)) for r in range(2) for c in (0, 2 ** 30, last - 32, last)]
    for r, c, n in at:
        x[r, c:c + n] = torch.randn((n,), generator=gen, device="cuda").half()
    return x, at


def _pieces(t, at):
    return [host(t[r, c:c + n])[None] for r, c, n in at]


def _scales_are(scales, at, ref):
    """Scale bytes of the blocks with values; 1 (step 2^-126) in every block of zeros."""
    for (r, c, _), (_, s, _) in zip(at, ref):
        assert int(scales[r, c // 32]) == int(s[0, 0]), (r, c)
    others = scales.clone()
    for r, c, _ in at:
        others[r, c // 32] = 1
    assert bool((others == 1).all())


@pytest.mark.parametrize("cols", WIDE)
def test_act8_of_the_widest_rows(cols):
    say(f"  act8 2 x {cols}")
    x, at = _wide(cols, 1)
    ref = [R.act8(p) for p in _pieces(x, at)]
    codes = torch.full((2, cols), 99, dtype=torch.int8, device="cuda")
    scales = torch.full(tcr.act8_scales_shape(2, cols), 99, dtype=torch.uint8, device="cuda")
    tcr.moe_act8_pack(x, codes, scales)
    _scales_are(scales, at, ref)
    for p, (q, _, _) in zip(_pieces(codes, at), ref):
        np.testing.assert_array_equal(p, q)
    x.fill_(7.0)
    tcr.moe_act8_unpack(codes, scales, x)
    for p, (_, _, v), (r, c, n) in zip(_pieces(x, at), ref, at):
        np.testing.assert_array_equal(p, v)
        x[r, c:c + n] = 0.0
    assert bool((x == 0).all())


@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu8_of_the_widest_rows(weighted):
    cols = WIDE[1]
    say(f"  swiglu8 2 x {cols} weighted {weighted}")
    (g, at), (u, _), (dh, _) = (_wide(cols, s) for s in (2, 3, 4))
    z, v, d = _pieces(g, at), _pieces(u, at), _pieces(dh, at)
    codes = [torch.full((2, cols), 99, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.full(tcr.act8_scales_shape(2, cols), 99, dtype=torch.uint8, device="cuda") for _ in range(2)]
    h = torch.full_like(g, 7.0)
    tcr.moe_swiglu_keep8(g, u, h, codes[0], scales[0], codes[1], scales[1])
    for i, p in enumerate(_pieces(h, at)):
        ref = R.swiglu(z[i], v[i])
        _within(torch.from_numpy(p), ref, _swiglu_tol(z[i], np.abs(ref), ref, "f16"), "h")
    z, v = [R.act8(p) for p in z], [R.act8(p) for p in v]
    for s, ref in zip(scales, (z, v)):
        _scales_are(s, at, ref)
    dg, du = g, u  # (their values are kept above)
    w = torch.tensor([0.75, -1.5], device="cuda")
    dw = torch.full((2,), 7.0, device="cuda") if weighted else None
    tcr.moe_swiglu_backward8(codes[0], scales[0], codes[1], scales[1], dh, dg, du, h=h, w_rows=w, dw=dw)
    rw, mag, tol = np.zeros(2), np.zeros(2), np.zeros(2)
    for i, (r, c, n) in enumerate(at):
        zi, vi = z[i][2], v[i][2]
        wi = np.array([[0.75, -1.5][r]])
        rg, ru, rh, rd = R.swiglu_backward(zi, vi, d[i], wi)
        a, s = np.abs(d[i] * wi[:, None]), R.sigmoid(zi)
        for name, t, ref, scale in (("dg", dg, rg, a * np.abs(vi) * s * (1 + np.abs(zi))),
                                    ("du", du, ru, a * np.abs(zi) * s), ("h8", h, rh, np.abs(rh))):
            _within(t[r, c:c + n][None], ref, _swiglu_tol(zi, scale, ref, "f16"), name)
        m = np.abs(d[i] * rh)
        rw[r] += rd[0]
        mag[r] += m.sum()
        tol[r] += (m * ((1.5 * np.abs(zi) + 6) * 2.0 ** -23)).sum()
    if weighted:  # at most 128 terms that are not zero, joined by a few more additions
        assert (np.abs(host(dw) - rw) <= tol + 150 * U * mag).all()
    for t in (dg, du, h):
        for r, c, n in at:
            t[r, c:c + n] = 0.0
        assert bool((t == 0).all())
