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


# More work than one pass of the largest grid, 2^20 workgroups. Positions run backwards
# through the expert rows, so r_tk = y_perm[T K - 1 - (t K + k)].
GRID = 1 << 20


def _slots_of(T, K, gen):
    """Random real slots first, then null ones; and which are real."""
    n = torch.randint(0, K + 1, (T, 1), generator=gen, device="cuda")
    real = torch.arange(K, device="cuda") < n
    p = (T * K - 1 - torch.arange(T * K, device="cuda")).view(T, K)
    return torch.where(real, p, -1).to(torch.int32), real


def _off(got, ref, mag, n, half):
    """Whether anything is off by more than a rounding and n float32 steps of mag."""
    tol = half * ref.abs() * (1 + 2.0 ** -6) + (n + 2) * U * mag + 1e-40
    return bool(((got.double() - ref).abs() > tol).any())


@pytest.mark.parametrize("T,d,null", [
    # wavefronts a token in the gradient: one, two and four
    (4 * GRID + 77, 8, tcr.MOE_NULL_ZERO), (2 * GRID + 77, 520, tcr.MOE_NULL_COPY), (GRID + 77, 1032, tcr.MOE_NULL_COPY),
    # the constant vector's sums over more chunks of 16 tokens than wavefronts
    (64 * GRID + 77, 8, tcr.MOE_NULL_CONSTANT)])
def test_more_tokens_than_the_largest_grid(T, d, null):
    say(f"  T = {T}, d = {d}, null kind {null}")
    K = 2
    gen = torch.Generator(device="cuda").manual_seed(d)

    def rnd(*s):
        return torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)

    dims = tcr.make_dims(T, d, 2, 2, K, 8, 0, tcr.MOE_BF16, null)
    slot, real = _slots_of(T, K, gen)
    w = torch.rand((T, K), generator=gen, device="cuda")
    y_perm, dy = rnd(T * K, d), rnd(T, d)
    src = {tcr.MOE_NULL_ZERO: None, tcr.MOE_NULL_COPY: dy, tcr.MOE_NULL_CONSTANT: rnd(d)}[null]
    y = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((T, d), 7.0, device="cuda")
    tcr.moe_combine_rows(dims, tcr.MOE_BF16, y_perm, slot, w, None, y, null_src=src)
    tcr.moe_permute_backward(dims, tcr.MOE_BF16, y_perm, slot, None, tcr.MOE_F32, dx)
    dyp = torch.full_like(y_perm, 7.0)
    wp, rs = torch.full((T * K,), 7.0, device="cuda"), torch.full((T * K,), 7, dtype=torch.int32, device="cuda")
    dtw = torch.full((T, K), 7.0, device="cuda")
    dnull = None if src is None else torch.full(src.shape, 7.0, device="cuda")
    ws = torch.empty((max(256, tcr.workspace_bytes(dims, tcr.MOE_WS_COMBINE_BACKWARD)),), dtype=torch.uint8,
                     device="cuda")
    tcr.moe_combine_backward(dims, tcr.MOE_BF16, dy, y_perm, slot, w, dyp, wp, rs, dtw, null_src=src, dnull=dnull, ws=ws)
    total, total_mag = (torch.zeros((d,), dtype=torch.float64, device="cuda") for _ in range(2))
    step = (1 << 27) // d
    for t0 in range(0, T, step):
        at = slice(t0, min(T, t0 + step))
        n = at.stop - t0

        def rows(p, c=d):  # of tokens at, [n][K][c]
            return p.view(T * K, c)[T * K - at.stop * K:T * K - t0 * K].flip(0).view(n, K, c)

        on, wt, g = real[at, :, None], w[at, :, None].double(), dy[at].double()
        r = torch.where(on, rows(y_perm).double(), 0.0)
        assert not _off(dx[at], r.sum(1), r.abs().sum(1), K, 2.0 ** -24), "dx"
        if src is not None:
            r = torch.where(on, r, src[at].double()[:, None] if null == tcr.MOE_NULL_COPY else src.double())
        assert not _off(y[at], (wt * r).sum(1), (wt * r).abs().sum(1), K, 2.0 ** -8), "y"
        gr = g[:, None] * r
        assert not _off(dtw[at], gr.sum(2), gr.abs().sum(2), -(-d // 64) + 14, 2.0 ** -24), "dtopk_w"
        del gr, r
        got, ref = rows(dyp).double(), wt * g[:, None]
        assert not _off(torch.where(on, got, 0.0), torch.where(on, ref, 0.0), ref.abs(), 0, 2.0 ** -8), "dy_perm"
        assert bool((got == 7.0)[~real[at]].all()), "dy_perm of no slot"
        flat = torch.arange(t0 * K, at.stop * K, device="cuda").view(n, K)
        assert torch.equal(rows(wp, 1)[..., 0], torch.where(real[at], w[at], 7.0)), "w_perm"
        assert torch.equal(rows(rs, 1)[..., 0], torch.where(real[at], flat, 7).to(torch.int32)), "row_slot"
        wn = torch.where(real[at], 0.0, w[at].double()).sum(1, keepdim=True)
        if null == tcr.MOE_NULL_COPY:
            assert not _off(dnull[at], wn * g, (wn * g).abs(), K + 1, 2.0 ** -24), "dnull"
        total += (wn * g).sum(0)
        total_mag += (wn * g).abs().sum(0)
    if null == tcr.MOE_NULL_CONSTANT:
        assert not _off(dnull, total, total_mag, K + 16, 2.0 ** -24), "dnull"


def _pow2(e):
    """2^e in float64, exact: e int64 in the range of normal numbers."""
    return ((e + 1023) << 52).view(torch.float64)


def _act8_of(x):
    """codes, scale bytes and values of [rows][cols <= 32], one block a row."""
    v = x.double()
    _, k = torch.frexp(v.abs().amax(1, keepdim=True))  # amax = m 2^k, m in [1/2, 1)
    e = (k.long() - 7).clamp(min=-126)
    q = torch.round(v * _pow2(-e)).clamp(-127, 127)
    return q, (e + 127)[:, 0], q * _pow2(e)


def _bwd_off(z, u, d, w, dg, du, dw, half):
    """Whether dg, du or dw (None: not asked for) are off (tolerances of _swiglu_tol)."""
    s = torch.sigmoid(z)
    wd = d * w[:, None]
    rel = (1.5 * z.abs() + 6) * 2.0 ** -23
    out = []
    for got, ref, scale in ((dg, wd * u * s * (1 + z * (1 - s)), wd.abs() * u.abs() * s * (1 + z.abs())),
                            (du, wd * z * s, wd.abs() * z.abs() * s)):
        tol = half * ref.abs() * (1 + 2.0 ** -6) + scale * (rel + 6 * U) + 1e-37
        out.append(bool(((got.double() - ref).abs() > tol).any()))
    if dw is not None:
        t = d * z * s * u
        tol = (t.abs() * rel).sum(1) + (z.shape[1] // 64 + 22) * U * t.abs().sum(1) + 1e-37
        out.append(bool(((dw.double() - t.sum(1)).abs() > tol).any()))
    return any(out)


def test_more_short_rows_than_the_largest_grid():
    """8 columns: four steps a row (of which one is on) in the step kernels, 32 rows a
    workgroup in the one with weight gradients."""
    rows, cols = 64 * GRID + 77, 8
    assert rows * 4 > GRID * 256 and rows > GRID * 32
    gen = torch.Generator(device="cuda").manual_seed(8)

    def rnd():
        return torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.bfloat16)

    def new(dt, *shape):
        return torch.full(shape or (rows, cols), 7, dtype=dt, device="cuda")

    g, u, dh = rnd(), rnd(), rnd()
    codes, scales = new(torch.int8), new(torch.uint8, rows, 1)
    kept = [new(torch.int8), new(torch.uint8, rows, 1), new(torch.int8), new(torch.uint8, rows, 1)]
    out, h, dg, du = (new(torch.bfloat16) for _ in range(4))
    w = torch.rand((rows,), generator=gen, device="cuda")
    tcr.moe_act8_pack(g, codes, scales)
    tcr.moe_act8_unpack(codes, scales, out)
    tcr.moe_swiglu_keep8(g, u, h, *kept)
    assert torch.equal(kept[0], codes) and torch.equal(kept[1], scales)
    tcr.moe_swiglu_backward8(*kept, dh, dg, du, w_rows=w)
    dg2, du2, dw = new(torch.bfloat16), new(torch.bfloat16), new(torch.float32, rows)
    tcr.moe_swiglu_backward8(*kept, dh, dg2, du2, w_rows=w, dw=dw)
    for r0 in range(0, rows, 1 << 24):
        at = slice(r0, r0 + (1 << 24))
        q, s, z = _act8_of(g[at])
        assert bool((codes[at] == q).all()) and bool((scales[at, 0] == s).all()) and bool((out[at] == z).all())
        qu, su, v = _act8_of(u[at])
        assert bool((kept[2][at] == qu).all()) and bool((kept[3][at, 0] == su).all())
        a, b = g[at].double(), u[at].double()
        ref = a * torch.sigmoid(a) * b
        tol = (2.0 ** -8 * (1 + 2.0 ** -6) + (1.5 * a.abs() + 6) * 2.0 ** -23 + 6 * U) * ref.abs() + 1e-37
        assert bool(((h[at].double() - ref).abs() <= tol).all())
        assert not _bwd_off(z, v, dh[at].double(), w[at].double(), dg[at], du[at], None, 2.0 ** -8)
        assert not _bwd_off(z, v, dh[at].double(), w[at].double(), dg2[at], du2[at], dw[at], 2.0 ** -8)


def test_more_rows_of_a_wavefront_than_the_largest_grid():
    """One wavefront a row, four rows a workgroup."""
    rows, F = 4 * GRID + 77, 264
    gen = torch.Generator(device="cuda").manual_seed(9)
    codes = [torch.randint(-127, 128, (rows, F), generator=gen, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.randint(119, 123, (rows, 9), generator=gen, dtype=torch.uint8, device="cuda") for _ in range(2)]
    dh = torch.randn((rows, F), generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.rand((rows,), generator=gen, device="cuda")
    dg, du = (torch.full((rows, F), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dw = torch.full((rows,), 7.0, device="cuda")
    tcr.moe_swiglu_backward8(codes[0], scales[0], codes[1], scales[1], dh, dg, du, w_rows=w, dw=dw)
    for r0 in range(0, rows, 1 << 19):
        at = slice(r0, r0 + (1 << 19))
        z, v = (c[at].double() * _pow2(s[at].long() - 127).repeat_interleave(32, 1)[:, :F]
                for c, s in zip(codes, scales))
        assert not _bwd_off(z, v, dh[at].double(), w[at].double(), dg[at], du[at], dw[at], 2.0 ** -8)


@pytest.mark.parametrize("d", [64, 520, 1032])
def test_slots_outside_the_rows_touch_nothing(d):
    """Positions past the capacity or below -1: the outputs in expert order hold what the
    slots inside name and are left alone elsewhere."""
    T, K, N = 6, 2, 8
    gen = torch.Generator(device="cuda").manual_seed(d)
    cap = T * K
    pos = torch.tensor([[cap, 2 ** 31 - 1], [-2, 3], [0, -1], [cap - 1, 5], [-1, -1], [7, -2 ** 31]], dtype=torch.int32)
    dims = tcr.make_dims(T, d, N, K, K, 8, 0, tcr.MOE_F32, tcr.MOE_NULL_COPY)
    y, dy, x = (torch.randn((n, d), generator=gen, device="cuda") for n in (cap, T, T))
    w = torch.rand((T, K), generator=gen, device="cuda")
    dyp, wp = torch.full((cap, d), 7.0, device="cuda"), torch.full((cap,), 7.0, device="cuda")
    rs, dtw = torch.full((cap,), 7, dtype=torch.int32, device="cuda"), torch.full((T, K), 7.0, device="cuda")
    dn = torch.full((T, d), 7.0, device="cuda")
    tcr.moe_combine_backward(dims, tcr.MOE_F32, dy, y, pos.cuda(), w, dyp, wp, rs, dtw, null_src=x, dnull=dn)
    want = dict(dyp=torch.full((cap, d), 7.0), wp=torch.full((cap,), 7.0), rs=torch.full((cap,), 7, dtype=torch.int32),
                dn=torch.zeros((T, d)))
    dyc, wc = dy.cpu(), w.cpu()
    for t in range(T):
        for k in range(K):
            p = int(pos[t, k])
            if 0 <= p < cap:  # one float32 product, the same on both sides
                want["dyp"][p], want["wp"][p], want["rs"][p] = wc[t, k] * dyc[t], wc[t, k], t * K + k
                ref, mag = (dy[t].double() * y[p].double()).sum(), (dy[t].double() * y[p].double()).abs().sum()
                assert not _off(dtw[t, k], ref, mag, -(-d // 64) + 14, 2.0 ** -24)
            elif p != -1:
                assert float(dtw[t, k]) == 0.0
    for t, wn in ((2, wc[2, 1]), (4, wc[4, 0] + wc[4, 1])):
        want["dn"][t] = wn * dyc[t]
    for name, got in (("dyp", dyp), ("wp", wp), ("rs", rs), ("dn", dn)):
        assert torch.equal(got.cpu(), want[name]), name


@pytest.mark.parametrize("kind", [tcr.MOE_NULL_ZERO, tcr.MOE_NULL_COPY, tcr.MOE_NULL_CONSTANT])
def test_every_output_of_a_replayed_combine_gradient(kind):
    """Each output is poisoned before each replay, and the inputs change between them."""
    T, d, N, K = 700, 1032, 8, 4
    gen = torch.Generator(device="cuda").manual_seed(5)
    dims = tcr.make_dims(T, d, N, K, K, 8, 0, tcr.MOE_BF16, kind)
    slot, _ = _slots_of(T, K, gen)
    w = torch.rand((T, K), generator=gen, device="cuda")

    def rnd(*s):
        return torch.randn(s, generator=gen, device="cuda").bfloat16()

    dy, yp = rnd(T, d), rnd(T * K, d)
    src = None if kind == tcr.MOE_NULL_ZERO else rnd(T, d) if kind == tcr.MOE_NULL_COPY else rnd(d)
    ws = torch.empty((max(256, tcr.workspace_bytes(dims, tcr.MOE_WS_COMBINE_BACKWARD)),), dtype=torch.uint8,
                     device="cuda")

    def outputs():
        o = [torch.empty_like(yp), torch.empty((T * K,), device="cuda"),
             torch.empty((T * K,), dtype=torch.int32, device="cuda"), torch.empty((T, K), device="cuda")]
        return o + ([torch.empty(src.shape, device="cuda")] if src is not None else [])

    def poison(o):
        for t in o:
            t.fill_(7)

    def call(o):
        tcr.moe_combine_backward(dims, tcr.MOE_BF16, dy, yp, slot, w, *o[:4], null_src=src,
                                 dnull=o[4] if src is not None else None, ws=ws)

    mine, eager = outputs(), outputs()
    call(mine)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(mine)
    for rep in range(3):
        dy.copy_(rnd(T, d))
        w.copy_(torch.rand((T, K), generator=gen, device="cuda"))
        poison(mine)
        poison(eager)
        graph.replay()
        torch.cuda.synchronize()
        call(eager)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(mine, eager)):
            assert torch.equal(a, b) and bool((a != 7).any()), (rep, i)
    del graph


@pytest.mark.parametrize("rows,F", [(70, 72), (3, 2056)])
def test_swiglu8_row_weights_and_skipped_slots(rows, F):
    """w_rows without dw scales dg and du alone; entries of row_slot outside dw are skipped."""
    gen = torch.Generator(device="cuda").manual_seed(F)
    g, u, dh = (torch.randn((rows, F), generator=gen, device="cuda") for _ in range(3))
    h, dg, du, dg1, du1 = (torch.empty_like(g) for _ in range(5))
    kept = [torch.empty((rows, F), dtype=torch.int8, device="cuda"),
            torch.empty(tcr.act8_scales_shape(rows, F), dtype=torch.uint8, device="cuda")]
    kept += [t.clone() for t in kept]
    tcr.moe_swiglu_keep8(g, u, h, *kept)
    w = torch.randn((rows,), generator=gen, device="cuda")
    tcr.moe_swiglu_backward8(*kept, dh, dg, du, w_rows=w)
    z, v = (torch.empty_like(g) for _ in range(2))
    tcr.moe_act8_unpack(kept[0], kept[1], z)
    tcr.moe_act8_unpack(kept[2], kept[3], v)
    assert not _bwd_off(z.double(), v.double(), dh.double(), w.double(), dg, du, None, 2.0 ** -24)
    dw = torch.full((rows + 2,), 7.0, device="cuda")
    full = torch.empty((rows,), device="cuda")
    slot = torch.arange(rows, dtype=torch.int32)
    slot[0], slot[1] = -1, rows + 1  # (rows + 1 is inside, rows is left free)
    slot[2] = rows + 2 if rows == 3 else 2 ** 31 - 1
    tcr.moe_swiglu_backward8(*kept, dh, dg1, du1, w_rows=w, dw=full)
    tcr.moe_swiglu_backward8(*kept, dh, dg1, du1, w_rows=w, dw=dw, row_slot=slot.cuda())
    want = torch.full((rows + 2,), 7.0, device="cuda")
    for p in range(rows):
        if 0 <= int(slot[p]) < rows + 2:
            want[int(slot[p])] = full[p]
    assert torch.equal(dw, want)
    assert not _bwd_off(z.double(), v.double(), dh.double(), w.double(), dg1, du1, full, 2.0 ** -24)


@pytest.mark.parametrize("rows,cols,act", [(40, 72, "f32"), (1100, 1008, "bf16")])
def test_swiglu8_blocks_that_are_not_finite(rows, cols, act):
    """A NaN or an infinity in g or u makes its block NaN in the backward pass and leaves
    every other block as it is."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
    gen = torch.Generator(device="cuda").manual_seed(6)
    g, u, dh = (torch.randn((rows, cols), generator=gen, device="cuda").to(dt) for _ in range(3))

    def step(g, u):
        h, dg, du, h8 = (torch.full_like(g, 7.0) for _ in range(4))
        kept = [torch.full((rows, cols), 7, dtype=torch.int8, device="cuda"),
                torch.full(tcr.act8_scales_shape(rows, cols), 7, dtype=torch.uint8, device="cuda")]
        kept += [t.clone() for t in kept]
        dw = torch.full((rows,), 7.0, device="cuda")
        tcr.moe_swiglu_keep8(g, u, h, *kept)
        tcr.moe_swiglu_backward8(*kept, dh, dg, du, h=h8, dw=dw)
        return h, kept, (dg, du, h8), dw

    clean = step(g, u)
    bad_g, bad_u = (torch.zeros((rows, cols), dtype=torch.bool, device="cuda") for _ in range(2))
    for t, mask, at in ((g, bad_g, [(0, 3, "nan"), (4, cols - 1, "inf"), (9, 40, "-inf")]),
                        (u, bad_u, [(1, 32, "nan"), (5, 0, "-inf"), (9, 40, "inf"), (rows - 1, cols - 8, "nan")])):
        for r, c, v in at:
            t[r, c] = float(v)
            mask[r, c // 32 * 32:c // 32 * 32 + 32] = True
    h, kept, outs, dw = step(g, u)
    for i, mask in ((0, bad_g), (2, bad_u)):
        blocks = mask[:, ::32]
        assert bool((kept[i][mask] == 0).all()) and torch.equal(kept[i][~mask], clean[1][i][~mask])
        assert bool((kept[i + 1][blocks] == 255).all()) and torch.equal(kept[i + 1][~blocks], clean[1][i + 1][~blocks])
    hit = torch.zeros_like(bad_g)  # h comes from g and u themselves
    for t in (g, u):
        hit |= ~torch.isfinite(t)
    assert torch.equal(h[~hit], clean[0][~hit]) and not bool(torch.isfinite(h[hit]).any())
    both = bad_g | bad_u
    # du = dh silu(z) does not depend on u
    for t, c, mask in zip(outs, clean[2], (both, bad_g, both)):
        assert bool(torch.isnan(t[mask]).all()) and torch.equal(t[~mask], c[~mask])
    bad_rows = both.any(1)
    assert bool(torch.isnan(dw[bad_rows]).all()) and torch.equal(dw[~bad_rows], clean[3][~bad_rows])
