"""GPU parity of the row operators (dispatch gradients, 8-bit activation checkpoints)
against their float64 definitions.

Tolerances, elementwise, with u = 2^-24 the float32 half step and H the output type's
half step, torch.finfo(t).eps / 2 of the value (bf16 2^-8, fp16 2^-11, fp32 2^-24):
  * a sum of n float32 terms in order: (n + 2) u sum |terms|, then one rounding H |ref|;
  * a dot over d columns: each lane adds at most ceil(d / 64) + 8 terms in order, six
    more additions join the lanes: (ceil(d / 64) + 16) u sum |terms|;
  * silu: the exponential's argument z log2 e is off by at most 1.5 |z| half steps times
    two, and the exponential, the sum and the reciprocal by a step each: the sigmoid's
    relative error is at most (1.5 |z| + 6) 2^-23.
A half-precision result below 2^-14 rounds in steps of 2^-24 (2^-25 off).
"""
import numpy as np
import pytest
import torch

import token_choice_routing_amd as tcr
from oracle import rows as R
from tests.gpu_util import say
from tests.test_oracle_rows import _slots

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"bf16": tcr.MOE_BF16, "f16": tcr.MOE_F16, "f32": tcr.MOE_F32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
KINDS = {"zero": tcr.MOE_NULL_ZERO, "copy": tcr.MOE_NULL_COPY, "constant": tcr.MOE_NULL_CONSTANT}


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def host(t):
    return t.double().cpu().numpy()


def rounded(rng, shape, dtype):
    """Random values of the type, on the device and as float64."""
    t = dev(rng.standard_normal(shape), torch.float64).to(TYPES[dtype])
    return t, host(t)


def close(got, ref, mag, n, dtype, what):
    got = host(got) if torch.is_tensor(got) else got
    tiny = 2.0 ** -25 if dtype == "f16" else 1e-40
    tol = HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -6) + (n + 2) * U * mag + tiny
    bad = ~(np.abs(got - ref) <= tol)
    worst = float((np.abs(got - ref) / tol).max()) if ref.size else 0.0
    say(f"  {what}: worst error {worst:.2f} of its tolerance")
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {worst} of the tolerance"


def dims(T, d, N, K, dtype, null="zero", M=None):
    return tcr.make_dims(T, d, N, K if M is None else M, K, 8, 0, CODES[dtype], KINDS[null])


ROUTED = [
    # T, d, N, K, rows, activations, null, shared
    (1, 8, 1, 1, "bf16", "bf16", "zero", False),
    (3, 512, 8, 2, "f32", "f32", "zero", True),
    (17, 520, 12, 6, "f16", "bf16", "copy", True),
    (65, 1032, 12, 5, "bf16", "f32", "constant", False),
    (130, 64, 40, 32, "bf16", "bf16", "copy", True),
    (33, 2048, 16, 8, "bf16", "bf16", "zero", True),
    (9, 2056, 16, 4, "f32", "bf16", "constant", True),
    (5, 4104, 8, 3, "f16", "f32", "copy", False),
    (200, 136, 64, 1, "f16", "f32", "zero", False),
]


def _routed(T, d, N, K, rows, act, null, seed=0):
    rng = np.random.default_rng(seed + T + d)
    sp = _slots(rng, T, K, N)
    if T > 2:
        sp[T // 2] = -1  # a token without real slots
    w = rng.random((T, K)).astype(np.float32)
    y, yh = rounded(rng, (T * min(K, N), d), rows)
    used = np.zeros(y.shape[0], bool)
    used[sp[sp >= 0]] = True
    y[torch.from_numpy(~used).cuda()] = float("nan")  # rows no slot names are never read
    src = srch = None
    if null != "zero":
        src, srch = rounded(rng, (T, d) if null == "copy" else (d,), act)
    return rng, sp, w, y, yh, used, src, srch


@pytest.mark.parametrize("T,d,N,K,rows,act,null,shared", ROUTED)
def test_combine_rows(T, d, N, K, rows, act, null, shared):
    rng, sp, w, y, yh, _, src, srch = _routed(T, d, N, K, rows, act, null)
    ys, ysh = rounded(rng, (T, d), rows) if shared else (None, None)
    ref, mag = R.combine(yh, sp, w.astype(np.float64), ysh, srch)
    out = torch.full((T, d), float("nan"), dtype=TYPES[act], device="cuda")
    D = dims(T, d, N, K, act, null)
    tcr.moe_combine_rows(D, CODES[rows], y, dev(sp, torch.int32), dev(w, torch.float32), ys, out, null_src=src)
    close(out, ref, mag, K, act, "y")


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_combine_rows_equals_combine(act):
    """Float32 rows: bit for bit what moe_combine writes."""
    rng, sp, w, y, _, _, src, _ = _routed(70, 1032, 12, 5, "f32", act, "copy")
    ys = dev(rng.standard_normal((70, 1032)), torch.float32)
    D = dims(70, 1032, 12, 5, act, "copy")
    a, b = (torch.empty((70, 1032), dtype=TYPES[act], device="cuda") for _ in range(2))
    args = (dev(sp, torch.int32), dev(w, torch.float32), ys)
    tcr.moe_combine_rows(D, tcr.MOE_F32, y, *args, a, null_src=src)
    tcr.moe_combine(D, y, *args, b, null_src=src)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,d,N,K,rows,act,null,shared", ROUTED)
def test_combine_backward(T, d, N, K, rows, act, null, shared):
    rng, sp, w, y, yh, used, src, srch = _routed(T, d, N, K, rows, act, null)
    dy, dyh = rounded(rng, (T, d), act)
    drows, dw, dnull, mag, nmag = R.combine_backward(dyh, yh, sp, w.astype(np.float64), srch)
    cap, D = y.shape[0], dims(T, d, N, K, act, null)
    dyp = torch.full((cap, d), 7.0, dtype=TYPES[rows], device="cuda")
    wp = torch.full((cap,), 7.0, device="cuda")
    rs = torch.full((cap,), 7, dtype=torch.int32, device="cuda")
    dtw = torch.full((T, K), float("nan"), device="cuda")
    dn = torch.full(srch.shape, float("nan"), device="cuda") if null != "zero" else None
    ws = torch.empty((max(256, tcr.workspace_bytes(D, tcr.MOE_WS_COMBINE_BACKWARD)),), dtype=torch.uint8,
                     device="cuda")
    tsp, tw = dev(sp, torch.int32), dev(w, torch.float32)
    tcr.moe_combine_backward(D, CODES[rows], dy, y, tsp, tw, dyp, wp, rs, dtw, null_src=src, dnull=dn, ws=ws)
    got = host(dyp)
    assert (got[~used] == 7.0).all()  # rows no slot names are left as they were
    close(got[used], drows[used], np.abs(drows[used]), 0, rows, "dy_perm")
    t, k = np.nonzero(sp >= 0)
    assert (host(wp)[sp[t, k]] == w[t, k]).all() and (host(wp)[~used] == 7.0).all()
    assert (host(rs)[sp[t, k]] == t * K + k).all() and (host(rs)[~used] == 7).all()
    close(dtw, dw, mag, -(-d // 64) + 14, "f32", "dtopk_w")
    if dn is not None:
        # a token's null weights are added first (K terms), then scaled; the constant's
        # sums run over 16 tokens in float32
        close(dn, dnull, nmag, K + (16 if null == "constant" else 1), "f32", "dnull")
    # expert outputs not kept: the null slots' weight gradients only
    part = torch.full((T, K), 7.0, device="cuda")
    tcr.moe_combine_backward(D, CODES[rows], dy, None, tsp, tw, None, None, None, part, null_src=src)
    assert (host(part)[sp >= 0] == 7.0).all()
    assert (host(part)[sp < 0] == host(dtw)[sp < 0]).all()


@pytest.mark.parametrize("T,d,N,K,rows,out,add", [
    (1, 8, 1, 1, "bf16", "bf16", False), (37, 520, 12, 6, "f16", "f16", True), (65, 1032, 12, 5, "bf16", "f32", True),
    (130, 64, 40, 32, "f32", "bf16", True), (33, 2048, 16, 8, "f32", "f32", True), (9, 4104, 16, 3, "bf16", "bf16", False),
])
def test_permute_backward(T, d, N, K, rows, out, add):
    rng, sp, _, y, yh, _, _, _ = _routed(T, d, N, K, rows, "f32", "zero")
    a = dev(rng.standard_normal((T, d)), torch.float32) if add else None
    ref, mag = R.permute_backward(yh, sp, host(a) if add else None)
    dx = torch.full((T, d), float("nan"), dtype=TYPES[out], device="cuda")
    tsp = dev(sp, torch.int32)
    D = dims(T, d, N, K, "bf16")
    tcr.moe_permute_backward(D, CODES[rows], y, tsp, a, CODES[out], dx)
    close(dx, ref, mag, K, out, "dx")
    if add and out == "f32":  # in place
        tcr.moe_permute_backward(D, CODES[rows], y, tsp, a, CODES[out], a)
        assert torch.equal(a, dx)


def test_slots_outside_the_rows():
    """Positions past the capacity or below -1 are skipped: no row read or written."""
    T, d, N, K = 6, 64, 8, 2
    rng, sp, w, y, yh, _, src, srch = _routed(T, d, N, K, "f32", "f32", "copy")
    sp[0], sp[1, 0], sp[5, 1] = [T * K, 2 ** 31 - 1], -2, -2 ** 31
    D, tsp, tw = dims(T, d, N, K, "f32", "copy"), dev(sp, torch.int32), dev(w, torch.float32)
    y = torch.nan_to_num(y)
    out, dx = (torch.empty((T, d), device="cuda") for _ in range(2))
    tcr.moe_combine_rows(D, tcr.MOE_F32, y, tsp, tw, None, out, null_src=src)
    ref, mag = R.combine(yh, sp, w.astype(np.float64), None, srch)
    close(out, ref, mag, K, "f32", "y")
    tcr.moe_permute_backward(D, tcr.MOE_F32, y, tsp, None, tcr.MOE_F32, dx)
    ref, mag = R.permute_backward(yh, sp, None)
    close(dx, ref, mag, K, "f32", "dx")
    dtw, dyp = torch.full((T, K), 7.0, device="cuda"), torch.full_like(y, 7.0)
    dy, dyh = rounded(rng, (T, d), "f32")
    tcr.moe_combine_backward(D, tcr.MOE_F32, dy, y, tsp, tw, dy_perm=dyp, dtopk_w=dtw, null_src=src)
    _, dw, _, mag, _ = R.combine_backward(dyh, yh, sp, w.astype(np.float64), srch)
    close(dtw, dw, mag, 20, "f32", "dtopk_w")


ACTS = [(1, 8, "f32"), (3, 24, "bf16"), (7, 32, "f16"), (5, 40, "bf16"), (64, 136, "f32"), (33, 1032, "f16"),
        (257, 776, "bf16"), (2, 8200, "bf16"), (1000, 72, "f32"),
        # 16 columns per lane, rows that end inside a block
        (1100, 1008, "bf16"), (700, 1552, "f16")]


def act_values(rng, rows, cols, dtype):
    """Blocks of unequal size, with zeros, exact half steps, clamped ends, tiny and huge ones."""
    a = rng.standard_normal((rows, cols)) * np.exp(2 * rng.standard_normal((rows, cols // 8)).repeat(8, 1))
    a[rng.random(a.shape) < 0.05] = 0.0
    half = rng.random(a.shape) < 0.1
    a[half] = np.ldexp(np.rint(a[half] * 128) + 0.5, -7)
    if rows > 2:
        a[1] = 0.0
        big = {"f32": 3.4e38, "bf16": 3.3e38, "f16": 65504.0}[dtype]
        a[2, :8] = [big, -big, 0.0, 1.0, big / 3, -big / 100, big / 127, big / 128]
    if rows > 4 and dtype != "f16":
        a[3] = np.ldexp(a[3], -130)  # subnormal
        a[4] = np.ldexp(a[4], -118)
    return dev(a, torch.float64).to(TYPES[dtype])


@pytest.mark.parametrize("rows,cols,dtype", ACTS)
def test_act8_is_exact(rows, cols, dtype):
    x = act_values(np.random.default_rng(rows * cols), rows, cols, dtype)
    q, s, v = R.act8(host(x))
    codes = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    scales = torch.full(tcr.act8_scales_shape(rows, cols), 99, dtype=torch.uint8, device="cuda")
    tcr.moe_act8_pack(x, codes, scales)
    np.testing.assert_array_equal(codes.cpu().numpy(), q)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    for t in ("f32", "bf16", dtype):
        out = torch.full((rows, cols), 7.0, dtype=TYPES[t], device="cuda")
        tcr.moe_act8_unpack(codes, scales, out)
        np.testing.assert_array_equal(host(out), v)


def test_act8_nonfinite_blocks():
    x = torch.ones((4, 72), device="cuda")
    x[0, 3], x[1, 40], x[2, 71] = float("nan"), float("inf"), -float("inf")
    codes = torch.empty((4, 72), dtype=torch.int8, device="cuda")
    scales = torch.empty((4, 3), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    tcr.moe_act8_pack(x, codes, scales)
    tcr.moe_act8_unpack(codes, scales, out)
    q, s, v = R.act8(host(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), q)
    np.testing.assert_array_equal(scales.cpu().numpy(), s)
    np.testing.assert_array_equal(host(out), v)


@pytest.mark.parametrize("live", [0, 1, 5, 9, 100, -3])
def test_act8_live_rows_and_spaced_rows(live):
    """Only rows below the device's count are touched; x and out may be column ranges."""
    wide = act_values(np.random.default_rng(1), 9, 160, "bf16")
    x = wide[:, 40:112]
    n = torch.tensor([3, live], dtype=torch.int32, device="cuda")[1:]
    codes = torch.full((9, 72), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((9, 3), 99, dtype=torch.uint8, device="cuda")
    tcr.moe_act8_pack(x, codes, scales, n_rows=n)
    m = min(max(live, 0), 9)
    q, s, v = R.act8(host(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), np.where(np.arange(9)[:, None] < m, q, 99))
    np.testing.assert_array_equal(scales.cpu().numpy(), np.where(np.arange(9)[:, None] < m, s, 99))
    out = torch.full((9, 160), 7.0, device="cuda")
    tcr.moe_act8_unpack(codes, scales, out[:, 80:152], n_rows=n)
    got = host(out)
    np.testing.assert_array_equal(got[:m, 80:152], v[:m])
    got[:m, 80:152] = 7.0
    assert (got == 7.0).all()


def _swiglu_tol(z, scale, h, dtype):
    rel = (1.5 * np.abs(z) + 6) * 2.0 ** -23
    tiny = 2.0 ** -25 if dtype == "f16" else 1e-37
    return HALF[dtype] * np.abs(h) * (1 + 2.0 ** -6) + scale * (rel + 6 * U) + tiny


def _within(got, ref, tol, what):
    got = host(got)
    worst = float((np.abs(got - ref) / tol).max())
    say(f"  {what}: worst error {worst:.2f} of its tolerance")
    assert (np.abs(got - ref) <= tol).all(), f"{what}: worst {worst} of the tolerance"


SWIGLU = [(400, 64, "bf16", "f32", "bf16", True), (90, 256, "f32", "f32", "f32", True), (50, 512, "bf16", "bf16", "bf16", True),
          (1, 8, "bf16", "bf16", "bf16", False), (5, 40, "f32", "f32", "f32", True),
          (33, 136, "f16", "f16", "f16", True), (130, 776, "bf16", "f32", "bf16", True),
          (64, 1544, "bf16", "bf16", "bf16", False), (7, 4104, "f32", "bf16", "f32", True),
          (300, 264, "f16", "f32", "bf16", False),
          # many rows take one wavefront each, few long ones four
          (2100, 528, "bf16", "bf16", "bf16", True), (1200, 912, "f16", "f16", "f16", False), (3, 2056, "f16", "f32", "f32", True)]


@pytest.mark.parametrize("rows,F,act,dht,out,weighted", SWIGLU)
def test_swiglu8(rows, F, act, dht, out, weighted):
    rng = np.random.default_rng(rows + F)
    spread = 3.0
    g, gh = rounded(rng, (rows, F), act)
    u, uh = rounded(rng, (rows, F), act)
    g = (g * spread).to(TYPES[act])
    gh = host(g)
    # g and u as the halves of one matrix
    gu = torch.cat([g, u], 1)
    h = torch.empty((rows, F), dtype=TYPES[act], device="cuda")
    cg, cu = (torch.empty((rows, F), dtype=torch.int8, device="cuda") for _ in range(2))
    sg, su = (torch.empty(tcr.act8_scales_shape(rows, F), dtype=torch.uint8, device="cuda") for _ in range(2))
    tcr.moe_swiglu_keep8(gu[:, :F], gu[:, F:], h, cg, sg, cu, su)
    ref = R.swiglu(gh, uh)
    _within(h, ref, _swiglu_tol(gh, np.abs(ref), ref, act), "h")
    qz, sz, z = R.act8(gh)
    qv, sv, v = R.act8(uh)
    for a, b in ((cg, qz), (sg, sz), (cu, qv), (su, sv)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    dh, dhh = rounded(rng, (rows, F), dht)
    w = rng.random(rows).astype(np.float32) if weighted else None
    slot = rng.permutation(rows + 3)[:rows].astype(np.int32) if weighted else None
    dgu = torch.empty((rows, 2 * F), dtype=TYPES[out], device="cuda")
    h8 = torch.empty((rows, F), dtype=TYPES[out], device="cuda")
    dw = torch.full((rows + 3,), 7.0, device="cuda") if weighted else None
    tw, ts = (dev(w, torch.float32), dev(slot, torch.int32)) if weighted else (None, None)
    tcr.moe_swiglu_backward8(cg, sg, cu, su, dh, dgu[:, :F], dgu[:, F:], h=h8, w_rows=tw, dw=dw, row_slot=ts)
    rg, ru, rh, rw = R.swiglu_backward(z, v, dhh, None if w is None else w.astype(np.float64))
    d = np.abs(dhh if w is None else dhh * w[:, None])
    s = R.sigmoid(z)
    _within(dgu[:, :F], rg, _swiglu_tol(z, d * np.abs(v) * s * (1 + np.abs(z)), rg, out), "dg")
    _within(dgu[:, F:], ru, _swiglu_tol(z, d * np.abs(z) * s, ru, out), "du")
    _within(h8, rh, _swiglu_tol(z, np.abs(rh), rh, out), "h8")
    if weighted:
        mag = np.abs(dhh * rh)
        tol = (mag * ((1.5 * np.abs(z) + 6) * 2.0 ** -23)).sum(1) + (F // 64 + 22) * U * mag.sum(1) + 1e-37
        got = host(dw)
        assert (np.abs(got[slot] - rw) <= tol).all()
        left = np.setdiff1d(np.arange(rows + 3), slot)
        assert (got[left] == 7.0).all()
        # by row, and without the optional outputs
        dw2 = torch.empty((rows,), device="cuda")
        dgu2 = torch.empty_like(dgu)
        tcr.moe_swiglu_backward8(cg, sg, cu, su, dh, dgu2[:, :F], dgu2[:, F:], w_rows=tw, dw=dw2)
        assert torch.equal(dw2, dw[torch.from_numpy(slot).long().cuda()])
        assert torch.equal(dgu2, dgu)


@pytest.mark.parametrize("rows,F,m", [(12, 104, 5), (12, 1048, 5), (2500, 520, 2049), (6, 1048, 0)])
def test_swiglu8_live_rows(rows, F, m):
    rng = np.random.default_rng(2)
    g, u, dh = (rounded(rng, (rows, F), "bf16")[0] for _ in range(3))
    g[m:] = float("nan")
    n = torch.tensor([m], dtype=torch.int32, device="cuda")

    def fresh(dt=torch.bfloat16):
        return torch.full((rows, F), 7, dtype=dt, device="cuda")

    h, h8, dg, du = (fresh() for _ in range(4))
    cg, cu = fresh(torch.int8), fresh(torch.int8)
    sg, su = (torch.full(tcr.act8_scales_shape(rows, F), 7, dtype=torch.uint8, device="cuda") for _ in range(2))
    dw = torch.full((rows,), 7.0, device="cuda")
    tcr.moe_swiglu_keep8(g, u, h, cg, sg, cu, su, n_rows=n)
    tcr.moe_swiglu_backward8(cg, sg, cu, su, dh, dg, du, h=h8, dw=dw, n_rows=n)
    for t in (h, h8, dg, du, cg, cu, sg, su, dw):
        assert bool((t[m:] == 7).all()) and bool(torch.isfinite(t[:m].float()).all())
    whole = [fresh() for _ in range(3)]
    tcr.moe_swiglu_backward8(cg, sg, cu, su, dh, whole[0], whole[1], h=whole[2])
    assert all(torch.equal(a[:m], b[:m]) for a, b in zip(whole, (dg, du, h8)))


def test_binding_refusals():
    """Tensors of another type, shape or layout than the call fixes are refused before it."""
    D = dims(6, 64, 8, 2, "bf16")
    x, rows = (torch.zeros((n, 64), dtype=torch.bfloat16, device="cuda") for n in (6, 12))
    sp, w = torch.zeros((6, 2), dtype=torch.int32, device="cuda"), torch.zeros((6, 2), device="cuda")
    B, F = tcr.MOE_BF16, tcr.MOE_F32
    wide = torch.zeros((12, 128), dtype=torch.bfloat16, device="cuda")[:, :64]
    for bad in (rows.float(), rows[:11], wide, rows.cpu()):
        with pytest.raises(ValueError, match="y_perm"):
            tcr.moe_combine_rows(D, B, bad, sp, w, None, x)
        with pytest.raises(ValueError, match="dx_perm"):
            tcr.moe_permute_backward(D, B, bad, sp, None, B, x)
        with pytest.raises(ValueError, match="dy_perm"):
            tcr.moe_combine_backward(D, B, x, rows, sp, w, dy_perm=bad)
    for bad in (sp.long(), sp[:5], sp.t().contiguous().t()):
        with pytest.raises(ValueError, match="slot_pos"):
            tcr.moe_combine_rows(D, B, rows, bad, w, None, x)
    with pytest.raises(ValueError, match="rows_dtype"):
        tcr.moe_combine_rows(D, 5, rows, sp, w, None, x)
    with pytest.raises(tcr.MoeError):
        tcr.moe_combine_rows(D, B, None, sp, w, None, x)
    with pytest.raises(ValueError, match="row_slot"):
        tcr.moe_combine_backward(D, B, x, rows, sp, w, row_slot=torch.zeros((12,), device="cuda"))
    with pytest.raises(ValueError, match="dx"):
        tcr.moe_permute_backward(D, F, rows.float(), sp, None, F, x)
    a, c, s = torch.zeros((5, 40), device="cuda"), torch.zeros((5, 40), dtype=torch.int8, device="cuda"), None
    s = torch.zeros((5, 2), dtype=torch.uint8, device="cuda")
    for args in ((a.double(), c, s), (a[0], c, s), (a.t(), c, s), (a, c[:4], s), (a, c, s[:, :1]), (a, c.float(), s),
                 (a.cpu(), c, s), (a.expand(5, 40)[:, ::2], c, s), (a[:1].expand(5, 40), c, s)):
        with pytest.raises(ValueError):
            tcr.moe_act8_pack(*args)
        with pytest.raises(ValueError):
            tcr.moe_act8_unpack(args[1], args[2], args[0])
    with pytest.raises(ValueError, match="n_rows"):
        tcr.moe_act8_pack(a, c, s, n_rows=torch.zeros((1,), dtype=torch.int64, device="cuda"))
    with pytest.raises(tcr.MoeError):  # rows spaced by no multiple of 8
        tcr.moe_act8_pack(torch.zeros((5, 44), device="cuda")[:, :40], c, s)
    with pytest.raises(tcr.MoeError):  # columns no multiple of 8
        tcr.moe_act8_pack(torch.zeros((5, 44), device="cuda"), torch.zeros((5, 44), dtype=torch.int8, device="cuda"), s)
    gu = torch.zeros((5, 80), device="cuda")
    with pytest.raises(ValueError, match="spacing"):
        tcr.moe_swiglu_keep8(gu[:, :40], a, a, c, s, c, s)
    with pytest.raises(ValueError, match="h:"):
        tcr.moe_swiglu_keep8(a, a, a.half(), c, s, c, s)
    with pytest.raises(ValueError, match="dw"):
        tcr.moe_swiglu_backward8(c, s, c, s, a, a, a, dw=torch.zeros((4,), device="cuda"))
    with pytest.raises(ValueError, match="dh"):
        tcr.moe_swiglu_backward8(c, s, c, s, gu[:, :40], a, a)
    with pytest.raises(ValueError, match="w_rows"):
        tcr.moe_swiglu_backward8(c, s, c, s, a, a, a, w_rows=torch.zeros((4,), device="cuda"))


def test_no_rows():
    """No tokens and no rows: accepted, nothing written."""
    D = dims(0, 64, 8, 2, "bf16", "constant")
    e = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    v, dn = e(64), torch.full((64,), 7.0, device="cuda")
    sp, w = e(0, 2, dtype=torch.int32), e(0, 2, dtype=torch.float32)
    tcr.moe_combine_rows(D, tcr.MOE_BF16, e(0, 64), sp, w, None, e(0, 64), null_src=v)
    tcr.moe_combine_backward(D, tcr.MOE_BF16, e(0, 64), e(0, 64), sp, w, e(0, 64), null_src=v, dnull=dn, ws=e(256))
    tcr.moe_permute_backward(D, tcr.MOE_BF16, e(0, 64), sp, None, tcr.MOE_BF16, e(0, 64))
    c, s = e(0, 64, dtype=torch.int8), e(0, 2, dtype=torch.uint8)
    tcr.moe_act8_pack(e(0, 64), c, s)
    tcr.moe_act8_unpack(c, s, e(0, 64))
    tcr.moe_swiglu_keep8(e(0, 64), e(0, 64), e(0, 64), c, s, c, s)
    tcr.moe_swiglu_backward8(c, s, c, s, e(0, 64), e(0, 64), e(0, 64), dw=e(0, dtype=torch.float32))
    torch.cuda.synchronize()
    assert bool((dn == 7.0).all())
