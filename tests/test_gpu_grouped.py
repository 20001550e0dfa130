"""Grouped products, their gradients, 4-bit weights and the product with them against the
float64 definitions (oracle/grouped.py).

Tolerances. 16-bit products are exact in float32 (22 bits at most), as are those of a 4-bit
weight (2 bits) with parts of a that have 8; a float32 product is off by half a step. A sum of
K terms takes K roundings at most, each within a step (2^-23; not half of one, the matrix
cores' adders may cut off) of a partial sum that no order makes larger than the sum of the
terms' magnitudes: K 2^-23 mag covers all. The result is rounded once more to its type: half a
step of the value, or of the smallest subnormal."""
import numpy as np
import pytest
import torch

import token_choice_routing_amd as tcr
from oracle import grouped as G
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SMALLEST = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}
KEEP = 776.0  # what outputs hold before a call (a value of every type)


def host(t):
    return t.detach().double().cpu().numpy()


def rounding(ref, dtype):
    return torch.finfo(TYPES[dtype]).eps / 2 * np.abs(ref) + SMALLEST[dtype]


def check(got, ref, mag, K, dtype, what):
    """Elements of ref that are NaN were not to be written."""
    got = host(got)
    tol = (K + 1) * 2.0 ** -23 * mag + rounding(ref, dtype)
    off = np.abs(got - ref) / tol
    untouched = np.isnan(ref)
    worst = float(off[~untouched].max()) if (~untouched).any() else 0.0
    say(f"  {what}: worst {worst:.3f} of the tolerance")
    assert (got[untouched] == KEEP).all(), f"{what}: rows outside the segments were written"
    assert np.isfinite(got).all() and worst <= 1.0, (what, worst)


def make(seed, counts, n, k, dtype, behind=3, T=None, first=0):
    """Rows in expert order with `first` rows before the first segment and some behind the
    last; NaN in every row that no segment has."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows = first + sum(counts) + behind
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]) + first, dtype=torch.int32, device="cuda")

    def normal(shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(TYPES[dtype])

    a = normal((rows if T is None else T, k))
    dy = normal((rows, n))
    a_rows = None
    if T is not None:
        a_rows = torch.randint(0, T, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    for t in (a, dy) if T is None else (dy,):
        t[:first] = float("nan")
        t[first + sum(counts):] = float("nan")
    return rows, off, a_rows, a, dy, normal((len(counts), n, k), k ** -0.5)


def kept(shape, dtype):
    return torch.full(shape, KEEP, dtype=TYPES[dtype], device="cuda")


def arrays(*ts):
    return [None if t is None else t.cpu().numpy() if t.dtype == torch.int32 else host(t) for t in ts]


# counts of rows an expert, n, k: single rows, empty experts, one row past a tile, sizes
# that are multiples of 8 only, many rows
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0, 2], 24, 40),
    ([5, 0, 64, 65, 1, 127, 129], 72, 136),
    ([16, 17, 15, 33, 0, 31], 264, 520),
    ([300, 0, 1, 257, 513], 328, 264),
    ([700], 512, 256),
    ([3] * 60, 136, 1016),
    ([0, 1, 2, 0, 70] * 51, 24, 40),  # MOE_MAX_EXPERTS
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_products(shape, dtype):
    counts, n, k = SHAPES[shape]
    for out in {dtype, "f32", "bf16"}:
        for gather in (False, True):
            say(f"product {counts} n {n} k {k} {dtype} -> {out} gather {gather}")
            rows, off, a_rows, a, dy, w = make(shape, counts, n, k, dtype, T=37 if gather else None)
            y = kept((rows, n), out)
            tcr.moe_grouped_mm(a, off, w, y, a_rows=a_rows)
            ha, hf, hw, hr, hd = arrays(a, off, w, a_rows, dy)
            ref, mag = G.product(ha, hf, hw, rows, hr)
            check(y, ref, mag, k, out, "out")
            da = kept((rows, k), out)
            tcr.moe_grouped_mm_dgrad(dy, off, w, da)
            ref, mag = G.data_gradient(hd, hf, hw)
            check(da, ref, mag, n, out, "da")
            dw = kept(w.shape, out)
            tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows)
            ref, mag = G.weight_gradient(hd, ha, hf, len(counts), None, hr)
            check(dw, ref, mag, max(counts), out, "dw")


# as many tiles as the 256 x 256 ones are taken for, with every number of 32-row blocks in them
MANY = [0, 1, 31, 33, 64, 65, 129, 160, 200, 255, 256, 257, 300, 400, 513, 3] * 4


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k,out", [(1032, 1040, "f32"), (1288, 1048, "bf16"), (1024, 2048, "f16")])
def test_many_tiles(n, k, out, gather, dtype):
    say(f"many tiles n {n} k {k} {dtype} -> {out} gather {gather}")
    rows, off, a_rows, a, dy, w = make(31, MANY, n, k, dtype, T=900 if gather else None)
    dw, add = kept(w.shape, out), None
    if n == 1288:
        add = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    y, da = kept((rows, n), out), kept((rows, k), out)
    tcr.moe_grouped_mm(a, off, w, y, a_rows=a_rows)
    tcr.moe_grouped_mm_dgrad(dy, off, w, da)
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows, dw_add=add)
    ha, hf, hw, hr, hd, hadd = arrays(a, off, w, a_rows, dy, add)
    check(y, *G.product(ha, hf, hw, rows, hr), k, out, "out")
    check(da, *G.data_gradient(hd, hf, hw), n, out, "da")
    check(dw, *G.weight_gradient(hd, ha, hf, len(MANY), hadd, hr), max(MANY) + 1, out, "dw")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,n,k", [([40, 0, 3], 72, 64), ([530, 300], 264, 520)])
def test_spaced_rows(dtype, counts, n, k):
    """Column ranges of wider matrices, as gate and up halves of one."""
    say(f"spaced rows {counts} n {n} k {k} {dtype}")
    rows, off, _, a, dy, w = make(7, counts, n, k, dtype, first=2)
    wide_a, wide_dy = kept((rows, 2 * k + 8), dtype), kept((rows, 2 * n + 16), dtype)
    wide_a[:, k:2 * k], wide_dy[:, 16:n + 16] = a, dy
    a, dy = wide_a[:, k:2 * k], wide_dy[:, 16:n + 16]
    ha, hf, hw, hd = arrays(a, off, w, dy)
    y, da, dw = kept((rows, 3 * n), "f32"), kept((rows, k + 24), dtype), kept(w.shape, "f32")
    tcr.moe_grouped_mm(a, off, w, y[:, n:2 * n])
    ref, mag = G.product(ha, hf, hw, rows)
    check(y[:, n:2 * n], ref, mag, k, "f32", "out")
    assert bool((y[:, :n] == KEEP).all()) and bool((y[:, 2 * n:] == KEEP).all())
    tcr.moe_grouped_mm_dgrad(dy, off, w, da[:, 8:k + 8])
    ref, mag = G.data_gradient(hd, hf, hw)
    check(da[:, 8:k + 8], ref, mag, n, dtype, "da")
    assert bool((da[:, :8] == KEEP).all()) and bool((da[:, k + 8:] == KEEP).all())
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw)
    ref, mag = G.weight_gradient(hd, ha, hf, len(counts))
    check(dw, ref, mag, max(counts), "f32", "dw")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts,n,k", [([9, 0, 70], 40, 72), ([0, 600, 260], 264, 256), ([0, 0], 16, 24)])
def test_weight_gradient_added(dtype, counts, n, k):
    say(f"added weight gradient {counts} n {n} k {k} {dtype}")
    rows, off, a_rows, a, dy, w = make(11, counts, n, k, dtype, T=50)
    add = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    ha, hf, hr, hd, hadd = arrays(a, off, a_rows, dy, add)
    ref, mag = G.weight_gradient(hd, ha, hf, len(counts), hadd, hr)
    dw = kept(w.shape, dtype)
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows, dw_add=add)
    check(dw, ref, mag, max(counts) + 1, dtype, "dw")
    tcr.moe_grouped_mm_wgrad(dy, a, off, add, a_rows=a_rows, dw_add=add)  # in place
    check(add, ref, mag, max(counts) + 1, "f32", "dw in place")


def test_without_offsets_and_without_rows():
    rows, off, _, a, dy, w = make(5, [77], 72, 40, "bf16", behind=0)
    ha, hw, hd = arrays(a, w, dy)
    y, da, dw = kept((77, 72), "f32"), kept((77, 40), "f32"), kept(w.shape, "f32")
    tcr.moe_grouped_mm(a, None, w, y)
    tcr.moe_grouped_mm_dgrad(dy, None, w, da)
    tcr.moe_grouped_mm_wgrad(dy, a, None, dw)
    check(y, *G.product(ha, None, hw, 77), 40, "f32", "out")
    check(da, *G.data_gradient(hd, None, hw), 72, "f32", "da")
    check(dw, *G.weight_gradient(hd, ha, None, 1), 77, "f32", "dw")
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    w2, add = torch.ones(2, 72, 40, device="cuda", dtype=torch.bfloat16), torch.full((2, 72, 40), 2.5, device="cuda")
    tcr.moe_grouped_mm(a[:0], zero, w2, y[:0])
    tcr.moe_grouped_mm_dgrad(dy[:0], zero, w2, da[:0])
    tcr.moe_grouped_mm_wgrad(dy[:0], a[:0], zero, w2)
    assert bool((w2 == 0).all())
    tcr.moe_grouped_mm_wgrad(dy[:0], a[:0], zero, w2, dw_add=add)
    assert bool((w2 == 2.5).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,k", [(40, 64), (264, 288)])
def test_offsets_and_row_numbers_outside(dtype, n, k):
    """Offsets are clamped into the rows, row numbers into the tokens."""
    rows, T = 90, 11
    say(f"offsets outside n {n} k {k} {dtype}")
    _, _, _, a, dy, w = make(2, [1, 1, 1], n, k, dtype, T=T)
    dy = torch.randn((rows, n), device="cuda").to(TYPES[dtype])
    off = torch.tensor([-7, 20, 20, 1 << 30], dtype=torch.int32, device="cuda")
    a_rows = torch.randint(-3, T + 3, (rows,), device="cuda", dtype=torch.int32)
    a_rows[0], a_rows[1] = -(1 << 31), (1 << 31) - 1
    ha, hf, hw, hr, hd = arrays(a, off, w, a_rows, dy)
    y, dw = kept((rows, n), "f32"), kept(w.shape, "f32")
    tcr.moe_grouped_mm(a, off, w, y, a_rows=a_rows)
    check(y, *G.product(ha, hf, hw, rows, hr), k, "f32", "out")
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows)
    check(dw, *G.weight_gradient(hd, ha, hf, 3, None, hr), 70, "f32", "dw")


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_stay_where_they_belong(dtype):
    counts, n, k = [40, 0, 300, 7], 136, 72
    say(f"not finite {dtype}")
    rows, off, _, a, dy, w = make(4, counts, n, k, dtype)
    ref_y, ref_da, ref_dw = kept((rows, n), "f32"), kept((rows, k), "f32"), kept(w.shape, "f32")

    def run(y, da, dw):
        tcr.moe_grouped_mm(a, off, w, y)
        tcr.moe_grouped_mm_dgrad(dy, off, w, da)
        tcr.moe_grouped_mm_wgrad(dy, a, off, dw)

    run(ref_y, ref_da, ref_dw)
    a[41, 3], dy[41, 5], a[39, 0] = float("nan"), float("inf"), float("-inf")
    w[1] = float("nan")  # an expert without rows
    w[3, 9, 11] = float("inf")
    y, da, dw = kept((rows, n), "f32"), kept((rows, k), "f32"), kept(w.shape, "f32")
    run(y, da, dw)
    same_y, same_da, same_dw = (torch.ones_like(t, dtype=torch.bool) for t in (y, da, dw))
    same_y[41], same_y[39] = False, False
    same_y[340:347, 9] = False
    same_da[41] = False
    same_da[340:347, 11] = False
    same_dw[2, :, 3], same_dw[2, 5], same_dw[0, :, 0] = False, False, False
    for got, ref, same in ((y, ref_y, same_y), (da, ref_da, same_da), (dw, ref_dw, same_dw)):
        assert bool((got[same] == ref[same]).all())
        assert not bool(torch.isfinite(got[~same]).all())
    assert bool(torch.isnan(y[41]).all()) and bool(torch.isnan(dw[2, :, 3]).all())


# ------------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 32), (7, 96), (3, 40, 544), (2, 1000, 2080)])
def test_weights4(dtype, shape):
    say(f"weights4 {shape} {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(9)
    w = torch.randn(shape, generator=gen, device="cuda")
    w *= torch.exp(2 * torch.randn((*shape[:-1], 1), generator=gen, device="cuda"))
    w = w.to(TYPES[dtype])
    flat = w.reshape(-1, shape[-1])
    flat[0, :8] = torch.tensor([0.0, -0.0, 1.0, 2.0, 4.0, 0.5, 0.25, -1.5])
    cs, ss = tcr.weights4_shapes(shape)
    codes = torch.full(cs, 99, dtype=torch.uint8, device="cuda")
    scales = torch.full(ss, 99, dtype=torch.uint8, device="cuda")
    out = kept(shape, dtype)
    tcr.moe_weights4_pack(w, codes, scales)
    tcr.moe_weights4_unpack(codes, scales, out)
    code, scale, v = G.pack4(host(flat))
    np.testing.assert_array_equal(codes.cpu().numpy().reshape(-1, shape[-1] // 2), G.bytes4(code))
    np.testing.assert_array_equal(scales.cpu().numpy().reshape(scale.shape), scale)
    np.testing.assert_array_equal(host(out).reshape(v.shape), v)


@pytest.mark.parametrize("dtype", TYPES)
def test_weights4_ties_ends_and_not_finite(dtype):
    """Every tie between two grid values and its neighbours at every exponent, the type's
    ends, and blocks that are not finite."""
    t = TYPES[dtype]
    fi = torch.finfo(t)
    lo, hi = {"f16": (-24, 15), "bf16": (-133, 127), "f32": (-149, 127)}[dtype]
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 4.0, 7.5, 3.0, 1.5, 0.5])
    for x in range(lo, hi + 1):
        v = torch.tensor(np.concatenate([ties, -ties]) * 2.0 ** (x - 2), dtype=torch.float64).to(t)
        rows.append(torch.cat([v, torch.zeros(4, dtype=t)]))
        if dtype != "bf16":
            rows.append(torch.cat([torch.nextafter(v, torch.zeros_like(v)), torch.zeros(4, dtype=t)]))
            rows.append(torch.cat([torch.nextafter(v, 100 * v), torch.zeros(4, dtype=t)]))
    for x in (fi.max, -fi.max, float("nan"), float("inf"), float("-inf"), 0.0, -0.0):
        rows.append(torch.full((32,), x, dtype=t))
        rows.append(torch.cat([torch.tensor([x], dtype=t), torch.ones(31, dtype=t)]))
        rows.append(torch.cat([torch.ones(31, dtype=t), torch.tensor([x], dtype=t)]))
    w = torch.stack(rows).cuda()
    w = torch.where(torch.isfinite(w) | (torch.arange(len(rows)) >= len(rows) - 21).cuda()[:, None], w, 0.0).to(t)
    n = w.shape[0]
    say(f"weights4 ends {dtype}: {n} rows")
    codes = torch.zeros((n, 16), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((n, 1), dtype=torch.uint8, device="cuda")
    out = torch.zeros((n, 32), dtype=torch.float32, device="cuda")
    tcr.moe_weights4_pack(w, codes, scales)
    tcr.moe_weights4_unpack(codes, scales, out)
    code, scale, v = G.pack4(host(w))
    np.testing.assert_array_equal(scales.cpu().numpy(), scale)
    np.testing.assert_array_equal(codes.cpu().numpy(), G.bytes4(code))
    np.testing.assert_array_equal(host(out), v)
    out = torch.zeros((n, 32), dtype=t, device="cuda")
    tcr.moe_weights4_unpack(codes, scales, out)
    np.testing.assert_array_equal(host(out), host(torch.from_numpy(v).to(t)))


def test_weights4_every_scale_and_code():
    """Scale bytes that packing never writes, as other programs may."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(16).reshape(256, 16)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").reshape(256, 1)
    h = codes.cpu().numpy()
    code = np.stack([h & 15, h >> 4], -1).reshape(256, 32)
    v = G.values4(code, scales.cpu().numpy())
    for name, t in TYPES.items():
        out = torch.zeros((256, 32), dtype=t, device="cuda")
        tcr.moe_weights4_unpack(codes, scales, out)
        np.testing.assert_array_equal(host(out), host(torch.from_numpy(v).to(t)))


def quantised(seed, groups, n, k, lo=118, hi=123):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (groups, n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(lo, hi, (groups, n, k // 32), generator=gen, device="cuda", dtype=torch.uint8)
    h = codes.cpu().numpy()
    return codes, scales, G.values4(np.stack([h & 15, h >> 4], -1).reshape(groups, n, k), scales.cpu().numpy())


# d silu / dz lies in (-0.1, 1.1); the sigmoid is off by up to (1.5 |z| + 6) 2^-23 of itself
def check_swiglu(got, g, mg, u, mu, K, dtype, what):
    ref = G.swiglu(g, u)
    eg, eu = (K + 1) * 2.0 ** -23 * mg, (K + 1) * 2.0 ** -23 * mu
    tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(G.swiglu(g, np.ones_like(g))) * eu
    tol += (1.5 * np.abs(g) + 10) * 2.0 ** -23 * np.abs(ref) + rounding(ref, dtype)
    got = host(got)
    live = ~np.isnan(ref)
    worst = float((np.abs(got - ref) / tol)[live].max()) if live.any() else 0.0
    say(f"  {what}: worst {worst:.3f} of the tolerance")
    assert (got[~live] == KEEP).all() and worst <= 1.0, (what, worst)


SHAPES4 = [
    ([1], 8, 32),
    ([0, 1, 0, 2], 24, 64),
    ([5, 0, 16, 17, 1, 33], 72, 160),
    ([1, 1, 1, 0, 2, 1, 4], 264, 544),
    ([3] * 60, 136, 1024),
    ([100, 0, 257], 40, 96),
    ([2, 0, 9], 16, 2080),
    ([0, 1, 2, 0, 70] * 51, 24, 64),  # MOE_MAX_EXPERTS
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", range(len(SHAPES4)))
def test_gemm4(shape, dtype):
    counts, n, k = SHAPES4[shape]
    c0, s0, w0 = quantised(shape, len(counts), n, k)
    c1, s1, w1 = quantised(shape + 100, len(counts), n, k)
    for out in {dtype, "f32", "bf16"}:
        for gather in (False, True):
            say(f"gemm4 {counts} n {n} k {k} {dtype} -> {out} gather {gather}")
            rows, off, a_rows, a, _, _ = make(shape, counts, n, k, dtype, T=13 if gather else None)
            ha, hf, hr = arrays(a, off, a_rows)
            (g, mg), (u, mu) = G.product(ha, hf, w0, rows, hr), G.product(ha, hf, w1, rows, hr)
            y = kept((rows, n), out)
            tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, c0, s0, y, a_rows=a_rows)
            check(y, g, mg, 3 * k, out, "down")
            y = kept((rows, n + 8), out)
            tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, a, off, c0, s0, y[:, :n], c1, s1, a_rows=a_rows)
            check_swiglu(y[:, :n], g, mg, u, mu, 3 * k, out, "gate/up")
            assert bool((y[:, n:] == KEEP).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_gemm4_scales_and_values_at_the_ends(dtype):
    """Large and small steps next to each other, blocks that are NaN, rows with an infinity,
    NaN or the type's largest value: in their outputs and nowhere else."""
    n, k, counts = 48, 128, [4, 3]
    say(f"gemm4 ends {dtype}")
    codes, scales, _ = quantised(1, 2, n, k, 60, 190)
    rows, off, _, a, _, _ = make(8, counts, n, k, dtype)
    a[3, 5] = torch.finfo(TYPES[dtype]).max * 2.0 ** -70 if dtype != "f16" else 65504.0
    h = codes.cpu().numpy()
    w = G.values4(np.stack([h & 15, h >> 4], -1).reshape(2, n, k), scales.cpu().numpy())
    y = kept((rows, n), "f32")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, y)
    ref, mag = G.product(host(a), off.cpu().numpy(), w, rows)
    check(y, ref, mag, 3 * k, "f32", "steps from 2^-67 to 2^62")
    codes, scales, _ = quantised(2, 2, n, k)
    scales[0, 7, 1] = 255
    h = codes.cpu().numpy()
    w = G.values4(np.stack([h & 15, h >> 4], -1).reshape(2, n, k), scales.cpu().numpy())
    a[1, 40], a[5, 100], a[6, 2] = float("inf"), float("nan"), torch.finfo(TYPES[dtype]).max / 1024
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, y)
    ha = host(a)
    got = host(y)
    assert np.isnan(got[:4, 7]).all() and np.isnan(got[5]).all()
    assert not np.isfinite(got[1]).any()
    ref, mag = G.product(np.where(np.isfinite(ha), ha, 0.0), off.cpu().numpy(), np.where(np.isnan(w), 0.0, w), rows)
    fine = np.ones(got.shape, bool)
    fine[:4, 7], fine[5], fine[1], fine[7:] = False, False, False, False
    tol = (3 * k + 1) * 2.0 ** -23 * mag + rounding(ref, "f32")
    assert (np.abs(got - ref) <= tol)[fine].all()


@pytest.mark.parametrize("dtype", TYPES)
def test_experts_packed_and_used_one_by_one(dtype):
    """Each expert's codes and scale bytes in their places, which begin at odd multiples of 8 for
    the scale bytes, equal those of all experts at once; and so do products with the last ones."""
    groups, n, k, rows = 5, 40, 96, 21
    say(f"experts one by one, {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(41)
    w = torch.randn((groups, n, k), generator=gen, device="cuda").to(TYPES[dtype])
    cs, ss = tcr.weights4_shapes(w.shape)
    sets = [(torch.full(cs, 99, dtype=torch.uint8, device="cuda"), torch.full(ss, 99, dtype=torch.uint8, device="cuda"),
             kept(w.shape, dtype)) for _ in range(2)]
    (c, s, v), (c1, s1, v1) = sets
    tcr.moe_weights4_pack(w, c, s)
    tcr.moe_weights4_unpack(c, s, v)
    for e in range(groups):
        assert s1[e].data_ptr() % 16 == (8 if e % 2 else 0)
        tcr.moe_weights4_pack(w[e], c1[e], s1[e])
        tcr.moe_weights4_unpack(c1[e], s1[e], v1[e])
    assert bool((c == c1).all()) and bool((s == s1).all()) and bool((v == v1).all())
    a = torch.randn((rows, k), generator=gen, device="cuda").to(TYPES[dtype])
    off = torch.tensor([0, 9, 9, 20, 20, 21], dtype=torch.int32, device="cuda")
    full, part = kept((rows, n), dtype), kept((rows, n), dtype)
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, a, off, c, s, full, c, s)
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, a, off[1:].clone(), c1[1:], s1[1:], part, c1[1:], s1[1:])
    assert bool((part[:9] == KEEP).all()) and bool((part[9:] == full[9:]).all())


# groups, rows of each and the wavefronts that share a reduction (n 256): four or one, of 16 or
# of 64 rows
SPLITS = [(1, 5), (1, 40), (128, 2), (120, 17)]
EXPONENTS = {"bf16": (0, -130, -100, -60, 60, 100, 118), "f16": (0, -14, -20, 4, 9),
             "f32": (0, -100, -60, 60, 100, 118)}


def check_extreme(got, ref, mag, K, top, what):
    """Products and sums as in check(), each operation further off by half the smallest float32
    (eight of them in a weight row with a byte above 252, whose sums are held divided by 8: `top`).
    Where the terms' magnitudes add up to 2^128, a partial sum may be infinite; below, none is."""
    got = host(got)
    tol = (3 * K + 1) * 2.0 ** -23 * mag + rounding(ref, "f32") + 3 * K * 2.0 ** -149 * np.where(top, 8, 1)
    finite = mag * (1 + 3 * K * 2.0 ** -23) < 2.0 ** 128
    nan = np.isnan(ref)
    assert np.isnan(got[nan]).all(), what
    with np.errstate(invalid="ignore"):
        off = np.abs(got - ref) / tol
    worst = float(off[finite & ~nan].max())
    say(f"  {what}: worst {worst:.3f} of the tolerance, {int((~finite).sum())} of {finite.size} may pass 2^128")
    assert worst <= 1.0, (what, worst)
    return finite


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("groups,each", SPLITS)
def test_gemm4_of_every_scale_byte(groups, each, dtype):
    """Weight row r has scale byte r, alone or next to other bytes, with rows of all sizes: no
    product or sum that a float32 can hold is lost."""
    n, k = 256, 160
    say(f"every scale byte, {groups} groups of {each} rows, {dtype}")
    rows = groups * each
    gen = torch.Generator(device="cuda").manual_seed(71)
    off = torch.arange(0, rows + 1, each, dtype=torch.int32, device="cuda")
    e = torch.tensor([EXPONENTS[dtype][i % len(EXPONENTS[dtype])] for i in range(rows)], device="cuda")
    a = torch.randn((rows, k), generator=gen, device="cuda", dtype=torch.float64) * torch.exp2(e.double())[:, None]
    a[:, 40:44] = 0.0
    a = a.to(TYPES[dtype])
    codes, _, _ = quantised(72, groups, n, k)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[None, :, None].expand(groups, n, 5).contiguous()
    other = torch.randint(0, 255, scales.shape, generator=gen, device="cuda", dtype=torch.uint8)
    for name, mixed in (("one byte a row", scales), ("first block", torch.cat((scales[..., :1], other[..., 1:]), 2)),
                        ("last block", torch.cat((other[..., :4] // 2, scales[..., 4:]), 2))):
        h, hs = codes.cpu().numpy(), mixed.cpu().numpy()
        w = G.values4(np.stack([h & 15, h >> 4], -1).reshape(groups, n, k), hs)
        y = kept((rows, n), "f32")
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, mixed, y)
        ref, mag = G.product(host(a), off.cpu().numpy(), w, rows)
        top = np.repeat(((hs == 253) | (hs == 254)).any(2), each, 0)
        assert check_extreme(y, ref, mag, k, top, name)[top].any()
    # up weights alone that reach 2^128: h = silu(g) u with u as above
    g_codes, g_scales, gw = quantised(73, groups, n, k, 80, 85)
    small = torch.where(a.abs() < 2, a, 0.0).to(a.dtype) if dtype != "f16" else (a.float() * 2.0 ** -12).half()
    ref_u, mag = G.product(host(small), off.cpu().numpy(), w, rows)
    ref_g, mag_g = G.product(host(small), off.cpu().numpy(), gw, rows)
    y = kept((rows, n), "f32")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, small, off, g_codes, g_scales, y, codes, mixed)
    # |silu(g)| <= |g|, and sigmoid(g) is 1/2 to within 2^-20 here
    assert np.abs(ref_g).max() < 2.0 ** -20
    fine = (mag * (1 + 3 * k * 2.0 ** -23) < 2.0 ** 128) & (mag_g * mag < 2.0 ** 126) & ~np.isnan(ref_u)
    tol = (8 * k + 40) * 2.0 ** -23 * mag_g * mag + 2.0 ** -20 * np.abs(ref_g * ref_u)
    tol += np.abs(ref_g) * 3 * k * 2.0 ** -146 + (np.abs(ref_u) + 1) * 3 * k * 2.0 ** -149
    err = np.abs(host(y) - ref_g * ref_u / 2)
    assert fine[:, 253:255].any() and (err <= tol)[fine].all()


@pytest.mark.parametrize("groups,each", SPLITS)
def test_gemm4_of_the_smallest_float32_rows(groups, each):
    """Rows down to float32's smallest subnormal, with all of their bits, next to ordinary ones and
    to elements that are not finite, and every scale byte."""
    n, k = 256, 160
    say(f"smallest rows, {groups} groups of {each} rows")
    rows = groups * each
    gen = torch.Generator(device="cuda").manual_seed(75)
    off = torch.arange(0, rows + 1, each, dtype=torch.int32, device="cuda")
    exponents = (-108, -112, -118, -124, -127, -133, -140, -147, 0)
    e = torch.tensor([exponents[i % len(exponents)] for i in range(rows)], device="cuda")
    a = torch.randn((rows, k), generator=gen, device="cuda", dtype=torch.float64) * torch.exp2(e.double())[:, None]
    a[:, 40:44] = 0.0
    a[-1] = torch.where(torch.arange(k, device="cuda") % 7 == 0, torch.exp2(e[-2].double() - 120), a[-1])
    a = a.float()
    codes, _, _ = quantised(76, groups, n, k)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda")[None, :, None].expand(groups, n, 5).contiguous()
    h, hs = codes.cpu().numpy(), scales.cpu().numpy()
    w = G.values4(np.stack([h & 15, h >> 4], -1).reshape(groups, n, k), hs)
    top = np.repeat(((hs == 253) | (hs == 254)).any(2), each, 0)
    y = kept((rows, n), "f32")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, y)
    ref, mag = G.product(host(a), off.cpu().numpy(), w, rows)
    check_extreme(y, ref, mag, k, top, "all bits of small rows")
    # without the largest scale bytes, and with an infinity and a NaN in two of the rows
    scales, top = scales.clamp(max=252), np.zeros_like(top)
    w = G.values4(np.stack([h & 15, h >> 4], -1).reshape(groups, n, k), scales.cpu().numpy())
    a[0, 3], a[1, 77] = float("inf"), float("nan")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, y)
    ref, mag = G.product(np.nan_to_num(host(a), posinf=0.0), off.cpu().numpy(), w, rows)
    check_extreme(y[2:], ref[2:], mag[2:], k, top[2:], "small rows next to others that are not finite")
    assert not np.isfinite(host(y)[0]).any() and np.isnan(host(y)[1]).all()


@pytest.mark.parametrize("groups,each", SPLITS)
def test_gemm4_rows_next_to_the_smallest_keep_their_bits(groups, each):
    """A row's outputs do not depend on whether a row or a weight row beside it is extreme."""
    n, k = 256, 160
    say(f"bits next to extremes, {groups} groups of {each} rows")
    rows = groups * each
    gen = torch.Generator(device="cuda").manual_seed(77)
    off = torch.arange(0, rows + 1, each, dtype=torch.int32, device="cuda")
    a = torch.randn((rows, k), generator=gen, device="cuda")
    codes, scales, _ = quantised(78, groups, n, k)
    first, second = kept((rows, n), "f32"), kept((rows, n), "f32")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, first)
    a[::each, 17] = 1e-37
    scales[:, 9::16, 2] = 254
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, second)
    same = torch.ones((rows, n), dtype=torch.bool, device="cuda")
    same[::each], same[:, 9::16] = False, False
    assert bool((first == second)[same].all()) and not bool((first == second)[~same].all())


@pytest.mark.parametrize("dtype", TYPES)
def test_gemm4_of_values_past_the_largest_float(dtype):
    """Weights of 2^128 and more: exact where the product is not too large, infinite where it
    is, 0 times a zero, NaN only with an infinity times a zero code or a NaN."""
    codes = torch.zeros((1, 16, 32), dtype=torch.uint8, device="cuda")
    codes[0, :8, :] = 0x77    # 6
    codes[0, 8:12, :] = 0xFF  # -6
    codes[0, 12:, 0] = 0x64   # 2 and 4, then zeros
    scales = torch.full((1, 16, 2), 254, dtype=torch.uint8, device="cuda")
    scales[0, 4:8] = 253
    a = torch.zeros((5, 64), device="cuda")
    a[1], a[2, 0], a[3, 1], a[4, 0] = 1.0, 2.0 ** -14, 1.0, float("inf")
    y = kept((5, 16), "f32")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a.to(TYPES[dtype]), None, codes, scales, y)
    got, inf = host(y), np.inf
    assert (got[0] == 0).all()
    assert (got[1] == [inf] * 8 + [-inf] * 4 + [inf] * 4).all()
    top = 6 * 2.0 ** 113
    assert (got[2] == [top] * 4 + [top / 2] * 4 + [-top] * 4 + [2.0 ** 114] * 4).all()
    assert (got[3] == [inf] * 8 + [-inf] * 4 + [inf] * 4).all()
    assert (got[4] == [inf] * 8 + [-inf] * 4 + [inf] * 4).all()


def test_gemm4_of_a_nan_with_any_payload():
    """A float32 NaN whose payload is in its last bits, of either sign, stays a NaN."""
    codes, scales, _ = quantised(4, 1, 16, 64)
    a = torch.ones((4, 64), device="cuda")
    a.view(torch.int32)[1, 9] = 0x7F800001
    a.view(torch.int32)[2, 33] = -0x7FFFFE  # 0xff800002
    y = kept((4, 16), "f32")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, None, codes, scales, y)
    assert bool(torch.isnan(y[1:3]).all()) and bool(torch.isfinite(y[::3]).all())


# Kernel forms that the sizes above leave out, with 256 CUs.
# At most 16 rows an expert, of the 16-bit product 256 in all, and at least 1024 items: a wavefront
# takes the whole reduction (of 16 rows). 968 columns end inside a panel of 128 (64 for gate/up): of its four wavefronts one has
# columns in part and one or more have none.
FEW_WHOLE = [0, 3, 9, 1, 5, 0, 2, 8, 4, 2, 16, 0] * 5
# More than 16 rows an expert: 64 rows an item, a wavefront with the whole reduction.
TALL_WHOLE = [17, 70, 0, 33, 64, 65, 1, 48, 20, 5, 16, 130]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k", [(968, 544), (1000, 72)])
def test_few_rows_with_the_whole_reduction(n, k, gather, out, dtype):
    say(f"few rows, whole reduction n {n} k {k} {dtype} -> {out} gather {gather}")
    rows, off, a_rows, a, _, w = make(51, FEW_WHOLE, n, k, dtype, T=40 if gather else None, first=1)
    assert rows <= 256 and (rows // 16 + len(FEW_WHOLE)) * (n // 32) >= 1024
    y = kept((rows, n + 8), out)
    tcr.moe_grouped_mm(a, off, w, y[:, :n], a_rows=a_rows)
    ha, hf, hw, hr = arrays(a, off, w, a_rows)
    check(y[:, :n], *G.product(ha, hf, hw, rows, hr), k, out, "out")
    assert bool((y[:, n:] == KEEP).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("groups", [7, 16, 64, 80])
def test_on_both_sides_of_few_rows(groups, dtype):
    """The most rows that count as few (4 an expert on average, or 256 of at most 16) and one row
    more, evenly and all of one expert."""
    n, k = 136, 200
    most = min(16 * groups, max(4 * groups, 256))
    for total in (most, most + 1):
        even = [total // groups + (e < total % groups) for e in range(groups)]
        for counts in (even, [0] * (groups - 1) + [total]):
            say(f"{total} rows of {groups} experts, {max(counts)} of one, {dtype}")
            rows, off, a_rows, a, _, w = make(53, counts, n, k, dtype, behind=0, T=90)
            y = kept((rows, n), dtype)
            tcr.moe_grouped_mm(a, off, w, y, a_rows=a_rows)
            ha, hf, hw, hr = arrays(a, off, w, a_rows)
            check(y, *G.product(ha, hf, hw, rows, hr), k, dtype, "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("counts,n,k", [(FEW_WHOLE, 968, 544), (TALL_WHOLE, 2056, 160)])
def test_gemm4_with_the_whole_reduction(counts, n, k, out, dtype):
    """A wavefront with the whole reduction of 16 or of 64 rows, plain and gate/up."""
    c0, s0, w0 = quantised(61, len(counts), n, k)
    c1, s1, w1 = quantised(62, len(counts), n, k)
    for gather in (False, True):
        say(f"gemm4, whole reduction {len(counts)} experts n {n} k {k} {dtype} -> {out} gather {gather}")
        rows, off, a_rows, a, _, _ = make(52, counts, n, k, dtype, T=70 if gather else None, first=1)
        per = 64 if rows > 16 * len(counts) else 16
        assert per == (16 if counts is FEW_WHOLE else 64) and (rows // per + len(counts)) * (n // 32) >= 1024
        ha, hf, hr = arrays(a, off, a_rows)
        (g, mg), (u, mu) = G.product(ha, hf, w0, rows, hr), G.product(ha, hf, w1, rows, hr)
        y = kept((rows, n), out)
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, c0, s0, y, a_rows=a_rows)
        check(y, g, mg, 3 * k, out, "down")
        y = kept((rows, n + 8), out)
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, a, off, c0, s0, y[:, :n], c1, s1, a_rows=a_rows)
        check_swiglu(y[:, :n], g, mg, u, mu, 3 * k, out, "gate/up")
        assert bool((y[:, n:] == KEEP).all())


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k,out,added", [(264, 520, "f32", False), (264, 520, "f32", True), (520, 136, "bf16", True),
                                           (136, 544, "f16", False)])
def test_many_tiles_of_float32(n, k, out, added, gather):
    """128 x 128 float32 tiles with every number of 32-row blocks, several row tiles and column
    tiles an expert, and many stages of the reduction in all three forms."""
    say(f"many tiles n {n} k {k} f32 -> {out} added {added} gather {gather}")
    rows, off, a_rows, a, dy, w = make(32, MANY, n, k, "f32", T=900 if gather else None)
    groups = len(MANY)
    assert (rows // 128 + groups) * (n // 128) >= 128 and groups * (n // 128) * (k // 128) >= 256
    dw, add = kept(w.shape, out), None
    if added:
        add = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    y, da = kept((rows, n), out), kept((rows, k), out)
    ha, hf, hw, hr, hd, hadd = arrays(a, off, w, a_rows, dy, add)
    tcr.moe_grouped_mm(a, off, w, y, a_rows=a_rows)
    check(y, *G.product(ha, hf, hw, rows, hr), k, out, "out")
    tcr.moe_grouped_mm_dgrad(dy, off, w, da)
    check(da, *G.data_gradient(hd, hf, hw), n, out, "da")
    ref, mag = G.weight_gradient(hd, ha, hf, groups, hadd, hr)
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows, dw_add=add)
    check(dw, ref, mag, max(MANY) + 1, out, "dw")
    if added:
        tcr.moe_grouped_mm_wgrad(dy, a, off, add, a_rows=a_rows, dw_add=add)
        check(add, ref, mag, max(MANY) + 1, "f32", "dw in place")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("gather", [False, True])
def test_large_weight_gradient_in_float32(gather, dtype):
    """256 x 256 tiles whose rows of the gradient are whole 128-byte lines, which are stored past
    the caches; and the same ones added to an earlier gradient, also in place."""
    n, k = 520, 544
    say(f"large weight gradient n {n} k {k} {dtype} -> f32 gather {gather}")
    rows, off, a_rows, a, dy, w = make(33, MANY, n, k, dtype, T=900 if gather else None)
    add = torch.randn(w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    ha, hf, hr, hd, hadd = arrays(a, off, a_rows, dy, add)
    dw = kept(w.shape, "f32")
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows)
    check(dw, *G.weight_gradient(hd, ha, hf, len(MANY), None, hr), max(MANY), "f32", "dw")
    ref, mag = G.weight_gradient(hd, ha, hf, len(MANY), hadd, hr)
    dw.fill_(KEEP)
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows, dw_add=add)
    check(dw, ref, mag, max(MANY) + 1, "f32", "dw added")
    tcr.moe_grouped_mm_wgrad(dy, a, off, add, a_rows=a_rows, dw_add=add)
    check(add, ref, mag, max(MANY) + 1, "f32", "dw in place")


# ------------------------------------------------------------------- past 32 bits

def test_rows_past_32_bit_offsets():
    """Segments at the end of matrices of more than 4 GB."""
    rows, n, k = 1_100_000, 2056, 64
    say("rows past 4 GB")
    gen = torch.Generator(device="cuda").manual_seed(17)
    off = torch.tensor([rows - 300, rows - 260, rows - 260, rows - 3], dtype=torch.int32, device="cuda")
    a = torch.randn((rows, k), generator=gen, device="cuda").bfloat16()
    dy = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    dy[rows - 300:] = torch.randn((300, n), generator=gen, device="cuda").bfloat16()
    w = (torch.randn((3, n, k), generator=gen, device="cuda") * 0.1).bfloat16()
    codes, scales, w4 = quantised(3, 3, n, k)
    y, da, dw = kept((rows, n), "bf16"), kept((rows, k), "f32"), kept(w.shape, "f32")
    tail = slice(rows - 300, rows)
    ha, hd, hw, hf = host(a[tail]), host(dy[tail]), host(w), off.cpu().numpy() - (rows - 300)
    tcr.moe_grouped_mm(a, off, w, y)
    check(y[tail], *G.product(ha, hf, hw, 300), k, "bf16", "out")
    y.fill_(KEEP)
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, y)
    check(y[tail], *G.product(ha, hf, w4, 300), k, "bf16", "out of 4-bit weights")
    assert bool((y[:rows - 300] == KEEP).all())
    tcr.moe_grouped_mm_dgrad(dy, off, w, da)
    check(da[tail], *G.data_gradient(hd, hf, hw), n, "f32", "da")
    assert bool((da[:rows - 300] == KEEP).all())
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw)
    check(dw, *G.weight_gradient(hd, ha, hf, 3), 257, "f32", "dw")


def test_gathered_rows_up_to_the_limit():
    """Row numbers at the end of the largest matrix that a_rows may name rows of."""
    lda = 2048
    tokens = 0xFFFFFF00 // (2 * lda) - 1
    say(f"{tokens} tokens of {lda}")
    a = torch.zeros((tokens, lda), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    a[-200:] = torch.randn((200, lda), generator=gen, device="cuda").bfloat16()
    a[:9] = torch.randn((9, lda), generator=gen, device="cuda").bfloat16()
    rows, n = 150, 264
    off = torch.tensor([0, 70, 140], dtype=torch.int32, device="cuda")
    a_rows = torch.randint(tokens - 200, tokens, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    a_rows[::7] = torch.randint(0, 9, (len(a_rows[::7]),), generator=gen, device="cuda", dtype=torch.int32)
    a_rows[3], a_rows[75] = tokens - 1, tokens + 5
    w = (torch.randn((2, n, lda), generator=gen, device="cuda") * 0.02).bfloat16()
    dy = torch.randn((rows, n), generator=gen, device="cuda").bfloat16()
    ends = a[a_rows.long().clamp(0, tokens - 1)]
    hx, hw, hd, hf = host(ends), host(w), host(dy), off.cpu().numpy()
    y, dw = kept((rows, n), "f32"), kept(w.shape, "f32")
    tcr.moe_grouped_mm(a, off, w, y, a_rows=a_rows)
    check(y, *G.product(hx, hf, hw, rows), lda, "f32", "out")
    tcr.moe_grouped_mm_wgrad(dy, a, off, dw, a_rows=a_rows)
    check(dw, *G.weight_gradient(hd, hx, hf, 2), 70, "f32", "dw")
    with pytest.raises(tcr.MoeError) as e:
        more = torch.empty((tokens + 1, lda), dtype=torch.bfloat16, device="cuda")
        tcr.moe_grouped_mm(more, off, w, y, a_rows=a_rows)
    assert e.value.status == tcr.MOE_ERR_UNSUPPORTED


# ------------------------------------------------------------------- how they are used

def test_two_streams_and_the_same_bits_again():
    counts, n, k = [300, 0, 41, 700], 264, 512
    rows, off, a_rows, a, dy, w = make(21, counts, n, k, "bf16", T=400)
    codes, scales, _ = quantised(5, 4, n, k)

    def outputs():
        return kept((rows, n), "bf16"), kept((rows, k), "f32"), kept(w.shape, "f32"), kept((rows, n), "f32")

    def run(o, stream=None):
        tcr.moe_grouped_mm(a, off, w, o[0], a_rows=a_rows, stream=stream)
        tcr.moe_grouped_mm_dgrad(dy, off, w, o[1], stream=stream)
        tcr.moe_grouped_mm_wgrad(dy, a, off, o[2], a_rows=a_rows, stream=stream)
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, a, off, codes, scales, o[3], a_rows=a_rows, stream=stream)

    ref, one, two = outputs(), outputs(), outputs()
    run(ref)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    run(one, s1)
    run(two, s2)
    torch.cuda.synchronize()
    for r, x, y in zip(ref, one, two):
        assert bool((r == x).all()) and bool((r == y).all())


def test_captured_in_a_graph():
    """Replays follow the inputs, the offsets and the row numbers of the moment."""
    n, k, T, rows = 136, 256, 60, 400
    gen = torch.Generator(device="cuda").manual_seed(2)
    a, dy = (torch.randn(s, generator=gen, device="cuda").bfloat16() for s in ((T, k), (rows, n)))
    w = torch.randn((3, n, k), generator=gen, device="cuda").bfloat16()
    codes, scales, _ = quantised(6, 3, n, k)
    off = torch.tensor([0, 10, 10, 300], dtype=torch.int32, device="cuda")
    a_rows = torch.randint(0, T, (rows,), generator=gen, device="cuda", dtype=torch.int32)

    def outputs():
        return kept((rows, n), "bf16"), kept((rows, k), "bf16"), kept(w.shape, "f32"), kept((rows, n), "bf16")

    def run(o):
        tcr.moe_grouped_mm(a, off, w, o[0], a_rows=a_rows)
        tcr.moe_grouped_mm_dgrad(dy, off, w, o[1])
        tcr.moe_grouped_mm_wgrad(dy, a, off, o[2], a_rows=a_rows)
        tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, a, off, codes, scales, o[3], codes, scales, a_rows=a_rows)

    got = outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(got)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    for i, ends in enumerate(([0, 10, 10, 300], [0, 0, 0, 0], [0, 1, 399, 400], [5, 6, 200, 201])):
        off.copy_(torch.tensor(ends, dtype=torch.int32))
        a.copy_(torch.randn((T, k), generator=gen, device="cuda"))
        a_rows.copy_(torch.randint(0, T, (rows,), generator=gen, device="cuda"))
        for t in got:
            t.fill_(KEEP)
        graph.replay()
        ref = outputs()
        run(ref)
        torch.cuda.synchronize()
        for r, g in zip(ref, got):
            assert bool((r == g).all()), i


def test_many_tiles_captured_in_a_graph():
    n, k = 1032, 1040
    rows, off, a_rows, a, dy, w = make(31, MANY, n, k, "bf16", T=900)

    def outputs():
        return kept((rows, n), "bf16"), kept((rows, k), "bf16"), kept(w.shape, "f32")

    def run(o):
        tcr.moe_grouped_mm(a, off, w, o[0], a_rows=a_rows)
        tcr.moe_grouped_mm_dgrad(dy, off, w, o[1])
        tcr.moe_grouped_mm_wgrad(dy, a, off, o[2], a_rows=a_rows)

    ref, got = outputs(), outputs()
    run(ref)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    for _ in range(3):
        for t in got:
            t.fill_(KEEP)
        graph.replay()
        run(ref)
        torch.cuda.synchronize()
        for r, g in zip(ref, got):
            assert bool((r == g).all())


def _dispatch(T, d, N, K, seed):
    """Routing of T random tokens as the layer's own entry points leave it."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, d), generator=gen, device="cuda").bfloat16()
    w_router = torch.randn((N + 1, d), generator=gen, device="cuda") * d ** -0.5
    dims = tcr.make_dims(T, d, N, N, K, 64)
    i32, cap = {"dtype": torch.int32, "device": "cuda"}, T * min(K, N)
    idx, wt = torch.zeros((T, K), **i32), torch.zeros((T, K), device="cuda")
    ws = [torch.empty(max(tcr.workspace_bytes(dims, q), 256), dtype=torch.uint8, device="cuda")
          for q in (tcr.MOE_WS_ROUTE, tcr.MOE_WS_PERMUTE)]
    tcr.moe_route(dims, x, w_router, topk_idx=idx, topk_w=wt, ws=ws[0])
    counts, off = torch.zeros(N, **i32), torch.zeros(N + 1, **i32)
    token, pos = torch.zeros(cap, **i32), torch.zeros((T, K), **i32)
    tcr.moe_permute(dims, idx, None, counts, off, token, pos, None, ws[1])
    return dims, x, off, token, pos, wt, cap


def _relative(got, ref):
    return float(np.sqrt(((host(got) - ref) ** 2).mean() / (ref ** 2).mean()))


@pytest.mark.parametrize("T", [1, 5, 64])
def test_a_decode_step_with_4_bit_experts(T):
    """Route, permute, gate/up and down with 4-bit weights, combine, against float64 on the
    values the codes stand for. bf16 h and expert rows: each rounding 2^-9 RMS of its value at
    most (half a step, uniform: 2^-8 / sqrt(12) < 2^-9), two of them and the output's: below
    3 2^-9 in all."""
    d, F, N, K = 256, 160, 16, 4
    dims, x, off, token, pos, wt, cap = _dispatch(T, d, N, K, 5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    packed = []
    for shape in ((N, F, d), (N, F, d), (N, d, F)):
        w = (torch.randn(shape, generator=gen, device="cuda") * shape[2] ** -0.5).bfloat16()
        cs, ss = tcr.weights4_shapes(shape)
        codes, scales, v = (torch.zeros(s, dtype=torch.uint8, device="cuda") for s in (cs, ss, ss))
        tcr.moe_weights4_pack(w, codes, scales)
        v = torch.zeros(shape, device="cuda")
        tcr.moe_weights4_unpack(codes, scales, v)
        packed.append((codes, scales, host(v)))
    (gc, gs, gv), (uc, us, uv), (dc, ds, dv) = packed
    h = torch.zeros((cap, F), dtype=torch.bfloat16, device="cuda")
    yp = torch.zeros((cap, d), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_GATE_UP, x, off, gc, gs, h, uc, us, a_rows=token)
    tcr.moe_grouped_gemm4(tcr.MOE_GEMM_DOWN, h, off, dc, ds, yp)
    tcr.moe_combine_rows(dims, tcr.MOE_BF16, yp, pos, wt, None, y)
    hx, hf, ht, hp, hw = arrays(x, off, token, pos, wt)
    ref = np.zeros((T, d))
    z = G.swiglu(G.product(hx, hf, gv, cap, ht)[0], G.product(hx, hf, uv, cap, ht)[0])
    rows, _ = G.product(z, hf, dv, cap)
    for t, s in np.ndindex(*hp.shape):
        if hp[t, s] >= 0:
            ref[t] += hw[t, s] * rows[hp[t, s]]
    if not ref.any():
        assert bool((y == 0).all())
        return
    off_by = _relative(y, ref)
    say(f"  decode step T {T}: {int(hf[-1])} rows, RMS error {off_by:.2e}")
    assert off_by <= 3 * 2.0 ** -9


@pytest.mark.parametrize("T", [3, 700])
def test_a_training_step_of_own_experts(T):
    """Dispatch, gate and up as halves of one product, 8-bit checkpoints, down, combine, and
    back: every product and gradient of this file next to the row operators, float32 rows,
    against float64 with the checkpoints' values in the backward."""
    from oracle import rows as R
    d, F, N, K = 128, 96, 8, 2
    dims, x, off, token, pos, wt, cap = _dispatch(T, d, N, K, 9)
    gen = torch.Generator(device="cuda").manual_seed(10)
    w1 = (torch.randn((N, 2 * F, d), generator=gen, device="cuda") * d ** -0.5)
    w2 = (torch.randn((N, d, F), generator=gen, device="cuda") * F ** -0.5)
    dy = torch.randn((T, d), generator=gen, device="cuda").bfloat16()
    xf, live = x.float(), off[N:]
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    gu, h, yp, y = f(cap, 2 * F), f(cap, F), f(cap, d), torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    cs = [(torch.zeros((cap, F), dtype=torch.int8, device="cuda"),
           torch.zeros(tcr.act8_scales_shape(cap, F), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    tcr.moe_grouped_mm(xf, off, w1, gu, a_rows=token)
    tcr.moe_swiglu_keep8(gu[:, :F], gu[:, F:], h, *cs[0], *cs[1], n_rows=live)
    tcr.moe_grouped_mm(h, off, w2, yp)
    tcr.moe_combine_rows(dims, tcr.MOE_F32, yp, pos, wt, None, y)
    dyp, wp, slot = f(cap, d), f(cap), torch.zeros(cap, dtype=torch.int32, device="cuda")
    tcr.moe_combine_backward(dims, tcr.MOE_F32, dy, None, pos, wt, dyp, wp, slot)
    dh, dgu, h8, dx = f(cap, F), f(cap, 2 * F), f(cap, F), f(T, d)
    dw1, dw2, dxp = f(N, 2 * F, d), f(N, d, F), f(cap, d)
    tcr.moe_grouped_mm_dgrad(dyp, off, w2, dh)
    tcr.moe_swiglu_backward8(*cs[0], *cs[1], dh, dgu[:, :F], dgu[:, F:], h=h8, n_rows=live)
    tcr.moe_grouped_mm_wgrad(dyp, h8, off, dw2)
    tcr.moe_grouped_mm_wgrad(dgu, xf, off, dw1, a_rows=token)
    tcr.moe_grouped_mm_dgrad(dgu, off, w1, dxp)
    tcr.moe_permute_backward(dims, tcr.MOE_F32, dxp, pos, None, tcr.MOE_F32, dx)
    hx, hf, ht, hp, hw, hw1, hw2, hdy = arrays(xf, off, token, pos, wt, w1, w2, dy)
    n = int(hf[-1])
    pre, _ = G.product(hx, hf, hw1, cap, ht)
    g, u = pre[:n, :F], pre[:n, F:]
    rows = np.zeros((cap, d))
    hh = np.full((cap, F), np.nan)
    hh[:n] = G.swiglu(g, u)
    rows, _ = G.product(hh, hf, hw2, cap)
    ref_y, ref_dyp = np.zeros((T, d)), np.zeros((cap, d))
    for t, s in np.ndindex(*hp.shape):
        if hp[t, s] >= 0:
            ref_y[t] += hw[t, s] * rows[hp[t, s]]
            ref_dyp[hp[t, s]] = hw[t, s] * hdy[t]
    # the checkpoints' own values (their codes are exact functions of g and u, so a g or u whose
    # float32 sum lies on the other side of a code's edge takes the neighbouring code)
    z, v = (host(c)[:n] * np.repeat(2.0 ** (s.cpu().numpy().astype(float) - 127), 32, 1)[:n, :F] for c, s in cs)
    for got, want in ((z, g), (v, u)):
        assert n == 0 or np.abs(got - want).max() <= 2.0 ** -6 * np.abs(want).max()
    q = 1 / (1 + np.exp(-z))
    ref_dh, _ = G.data_gradient(ref_dyp, hf, hw2)
    ref_dh = ref_dh[:n]
    ref_dgu, ref_h8 = np.zeros((cap, 2 * F)), np.zeros((cap, F))
    ref_dgu[:n, :F], ref_dgu[:n, F:], ref_h8[:n] = ref_dh * v * (q + z * q * (1 - q)), ref_dh * z * q, z * q * v
    ref_dw2, _ = G.weight_gradient(ref_dyp, ref_h8, hf, N)
    ref_dw1, _ = G.weight_gradient(ref_dgu, hx, hf, N, None, ht)
    ref_dxp, _ = G.data_gradient(ref_dgu, hf, hw1)
    ref_dx = np.zeros((T, d))
    for t, s in np.ndindex(*hp.shape):
        if hp[t, s] >= 0:
            ref_dx[t] += ref_dxp[hp[t, s]]
    assert _relative(y, ref_y) <= 2.0 ** -8  # one rounding to bf16
    # float32 throughout: sums of at most 2 F = 192 terms, or T rows, at 2^-23 RMS a term or less
    for name, got, want in (("dw2", dw2, ref_dw2), ("dw1", dw1, ref_dw1), ("dx", dx, ref_dx)):
        err = _relative(got, want)
        say(f"  training step T {T}: {name} RMS error {err:.2e}")
        assert err <= 2.0 ** -15, name
