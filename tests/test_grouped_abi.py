"""Host-side checks of the grouped products and the 4-bit weights: the C ABI and the binding
refuse bad arguments before anything reaches the GPU, and calls without rows are no-ops. No
kernel runs."""
import pytest
import torch

import token_choice_routing_amd as tcr
from token_choice_routing_amd import (MOE_BF16, MOE_ERR_ALIGN, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_F16, MOE_F32,
                                      MOE_GEMM_DOWN, MOE_GEMM_GATE_UP, MOE_OK)

FAKE = 0x7f0000001000  # 16-byte aligned, never dereferenced: validation fails first
MIS = FAKE + 4
BIG = (1 << 20) + 8


@pytest.fixture(scope="module")
def lib():
    return tcr.load_library()


def _mm(lib, dt=MOE_BF16, G=4, n=64, k=32, rows=10, a=FAKE, lda=32, ar=None, an=0, off=FAKE, w=FAKE, ot=MOE_F32,
        out=FAKE, ldo=64):
    return lib.moe_grouped_mm(dt, G, n, k, rows, a, lda, ar, an, off, w, ot, out, ldo, None)


def _dgrad(lib, dt=MOE_BF16, G=4, n=64, k=32, rows=10, dy=FAKE, ldy=64, off=FAKE, w=FAKE, ot=MOE_F32, out=FAKE,
           ldo=32):
    return lib.moe_grouped_mm_dgrad(dt, G, n, k, rows, dy, ldy, off, w, ot, out, ldo, None)


def _wgrad(lib, dt=MOE_BF16, G=4, n=64, k=32, rows=10, dy=FAKE, ldy=64, a=FAKE, lda=32, ar=None, an=0, off=FAKE,
           add=None, ot=MOE_F32, out=FAKE):
    return lib.moe_grouped_mm_wgrad(dt, G, n, k, rows, dy, ldy, a, lda, ar, an, off, add, ot, out, None)


def _gemm4(lib, op=MOE_GEMM_GATE_UP, dt=MOE_BF16, G=4, n=64, k=32, rows=10, a=FAKE, lda=32, ar=None, an=0, off=FAKE,
           c0=FAKE, s0=FAKE, c1=FAKE, s1=FAKE, ot=MOE_F32, out=FAKE, ldo=64):
    return lib.moe_grouped_gemm4(op, dt, G, n, k, rows, a, lda, ar, an, off, c0, s0, c1, s1, ot, out, ldo, None)


CALLS = {"mm": _mm, "dgrad": _dgrad, "wgrad": _wgrad, "gemm4": _gemm4}


def test_declared(lib):
    names = {"moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad", "moe_grouped_gemm4",
             "moe_weights4_pack", "moe_weights4_unpack"}
    assert names <= set(tcr.header_functions())
    for n in names:
        assert hasattr(lib, n) and callable(getattr(tcr, n))


@pytest.mark.parametrize("op", CALLS)
def test_common_checks(lib, op):
    call = CALLS[op]
    for kw in (dict(dt=3), dict(dt=-1), dict(ot=3), dict(G=0), dict(n=0), dict(n=60), dict(k=0), dict(k=36),
               dict(rows=-1), dict(out=None), dict(off=None)):
        assert call(lib, **kw) == MOE_ERR_ARG, kw
    for kw in (dict(out=MIS), dict(off=MIS)):
        assert call(lib, **kw) == MOE_ERR_ALIGN, kw
    ld = {"mm": ("lda", "ldo"), "dgrad": ("ldy", "ldo"), "wgrad": ("ldy", "lda"), "gemm4": ("lda", "ldo")}[op]
    for name in ld:
        assert call(lib, **{name: 24}) == MOE_ERR_ARG, name   # shorter than the row
        assert call(lib, **{name: 68}) == MOE_ERR_ARG, name   # not a multiple of 8
        assert call(lib, **{name: 1 << 22}) == MOE_ERR_UNSUPPORTED, name
    for kw in (dict(G=256), dict(rows=(1 << 31) - 512), dict(n=BIG, ldo=BIG, ldy=BIG), dict(rows=1 << 30, G=255)):
        kw = {a: b for a, b in kw.items() if a in call.__code__.co_varnames}
        assert call(lib, **kw) == MOE_ERR_UNSUPPORTED, kw
    # more pieces than 31 bits count: of rows and columns, of a weight gradient's two sides
    wide = dict(n=1 << 20, ldo=1 << 20, ldy=1 << 20)
    for kw in (dict(rows=1 << 17, G=255, **wide), dict(rows=1, G=255, k=1 << 20, lda=1 << 20, **wide)):
        kw = {a: b for a, b in kw.items() if a in call.__code__.co_varnames}
        if op == "dgrad":
            kw["ldo"] = kw.get("k", 32)
        assert call(lib, **kw) == MOE_ERR_UNSUPPORTED, kw
    if op != "wgrad":  # a weight gradient of no rows writes the experts' sums
        for G, off in ((4, FAKE), (1, None)):
            assert call(lib, rows=0, G=G, off=off) == MOE_OK


@pytest.mark.parametrize("op", ["mm", "wgrad", "gemm4"])
def test_gathered_rows(lib, op):
    call = CALLS[op]
    assert call(lib, a=None) == MOE_ERR_ARG
    assert call(lib, a=MIS) == MOE_ERR_ALIGN
    assert call(lib, ar=MIS, an=5) == MOE_ERR_ALIGN
    assert call(lib, ar=FAKE, an=0) == MOE_ERR_ARG
    assert call(lib, ar=FAKE, an=-1) == MOE_ERR_ARG
    # (an + 1) rows of lda elements in 4 GB
    an = (1 << 32) // (1024 * 2)
    assert call(lib, ar=FAKE, an=an, lda=1024) == MOE_ERR_UNSUPPORTED
    assert call(lib, ar=FAKE, an=an // 2, lda=1024, dt=MOE_F32) == MOE_ERR_UNSUPPORTED
    assert call(lib, ar=FAKE, an=1 << 62, lda=1024) == MOE_ERR_UNSUPPORTED


def test_operands(lib):
    assert _mm(lib, w=None) == MOE_ERR_ARG and _mm(lib, w=MIS) == MOE_ERR_ALIGN
    assert _dgrad(lib, w=None) == MOE_ERR_ARG and _dgrad(lib, w=MIS) == MOE_ERR_ALIGN
    assert _dgrad(lib, dy=None) == MOE_ERR_ARG and _wgrad(lib, dy=MIS) == MOE_ERR_ALIGN
    assert _wgrad(lib, add=MIS) == MOE_ERR_ALIGN
    assert _wgrad(lib, add=FAKE, out=FAKE, ot=MOE_BF16) == MOE_ERR_ARG  # in place: float32 only
    for name in ("c0", "s0", "c1", "s1"):
        assert _gemm4(lib, **{name: None}) == MOE_ERR_ARG
        assert _gemm4(lib, **{name: MIS}) == MOE_ERR_ALIGN
    assert _gemm4(lib, op=2) == MOE_ERR_ARG
    assert _gemm4(lib, k=40, lda=40) == MOE_ERR_ARG  # whole blocks of 32
    assert _gemm4(lib, op=MOE_GEMM_DOWN, c1=None, s1=None, rows=0) == MOE_OK


def test_weights4_checks(lib):
    def pack(rows=4, cols=64, dt=MOE_F16, w=FAKE, c=FAKE, s=FAKE):
        return lib.moe_weights4_pack(rows, cols, dt, w, c, s, None)

    def unpack(rows=4, cols=64, dt=MOE_F16, w=FAKE, c=FAKE, s=FAKE):
        return lib.moe_weights4_unpack(rows, cols, dt, c, s, w, None)

    for call in (pack, unpack):
        for kw in (dict(rows=-1), dict(cols=0), dict(cols=48), dict(dt=3), dict(w=None), dict(c=None), dict(s=None)):
            assert call(**kw) == MOE_ERR_ARG, kw
        for kw in (dict(w=MIS), dict(c=MIS), dict(s=MIS)):
            assert call(**kw) == MOE_ERR_ALIGN, kw
        assert call(rows=1 << 40) == MOE_ERR_UNSUPPORTED
        assert call(rows=1 << 34) == MOE_ERR_UNSUPPORTED
        assert call(rows=0) == MOE_OK


def test_weights4_sizes_whose_product_passes_64_bits(lib):
    """rows * cols of 2^40 and more are refused, also where the product as 64 bits is small or
    negative, and the largest size below that is not."""
    most = 2 ** 31 - 32
    sizes = [((1 << 40) // 64, 64), ((1 << 40) // most + 1, most), (1 << 39, 1 << 26), (1 << 38, 1 << 26),
             (1 << 39, 1 << 24), ((1 << 40) - 1, most), ((1 << 63) - 1, 32), ((1 << 63) - 1, most)]
    for rows, cols in sizes:
        assert rows * cols >= 1 << 40
        assert lib.moe_weights4_pack(rows, cols, MOE_F32, FAKE, FAKE, FAKE, None) == MOE_ERR_UNSUPPORTED, (rows, cols)
        assert lib.moe_weights4_unpack(rows, cols, MOE_F32, FAKE, FAKE, FAKE, None) == MOE_ERR_UNSUPPORTED, (rows, cols)
    # (a misaligned pointer, which is looked at after the sizes)
    for rows, cols in (((1 << 40) // 64 - 1, 64), ((1 << 40) // most, most), (1 << 34, 32)):
        assert rows * cols < 1 << 40
        assert lib.moe_weights4_pack(rows, cols, MOE_F32, MIS, FAKE, FAKE, None) == MOE_ERR_ALIGN, (rows, cols)


def test_scale_bytes_at_multiples_of_8(lib):
    """Where one expert's scale bytes begin among those of all."""
    for s, status in ((FAKE + 8, MOE_OK), (FAKE + 24, MOE_OK), (FAKE + 2, MOE_ERR_ALIGN), (FAKE + 12, MOE_ERR_ALIGN)):
        assert lib.moe_weights4_pack(0, 64, MOE_F16, FAKE, FAKE, s, None) == status
        assert lib.moe_weights4_unpack(0, 64, MOE_F16, FAKE, s, FAKE, None) == status
        assert _gemm4(lib, s0=s, rows=0) == status
        assert _gemm4(lib, s1=s, rows=0) == status
    assert lib.moe_weights4_pack(0, 64, MOE_F16, FAKE, FAKE + 8, FAKE, None) == MOE_ERR_ALIGN


def test_binding_refuses():
    """Tensors on the host, of another type or shape, or missing."""
    z = torch.zeros
    a, w, off, out = z(6, 32), z(2, 8, 32), z(3, dtype=torch.int32), z(6, 8)
    codes, scales = z(2, 8, 16, dtype=torch.uint8), z(2, 8, 1, dtype=torch.uint8)
    for call in (lambda: tcr.moe_grouped_mm(a, off, w, out), lambda: tcr.moe_grouped_mm(a, off, w[0], out),
                 lambda: tcr.moe_grouped_mm(None, off, w, out), lambda: tcr.moe_grouped_mm_dgrad(out, off, w, a),
                 lambda: tcr.moe_grouped_mm_wgrad(out, a, off, w), lambda: tcr.moe_weights4_pack(w, codes, scales),
                 lambda: tcr.moe_weights4_pack(w.int(), codes, scales),
                 lambda: tcr.moe_weights4_unpack(codes, scales, w),
                 lambda: tcr.moe_grouped_gemm4(MOE_GEMM_DOWN, a, off, codes, scales, out),
                 lambda: tcr.moe_grouped_gemm4(MOE_GEMM_DOWN, a, off, None, scales, out)):
        with pytest.raises(ValueError):
            call()
