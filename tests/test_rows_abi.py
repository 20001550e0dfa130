"""Host-side checks of the row operators (dispatch gradients, 8-bit activation
checkpoints): the C ABI and the binding refuse bad arguments before anything reaches
the GPU, and calls without rows are no-ops. No kernel runs."""
import ctypes

import pytest
import torch

import token_choice_routing_amd as tcr
from token_choice_routing_amd import (MOE_BF16, MOE_ERR_ALIGN, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED,
                                      MOE_ERR_WORKSPACE, MOE_F16, MOE_F32, MOE_OK, make_dims)

FAKE = 0x7f0000001000  # 16-byte aligned, never dereferenced: validation fails first
MIS = FAKE + 4


@pytest.fixture(scope="module")
def lib():
    return tcr.load_library()


def _dims(**kw):
    base = dict(T=64, d_model=64, n_experts=8, n_null=8, top_k=2, d_ff=64, d_ff_shared=0, dtype=MOE_BF16)
    base.update(kw)
    return make_dims(**base)


def test_declared(lib):
    names = {"moe_combine_rows", "moe_combine_backward", "moe_permute_backward", "moe_act8_pack",
             "moe_act8_unpack", "moe_swiglu_keep8", "moe_swiglu_backward8"}
    assert names <= set(tcr.header_functions())
    for n in names:
        assert hasattr(lib, n) and callable(getattr(tcr, n))


def test_combine_rows_checks(lib):
    def call(d, rt=MOE_BF16, yp=FAKE, sp=FAKE, w=FAKE, ys=None, ns=None, y=FAKE):
        return lib.moe_combine_rows(ctypes.byref(d), rt, yp, sp, w, ys, ns, y, None)

    d = _dims()
    for kw in (dict(yp=None), dict(sp=None), dict(w=None), dict(y=None), dict(rt=3), dict(rt=-1)):
        assert call(d, **kw) == MOE_ERR_ARG, kw
    for kw in (dict(yp=MIS), dict(sp=MIS), dict(w=MIS), dict(y=MIS), dict(ys=MIS)):
        assert call(d, **kw) == MOE_ERR_ALIGN, kw
    for kind in (tcr.MOE_NULL_COPY, tcr.MOE_NULL_CONSTANT):
        assert call(_dims(null_kind=kind)) == MOE_ERR_ARG
        assert call(_dims(null_kind=kind), ns=MIS) == MOE_ERR_ALIGN
    assert call(_dims(dtype=MOE_F16)) == MOE_ERR_ARG  # half is a type of rows, not of a layer
    assert call(_dims(d_model=(1 << 30) + 8, T=1)) == MOE_ERR_UNSUPPORTED
    assert call(_dims(T=0)) == MOE_OK
    assert lib.moe_combine_rows(None, 0, FAKE, FAKE, FAKE, None, None, FAKE, None) == MOE_ERR_ARG


def test_permute_backward_checks(lib):
    def call(d, rt=MOE_BF16, dp=FAKE, sp=FAKE, add=None, dt=MOE_F32, dx=FAKE + 64):
        return lib.moe_permute_backward(ctypes.byref(d), rt, dp, sp, add, dt, dx, None)

    d = _dims()
    for kw in (dict(dp=None), dict(sp=None), dict(dx=None), dict(rt=3), dict(dt=3)):
        assert call(d, **kw) == MOE_ERR_ARG, kw
    for kw in (dict(dp=MIS), dict(sp=MIS), dict(dx=MIS), dict(add=MIS)):
        assert call(d, **kw) == MOE_ERR_ALIGN, kw
    # accumulating in place needs the added gradient's own type
    assert call(d, add=FAKE, dx=FAKE, dt=MOE_BF16) == MOE_ERR_ARG
    assert call(_dims(d_model=(1 << 30) + 8, T=1)) == MOE_ERR_UNSUPPORTED
    assert call(_dims(T=0), add=FAKE, dx=FAKE) == MOE_OK


def test_combine_backward_checks(lib):
    def call(d, rt=MOE_BF16, dy=FAKE, yp=FAKE, sp=FAKE, w=FAKE, ns=None, dyp=FAKE, wp=None, rs=None, dw=FAKE,
             dn=None, ws=None, nbytes=0):
        return lib.moe_combine_backward(ctypes.byref(d), rt, dy, yp, sp, w, ns, dyp, wp, rs, dw, dn, ws, nbytes, None)

    d = _dims()
    for kw in (dict(dy=None), dict(sp=None), dict(w=None), dict(rt=7)):
        assert call(d, **kw) == MOE_ERR_ARG, kw
    for kw in (dict(dy=MIS), dict(yp=MIS), dict(sp=MIS), dict(w=MIS), dict(dyp=MIS), dict(wp=MIS), dict(rs=MIS),
               dict(dw=MIS)):
        assert call(d, **kw) == MOE_ERR_ALIGN, kw
    dc = _dims(null_kind=tcr.MOE_NULL_CONSTANT)
    assert call(dc) == MOE_ERR_ARG
    need = tcr.workspace_bytes(dc, tcr.MOE_WS_COMBINE_BACKWARD)
    assert need > 0 and tcr.workspace_bytes(d, tcr.MOE_WS_COMBINE_BACKWARD) == 0
    assert call(dc, ns=FAKE, dn=FAKE, ws=FAKE, nbytes=need - 1) == MOE_ERR_WORKSPACE
    assert call(dc, ns=FAKE, dn=FAKE) == MOE_ERR_WORKSPACE
    assert call(dc, ns=FAKE, dn=FAKE, ws=MIS, nbytes=need) == MOE_ERR_ALIGN
    assert call(dc, ns=FAKE, dn=MIS) == MOE_ERR_ALIGN
    assert call(_dims(T=0)) == MOE_OK


def test_act8_checks(lib):
    def pack(rows=4, cols=64, dt=MOE_BF16, x=FAKE, ld=64, n=None, c=FAKE, s=FAKE):
        return lib.moe_act8_pack(rows, cols, dt, x, ld, n, c, s, None)

    def unpack(rows=4, cols=64, dt=MOE_BF16, out=FAKE, ld=64, n=None, c=FAKE, s=FAKE):
        return lib.moe_act8_unpack(rows, cols, dt, c, s, n, out, ld, None)

    for call, data in ((pack, "x"), (unpack, "out")):
        for kw in (dict(rows=-1), dict(cols=0), dict(cols=12), dict(dt=3), dict(ld=56), dict(ld=68),
                   {data: None}, dict(c=None), dict(s=None)):
            assert call(**kw) == MOE_ERR_ARG, kw
        for kw in ({data: MIS}, dict(c=MIS), dict(s=MIS), dict(n=FAKE + 2)):
            assert call(**kw) == MOE_ERR_ALIGN, kw
        assert call(rows=1 << 40) == MOE_ERR_UNSUPPORTED
        assert call(rows=1 << 36) == MOE_ERR_UNSUPPORTED
        assert call(rows=0) == MOE_OK


def test_swiglu8_checks(lib):
    def keep(rows=4, F=64, dt=MOE_BF16, g=FAKE, u=FAKE, ld=64, n=None, h=FAKE, cg=FAKE, sg=FAKE, cu=FAKE, su=FAKE):
        return lib.moe_swiglu_keep8(rows, F, dt, g, u, ld, n, h, cg, sg, cu, su, None)

    def bwd(rows=4, F=64, cg=FAKE, sg=FAKE, cu=FAKE, su=FAKE, n=None, dt=MOE_F32, dh=FAKE, w=None, rs=None, ns=4,
            ot=MOE_BF16, dg=FAKE, du=FAKE, ld=128, h=None, dw=None):
        return lib.moe_swiglu_backward8(rows, F, cg, sg, cu, su, n, dt, dh, w, rs, ns, ot, dg, du, ld, h, dw, None)

    for kw in (dict(rows=-1), dict(F=4), dict(F=20), dict(dt=5), dict(ld=60), dict(g=None), dict(u=None),
               dict(h=None), dict(cg=None), dict(sg=None), dict(cu=None), dict(su=None)):
        assert keep(**kw) == MOE_ERR_ARG, kw
    for kw in (dict(g=MIS), dict(u=MIS), dict(h=MIS), dict(cg=MIS), dict(sg=MIS), dict(cu=MIS), dict(su=MIS),
               dict(n=FAKE + 1)):
        assert keep(**kw) == MOE_ERR_ALIGN, kw
    assert keep(rows=0) == MOE_OK
    for kw in (dict(rows=-1), dict(F=20), dict(dt=5), dict(ot=5), dict(ld=60), dict(dg=None), dict(du=None),
               dict(dh=None), dict(cg=None), dict(sg=None), dict(cu=None), dict(su=None), dict(dw=FAKE, ns=-1)):
        assert bwd(**kw) == MOE_ERR_ARG, kw
    for kw in (dict(dg=MIS), dict(du=MIS), dict(dh=MIS), dict(h=MIS), dict(dw=MIS), dict(w=MIS), dict(rs=MIS)):
        assert bwd(**kw) == MOE_ERR_ALIGN, kw
    assert bwd(rows=0) == MOE_OK


def test_binding_refuses_host_tensors():
    """Every tensor argument has to be on the device: nothing of the host's is read."""
    d = _dims(T=4, top_k=2)
    f = torch.zeros
    slots, w = f((4, 2), dtype=torch.int32), f((4, 2))
    x, rows = f((4, 64), dtype=torch.bfloat16), f((8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tcr.moe_combine_rows(d, MOE_BF16, rows, slots, w, None, x)
    with pytest.raises(ValueError):
        tcr.moe_combine_backward(d, MOE_BF16, x, rows, slots, w)
    with pytest.raises(ValueError):
        tcr.moe_permute_backward(d, MOE_BF16, rows, slots, None, MOE_F32, f((4, 64)))
    with pytest.raises(ValueError):
        tcr.moe_act8_pack(x, f((4, 64), dtype=torch.int8), f((4, 2), dtype=torch.uint8))
    with pytest.raises(ValueError):
        tcr.moe_combine_rows(d, 9, rows, slots, w, None, x)


def test_training_pair8_checks(lib):
    """The 8-bit training pair refuses what moe_layer_backward does not cover, and bad
    pointers, states and workspaces, before anything is launched."""
    big = 1 << 40
    p = tcr.LayerParams(FAKE, FAKE, 0.0, None, FAKE, FAKE, FAKE, None, None, None)
    g = tcr.LayerGrads(FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None)
    d = _dims()
    st, ws = tcr.workspace_bytes(d, tcr.MOE_WS_STATE8), tcr.workspace_bytes(d, tcr.MOE_WS_TRAIN8)
    R, F = 64 * 2, 64
    assert 2 * R * F * 33 // 32 <= st < tcr.workspace_bytes(d, tcr.MOE_WS_BACKWARD)
    assert tcr.workspace_bytes(_dims(dtype=MOE_F32), tcr.MOE_WS_STATE8) == 0

    def fwd(d, p=p, y=FAKE, aux=None, s=FAKE, sb=big, w=FAKE, wb=big):
        return lib.moe_layer_forward_train8(ctypes.byref(d), ctypes.byref(p) if p else None, y,
                                            ctypes.byref(aux) if aux else None, s, sb, w, wb, None)

    def bwd(d, dy=FAKE, g=g, s=FAKE, sb=big, w=FAKE, wb=big):
        return lib.moe_layer_backward_saved8(ctypes.byref(d), ctypes.byref(p), dy, 0.02, 0.001,
                                             ctypes.byref(g) if g else None, s, sb, w, wb, None)

    for call in (fwd, bwd):
        assert call(_dims(dtype=MOE_F32)) == MOE_ERR_UNSUPPORTED
        assert call(_dims(null_kind=tcr.MOE_NULL_COPY)) == MOE_ERR_UNSUPPORTED
        assert call(d, sb=st - 1) == MOE_ERR_WORKSPACE
        assert call(d, s=None) == MOE_ERR_WORKSPACE
        assert call(d, s=MIS) == MOE_ERR_ALIGN
        assert call(d, wb=ws - 1) == MOE_ERR_WORKSPACE
        assert call(d, w=None) == MOE_ERR_WORKSPACE
        assert call(_dims(T=0)) == MOE_OK
    assert fwd(d, p=None) == MOE_ERR_ARG
    assert fwd(d, y=None) == MOE_ERR_ARG
    a = tcr.AuxOut()
    a.logits = FAKE
    assert fwd(d, aux=a) == MOE_ERR_ARG
    assert bwd(d, g=None) == MOE_ERR_ARG
    assert bwd(d, dy=None) == MOE_ERR_ARG
    assert bwd(d, dy=MIS) == MOE_ERR_ALIGN
