"""The row operators as a training step of a user's own experts runs them, against the
float64 formulas; the same step captured in a HIP graph, on two streams at once, and at
sizes whose offsets pass 32 bits.

Tolerances of the chain (float32 throughout): every value is a product chain of float32
GEMMs over at most 128 terms; their RMS error is near sqrt(128) 2^-24 = 7e-7 of the
result's RMS a GEMM, three GEMMs and the elementwise steps stay below 1e-5. Checkpoint
values enter both sides as the ones the kernels kept."""
import numpy as np
import pytest
import torch

import token_choice_routing_amd as tcr
from oracle import rows as R
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

f32, i32 = torch.float32, torch.int32


class Step:
    """One MoE layer with expert GEMMs by torch, every other step by the library."""

    def __init__(self, T=77, d=64, F=104, N=6, M=6, K=3, kind=tcr.MOE_NULL_COPY, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.d, self.F, self.N, self.K = T, d, F, N, K
        self.dims = tcr.make_dims(T, d, N, M, K, F, 0, tcr.MOE_F32, kind)

        def rnd(*s):
            return torch.randn(s, generator=g, device="cuda")

        def new(*s, dtype=f32):
            return torch.zeros(s, dtype=dtype, device="cuda")

        self.x, self.dy = rnd(T, d), rnd(T, d)
        self.wr = rnd(N + 1, d) / d ** 0.5
        self.wg, self.wu, self.wd = (rnd(N, F, d) / d ** 0.5, rnd(N, F, d) / d ** 0.5, rnd(N, d, F) / F ** 0.5)
        cap = self.cap = T * min(K, N)
        self.topk, self.slot = new(T, K, dtype=i32), new(T, K, dtype=i32)
        self.w = new(T, K)
        self.counts, self.offsets, self.perm = new(N, dtype=i32), new(N + 1, dtype=i32), new(cap, dtype=i32)
        self.ws = new(max(256, tcr.workspace_bytes(self.dims, tcr.MOE_WS_PERMUTE)), dtype=torch.uint8)
        self.xp, self.yp, self.dyp, self.dxp, self.U = (new(cap, d), new(cap, d), new(cap, d), new(cap, d), new(cap, F))
        self.gu, self.dgu = new(cap, 2 * F), new(cap, 2 * F)
        self.h, self.h8 = new(cap, F), new(cap, F)
        nb = tcr.act8_scales_shape(cap, F)
        self.kept = (new(cap, F, dtype=torch.int8), new(*nb, dtype=torch.uint8),
                     new(cap, F, dtype=torch.int8), new(*nb, dtype=torch.uint8))
        self.wp, self.rs = new(cap), new(cap, dtype=i32)
        self.y, self.dx, self.dnull, self.dtw = new(T, d), new(T, d), new(T, d), new(T, K)
        self.seg = None

    def route(self):
        tcr.moe_route(self.dims, self.x, self.wr, topk_idx=self.topk, topk_w=self.w)
        tcr.moe_permute(self.dims, self.topk, self.x, self.counts, self.offsets, self.perm, self.slot, self.xp, self.ws)

    def segments(self):
        o = self.offsets.tolist()
        self.seg = [(e, o[e], o[e + 1]) for e in range(self.N) if o[e + 1] > o[e]]

    def run(self, seg):
        F, n = self.F, self.offsets[self.N:]
        self.route()
        for e, a, b in seg:
            self.gu[a:b, :F] = self.xp[a:b] @ self.wg[e].T
            self.gu[a:b, F:] = self.xp[a:b] @ self.wu[e].T
        tcr.moe_swiglu_keep8(self.gu[:, :F], self.gu[:, F:], self.h, *self.kept, n_rows=n)
        for e, a, b in seg:
            self.yp[a:b] = self.h[a:b] @ self.wd[e].T
        tcr.moe_combine_rows(self.dims, tcr.MOE_F32, self.yp, self.slot, self.w, None, self.y, null_src=self.x)
        # backward; the expert outputs yp are not used
        tcr.moe_combine_backward(self.dims, tcr.MOE_F32, self.dy, None, self.slot, self.w, self.dyp, self.wp, self.rs,
                                 self.dtw, null_src=self.x, dnull=self.dnull)
        for e, a, b in seg:
            self.U[a:b] = self.dy[self.perm[a:b].long()] @ self.wd[e]
        tcr.moe_swiglu_backward8(*self.kept, self.U, self.dgu[:, :F], self.dgu[:, F:], h=self.h8, w_rows=self.wp,
                                 dw=self.dtw.view(-1), row_slot=self.rs, n_rows=n)
        for e, a, b in seg:
            self.dxp[a:b] = self.dgu[a:b, :F] @ self.wg[e] + self.dgu[a:b, F:] @ self.wu[e]
        tcr.moe_permute_backward(self.dims, tcr.MOE_F32, self.dxp, self.slot, self.dnull, tcr.MOE_F32, self.dx)

    OUT = ("y", "dx", "dtw", "dyp", "h8", "dgu", "dnull")

    def outputs(self):
        return {k: getattr(self, k).clone() for k in self.OUT}


def _rms(a):
    return float(np.sqrt(np.mean(np.square(a))))


def test_training_step_of_own_experts():
    s = Step()
    s.route()
    s.segments()
    s.run(s.seg)
    h = lambda t: t.double().cpu().numpy()  # noqa: E731
    x, dy, w, slot = h(s.x), h(s.dy), h(s.w), s.slot.cpu().numpy()
    real = int(s.offsets[s.N])
    z, u = (torch.empty((s.cap, s.F), device="cuda") for _ in range(2))
    tcr.moe_act8_unpack(s.kept[0], s.kept[1], z)
    tcr.moe_act8_unpack(s.kept[2], s.kept[3], u)
    z, u = h(z), h(u)
    perm = s.perm.cpu().numpy()
    yp, yp8, dxp = np.zeros((s.cap, s.d)), np.zeros((s.cap, s.d)), np.zeros((s.cap, s.d))
    h8 = np.zeros((s.cap, s.F))
    wp = np.zeros(s.cap)
    for t in range(s.T):
        for k in range(s.K):
            if slot[t, k] >= 0:
                wp[slot[t, k]] = w[t, k]
    for e, a, b in s.seg:
        wg, wu, wd = h(s.wg[e]), h(s.wu[e]), h(s.wd[e])
        g1, u1 = x[perm[a:b]] @ wg.T, x[perm[a:b]] @ wu.T
        step = np.ldexp(1.0, s.kept[1][a:b].cpu().numpy().astype(int) - 127).repeat(32, 1)[:, :s.F]
        assert (np.abs(z[a:b] - g1) <= step * 1.001).all()  # the checkpoint is of this g
        yp[a:b] = R.swiglu(g1, u1) @ wd.T
        h8[a:b] = R.swiglu(z[a:b], u[a:b])
        yp8[a:b] = h8[a:b] @ wd.T
        dg, du, _, _ = R.swiglu_backward(z[a:b], u[a:b], dy[perm[a:b]] @ wd, wp[a:b])
        dxp[a:b] = dg @ wg + du @ wu
    y, _ = R.combine(yp, slot, w, None, x)
    _, dtw, dnull, _, _ = R.combine_backward(dy, yp8, slot, w, x)
    dx, _ = R.permute_backward(dxp, slot, dnull)
    assert 0 < real < s.T * s.K and (slot < 0).any()
    for name, ref in (("y", y), ("dtw", dtw), ("dnull", dnull), ("dx", dx)):
        err = _rms(h(getattr(s, name)) - ref) / _rms(ref)
        say(f"  {name}: RMS(err)/RMS = {err:.2e}")
        assert err <= 1e-5, name
    assert _rms(h(s.h8)[:real] - h8[:real]) <= 1e-5 * _rms(h8[:real])
    # (the weight gradients take h8: dW_down = dyp^T h8)
    dwd = np.zeros((s.N, s.d, s.F))
    for e, a, b in s.seg:
        dwd[e] = (wp[a:b, None] * dy[perm[a:b]]).T @ h8[a:b]
        got = h(s.dyp[a:b].T @ s.h8[a:b])
        assert _rms(got - dwd[e]) <= 1e-5 * _rms(dwd[e])


def test_training_step_replays_in_a_hip_graph():
    s = Step(seed=1)
    s.route()
    s.segments()
    s.run(s.seg)
    ref = s.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run(s.seg)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(s.seg)
    for rep in range(3):
        for k in s.OUT:
            getattr(s, k).fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        real = int(s.offsets[s.N])
        for k, v in ref.items():
            n = real if k in ("dyp", "h8", "dgu") else None
            assert torch.equal(getattr(s, k)[:n], v[:n]), (rep, k)
        s.run(s.seg)  # eager work between the replays
        torch.cuda.synchronize()
    del graph


@pytest.mark.parametrize("kind", [tcr.MOE_NULL_ZERO, tcr.MOE_NULL_CONSTANT])
def test_constant_vector_gradient_in_a_graph_and_on_two_streams(kind):
    """moe_combine_backward with a workspace: two calls at once on two streams, each with
    its own workspace, and a captured one."""
    T, d, N, K = 3000, 264, 8, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    dims = tcr.make_dims(T, d, N, K, K, 8, 0, tcr.MOE_BF16, kind)
    rng = np.random.default_rng(3)
    from tests.test_oracle_rows import _slots
    slot = torch.from_numpy(_slots(rng, T, K, N)).to("cuda", i32)
    w = torch.rand((T, K), generator=gen, device="cuda")
    v = torch.randn((d,), generator=gen, device="cuda").bfloat16()
    yp = torch.randn((T * K, d), generator=gen, device="cuda").bfloat16()
    need = max(256, tcr.workspace_bytes(dims, tcr.MOE_WS_COMBINE_BACKWARD))
    sets = []
    for i in range(2):
        sets.append(dict(dy=torch.randn((T, d), generator=gen, device="cuda").bfloat16(),
                         dyp=torch.zeros_like(yp), dtw=torch.zeros((T, K), device="cuda"),
                         dn=torch.zeros((d,), device="cuda"), ws=torch.empty((need,), dtype=torch.uint8, device="cuda")))

    def call(s, stream=None):
        tcr.moe_combine_backward(dims, tcr.MOE_BF16, s["dy"], yp, slot, w, s["dyp"], None, None, s["dtw"],
                                 null_src=v, dnull=s["dn"], ws=s["ws"], stream=stream)

    ref = []
    for s in sets:
        call(s)
        torch.cuda.synchronize()
        ref.append({k: s[k].clone() for k in ("dyp", "dtw", "dn")})
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s in sets:
            for k in ref[0]:
                s[k].zero_()
        torch.cuda.synchronize()
        for s, st in zip(sets, streams):
            call(s, st)
        torch.cuda.synchronize()
        for s, r in zip(sets, ref):
            for k, t in r.items():
                assert torch.equal(s[k], t), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(sets[0])
    for rep in range(3):
        sets[0]["dn"].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sets[0]["dn"], ref[0]["dn"]) or kind == tcr.MOE_NULL_ZERO, rep
        call(sets[1])
        torch.cuda.synchronize()
    del graph


def test_offsets_past_32_bits():
    """More than 2^31 elements (and 2^32 bytes) behind one pointer: the far rows."""
    T, d, N, K = 140000, 2048, 16, 8
    dims = tcr.make_dims(T, d, N, K, K, 8, 0, tcr.MOE_BF16)
    cap = T * K  # 2.3e9 elements of y_perm
    assert cap * d > 2 ** 31
    rng = np.random.default_rng(0)
    tokens = [0, 1, T // 2, T - 2, T - 1]
    slot = torch.full((T, K), -1, dtype=i32, device="cuda")
    pos = np.concatenate([rng.choice(cap - 64, 3 * len(tokens) - 4, replace=False), [cap - 1, cap - 2, 0, cap - 30]])
    for i, t in enumerate(tokens):
        slot[t, :3] = torch.from_numpy(pos[3 * i:3 * i + 3].astype(np.int32)).cuda()
    w = torch.rand((T, K), device="cuda")
    yp = torch.empty((cap, d), dtype=torch.bfloat16, device="cuda")
    idx = torch.from_numpy(pos).cuda()
    yp[idx] = torch.randn((len(pos), d), device="cuda").bfloat16()
    dy = torch.randn((T, d), device="cuda").bfloat16()
    y, dx = torch.empty_like(dy), torch.empty((T, d), device="cuda")
    dtw, wp = torch.empty((T, K), device="cuda"), torch.empty((cap,), device="cuda")
    tcr.moe_combine_rows(dims, tcr.MOE_BF16, yp, slot, w, None, y)
    tcr.moe_permute_backward(dims, tcr.MOE_BF16, yp, slot, None, tcr.MOE_F32, dx)
    for t in tokens:
        rows = yp[slot[t, :3].long()].double()
        ref = (w[t, :3, None].double() * rows).sum(0)
        mag = (w[t, :3, None].double() * rows).abs().sum(0)
        assert bool(((y[t].double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + 5 * 2.0 ** -24 * mag).all())
        ref, mag = rows.sum(0), rows.abs().sum(0)
        assert bool(((dx[t].double() - ref).abs() <= 5 * 2.0 ** -24 * mag).all())
    assert bool((y[2] == 0).all()) and bool((dx[T - 3] == 0).all())
    ref_dot = {t: (yp[slot[t, :3].long()].double() * dy[t].double()).sum(1) for t in tokens}
    mag_dot = {t: (yp[slot[t, :3].long()].double() * dy[t].double()).abs().sum(1) for t in tokens}
    dyp = torch.empty_like(yp)
    tcr.moe_combine_backward(dims, tcr.MOE_BF16, dy, yp, slot, w, dyp, wp, None, dtw)
    for t in tokens:
        p = slot[t, :3].long()
        ref = w[t, :3, None].double() * dy[t].double()
        assert bool(((dyp[p].double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01).all())
        assert torch.equal(wp[p], w[t, :3])
        assert bool(((dtw[t, :3].double() - ref_dot[t]).abs() <= 48 * 2.0 ** -24 * mag_dot[t]).all())
    assert bool((dtw[3] == 0).all())
    del yp, dyp
    # checkpoints of 2.3e9 elements
    rows, cols = 1100000, 2056
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    far = torch.tensor([0, 5, rows // 2, rows - 2, rows - 1], device="cuda")
    x[far] = torch.randn((5, cols), device="cuda").bfloat16()
    codes = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    scales = torch.empty(tcr.act8_scales_shape(rows, cols), dtype=torch.uint8, device="cuda")
    tcr.moe_act8_pack(x, codes, scales)
    q, s, v = R.act8(x[far].double().cpu().numpy())
    np.testing.assert_array_equal(codes[far].cpu().numpy(), q)
    np.testing.assert_array_equal(scales[far].cpu().numpy(), s)
    x.fill_(7.0)
    tcr.moe_act8_unpack(codes, scales, x)
    np.testing.assert_array_equal(x[far].double().cpu().numpy(), v)
    dg = torch.empty_like(x)
    dw = torch.empty((rows,), device="cuda")
    tcr.moe_swiglu_backward8(codes, scales, codes, scales, x, dg, codes.new_empty((rows, cols), dtype=torch.bfloat16),
                             dw=dw)
    rg, _, _, rw = R.swiglu_backward(v, v, v)
    got = dg[far].double().cpu().numpy()
    assert np.abs(got - rg).max() <= 2.0 ** -8 * np.abs(rg).max() * 1.01
    np.testing.assert_allclose(dw[far].double().cpu().numpy(), rw, rtol=1e-4)
