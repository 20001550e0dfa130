"""GPU parity of the layer's 8-bit training pair, moe_layer_forward_train8 and
moe_layer_backward_saved8.

y is moe_layer_forward's bit for bit. The checkpoints are read from the state: each
block's step must be the one of its exact g or u and each value within half a step of it
(a step where clamped), give or take the float32 GEMM's own error, at most
d 2^-24 sum |x w|. The gradients are then held, with the backward's own tolerances, to the
float64 backward oracle in which every expert's g and u are those values: nothing but the
backward's bf16 and float32 roundings is left between the two.

Against the exact gradients the 8-bit values themselves count. A block of 32 normal
values has a largest value below 3 sigma in the mean square, its step is at most 2^-6 of
that and the error's RMS a step / sqrt(12): 0.0135 sigma at most. du = dh silu(z) and
h = silu(z) u carry that of z (times silu', at most 1.1) and u: relative RMS at most
sqrt(2) 0.0135 1.1 = 2.1%; with the bf16 roundings (0.3%) 3e-2 holds with room."""
import numpy as np
import pytest
import torch

from oracle import moe_backward as B
from oracle import moe_oracle as O
from oracle import rows as R
from tests.gpu_util import say, vals
from tests.test_gpu_backward import CASES, TRAIN_CASES, _check, _ratios
from token_choice_routing_amd.layer import MoeLayer, to_device, to_host
from workloads import bf16_round, generate
from workloads.configs import Config

pytestmark = pytest.mark.gpu

PAIR = dict(CASES, **TRAIN_CASES,
            # the keeping gate/up launch on d_ff and d_ff_shared that are not multiples of
            # 16 or 32: short last blocks, 8-byte code stores
            keep_ragged=dict(T=2048, d_model=128, n_experts=4, n_null=4, top_k=2, d_ff=168, d_ff_shared=104),
            one_token=dict(T=1, d_model=64, n_experts=8, n_null=8, top_k=4, d_ff=40, d_ff_shared=24))


def _state(layer):
    """Values and steps of the checkpoints in layer.state8: routed g, u, shared g, u."""
    c, T = layer.cfg, layer.T
    TK, rows = T * c.top_k, T * min(c.top_k, c.n_experts)
    raw, at = layer.state8.cpu().numpy(), 0

    def take(n):
        nonlocal at
        piece, at = raw[at:at + n], at + (n + 255) // 256 * 256
        return piece

    for n in (T * (c.n_experts + 1), TK, TK, c.n_experts + 1, rows, TK, c.n_experts + c.n_null):
        take(4 * n)
    out = []
    for r, F in ((rows, c.d_ff), (rows, c.d_ff), (T, c.d_ff_shared), (T, c.d_ff_shared)):
        nb = -(-F // 32)
        q = take(r * F).view(np.int8).reshape(r, F).astype(np.float64)
        step = np.ldexp(1.0, take(r * nb).reshape(r, nb).astype(int) - 127).repeat(32, 1)[:, :F]
        out.append((q * step, step))
    return out


def _check_kept(v, kept, slack, what):
    """kept = (values, steps) against the exact values v, known to within slack."""
    val, step = kept
    assert (step > 0).all()
    clamped = np.abs(v) + slack > 127.5 * step
    assert (np.abs(v - val) <= np.where(clamped, step, step / 2) + slack).all(), what
    for c in range(0, v.shape[1], 32):
        amax, s = np.abs(v[:, c:c + 32]).max(1), slack[:, c:c + 32].max(1)
        # 2^6 steps <= amax < 2^7 steps
        assert (64 * step[:, c] <= amax + s).all() and (amax - s < 128 * step[:, c]).all(), what


class _Kept:
    """The oracle's experts on the kept g and u: the forward and the backward oracle visit
    the routed rows in expert order, then the shared expert's."""

    def __init__(self, layer, real_rows):
        self.g, self.u, self.gs, self.us = _state(layer)
        self.rows, self.at = real_rows, {"ffn": 0, "bwd": 0}

    def _next(self, who, a, wg, wu):
        n, i = a.shape[0], self.at[who]
        shared = i >= self.rows
        g, u = (self.gs, self.us) if shared else (self.g, self.u)
        i = 0 if shared else i
        self.at[who] += n
        g, u = [(x[0][i:i + n], x[1][i:i + n]) for x in (g, u)]
        for k, w in ((g, wg), (u, wu)):
            slack = a.shape[1] * 2.0 ** -24 * (np.abs(a) @ np.abs(w).T)
            _check_kept(a @ w.T, k, slack, f"{who} rows {i}..{i + n} shared {shared}")
        return g[0], u[0]

    def ffn(self, a, w_gate, w_up, w_down):
        g, u = self._next("ffn", np.asarray(a, np.float64), O._vals(w_gate), O._vals(w_up))
        return R.swiglu(g, u) @ O._vals(w_down).T

    def backward(self, a, w_gate, w_up, w_down, dY):
        a = np.asarray(a, np.float64)
        wg, wu, wd = O._vals(w_gate), O._vals(w_up), O._vals(w_down)
        g, u = self._next("bwd", a, wg, wu)
        dg, du, h, _ = R.swiglu_backward(g, u, dY @ wd)
        return dict(dw_gate=dg.T @ a, dw_up=du.T @ a, dw_down=dY.T @ h, da=dg @ wg + du @ wu)


def _layer(case, seed=0, null_bias=None):
    cfg = Config(name=f"train8_{case}", dtype="bf16", w_std=None, seed=seed, **PAIR[case])
    wl = generate(cfg)
    if null_bias is not None:
        wl.null_bias_tok = np.full(cfg.T, null_bias, dtype=np.float32)
    dy = bf16_round(np.random.default_rng(seed + 7).standard_normal((cfg.T, cfg.d_model)).astype(np.float32))
    say(f"  8-bit pair {case} T={cfg.T} d={cfg.d_model} F={cfg.d_ff} Fs={cfg.d_ff_shared} null bias {null_bias}")
    return cfg, wl, MoeLayer(wl), dy


@pytest.mark.parametrize("case", list(PAIR))
def test_pair_matches_the_oracle_with_8bit_preactivations(case, monkeypatch):
    cfg, wl, layer, dy_bits = _layer(case)
    layer.forward()
    out = layer.results()
    aux = {k: getattr(layer, k).clone() for k in ("counts", "P", "scalars")}
    y = layer.y.clone()
    layer.y.zero_()
    layer.forward_train8()
    torch.cuda.synchronize()
    assert torch.equal(layer.y, y), "forward_train8 y differs from the forward's"
    for k, v in aux.items():
        assert torch.equal(getattr(layer, k), v), k
    dy = to_device(dy_bits)
    layer.ws_train8.fill_(255)  # nothing of the forward's workspace is needed
    got = {k: to_host(v) if v is not None else None for k, v in layer.backward_saved8(dy, 2e-2, 1e-3).items()}
    kept = _Kept(layer, int(out["offsets"][cfg.n_experts]))
    monkeypatch.setattr(B, "_swiglu_backward", kept.backward)
    monkeypatch.setattr(O, "swiglu_ffn", kept.ffn)
    ref = B.layer_backward(wl, vals(dy_bits), 2e-2, 1e-3, logits=out["logits"].astype(np.float64))
    if cfg.T > 1:
        _check(cfg, got, ref)
    else:
        for k in ("dx", "dw_gate", "dw_up", "dw_down", "dws_gate", "dws_up", "dws_down"):
            assert _ratios(got[k], ref[k])[0] <= 1e-2, k
    # the state is only read: a second backward gives the same bits
    again = layer.backward_saved8(dy, 2e-2, 1e-3)
    for k, v in again.items():
        if v is not None:
            np.testing.assert_array_equal(to_host(v), got[k], err_msg=k)


@pytest.mark.parametrize("null_bias", [1e3, np.inf])
def test_pair_without_routed_rows(null_bias):
    cfg, _, layer, dy_bits = _layer("keep_fused", null_bias=null_bias)
    layer.forward()
    y = layer.y.clone()
    layer.forward_train8()
    assert torch.equal(layer.y, y)
    dy = to_device(dy_bits)
    ref = {k: v.clone() for k, v in layer.backward(dy, 2e-2, 1e-3).items()}
    got = layer.backward_saved8(dy, 2e-2, 1e-3)
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert bool((got[k] == 0).all()), k
    assert torch.equal(got["dw_router"], ref["dw_router"])
    for k in ("dx", "dws_gate", "dws_up", "dws_down"):
        r = _ratios(to_host(got[k]), to_host(ref[k]).astype(np.float64))[0]
        assert r <= 3e-2, (k, r)


def test_layers_share_a_workspace():
    """Two layers, forwards first and backwards in reverse, one workspace between them."""
    a, b = _layer("keep_fused", seed=1), _layer("small", seed=2)
    alone = []
    for _, _, layer, dy in (a, b):
        layer.forward_train8()
        g = layer.backward_saved8(to_device(dy), 2e-2, 1e-3)
        alone.append({k: v.clone() for k, v in g.items() if v is not None})
    ws = max((a[2].ws_train8, b[2].ws_train8), key=lambda t: t.numel())
    for _, _, layer, _ in (a, b):
        layer.state8.fill_(255)
        layer.forward_train8(ws=ws)
    for (_, _, layer, dy), ref in zip((b, a), (alone[1], alone[0])):
        g = layer.backward_saved8(to_device(dy), 2e-2, 1e-3, ws=ws)
        for k, v in ref.items():
            assert torch.equal(g[k], v), k


def test_pair_replays_in_a_hip_graph():
    _, _, layer, dy_bits = _layer("keep_fused", seed=4)
    dy = to_device(dy_bits)
    layer.forward_train8()
    ref = {k: v.clone() for k, v in layer.backward_saved8(dy, 2e-2, 1e-3).items()}
    y = layer.y.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward_train8()
        layer.backward_saved8(dy, 2e-2, 1e-3)
    for rep in range(3):
        layer.y.zero_()
        for v in layer.grads.values():
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, y), rep
        for k, v in ref.items():
            assert torch.equal(layer.grads[k], v), (rep, k)
        layer.forward_train8()  # eager calls between the replays
        layer.backward_saved8(dy, 2e-2, 1e-3)
    del graph


def test_pair_full_size_headline_shape():
    """At the Qwen3-1.7B rho = 0.25 shape: y equals the forward's, every gradient is the
    stateless backward's within the 8-bit bound."""
    from workloads import CONFIGS
    cfg = CONFIGS["qwen3_1p7b_rho0p25"]
    say(f"  8-bit pair full size {cfg.name}")
    layer = MoeLayer(generate(cfg))
    layer.forward(aux=False)
    y = layer.y.clone()
    gen = torch.Generator(device="cuda").manual_seed(5)
    dy = torch.randn((layer.T, cfg.d_model), generator=gen, device="cuda").to(torch.bfloat16)
    ref = {k: v.clone() for k, v in layer.backward(dy, 2e-2, 1e-3).items() if v is not None}
    layer.forward_train8()
    assert torch.equal(layer.y, y)
    got = layer.backward_saved8(dy, 2e-2, 1e-3)
    for k, v in ref.items():
        r = float((got[k] - v).double().pow(2).mean().sqrt() / v.double().pow(2).mean().sqrt())
        say(f"  {k}: RMS(8-bit - exact) / RMS = {r:.3e}")
        assert r <= 3e-2, k
