"""The layer's 8-bit training pair with weights that are not finite: the gate/up launch
that encodes in its epilogue (256 x 256 tiles) and the packed path. A NaN or an infinity
in an expert's pre-activations makes its blocks NaN in the state and that expert's
gradients NaN; y stays the forward's, and what does not depend on the expert is left as
it is."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_train8 import PAIR, _state
from token_choice_routing_amd.layer import MoeLayer, to_device
from workloads import bf16_round, generate
from workloads.configs import Config

pytestmark = pytest.mark.gpu

NAN, INF = 0x7FC0, 0x7F80  # bf16 bit patterns


def _run(cfg, wl):
    layer = MoeLayer(wl)
    layer.forward()
    y, offsets = layer.y.clone(), layer.offsets.cpu().numpy()
    layer.forward_train8()
    same = (layer.y == y) | (torch.isnan(layer.y) & torch.isnan(y))
    assert bool(same.all()), "forward_train8 y differs from the forward's"
    dy = to_device(bf16_round(np.random.default_rng(7).standard_normal((cfg.T, cfg.d_model)).astype(np.float32)))
    grads = {k: v.clone() for k, v in layer.backward_saved8(dy, 2e-2, 1e-3).items() if v is not None}
    return _state(layer), offsets, grads


@pytest.mark.parametrize("case", ["keep_ragged", "small"])
def test_weights_that_are_not_finite(case):
    cfg = Config(name=f"train8_nonfinite_{case}", dtype="bf16", w_std=None, seed=3, **PAIR[case])
    wl = generate(cfg)
    say(f"  {case}: T={cfg.T} F={cfg.d_ff} Fs={cfg.d_ff_shared}")
    clean, offsets, ref = _run(cfg, wl)
    # expert 0: one gate row NaN (the block of column 5), expert 1: one up value infinite
    # (the last block, a short one in keep_ragged)
    wl.w_gate[0, 5, :] = NAN
    wl.w_up[1, cfg.d_ff - 1, 0] = INF
    state, off, got = _run(cfg, wl)
    assert (off == offsets).all()  # the router does not see the experts' weights
    a, b, c = offsets[:3]
    assert b > a and c > b
    real = offsets[cfg.n_experts]
    last = (cfg.d_ff - 1) // 32 * 32
    for i, (r0, r1, col) in ((0, (a, b, 0)), (1, (b, c, last))):
        val, step = state[i]
        hit = np.zeros(val.shape, bool)
        hit[r0:r1, col:col + 32] = True
        assert (step[hit] == 2.0 ** 128).all() and (val[hit] == 0).all()  # byte 255, codes 0
        hit[real:] = True  # rows behind the real slots are not written
        assert (step[~hit] == clean[i][1][~hit]).all() and (val[~hit] == clean[i][0][~hit]).all()
    for i in (2, 3):  # the shared expert's
        assert all((x == y).all() for x, y in zip(state[i], clean[i]))
    # gradients of the other experts' weights: the same bits; those of the two: not finite,
    # but for du = dh silu(g), which does not depend on u
    for k in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(got[k][2:], ref[k][2:]), k
        assert not bool(torch.isfinite(got[k][0]).all()), k
        if k == "dw_up":
            assert torch.equal(got[k][1], ref[k][1])
        else:
            assert not bool(torch.isfinite(got[k][1]).all()), k
    for k in ("dws_gate", "dws_up", "dws_down"):
        if k in ref:
            assert torch.equal(got[k], ref[k]), k
