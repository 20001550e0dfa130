"""MoeLayer's backwards from kept state ask for the forward that keeps it. Host only: the
library's calls are replaced by recorders, so that nothing is launched."""
import pytest
import torch

import token_choice_routing_amd.layer as L
from token_choice_routing_amd import MOE_WS_BACKWARD, MOE_WS_STATE8, workspace_bytes
from workloads import generate
from workloads.configs import Config

CFG = Config(name="state", T=16, d_model=64, n_experts=4, n_null=4, top_k=2, d_ff=64, d_ff_shared=0, dtype="bf16",
             w_std=None)


@pytest.fixture
def layer(monkeypatch):
    layer = L.MoeLayer(generate(CFG), device="cpu")
    layer.calls = []
    for name in ("moe_layer_forward_train", "moe_layer_backward_saved", "moe_layer_forward_train8",
                 "moe_layer_backward_saved8", "moe_layer_backward"):
        def call(dims, params, *args, name=name, **kw):
            layer.calls.append((name, args))
        monkeypatch.setattr(L, name, call)
    return layer


PAIRS = [("forward_train", "backward_saved", "ws_bwd", MOE_WS_BACKWARD),
         ("forward_train8", "backward_saved8", "state8", MOE_WS_STATE8)]


@pytest.mark.parametrize("forward,backward,buffer,which", PAIRS)
def test_backward_needs_its_forward(layer, forward, backward, buffer, which):
    dy = torch.zeros((CFG.T, CFG.d_model), dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match=f"no state of a forward: {forward}"):
        getattr(layer, backward)(dy)
    # buffers that exist for another reason are not a forward's state
    layer.backward(dy)
    for other in PAIRS:
        if other[0] != forward:
            getattr(layer, other[0])()
    layer._buffer(buffer, which)
    layer.calls.clear()
    with pytest.raises(RuntimeError, match=f"no state of a forward: {forward}"):
        getattr(layer, backward)(dy)
    assert layer.calls == []
    getattr(layer, forward)()
    state = getattr(layer, buffer)
    assert state.numel() >= workspace_bytes(layer.dims, which)
    for _ in range(2):  # the state is only read
        assert getattr(layer, backward)(dy) is layer.grads
        assert any(a is state for a in layer.calls[-1][1])


@pytest.mark.parametrize("forward,backward,buffer,which", PAIRS)
def test_forward_that_fails_leaves_no_state(layer, monkeypatch, forward, backward, buffer, which):
    dy = torch.zeros((CFG.T, CFG.d_model), dtype=torch.bfloat16)
    getattr(layer, forward)()

    def fail(*a, **kw):
        raise RuntimeError("launch failed")

    monkeypatch.setattr(L, f"moe_layer_{forward}", fail)
    with pytest.raises(RuntimeError, match="launch failed"):
        getattr(layer, forward)()
    with pytest.raises(RuntimeError, match="no state of a forward"):
        getattr(layer, backward)(dy)


@pytest.mark.parametrize("forward,backward,buffer,which", PAIRS)
def test_state_that_was_freed(layer, forward, backward, buffer, which):
    getattr(layer, forward)()
    setattr(layer, buffer, None)
    with pytest.raises(RuntimeError, match="no state of a forward"):
        getattr(layer, backward)(torch.zeros((CFG.T, CFG.d_model), dtype=torch.bfloat16))
    # a buffer allocated in its place does not hold the state either
    layer._buffer(buffer, which)
    with pytest.raises(RuntimeError, match="no state of a forward"):
        getattr(layer, backward)(torch.zeros((CFG.T, CFG.d_model), dtype=torch.bfloat16))
