"""What the expert layer's plan refuses of its kinds of weights, and the calls that it makes."""
import pytest
import torch

from combine_mp_layout_gb300 import binding as B
from combine_mp_layout_gb300.pipeline import MoELayerPlan

SIZE = (2, 4, 2, 8, 64, 32)


@pytest.fixture(autouse=True)
def sizes(monkeypatch):
    monkeypatch.setattr(B, "mp_route_workspace_size", lambda R, N, E: 64)


@pytest.mark.parametrize("bad", [
    dict(weights="fp8"), dict(weights="e4m3"),  # (64 and 32 are no multiples of 128)
    dict(weights="mxfp4"), dict(weights="mxfp4", train=True),
    dict(weights="bf16", grad_dtype=torch.float16),
    dict(weights="mxfp4", train=False, grad_dtype=torch.float32)])
def test_refusals(bad):
    with pytest.raises(ValueError):
        MoELayerPlan(*SIZE, device="cpu", **bad)


@pytest.mark.parametrize("size,weights", [((2, 4, 2, 8, 60, 32), "bf16"),
                                          ((2, 4, 2, 8, 64, 36), "bf16"),
                                          ((2, 4, 2, 8, 72, 32), "mxfp4"),
                                          ((2, 4, 2, 8, 64, 40), "mxfp4")])
def test_refuses_partial_blocks(size, weights):
    with pytest.raises(ValueError):
        MoELayerPlan(*size, device="cpu", weights=weights, train=False)


def test_e4m3_gradients_stay_bf16():
    with pytest.raises(ValueError):
        MoELayerPlan(2, 4, 2, 8, 128, 128, device="cpu", grad_dtype=torch.float32)


@pytest.mark.parametrize("weights", ["e4m3", "bf16", "mxfp4"])
def test_operators_called(monkeypatch, weights):
    calls = []
    for name in dir(B):
        if name.startswith("mp_") and not name.endswith("size"):
            monkeypatch.setattr(B, name, lambda *a, name=name, **k: calls.append(name) or 0)
    monkeypatch.setattr(B, "_arr", lambda *a: 0)
    train = weights != "mxfp4"
    plan = MoELayerPlan(2, 4, 2, 8, 128, 128, device="cpu", weights=weights, train=train)
    plan.forward(None, None, None, None, None, None)
    tail = {"e4m3": "e4m3", "bf16": "bf16", "mxfp4": "mxfp4"}[weights]
    gate = "e4m3" if weights == "e4m3" else "bf16"
    assert calls == ["mp_route", "mp_dispatch_ll_quant" if weights == "e4m3" else "mp_dispatch_ll",
                     "mp_ll_row_weights", "mp_expert_matmul_" + tail, "mp_swiglu_" + gate,
                     "mp_expert_matmul_" + tail, "mp_combine_ll"]
    if train:
        calls.clear()
        plan.backward(None, None, None, None, None, None)
        d, w = "mp_expert_matmul_dgrad_" + tail, "mp_expert_matmul_wgrad_" + tail
        assert calls == ["mp_dispatch_ll_rows" + ("_quant" if weights == "e4m3" else ""), d, w,
                         "mp_swiglu_backward_" + gate, w, d, "mp_combine_ll",
                         "mp_ll_row_weights_backward", "mp_route_backward"]
