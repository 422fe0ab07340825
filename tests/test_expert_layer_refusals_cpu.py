"""What the expert layer's plan refuses after it was made."""
import pytest

from combine_mp_layout_gb300 import binding as B
from combine_mp_layout_gb300.pipeline import MoELayerPlan


@pytest.mark.parametrize("weights", ["e4m3", "bf16", "mxfp4"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_of_a_plan_for_the_forward_pass_alone(monkeypatch, weights, accumulate):
    """Refused before any operator is called."""
    monkeypatch.setattr(B, "mp_route_workspace_size", lambda R, N, E: 64)
    calls = []
    for name in dir(B):
        if name.startswith("mp_") and not name.endswith("size"):
            monkeypatch.setattr(B, name, lambda *a, name=name, **k: calls.append(name) or 0)
    monkeypatch.setattr(B, "_arr", lambda *a: 0)
    plan = MoELayerPlan(2, 4, 2, 8, 128, 128, device="cpu", weights=weights, train=False)
    plan.forward(None, None, None, None, None, None)
    calls.clear()
    with pytest.raises(ValueError, match="train=False"):
        plan.backward(None, None, None, None, None, None, accumulate=accumulate)
    assert calls == []
