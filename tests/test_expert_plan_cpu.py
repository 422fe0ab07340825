"""The expert layer's plan refuses tokens that the dispatch, which takes addresses, would misread."""
import pytest
import torch

from combine_mp_layout_gb300 import binding as B
from combine_mp_layout_gb300.pipeline import MoELayerPlan

R, N, K, E, H, I = 2, 4, 2, 8, 256, 128


class OnCuda(torch.Tensor):
    """A tensor that says it is on a GPU; nothing of it is read."""
    is_cuda = True


def on_cuda(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnCuda)


@pytest.fixture
def plan(monkeypatch):
    monkeypatch.setattr(B, "mp_route_workspace_size", lambda R, N, E: 64)
    for name in ("mp_route", "mp_dispatch_ll_rows_quant"):
        def reached(*a, name=name):
            raise AssertionError("%s was called" % name)
        monkeypatch.setattr(B, name, reached)
    return MoELayerPlan(R, N, K, E, H, I, device="cpu")


@pytest.mark.parametrize("bad,error", [
    (on_cuda(R, N, H, dtype=torch.float32), TypeError),
    (on_cuda(R, N, H, dtype=torch.float16), TypeError),
    (torch.zeros((R, N, H), dtype=torch.bfloat16), TypeError),
    (on_cuda(R, N, H // 2), ValueError), (on_cuda(R, N - 1, H), ValueError),
    (on_cuda(R, N, 2 * H)[..., :H], ValueError)])
def test_plan_refuses_other_tokens(plan, bad, error):
    with pytest.raises(error):
        plan.forward(bad, None, None, None, None, None)
    with pytest.raises(error):
        plan.backward(bad, None, None, None, None, None)


def test_plan_takes_dense_bf16_tokens(plan):
    for good in (on_cuda(R, N, H), on_cuda(R * N, H), on_cuda(R + 1, N, H)):
        with pytest.raises(AssertionError, match="mp_route was called"):
            plan.forward(good, None, None, None, None, None)
        with pytest.raises(AssertionError, match="mp_dispatch_ll_rows_quant was called"):
            plan.backward(good, None, None, None, None, None)
