"""The whole expert layer with bf16 and with 4-bit weights against 64 bits, with the kernels'
choice of experts.

Tolerance: every array between the operators is rounded to bf16, 2^-8 / sqrt(3) of a value in the
2-norm.  Forward these are gate and up (which the activation multiplies: at most twice their
relative error), its output, the down product and the combined rows: below 2^-8 * sqrt(7 / 3);
the gradients pass through at most six roundings more, the activation's derivative among them:
2^-8 * sqrt(7 / 3 + 6 * 4 / 3) is below 2^-6.  With few tokens one expert's rows may weigh more
than others: a factor of two.

The logits' gradients are not bounded by their own size: the gradient of a routing weight is a sum
over the inner channels, and the logits' are differences of these, so both can cancel.  A term's
error is its roundings' (at most 2^-5 of it, as above), independent of the others', so the sum's
is 2^-5 of the terms' 2-norm; a logit's gradient is scale * p_j * (dw_j - sum_k p_k dw_k), so its
error is within scale * 2 * 2^-5 of the token's largest such norm.
"""
import math

import pytest
import torch

from combine_mp_layout_gb300 import binding as B
from combine_mp_layout_gb300.pipeline import MoELayerPlan

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16
TOL = 2.0 ** -5


class Problem:
    def __init__(self, R, N, K, E, H, I, seed, weights="bf16"):
        from combine_mp_layout_gb300.moe_layer import quantise_weights_mxfp4
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device=DEV)
        self.R, self.N, self.K, self.E, self.H, self.I = R, N, K, E, H, I
        self.x, self.d_out = rand(R, N, H).to(BF), rand(R, N, H).to(BF)
        self.logits, self.d_loss = rand(R, N, E) * 1.5, rand(R)
        self.active = (torch.rand((R, N), generator=g, device=DEV) < 0.9).to(torch.uint8)
        self.active[0, 0] = 1
        up, down = rand(E, 2 * I, H) / math.sqrt(H), rand(E, H, I) / math.sqrt(I)
        if weights == "bf16":
            self.up, self.down = (up.to(BF), None), (down.to(BF), None)
            self.up64, self.down64 = self.up[0].double(), self.down[0].double()
        else:
            from tests.test_expert_bf16_gpu import fp4_ref
            self.up, self.down = quantise_weights_mxfp4(up), quantise_weights_mxfp4(down)
            self.up64, self.down64 = fp4_ref(*self.up), fp4_ref(*self.down)

    def reference(self, plan, scale, coef):
        """Output and gradients in 64 bits, the choice of experts being the plan's, and per token
        the largest 2-norm of the terms of a routing weight's gradient."""
        from tests.test_expert_ops_gpu import objective_ref
        xd, ld, up, down = (t.double().requires_grad_(True)
                            for t in (self.x, self.logits, self.up64, self.down64))
        lost = ~self.active.bool()[..., None]
        masked = torch.where(lost, torch.full_like(ld, -math.inf), ld)
        R, N, K, I = self.R, self.N, self.K, self.I
        _, w, loss = objective_ref(masked, plan.topk_idx, plan.num_tokens_per_expert,
                                   plan.num_routed, B.MP_SOFTMAX, True, scale, coef,
                                   torch.zeros((R, N, K), device=DEV), torch.zeros(R, device=DEV), K)
        out = torch.zeros((R, N, self.H), dtype=torch.float64, device=DEV)
        size = torch.zeros((R, N), dtype=torch.float64, device=DEV)
        for k in range(K):
            e = plan.topk_idx[..., k].long()
            ec = e.clamp(min=0)
            a, u = torch.einsum("rnh,rnih->rni", xd, up[ec]).split(I, -1)
            z = a * torch.sigmoid(a) * u
            dz = torch.einsum("rnh,rnhi->rni", self.d_out.double(), down[ec])
            size = torch.maximum(size, torch.where(e >= 0, (dz * z).detach().norm(dim=-1), 0.0))
            z = z * w[..., k:k + 1]
            out = out + torch.where((e >= 0)[..., None],
                                    torch.einsum("rni,rnhi->rnh", z, down[ec]), 0.0)
        total = (out * self.d_out.double()).sum() + (loss * self.d_loss.double()).sum()
        return (out.detach(),) + torch.autograd.grad(total, (xd, ld, up, down)) + (size,)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("R,N,K,E,H,I", [(2, 37, 2, 8, 256, 384), (1, 1, 2, 4, 136, 72),
                                         (2, 150, 3, 6, 264, 200)])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_layer_bf16(R, N, K, E, H, I, grad):
    p = Problem(R, N, K, E, H, I, 1)
    plan = MoELayerPlan(R, N, K, E, H, I, scale=1.5, loss_coef=0.1, weights="bf16", grad_dtype=grad)
    plan.forward(p.x, p.logits, *p.up, *p.down, active=p.active)
    plan.backward(p.d_out, p.logits, *p.up, *p.down, d_balance_loss=p.d_loss, active=p.active)
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    out, dx, dlog, dup, ddown, size = p.reference(plan, 1.5, 0.1)
    assert off(plan.out, out) <= TOL
    for got, want in ((plan.d_x, dx), (plan.d_w_gate_up, dup), (plan.d_w_down, ddown)):
        assert got.dtype is (grad if got is not plan.d_x else BF)
        assert off(got, want) <= TOL
    live = p.active.bool()
    bound = TOL * (dlog.abs() + 2 * 1.5 * size[..., None])
    assert bool(((plan.d_logits.double() - dlog).abs() <= bound)[live].all())
    assert float(plan.d_logits[~live].abs().max() if bool((~live).any()) else 0.0) == 0.0


def test_layer_bf16_gradients_of_two_batches_add_up():
    R, N, K, E, H, I = 2, 40, 2, 8, 256, 128
    one, two = Problem(R, N, K, E, H, I, 2), Problem(R, N, K, E, H, I, 3)
    two.up, two.down = one.up, one.down
    plan = MoELayerPlan(R, N, K, E, H, I, weights="bf16", grad_dtype=torch.float32)

    def step(p, accumulate):
        plan.forward(p.x, p.logits, *p.up, *p.down, active=p.active)
        plan.backward(p.d_out, p.logits, *p.up, *p.down, active=p.active, accumulate=accumulate)
        torch.cuda.synchronize()
        return plan.d_w_gate_up.clone(), plan.d_w_down.clone()
    alone = [step(p, False) for p in (one, two)]
    step(one, False)
    both = step(two, True)
    for a, b, c in zip(alone[0], alone[1], both):
        assert torch.equal(a + b, c)  # one fp32 addition
    assert plan.device_error() == 0
    with pytest.raises(ValueError):
        MoELayerPlan(R, N, K, E, H, I, weights="bf16").backward(
            one.d_out, one.logits, *one.up, *one.down, accumulate=True)


@pytest.mark.parametrize("R,N,K,E,H,I", [(2, 37, 2, 8, 256, 384), (1, 1, 2, 4, 160, 96),
                                         (2, 150, 3, 6, 288, 224)])
def test_layer_mxfp4(R, N, K, E, H, I):
    p = Problem(R, N, K, E, H, I, 4, weights="mxfp4")
    plan = MoELayerPlan(R, N, K, E, H, I, scale=1.5, weights="mxfp4", train=False)
    plan.forward(p.x, p.logits, *p.up, *p.down, active=p.active)
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    assert off(plan.out, p.reference(plan, 1.5, 0.01)[0]) <= TOL


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_layer_in_a_graph_and_two_plans_at_once(weights):
    """Captured layers share nothing: replays of two plans on two streams give what each gives
    alone, and so do further replays with other tokens in the same buffers."""
    R, N, K, E, H, I = 1, 24, 2, 8, 256, 128
    train = weights == "bf16"
    probs = [Problem(R, N, K, E, H, I, s, weights=weights) for s in (5, 6)]
    plans = [MoELayerPlan(R, N, K, E, H, I, weights=weights, train=train) for _ in probs]

    def step(plan, p):
        plan.forward(p.x, p.logits, *p.up, *p.down, active=p.active)
        if train:
            plan.backward(p.d_out, p.logits, *p.up, *p.down, active=p.active)

    def outputs(plan):
        return [plan.out] + ([plan.d_x, plan.d_logits, plan.d_w_gate_up, plan.d_w_down]
                             if train else [])
    graphs = []
    for plan, p in zip(plans, probs):
        step(plan, p)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(plan, p)
        graphs.append(graph)
    for turn in range(3):
        if turn == 2:
            for p in probs:
                p.x.neg_()
        want = []
        for plan, p in zip(plans, probs):
            step(plan, p)
            torch.cuda.synchronize()
            want.append([t.clone() for t in outputs(plan)])
            for t in outputs(plan):
                t.zero_()
        streams = [torch.cuda.Stream() for _ in plans]
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for plan, w in zip(plans, want):
            assert all(torch.equal(a, b) for a, b in zip(outputs(plan), w))
    assert all(plan.device_error() == 0 for plan in plans)


@pytest.mark.parametrize("weights", ["bf16", "mxfp4"])
def test_layer_example(weights, capsys):
    from combine_mp_layout_gb300 import moe_layer
    moe_layer.main(["--ranks", "2", "--tokens", "16", "--hidden", "256", "--inner", "128",
                    "--experts", "8", "--topk", "2", "--steps", "1", "--weights", weights])
    text = capsys.readouterr().out
    assert "balance loss" in text and ("d_w_down" in text) == (weights == "bf16")
