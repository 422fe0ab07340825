"""One expert layer, forward and backward, on synthetic inputs.

    python -m combine_mp_layout_gb300.moe_layer [--tokens 512] [--ranks 8] [--hidden 4096]
        [--inner 2048] [--experts 64] [--topk 6] [--scoring softmax]

Draws tokens, a router and experts, quantises the experts' weights (e4m3, one fp32 scale per
128 x 128 block), runs ``pipeline.MoELayerPlan`` and prints the balance loss, the size of the
output and of the gradients, and the time of a pass.
"""
from __future__ import annotations

import argparse

import torch

from . import binding as B
from .pipeline import MoELayerPlan


def quantise_weights(w: torch.Tensor):
    """[E][N][K] to e4m3 codes and one fp32 scale per 128 x 128 block (amax / 448)."""
    E, N, K = w.shape
    nb, kb = -(-N // B.SCALE_BLOCK), K // B.SCALE_BLOCK
    padded = torch.zeros((E, nb * B.SCALE_BLOCK, K), dtype=torch.float32, device=w.device)
    padded[:, :N] = w
    blocks = padded.view(E, nb, B.SCALE_BLOCK, kb, B.SCALE_BLOCK)
    scales = blocks.abs().amax((2, 4)) / 448.0
    scales = torch.where(scales > 0, scales, torch.ones_like(scales))
    codes = (blocks / scales[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(E, -1, K)[:, :N].contiguous(), scales.contiguous()


def main(argv=None) -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=512, help="tokens per rank")
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=6)
    ap.add_argument("--scoring", choices=("softmax", "sigmoid"), default="softmax")
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args(argv)
    R, N, H, I, E, K = a.ranks, a.tokens, a.hidden, a.inner, a.experts, a.topk
    torch.manual_seed(0)
    dev = "cuda"
    x = torch.randn((R, N, H), device=dev).to(torch.bfloat16)
    router = torch.randn((H, E), device=dev) / H ** 0.5
    logits = x.float() @ router
    gate_up = quantise_weights(torch.randn((E, 2 * I, H), device=dev) / H ** 0.5)
    down = quantise_weights(torch.randn((E, H, I), device=dev) / I ** 0.5)
    d_out = torch.randn((R, N, H), device=dev).to(torch.bfloat16)
    d_loss = torch.ones(R, device=dev)
    plan = MoELayerPlan(R, N, K, E, H, I, scoring=a.scoring, device=dev)

    def step():
        plan.forward(x, logits, *gate_up, *down)
        plan.backward(d_out, logits, *gate_up, *down, d_balance_loss=d_loss)
    for _ in range(3):
        step()
    t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    t0.record()
    for _ in range(a.steps):
        step()
    t1.record()
    torch.cuda.synchronize()
    err = plan.device_error()
    if err:
        raise B.MPError(err, "moe_layer")
    print("balance loss per rank: " + " ".join("%.5f" % v for v in plan.balance_loss.tolist()))
    for name in ("out", "d_x", "d_logits", "d_w_gate_up", "d_w_down"):
        print("%-12s rms %.5f" % (name, getattr(plan, name).float().square().mean().sqrt()))
    print("forward + backward: %.3f ms for %d tokens" % (t0.elapsed_time(t1) / a.steps, R * N))


if __name__ == "__main__":
    main()
