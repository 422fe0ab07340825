"""Buffer allocation and call sequencing around the C ABI (torch is used for
device memory and streams only; every computation is a library kernel).

``EPPlan`` owns the device buffers of one (R, N, K, E, H, dtype) problem and
runs mp_layout -> mp_dispatch -> mp_combine on them; ``RSVPlan`` does the same
for mp_reducescatterv / mp_allgatherv; ``MoELayerPlan`` for a whole expert layer
(router, low-latency e4m3 dispatch, the experts' gated products, combine) and its
gradient.
"""
from __future__ import annotations

import torch

from . import binding as B


def _i32(n, dev):
    return torch.zeros(n, dtype=torch.int32, device=dev)


class EPPlan:
    def __init__(self, R: int, N: int, K: int, E: int, H: int, dtype: str = "bf16",
                 recv_capacity: int | None = None, device="cuda"):
        if dtype not in ("bf16", "e4m3"):
            raise ValueError("dtype must be bf16 or e4m3")
        self.R, self.N, self.K, self.E, self.H, self.dtype = R, N, K, E, H, dtype
        self.device = torch.device(device)
        dev = self.device
        self.cap = R * N * min(R, K) if recv_capacity is None else int(recv_capacity)
        ws = B.mp_workspace_size(R, N, E)
        if ws == 0:
            raise ValueError("invalid problem shape R=%d N=%d E=%d" % (R, N, E))
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=dev)
        self.dev_err = _i32(1, dev)
        # inputs
        self.topk_idx = torch.full((R, N, K), -1, dtype=torch.int32, device=dev)
        self.topk_weights = torch.zeros((R, N, K), dtype=torch.float32, device=dev)
        xdt = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
        self.x = torch.zeros((R, N, H), dtype=xdt, device=dev)
        self.x_scales = (torch.zeros((R, N, H // B.SCALE_BLOCK), dtype=torch.float32, device=dev)
                         if dtype == "e4m3" else None)
        # layout outputs
        self.num_tokens_per_rank = _i32((R, R), dev)
        self.num_tokens_per_expert = _i32((R, E), dev)
        self.is_token_in_rank = torch.zeros((R, N), dtype=torch.int32, device=dev)
        # dispatch outputs
        c1 = max(self.cap, 1)
        self.recv_x = torch.zeros((c1, H), dtype=xdt, device=dev)
        self.recv_scales = (torch.zeros((c1, H // B.SCALE_BLOCK), dtype=torch.float32, device=dev)
                            if dtype == "e4m3" else None)
        self.recv_src_rank = _i32(c1, dev)
        self.recv_src_idx = _i32(c1, dev)
        self.recv_topk_idx = _i32((c1, K), dev)
        self.recv_topk_weights = torch.zeros((c1, K), dtype=torch.float32, device=dev)
        self.dest_offsets = _i32(R + 1, dev)
        self.rank_prefix = _i32((R, R), dev)
        self.num_recv_tokens_per_expert = _i32((R, E // R), dev)
        self.send_row = _i32((R, N, R), dev)
        # combine output
        self.out = torch.zeros((R, N, H), dtype=torch.bfloat16, device=dev)

    def load(self, inp, non_blocking: bool = False) -> None:
        """Copy a workloads.EPInputs (CPU tensors / arrays) into the device inputs."""
        self.topk_idx.copy_(torch.as_tensor(inp.topk_idx), non_blocking=non_blocking)
        self.topk_weights.copy_(torch.as_tensor(inp.topk_weights), non_blocking=non_blocking)
        self.x.copy_(inp.x, non_blocking=non_blocking)
        if self.x_scales is not None:
            self.x_scales.copy_(inp.x_scales, non_blocking=non_blocking)

    def layout(self, stream=None) -> int:
        return B.mp_layout(self.R, self.N, self.K, self.E, self.topk_idx,
                           self.num_tokens_per_rank, self.num_tokens_per_expert,
                           self.is_token_in_rank, self.dev_err, self.workspace, stream)

    def dispatch(self, stream=None) -> int:
        return B.mp_dispatch(
            self.R, self.N, self.K, self.E, self.H,
            B.MP_BF16 if self.dtype == "bf16" else B.MP_E4M3, self.x, self.x_scales,
            self.topk_idx, self.topk_weights, self.is_token_in_rank, self.num_tokens_per_rank,
            self.num_tokens_per_expert, self.cap, self.recv_x, self.recv_scales,
            self.recv_src_rank, self.recv_src_idx, self.recv_topk_idx, self.recv_topk_weights,
            self.dest_offsets, self.rank_prefix, self.num_recv_tokens_per_expert, self.send_row,
            self.dev_err, self.workspace, stream)

    def layout_and_offsets(self, stream=None) -> int:
        """mp_layout + mp_dispatch_offsets in one call (one cooperative launch when the
        problem fits one resident grid)."""
        return B.mp_layout_and_offsets(
            self.R, self.N, self.K, self.E, self.topk_idx, self.topk_weights, self.cap,
            self.num_tokens_per_rank, self.num_tokens_per_expert, self.is_token_in_rank,
            self.recv_src_rank, self.recv_src_idx, self.recv_topk_idx, self.recv_topk_weights,
            self.dest_offsets, self.rank_prefix, self.num_recv_tokens_per_expert, self.send_row,
            self.dev_err, self.workspace, stream)

    def layout_dispatch(self, stream=None) -> int:
        """The whole dispatch in one call (mp_layout_dispatch): layout, receive offsets
        and row copy, the copy launched as a programmatic dependent of the offsets."""
        return B.mp_layout_dispatch(
            self.R, self.N, self.K, self.E, self.H,
            B.MP_BF16 if self.dtype == "bf16" else B.MP_E4M3, self.x, self.x_scales,
            self.topk_idx, self.topk_weights, self.cap, self.num_tokens_per_rank,
            self.num_tokens_per_expert, self.is_token_in_rank, self.recv_x, self.recv_scales,
            self.recv_src_rank, self.recv_src_idx, self.recv_topk_idx, self.recv_topk_weights,
            self.dest_offsets, self.rank_prefix, self.num_recv_tokens_per_expert, self.send_row,
            self.dev_err, self.workspace, stream)

    def dispatch_offsets(self, stream=None) -> int:
        return B.mp_dispatch_offsets(
            self.R, self.N, self.K, self.E, self.topk_idx, self.topk_weights,
            self.is_token_in_rank, self.num_tokens_per_rank, self.num_tokens_per_expert,
            self.cap, self.recv_src_rank, self.recv_src_idx, self.recv_topk_idx,
            self.recv_topk_weights, self.dest_offsets, self.rank_prefix,
            self.num_recv_tokens_per_expert, self.send_row, self.dev_err, self.workspace, stream)

    def dispatch_rows(self, x: torch.Tensor | None = None, x_scales=None, recv_x=None,
                      recv_scales=None, stream=None) -> int:
        """Copy rows with the current send_row (default: this plan's own x / recv_x)."""
        x = self.x if x is None else x
        return B.mp_dispatch_rows(
            self.R, self.N, self.H, B.MP_BF16 if self.dtype == "bf16" else B.MP_E4M3, x,
            self.x_scales if x_scales is None else x_scales, self.send_row, self.cap,
            self.recv_x if recv_x is None else recv_x,
            self.recv_scales if recv_scales is None else recv_scales, stream)

    def combine(self, y: torch.Tensor | None = None, stream=None) -> int:
        """Combine y (default: recv_x, i.e. identity experts) back into self.out."""
        y = self.recv_x if y is None else y
        if y.dtype != torch.bfloat16 or y.dim() != 2 or y.shape[1] != self.H:
            raise ValueError("combine takes bf16 rows [rows][H] (an e4m3 plan needs its "
                             "expert outputs as y)")
        return B.mp_combine(self.R, self.N, self.H, y, y.shape[0], self.send_row, self.out,
                            self.dev_err, stream)

    def step(self, y: torch.Tensor | None = None, stream=None) -> None:
        """One pass of the hot path: layout -> dispatch -> combine as two calls (the whole
        dispatch in one call, then combine)."""
        B.check(self.layout_dispatch(stream), "mp_layout_dispatch")
        B.check(self.combine(y, stream), "mp_combine")

    def step_three_calls(self, y: torch.Tensor | None = None, stream=None) -> None:
        """The same pass as three calls: layout and receive offsets, row copy, combine."""
        B.check(self.layout_and_offsets(stream), "mp_layout_and_offsets")
        B.check(self.dispatch_rows(stream=stream), "mp_dispatch_rows")
        B.check(self.combine(y, stream), "mp_combine")

    def num_recv(self) -> int:
        return int(self.dest_offsets[self.R].item())

    def device_error(self) -> int:
        return int(self.dev_err.item())


class RSVPlan:
    def __init__(self, R: int, H: int, sizes, device="cuda"):
        self.R, self.H = R, H
        self.sizes = [int(s) for s in sizes]
        self.S = sum(self.sizes)
        dev = torch.device(device)
        self.x = torch.zeros((R, self.S, H), dtype=torch.bfloat16, device=dev)
        self.rs_out = torch.zeros((self.S, H), dtype=torch.bfloat16, device=dev)
        self.shards = torch.zeros((self.S, H), dtype=torch.bfloat16, device=dev)
        self.ag_out = torch.zeros((R, self.S, H), dtype=torch.bfloat16, device=dev)

    def reducescatterv(self, stream=None) -> int:
        return B.mp_reducescatterv(self.R, self.H, self.sizes, self.x, self.rs_out, stream)

    def allgatherv(self, stream=None) -> int:
        return B.mp_allgatherv(self.R, self.H * 2, self.sizes, self.shards, self.ag_out, stream)


class MoELayerPlan:
    """One expert layer: tokens x [R][N][H] and router logits [R][N][E] in, bf16 [R][N][H] out.

    Expert e computes w_down[e] (silu(g) * u), (g, u) = w_gate_up[e] x, on e4m3 rows; its
    weights are e4m3 with one fp32 scale per 128 x 128 block: w_gate_up [E][2I][H] (the gate's
    channels first) and w_down [E][H][I].  ``forward`` leaves what ``backward`` needs in the
    plan's buffers.

    The weights' gradients are sums in fp32 of products of e4m3 rows held in f16: relative to
    the largest scale of their 128 channels in the expert's rows, so rows whose scale is
    below 2^-19 of it lose bits and below 2^-30 are lost (``mp_expert_matmul_wgrad_e4m3``).
    """

    def __init__(self, R: int, N: int, K: int, E: int, H: int, I: int, scoring: str = "softmax",
                 normalize: bool = True, scale: float = 1.0, loss_coef: float = 0.01,
                 logits_dtype=torch.float32, recv_capacity: int | None = None, train: bool = True,
                 device="cuda"):
        if scoring not in ("softmax", "sigmoid"):
            raise ValueError("scoring must be softmax or sigmoid")
        if H % B.SCALE_BLOCK or I % B.SCALE_BLOCK:
            raise ValueError("H and I must be multiples of %d" % B.SCALE_BLOCK)
        self.R, self.N, self.K, self.E, self.H, self.I = R, N, K, E, H, I
        self.scoring = B.MP_SOFTMAX if scoring == "softmax" else B.MP_SIGMOID
        self.normalize, self.scale, self.loss_coef = normalize, scale, loss_coef
        dev = self.device = torch.device(device)
        self.cap = cap = R * N * K if recv_capacity is None else int(recv_capacity)
        ws = B.mp_route_workspace_size(R, N, E)
        if ws == 0:
            raise ValueError("invalid problem shape R=%d N=%d E=%d" % (R, N, E))

        def buf(shape, dtype):
            return torch.zeros(shape, dtype=dtype, device=dev)
        f32, bf16, f8, nb = torch.float32, torch.bfloat16, torch.float8_e4m3fn, B.SCALE_BLOCK
        self.workspace = buf(ws, torch.uint8)
        self.dev_err = _i32(1, dev)
        # router
        self.topk_idx, self.topk_weights = _i32((R, N, K), dev), buf((R, N, K), f32)
        self.num_tokens_per_expert, self.num_routed = _i32((R, E), dev), _i32(R, dev)
        self.balance_loss = buf(R, f32)
        # expert-major rows
        self.expert_offsets, self.expert_src_offsets = _i32(E + 1, dev), _i32((E, R), dev)
        self.recv_src_token, self.slot_row = _i32(max(cap, 1), dev), _i32((R, N, K), dev)
        self.recv_x, self.recv_scales = buf((cap, H), f8), buf((cap, H // nb), f32)
        self.row_weights = buf(cap, f32)
        # experts
        self.gate_up = buf((cap, 2 * I), bf16)
        self.z, self.z_scales = buf((cap, I), f8), buf((cap, I // nb), f32)
        self.y = buf((cap, H), bf16)
        self.ones = torch.ones((R, N, K), dtype=f32, device=dev)
        self.out = buf((R, N, H), bf16)
        if train:
            self.dy, self.dy_scales = buf((cap, H), f8), buf((cap, H // nb), f32)
            self.dz = buf((cap, I), bf16)
            self.d_gate_up = buf((cap, 2 * I), f8)
            self.d_gate_up_scales = buf((cap, 2 * I // nb), f32)
            self.d_row_weights = buf(cap, f32)
            self.d_rows = buf((cap, H), bf16)
            self.d_x = buf((R, N, H), bf16)
            self.d_w_gate_up, self.d_w_down = buf((E, 2 * I, H), bf16), buf((E, H, I), bf16)
            self.d_topk_weights = buf((R, N, K), f32)
            self.d_logits = buf((R, N, E), logits_dtype)

    @property
    def _num_rows(self):
        return self.expert_offsets[self.E:]

    def forward(self, x, logits, w_gate_up, w_gate_up_scales, w_down, w_down_scales, bias=None,
                active=None, stream=None):
        """The layer's output (self.out); self.balance_loss holds the loss per rank."""
        R, N, K, E, H, I, cap = (self.R, self.N, self.K, self.E, self.H, self.I, self.cap)
        # (the dispatches read what stands at an address, whatever it is)
        B._arr(x, "x", torch.bfloat16, R * N * H)
        B.check(B.mp_route(R, N, K, E, self.scoring, logits, bias, active, self.normalize,
                           self.scale, self.loss_coef, self.topk_idx, self.topk_weights,
                           self.num_tokens_per_expert, self.num_routed, self.balance_loss,
                           self.dev_err, self.workspace, stream), "mp_route")
        # (small batches: the dispatch that counts for itself is one kernel)
        counts = self.num_tokens_per_expert if R * N * K > 16384 else None
        B.check(B.mp_dispatch_ll_quant(R, N, K, E, H, B.MP_Q_E4M3, 0, x, self.topk_idx, counts,
                                       cap, self.expert_offsets, self.expert_src_offsets,
                                       self.recv_src_token, self.slot_row, self.recv_x,
                                       self.recv_scales, self.dev_err, stream),
                "mp_dispatch_ll_quant")
        B.check(B.mp_ll_row_weights(R, N, K, self.topk_weights, self.slot_row, cap,
                                    self.row_weights, stream), "mp_ll_row_weights")
        B.check(B.mp_expert_matmul_e4m3(E, cap, 2 * I, H, self.recv_x, self.recv_scales, w_gate_up,
                                        w_gate_up_scales, self.expert_offsets, self.gate_up,
                                        self.dev_err, stream), "mp_expert_matmul_e4m3")
        B.check(B.mp_swiglu_e4m3(cap, I, self.gate_up, self.row_weights, self._num_rows, self.z,
                                 self.z_scales, stream), "mp_swiglu_e4m3")
        B.check(B.mp_expert_matmul_e4m3(E, cap, H, I, self.z, self.z_scales, w_down, w_down_scales,
                                        self.expert_offsets, self.y, self.dev_err, stream),
                "mp_expert_matmul_e4m3")
        B.check(B.mp_combine_ll(R, N, K, H, self.y, cap, self.slot_row, self.ones, self.out,
                                self.dev_err, stream), "mp_combine_ll")
        return self.out

    def backward(self, d_out, logits, w_gate_up, w_gate_up_scales, w_down, w_down_scales,
                 d_balance_loss=None, active=None, stream=None):
        """Gradients of a forward pass, from the output's (and the losses'): d_x, d_logits,
        d_w_gate_up, d_w_down of the plan."""
        R, N, K, E, H, I, cap = (self.R, self.N, self.K, self.E, self.H, self.I, self.cap)
        B._arr(d_out, "d_out", torch.bfloat16, R * N * H)
        B.check(B.mp_dispatch_ll_rows_quant(R, N, K, H, B.MP_Q_E4M3, d_out, self.slot_row, cap,
                                            self.dy, self.dy_scales, stream),
                "mp_dispatch_ll_rows_quant")
        B.check(B.mp_expert_matmul_dgrad_e4m3(E, cap, H, I, self.dy, self.dy_scales, w_down,
                                              w_down_scales, self.expert_offsets, self.dz,
                                              self.dev_err, stream), "mp_expert_matmul_dgrad_e4m3")
        B.check(B.mp_expert_matmul_wgrad_e4m3(E, cap, H, I, self.dy, self.dy_scales, self.z,
                                              self.z_scales, self.expert_offsets, self.d_w_down,
                                              self.dev_err, stream), "mp_expert_matmul_wgrad_e4m3")
        B.check(B.mp_swiglu_backward_e4m3(cap, I, self.gate_up, self.row_weights, self.dz,
                                          self._num_rows, self.d_gate_up, self.d_gate_up_scales,
                                          self.d_row_weights, stream), "mp_swiglu_backward_e4m3")
        B.check(B.mp_expert_matmul_wgrad_e4m3(E, cap, 2 * I, H, self.d_gate_up,
                                              self.d_gate_up_scales, self.recv_x,
                                              self.recv_scales, self.expert_offsets,
                                              self.d_w_gate_up, self.dev_err, stream),
                "mp_expert_matmul_wgrad_e4m3")
        B.check(B.mp_expert_matmul_dgrad_e4m3(E, cap, 2 * I, H, self.d_gate_up,
                                              self.d_gate_up_scales, w_gate_up, w_gate_up_scales,
                                              self.expert_offsets, self.d_rows, self.dev_err,
                                              stream), "mp_expert_matmul_dgrad_e4m3")
        B.check(B.mp_combine_ll(R, N, K, H, self.d_rows, cap, self.slot_row, self.ones, self.d_x,
                                self.dev_err, stream), "mp_combine_ll")
        B.check(B.mp_ll_row_weights_backward(R, N, K, self.d_row_weights, cap, self.slot_row,
                                             self.d_topk_weights, stream),
                "mp_ll_row_weights_backward")
        B.check(B.mp_route_backward(R, N, K, E, self.scoring, logits, active, self.normalize,
                                    self.scale, self.loss_coef, self.topk_idx,
                                    self.d_topk_weights, self.num_tokens_per_expert,
                                    self.num_routed, d_balance_loss, self.d_logits, stream),
                "mp_route_backward")
        return self.d_x, self.d_logits, self.d_w_gate_up, self.d_w_down

    def device_error(self) -> int:
        return int(self.dev_err.item())
