"""What is measured of the expert layer's own operators: the router with its balance loss
(mp_route, mp_route_backward), the experts' products on e4m3 rows with one fp32 scale per
block of 128 (mp_expert_matmul_e4m3 and its two gradients) and the gated activation between
them (mp_swiglu_e4m3, mp_swiglu_backward_e4m3).

With ``own`` false ``run`` computes an operator from elementary torch operations in 32 bits,
rounded once at the end; with ``own`` true it makes the library's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BLOCK = 128          # channels per fp32 scale of an e4m3 tensor
E4M3_MAX = 448.0
TINY = 2.0 ** -126   # a block whose scale would be below this has scale 1 (all its codes are 0)
LOSS_COEF = 0.01     # of the balance loss
WEIGHT_SCALE = 2.5   # factor on the sigmoid router's weights


def listed():
    return [
        # one decode step's router: latency alone
        dict(name="route 8x64", op="route", R=1, N=8, E=64, K=6, scoring="softmax", dtype="fp32",
             masked=False),
        # the router of one training step of the DeepSeek-V3-shaped workload
        dict(name="route 8x4096x256", op="route", R=8, N=4096, E=256, K=8, scoring="sigmoid",
             dtype="fp32", masked=False),
        # its gradient
        dict(name="route bwd 8x4096x256", op="route_bwd", R=8, N=4096, E=256, K=8,
             scoring="sigmoid", dtype="fp32", masked=False),
        # the gradient in the skewed workload's shape: bf16 logits, padding, an odd batch
        dict(name="route bwd 16x2047x64", op="route_bwd", R=16, N=2047, E=64, K=6,
             scoring="softmax", dtype="bf16", masked=True),
        # the activation of one decode step: a few rows
        dict(name="swiglu 64x2048", op="swiglu", rows=64, I=2048, weighted=False),
        # the activation of one rank's experts in the DeepSeek-V3-shaped workload
        dict(name="swiglu 32768x2048", op="swiglu", rows=32768, I=2048, weighted=True),
        # its gradient, that of the routing weights too
        dict(name="swiglu bwd 32768x2048", op="swiglu_bwd", rows=32768, I=2048, weighted=True),
        # one token through one dense projection: the weights' bytes alone count
        dict(name="matmul 1x4096x7168", op="matmul", rows=1, E=1, N=4096, K=7168, skew=False),
        # a decode batch over one rank's experts (about 31 rows each, an odd total)
        dict(name="matmul 999/32x4096x7168", op="matmul", rows=999, E=32, N=4096, K=7168,
             skew=False),
        # a training or prefill batch over one rank's experts: gate and up projection
        dict(name="matmul 32768/32x4096x7168", op="matmul", rows=32768, E=32, N=4096, K=7168,
             skew=False),
        # the gradient through the down projection: rows of 7168 channels back to 2048
        dict(name="dgrad 32768/32x7168x2048", op="dgrad", rows=32768, E=32, N=7168, K=2048,
             skew=False),
        # the gradient of the gate and up weights
        dict(name="wgrad 32768/32x4096x7168", op="wgrad", rows=32768, E=32, N=4096, K=7168,
             skew=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "swiglu", "swiglu_bwd", "matmul", "dgrad", "wgrad"])
    if op in ("route", "route_bwd"):
        R = rng.choice([1, 2, 3, 4, 8, 16])
        E = _log(rng, 8, 512)
        return dict(op=op, R=R, N=_log(rng, 1, 32768 // R), E=E, K=rng.randint(1, min(8, E)),
                    scoring=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]),
                    masked=rng.random() < 0.5)
    if op in ("swiglu", "swiglu_bwd"):
        I = BLOCK * _log(rng, 1, 32)
        return dict(op=op, rows=_log(rng, 1, 32768 * 2048 // max(I, 2048)), I=I,
                    weighted=rng.random() < 0.5)
    while True:
        E, N, K = _log(rng, 1, 64), 16 * _log(rng, 8, 448), BLOCK * _log(rng, 1, 56)
        if op != "matmul":
            N = BLOCK * max(1, N // BLOCK)
        rows = _log(rng, 1, 32768)
        if N == 3072 or K == 3072 or E * N * K > 32 * 4096 * 7168:
            continue
        if rows * N * K <= 32768 * 4096 * 7168:
            return dict(op=op, rows=rows, E=E, N=N, K=K, skew=rows <= 4096 and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _quantised_rows(rows, C, g, size):
    """Normal rows as a quantiser leaves them: codes that fill e4m3's range, a scale per block."""
    x = torch.randn((rows, C // BLOCK, BLOCK), generator=g, device="cuda")
    amax = x.abs().amax(-1, keepdim=True)
    return _e4m3(x * (E4M3_MAX / amax)).view(rows, C), (amax * (size / E4M3_MAX)).view(rows, -1)


def _quantised_weights(E, N, K, g):
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):  # a block of 128 x 128 normal values spans about 4 standard deviations
        codes[e] = _e4m3(torch.randn((N, K), generator=g, device="cuda") * (E4M3_MAX / 4.0))
    scales = torch.rand((E, -(-N // BLOCK), K // BLOCK), generator=g, device="cuda") + 0.5
    return codes, scales * (4.0 / E4M3_MAX / math.sqrt(K))


def _expert_counts(case, seed):
    rng = np.random.default_rng(seed)
    p = np.arange(1, case["E"] + 1, dtype=np.float64) ** (-1.2 if case["skew"] else 0.0)
    return rng.multinomial(case["rows"], p / p.sum()).astype(np.int64)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    dev = dict(device="cuda")
    s["dev_err"] = torch.zeros(1, dtype=torch.int32, **dev)
    if op in ("route", "route_bwd"):
        R, N, E, K = (case[k] for k in "RNEK")
        # some experts are liked more than others, as in an unfinished training
        logits = (torch.randn((R, N, E), generator=g, **dev) * 1.5
                  + torch.randn(E, generator=g, **dev) * 0.5)
        s["logits"] = logits.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16)
        s["bias"] = (torch.randn(E, generator=g, **dev) * 0.05
                     if case["scoring"] == "sigmoid" else None)
        s["active"] = ((torch.rand((R, N), generator=g, **dev) < 0.9).to(torch.uint8)
                       if case["masked"] else None)
        s["normalize"] = True
        s["scale"] = WEIGHT_SCALE if case["scoring"] == "sigmoid" else 1.0
        s["topk_idx"] = torch.zeros((R, N, K), dtype=torch.int32, **dev)
        s["topk_weights"] = torch.zeros((R, N, K), **dev)
        s["counts"] = torch.zeros((R, E), dtype=torch.int32, **dev)
        s["routed"] = torch.zeros(R, dtype=torch.int32, **dev)
        s["loss"] = torch.zeros(R, **dev)
        if op == "route_bwd":  # what the forward pass left, and the gradients that arrive
            idx, w, counts, routed, loss = _route_plain(s)
            s["topk_idx"], s["topk_weights"] = idx, w
            s["counts"], s["routed"] = counts, routed
            s["d_topk_weights"] = torch.randn((R, N, K), generator=g, **dev)
            s["d_loss"] = torch.rand(R, generator=g, **dev) + 0.5
            s["d_logits"] = torch.zeros_like(s["logits"])
        return s
    if op in ("swiglu", "swiglu_bwd"):
        rows, I = case["rows"], case["I"]
        s["gate_up"] = torch.randn((rows, 2 * I), generator=g, **dev).to(torch.bfloat16)
        s["row_weights"] = torch.rand(rows, generator=g, **dev) if case["weighted"] else None
        s["num_rows"] = torch.full((1,), rows, dtype=torch.int32, **dev)
        if op == "swiglu":
            s["out"] = torch.zeros((rows, I), dtype=torch.float8_e4m3fn, **dev)
            s["out_scales"] = torch.zeros((rows, I // BLOCK), **dev)
        else:
            s["d_out"] = torch.randn((rows, I), generator=g, **dev).to(torch.bfloat16)
            s["d_gate_up"] = torch.zeros((rows, 2 * I), dtype=torch.float8_e4m3fn, **dev)
            s["d_gate_up_scales"] = torch.zeros((rows, 2 * I // BLOCK), **dev)
            s["d_row_weights"] = torch.zeros(rows, **dev) if case["weighted"] else None
        return s
    rows, E, N, K = (case[k] for k in ("rows", "E", "N", "K"))
    counts = _expert_counts(case, seed)
    s["most"] = int(counts.max())
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    if op in ("matmul", "wgrad"):
        s["a"], s["a_scales"] = _quantised_rows(rows, K, g, 4.0)
    if op in ("dgrad", "wgrad"):
        s["dy"], s["dy_scales"] = _quantised_rows(rows, N, g, 0.1)
    if op in ("matmul", "dgrad"):
        s["w"], s["w_scales"] = _quantised_weights(E, N, K, g)
        s["out"] = torch.zeros((rows, N if op == "matmul" else K), dtype=torch.bfloat16, **dev)
    else:
        s["out"] = torch.zeros((E, N, K), dtype=torch.bfloat16, **dev)
    return s


# ---------------------------------------------------------------- the plain forms

def _scores(s):
    """(tokens that count, experts they may go to, scores, shares, selection keys)."""
    x = s["logits"].float()
    ok = ~(torch.isnan(x) | (x == math.inf)).any(-1)
    if s["active"] is not None:
        ok = ok & (s["active"] != 0)
    allowed = (x > -math.inf) & ok.unsqueeze(-1)
    if s["scoring"] == "softmax":
        m = torch.where(allowed, x, -math.inf).amax(-1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        score = torch.where(allowed, torch.exp(torch.where(allowed, x, m) - m), 0.0)
        total = score.sum(-1, keepdim=True)
        score = score / torch.where(total > 0, total, 1.0)
        return allowed, score, score, torch.where(allowed, x, -math.inf)
    score = torch.where(allowed, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    total = score.sum(-1, keepdim=True)
    share = score / torch.where(total > 0, total, 1.0)
    key = score + s["bias"] if s["bias"] is not None else score
    return allowed, score, share, torch.where(allowed, key, -math.inf)


def _route_plain(s):
    R, N, E, K = (s[k] for k in "RNEK")
    allowed, score, share, key = _scores(s)
    key, order = torch.sort(key, dim=-1, descending=True, stable=True)  # ties: the lowest index
    chosen = key[..., :K] > -math.inf
    idx = order[..., :K]
    w = torch.where(chosen, torch.gather(score, -1, idx), 0.0)
    if s["normalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    w = w * s["scale"]
    counts = torch.zeros((R, E), dtype=torch.int32, device=idx.device)
    counts.scatter_add_(1, idx.reshape(R, N * K), chosen.to(torch.int32).reshape(R, N * K))
    token = chosen.any(-1)
    routed = token.sum(1).to(torch.int32)
    mass = torch.where(token.unsqueeze(-1), share, 0.0).sum(1)
    t = routed.clamp(min=1).float()
    loss = LOSS_COEF * E / K * (counts.float() * mass).sum(-1) / (t * t)
    return torch.where(chosen, idx, -1).to(torch.int32), w, counts, routed, loss


def _route_bwd_plain(s):
    R, N, E, K = (s[k] for k in "RNEK")
    allowed, score, share, _ = _scores(s)
    idx = s["topk_idx"].long()
    chosen = idx >= 0
    at = idx.clamp(min=0)
    picked = torch.where(chosen, torch.gather(score, -1, at), 0.0)
    dw = torch.where(chosen, s["d_topk_weights"], 0.0) * s["scale"]
    if s["normalize"]:
        total = picked.sum(-1, keepdim=True)
        inv = torch.where(total > 0, 1.0 / torch.where(total > 0, total, 1.0), 0.0)
        dw = (dw - (dw * picked).sum(-1, keepdim=True) * inv) * inv
    dw = torch.where(chosen, dw, 0.0)
    d_score = torch.zeros_like(score).scatter_add_(-1, at, dw)
    t = s["routed"].clamp(min=1).float()
    d_share = (s["d_loss"] * LOSS_COEF * E / K / (t * t)).unsqueeze(-1) * s["counts"].float()
    d_share = d_share.unsqueeze(1) * chosen.any(-1, keepdim=True)
    if s["scoring"] == "softmax":
        d = d_score + d_share
        return (share * (d - (share * d).sum(-1, keepdim=True))).to(s["logits"].dtype)
    total = score.sum(-1, keepdim=True)
    d = d_score + (d_share - (share * d_share).sum(-1, keepdim=True)) / torch.where(
        total > 0, total, 1.0)
    return (d * score * (1.0 - score)).to(s["logits"].dtype)


def _quantise(x):
    rows, C = x.shape
    x = x.view(rows, C // BLOCK, BLOCK)
    scale = x.abs().amax(-1, keepdim=True) / E4M3_MAX
    scale = torch.where(scale >= TINY, scale, 1.0)
    return _e4m3(x / scale).view(rows, C), scale.view(rows, -1)


def _swiglu_plain(s):
    g, u = s["gate_up"].float().chunk(2, -1)
    z = g / (1.0 + torch.exp(-g)) * u
    if s["row_weights"] is not None:
        z = z * s["row_weights"].unsqueeze(-1)
    return _quantise(z)


def _swiglu_bwd_plain(s):
    g, u = s["gate_up"].float().chunk(2, -1)
    d = s["d_out"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig
    dw = (d * act * u).sum(-1) if s["row_weights"] is not None else None
    if s["row_weights"] is not None:
        d = d * s["row_weights"].unsqueeze(-1)
    dg = d * u * sig * (1.0 + g * (1.0 - sig))
    codes, scales = _quantise(torch.cat([dg, d * act], -1))
    return (codes, scales) if dw is None else (codes, scales, dw)


def _rows_fp32(codes, scales):
    rows, C = codes.shape
    return (codes.float().view(rows, C // BLOCK, BLOCK) * scales.unsqueeze(-1)).view(rows, C)


def _weights_fp32(w, scales):
    E, N, K = w.shape
    wide = scales.repeat_interleave(BLOCK, 1)[:, :N]
    return (w.float().view(E, N, K // BLOCK, BLOCK) * wide.unsqueeze(-1)).view(E, N, K)


def _padded(x, s):
    """[E, most, C]: each expert's rows, zeros after its last one."""
    off = s["offsets"].long()
    at = off[:-1].unsqueeze(1) + torch.arange(s["most"], device=x.device)
    there = at < off[1:].unsqueeze(1)
    return x[at.clamp(max=x.shape[0] - 1)] * there.unsqueeze(-1), there


def _matmul_plain(s):
    if s["op"] == "wgrad":
        dy, _ = _padded(_rows_fp32(s["dy"], s["dy_scales"]), s)
        a, _ = _padded(_rows_fp32(s["a"], s["a_scales"]), s)
        return torch.bmm(dy.transpose(1, 2), a).to(torch.bfloat16)
    w = _weights_fp32(s["w"], s["w_scales"])
    if s["op"] == "matmul":
        x, there = _padded(_rows_fp32(s["a"], s["a_scales"]), s)
        return torch.bmm(x, w.transpose(1, 2))[there].to(torch.bfloat16)
    x, there = _padded(_rows_fp32(s["dy"], s["dy_scales"]), s)
    return torch.bmm(x, w)[there].to(torch.bfloat16)


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from combine_mp_layout_gb300 import binding as B
    op = s["op"]
    if op in ("route", "route_bwd"):
        R, N, E, K = (s[k] for k in "RNEK")
        scoring = B.MP_SOFTMAX if s["scoring"] == "softmax" else B.MP_SIGMOID
        if op == "route":
            if "workspace" not in s:
                s["workspace"] = torch.zeros(B.mp_route_workspace_size(R, N, E),
                                             dtype=torch.uint8, device="cuda")
            B.check(B.mp_route(R, N, K, E, scoring, s["logits"], s["bias"], s["active"],
                               s["normalize"], s["scale"], LOSS_COEF, s["topk_idx"],
                               s["topk_weights"], s["counts"], s["routed"], s["loss"],
                               s["dev_err"], s["workspace"]), "mp_route")
            return s["topk_idx"], s["topk_weights"], s["counts"], s["routed"], s["loss"]
        B.check(B.mp_route_backward(R, N, K, E, scoring, s["logits"], s["active"], s["normalize"],
                                    s["scale"], LOSS_COEF, s["topk_idx"], s["d_topk_weights"],
                                    s["counts"], s["routed"], s["d_loss"], s["d_logits"]),
                "mp_route_backward")
        return s["d_logits"]
    if op == "swiglu":
        B.check(B.mp_swiglu_e4m3(s["rows"], s["I"], s["gate_up"], s["row_weights"], s["num_rows"],
                                 s["out"], s["out_scales"]), "mp_swiglu_e4m3")
        return s["out"], s["out_scales"]
    if op == "swiglu_bwd":
        B.check(B.mp_swiglu_backward_e4m3(s["rows"], s["I"], s["gate_up"], s["row_weights"],
                                          s["d_out"], s["num_rows"], s["d_gate_up"],
                                          s["d_gate_up_scales"], s["d_row_weights"]),
                "mp_swiglu_backward_e4m3")
        out = (s["d_gate_up"], s["d_gate_up_scales"])
        return out if s["d_row_weights"] is None else out + (s["d_row_weights"],)
    size = (s["E"], s["rows"], s["N"], s["K"])
    if op == "matmul":
        B.check(B.mp_expert_matmul_e4m3(*size, s["a"], s["a_scales"], s["w"], s["w_scales"],
                                        s["offsets"], s["out"], s["dev_err"]),
                "mp_expert_matmul_e4m3")
    elif op == "dgrad":
        B.check(B.mp_expert_matmul_dgrad_e4m3(*size, s["dy"], s["dy_scales"], s["w"],
                                              s["w_scales"], s["offsets"], s["out"],
                                              s["dev_err"]), "mp_expert_matmul_dgrad_e4m3")
    else:
        B.check(B.mp_expert_matmul_wgrad_e4m3(*size, s["dy"], s["dy_scales"], s["a"],
                                              s["a_scales"], s["offsets"], s["out"],
                                              s["dev_err"]), "mp_expert_matmul_wgrad_e4m3")
    return s["out"]


def run(s):
    if own:
        return _run_own(s)
    return {"route": _route_plain, "route_bwd": _route_bwd_plain, "swiglu": _swiglu_plain,
            "swiglu_bwd": _swiglu_bwd_plain}.get(s["op"], _matmul_plain)(s)


# ---------------------------------------------------------------- the work, and 64 bits

def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        T, E, K = case["R"] * case["N"], case["E"], case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        table = 8 * T * K + (T if case["masked"] else 0) + 4 * case["R"] * (E + 2)
        return dict(bytes=T * E * size * (1 if op == "route" else 2) + table, flops=8 * T * E)
    if op in ("swiglu", "swiglu_bwd"):
        rows, I = case["rows"], case["I"]
        w = 4 * rows if case["weighted"] else 0
        if op == "swiglu":
            return dict(bytes=rows * (4 * I + I + I // 32) + w, flops=8 * rows * I)
        return dict(bytes=rows * (4 * I + 2 * I + 2 * I + I // 16) + 2 * w, flops=16 * rows * I)
    rows, E, N, K = (case[k] for k in ("rows", "E", "N", "K"))
    used = E * (1.0 - (1.0 - 1.0 / E) ** rows)  # experts that get a row
    flops = 2 * rows * N * K
    if op == "wgrad":
        return dict(bytes=rows * (N + K) * (1 + 1 / 32) + 2 * E * N * K, flops=flops)
    src, dst = (K, N) if op == "matmul" else (N, K)
    return dict(bytes=rows * (src * (1 + 1 / 32) + 2 * dst) + used * N * K, flops=flops)


def _exact_rows(codes, scales):
    return codes.double() * torch.repeat_interleave(scales.double(), BLOCK, dim=1)


def _exact_matmul(s):
    off = s["offsets"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        if s["op"] == "wgrad":
            out[e] = (_exact_rows(s["dy"][lo:hi], s["dy_scales"][lo:hi]).t()
                      @ _exact_rows(s["a"][lo:hi], s["a_scales"][lo:hi]))
            continue
        sc = s["w_scales"][e].double()
        w = s["w"][e].double()
        w *= sc.repeat_interleave(BLOCK, 0)[:s["N"]].repeat_interleave(BLOCK, 1)
        if s["op"] == "matmul":
            out[lo:hi] = _exact_rows(s["a"][lo:hi], s["a_scales"][lo:hi]) @ w.t()
        else:
            out[lo:hi] = _exact_rows(s["dy"][lo:hi], s["dy_scales"][lo:hi]) @ w
    return out


def _exact_quantised(z):
    """Values over their block's scale (what a code rounds), and the scales."""
    rows, C = z.shape
    b = z.reshape(rows, C // BLOCK, BLOCK)
    scale = b.abs().max(-1).values / E4M3_MAX
    scale[scale < TINY] = 1.0
    return (b / scale[..., None]).reshape(rows, C), scale


def _exact_router_terms(s):
    x = s["logits"].double()
    live = torch.isfinite(x) | (x == -math.inf)
    live = live.all(-1)
    if s["active"] is not None:
        live &= s["active"].bool()
    if s["scoring"] == "softmax":
        score = torch.softmax(x, -1)
        share = score
    else:
        score = torch.sigmoid(x)
        share = score / score.sum(-1, keepdim=True)
    return x, live, score, share


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("matmul", "dgrad", "wgrad"):
        return _exact_matmul(s)
    if op == "swiglu":
        g, u = s["gate_up"].double().split(case["I"], -1)
        z = torch.sigmoid(g) * g * u
        if s["row_weights"] is not None:
            z = z * s["row_weights"].double()[:, None]
        return _exact_quantised(z)
    if op == "swiglu_bwd":
        g, u = s["gate_up"].double().split(case["I"], -1)
        d, sig = s["d_out"].double(), torch.sigmoid(g)
        w = (s["row_weights"].double() if s["row_weights"] is not None
             else torch.ones(case["rows"], dtype=torch.float64, device="cuda"))[:, None]
        dz = torch.cat([d * w * u * (sig + g * sig * torch.sigmoid(-g)), d * w * g * sig], -1)
        out = _exact_quantised(dz)
        return out if s["row_weights"] is None else out + ((d * g * sig * u).sum(-1),)
    R, N, E, K = (case[k] for k in "RNEK")
    x, live, score, share = _exact_router_terms(s)
    if op == "route":
        key = x if case["scoring"] == "softmax" else score + s["bias"].double()
        top = torch.topk(key, K, dim=-1).indices
        w = score.gather(-1, top)
        w = w / w.sum(-1, keepdim=True) * s["scale"] * live[..., None]
        hits = torch.nn.functional.one_hot(top, E).sum(-2) * live[..., None]
        t = live.sum(1).double()
        f, mean = hits.sum(1).double(), (share * live[..., None]).sum(1)
        loss = LOSS_COEF * E / K * (f * mean).sum(-1) / t.clamp(min=1) ** 2
        return None, w, None, None, loss
    # the gradient of the weights' and the loss's sum, by automatic differentiation in 64 bits
    x = x.detach().requires_grad_(True)
    score = torch.softmax(x, -1) if case["scoring"] == "softmax" else torch.sigmoid(x)
    share = score / score.sum(-1, keepdim=True)
    w = score.gather(-1, s["topk_idx"].long().clamp(min=0))
    w = w / w.sum(-1, keepdim=True) * s["scale"]
    total = (w * s["d_topk_weights"].double() * live[..., None]).sum()
    t = s["routed"].double().clamp(min=1)
    loss = LOSS_COEF * E / K * (s["counts"].double() * (share * live[..., None]).sum(1)).sum(-1)
    total = total + (loss / t ** 2 * s["d_loss"].double()).sum()
    return torch.autograd.grad(total, x)[0]
