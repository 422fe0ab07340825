"""What is measured of the expert layer on bf16 rows: the experts' products with bf16 weights
and their two gradients (mp_expert_matmul_bf16, _dgrad_bf16, _wgrad_bf16), the products with
4-bit weights (mp_expert_matmul_mxfp4: e2m1 codes, one UE8M0 scale per 32) and the gated
activation between two products with its gradient (mp_swiglu_bf16, mp_swiglu_backward_bf16).

With ``own`` false ``run`` computes an operator from elementary torch operations in 32 bits,
rounded once at the end; with ``own`` true it makes the library's calls.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

GROUP = 32            # channels per scale of a 4-bit weight
EXACT_FLOPS = 1.5e13  # the most that 64 bits are computed for: about 15 s


def listed():
    return [
        # one token through one dense projection: the weights' bytes alone count
        dict(name="matmul 1x4096x7168", op="matmul", rows=1, E=1, N=4096, K=7168, skew=False,
             out="bf16"),
        # a decode batch over one rank's experts (about 31 rows each, an odd total)
        dict(name="matmul 999/32x4096x7168", op="matmul", rows=999, E=32, N=4096, K=7168,
             skew=False, out="bf16"),
        # a training or prefill batch over one rank's experts: gate and up projection
        dict(name="matmul 32768/32x4096x7168", op="matmul", rows=32768, E=32, N=4096, K=7168,
             skew=False, out="bf16"),
        # the gradient through the down projection: rows of 7168 channels back to 2048
        dict(name="dgrad 32768/32x7168x2048", op="dgrad", rows=32768, E=32, N=7168, K=2048,
             skew=False, out="bf16"),
        # the gradient of the gate and up weights
        dict(name="wgrad 32768/32x4096x7168", op="wgrad", rows=32768, E=32, N=4096, K=7168,
             skew=False, out="bf16"),
        # the skewed workload's down projection, a small batch: fp32 gradients, many experts
        # with a few rows or none
        dict(name="wgrad fp32 4095/64x4096x2048", op="wgrad", rows=4095, E=64, N=4096, K=2048,
             skew=True, out="fp32"),
        # one token through one dense projection of 4-bit weights
        dict(name="mxfp4 1x4096x7168", op="mxfp4", rows=1, E=1, N=4096, K=7168, skew=False,
             out="bf16"),
        # a small decode batch over one rank's experts: about two rows each
        dict(name="mxfp4 61/32x4096x7168", op="mxfp4", rows=61, E=32, N=4096, K=7168, skew=False,
             out="bf16"),
        # a prefill batch through the down projection: about 256 rows each
        dict(name="mxfp4 8191/32x7168x2048", op="mxfp4", rows=8191, E=32, N=7168, K=2048,
             skew=False, out="bf16"),
        # the activation of one decode step: a few rows
        dict(name="swiglu 64x2048", op="swiglu", rows=64, I=2048, weighted=False),
        # the activation of one rank's experts in the DeepSeek-V3-shaped workload
        dict(name="swiglu 32768x2048", op="swiglu", rows=32768, I=2048, weighted=True),
        # its gradient, that of the routing weights too
        dict(name="swiglu bwd 32768x2048", op="swiglu_bwd", rows=32768, I=2048, weighted=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "dgrad", "wgrad", "mxfp4", "mxfp4", "swiglu",
                     "swiglu_bwd"])
    if op in ("swiglu", "swiglu_bwd"):
        I = 8 * _log(rng, 8, 512)
        return dict(op=op, rows=_log(rng, 1, 32768 * 2048 // max(I, 2048)), I=I,
                    weighted=rng.random() < 0.5)
    step = GROUP if op == "mxfp4" else 8
    while True:
        E, N, K = _log(rng, 1, 64), 8 * _log(rng, 16, 896), step * _log(rng, 128 // step,
                                                                        7168 // step)
        rows = _log(rng, 1, 32768)
        if E * N * K <= 32 * 4096 * 7168 and rows * N * K <= 32768 * 4096 * 7168:
            return dict(op=op, rows=rows, E=E, N=N, K=K, skew=rows <= 4096 and rng.random() < 0.5,
                        out=rng.choice(["bf16", "fp32"]) if op == "wgrad" else "bf16")


# ---------------------------------------------------------------- inputs

def _bf16(shape, g, size=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in (out if len(shape) == 3 else [out]):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(size))
    return out


def _mxfp4(w):
    """Rows of w as a microscaling quantiser leaves them: codes (two a byte, the even channel in
    the low four bits) and the scales' exponents."""
    N, K = w.shape
    b = w.view(N, K // GROUP, GROUP)
    exp = torch.floor(torch.log2(b.abs().amax(-1))).to(torch.int32) - 2  # 2: of the largest, 6
    m = (b * torch.exp2(-exp.float()).unsqueeze(-1)).clamp(-6.0, 6.0)
    mag = m.abs()
    # steps of 1/2 up to 2, of 1 up to 4, then 4 and 6
    q = torch.where(mag < 2.0, torch.round(mag * 2.0),
                    torch.where(mag < 4.0, torch.round(mag) + 2.0, torch.round(mag * 0.5) + 4.0))
    code = (q.to(torch.uint8) | ((m < 0).to(torch.uint8) << 3)).view(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), (exp + 127).to(torch.uint8)


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
    if op in ("swiglu", "swiglu_bwd"):
        rows, I = case["rows"], case["I"]
        s["gate_up"] = _bf16((rows, 2 * I), g)
        s["row_weights"] = torch.rand(rows, generator=g, **dev) if case["weighted"] else None
        s["num_rows"] = torch.full((1,), rows, dtype=torch.int32, **dev)
        if op == "swiglu":
            s["out_rows"] = torch.zeros((rows, I), dtype=torch.bfloat16, **dev)
        else:
            s["d_out"] = _bf16((rows, I), g)
            s["d_gate_up"] = torch.zeros((rows, 2 * I), dtype=torch.bfloat16, **dev)
            s["d_row_weights"] = torch.zeros(rows, **dev) if case["weighted"] else None
        return s
    rows, E, N, K = (case[k] for k in ("rows", "E", "N", "K"))
    counts = _expert_counts(case, seed)
    s["most"] = int(counts.max())
    s["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    if op in ("matmul", "mxfp4", "wgrad"):
        s["a"] = _bf16((rows, K), g)
    if op in ("dgrad", "wgrad"):
        s["dy"] = _bf16((rows, N), g, 0.1)
    if op in ("matmul", "dgrad"):
        s["w"] = _bf16((E, N, K), g, 1.0 / math.sqrt(K))
    if op == "mxfp4":
        s["w"] = torch.empty((E, N, K // 2), dtype=torch.uint8, **dev)
        s["w_scales"] = torch.empty((E, N, K // GROUP), dtype=torch.uint8, **dev)
        for e in range(E):
            s["w"][e], s["w_scales"][e] = _mxfp4(torch.randn((N, K), generator=g, **dev)
                                                 / math.sqrt(K))
    if op == "wgrad":
        s["out_rows"] = torch.zeros((E, N, K), dtype=torch.float32 if case["out"] == "fp32"
                                    else torch.bfloat16, **dev)
    else:
        s["out_rows"] = torch.zeros((rows, K if op == "dgrad" else N), dtype=torch.bfloat16, **dev)
    return s


# ---------------------------------------------------------------- the plain forms

def _padded(x, s):
    """[E, most, C]: each expert's rows in 32 bits, zeros after its last one."""
    off = s["offsets"].long()
    at = off[:-1].unsqueeze(1) + torch.arange(s["most"], device=x.device)
    there = at < off[1:].unsqueeze(1)
    return x[at.clamp(max=x.shape[0] - 1)].float() * there.unsqueeze(-1), there


def _fp4_weights(s):
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0,
                           -3.0, -4.0, -6.0], device="cuda")
    E, N, half = s["w"].shape
    w = torch.empty((E, N, 2 * half), device="cuda")
    for e in range(E):
        code = s["w"][e].int()
        w[e] = torch.stack([values[code & 15], values[code >> 4]], -1).view(N, -1)
        w[e].view(N, -1, GROUP).mul_(torch.exp2(s["w_scales"][e].float() - 127.0).unsqueeze(-1))
    return w


def _matmul_plain(s):
    if s["op"] == "wgrad":
        dy, a = _padded(s["dy"], s)[0], _padded(s["a"], s)[0]
        return torch.bmm(dy.transpose(1, 2), a).to(s["out_rows"].dtype)
    w = _fp4_weights(s) if s["op"] == "mxfp4" else s["w"].float()
    if s["op"] == "dgrad":
        x, there = _padded(s["dy"], s)
        return torch.bmm(x, w)[there].to(torch.bfloat16)
    x, there = _padded(s["a"], s)
    return torch.bmm(x, w.transpose(1, 2))[there].to(torch.bfloat16)


def _swiglu_plain(s):
    g, u = s["gate_up"].float().chunk(2, -1)
    z = g / (1.0 + torch.exp(-g)) * u
    if s["row_weights"] is not None:
        z = z * s["row_weights"].unsqueeze(-1)
    return z.to(torch.bfloat16)


def _swiglu_bwd_plain(s):
    g, u = s["gate_up"].float().chunk(2, -1)
    d = s["d_out"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = g * sig
    dw = (d * act * u).sum(-1) if s["row_weights"] is not None else None
    if s["row_weights"] is not None:
        d = d * s["row_weights"].unsqueeze(-1)
    dg = d * u * sig * (1.0 + g * (1.0 - sig))
    d_gate_up = torch.cat([dg, d * act], -1).to(torch.bfloat16)
    return d_gate_up if dw is None else (d_gate_up, dw)


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from combine_mp_layout_gb300 import binding as B
    op = s["op"]
    if op == "swiglu":
        B.check(B.mp_swiglu_bf16(s["rows"], s["I"], s["gate_up"], s["row_weights"],
                                 s["num_rows"], s["out_rows"]), "mp_swiglu_bf16")
        return s["out_rows"]
    if op == "swiglu_bwd":
        B.check(B.mp_swiglu_backward_bf16(s["rows"], s["I"], s["gate_up"], s["row_weights"],
                                          s["d_out"], s["num_rows"], s["d_gate_up"],
                                          s["d_row_weights"]), "mp_swiglu_backward_bf16")
        return s["d_gate_up"] if s["d_row_weights"] is None else (s["d_gate_up"],
                                                                  s["d_row_weights"])
    size = (s["E"], s["rows"], s["N"], s["K"])
    if op == "matmul":
        B.check(B.mp_expert_matmul_bf16(*size, s["a"], s["w"], s["offsets"], s["out_rows"],
                                        s["dev_err"]), "mp_expert_matmul_bf16")
    elif op == "dgrad":
        B.check(B.mp_expert_matmul_dgrad_bf16(*size, s["dy"], s["w"], s["offsets"], s["out_rows"],
                                              s["dev_err"]), "mp_expert_matmul_dgrad_bf16")
    elif op == "wgrad":  # the gradient's type is that of its buffer; not added to what stands there
        B.check(B.mp_expert_matmul_wgrad_bf16(*size, s["dy"], s["a"], s["offsets"], False,
                                              s["out_rows"], s["dev_err"]),
                "mp_expert_matmul_wgrad_bf16")
    else:
        B.check(B.mp_expert_matmul_mxfp4(*size, s["a"], s["w"], s["w_scales"], s["offsets"],
                                         s["out_rows"], s["dev_err"]), "mp_expert_matmul_mxfp4")
    return s["out_rows"]


def run(s):
    if own:
        return _run_own(s)
    return {"swiglu": _swiglu_plain, "swiglu_bwd": _swiglu_bwd_plain}.get(s["op"],
                                                                          _matmul_plain)(s)


# ---------------------------------------------------------------- the work, and 64 bits

def work(case):
    op = case["op"]
    if op in ("swiglu", "swiglu_bwd"):
        rows, I = case["rows"], case["I"]
        w = 4 * rows if case["weighted"] else 0
        if op == "swiglu":
            return dict(bytes=rows * 6 * I + w, flops=8 * rows * I)
        return dict(bytes=rows * 10 * I + 2 * w, flops=16 * rows * I)
    rows, E, N, K = (case[k] for k in ("rows", "E", "N", "K"))
    p = np.arange(1, E + 1, dtype=np.float64) ** (-1.2 if case["skew"] else 0.0)
    used = float((1.0 - (1.0 - p / p.sum()) ** rows).sum())  # experts that get a row
    flops = 2 * rows * N * K
    if op == "wgrad":
        return dict(bytes=2 * rows * (N + K) + (4 if case["out"] == "fp32" else 2) * E * N * K,
                    flops=flops)
    weight = 0.5 + 1.0 / GROUP if op == "mxfp4" else 2.0
    return dict(bytes=2 * rows * (N + K) + used * N * K * weight, flops=flops)


def _exact_fp4(codes, exponents):
    """e2m1 from its fields: sign, two bits of exponent (bias 1), one of mantissa."""
    c = torch.stack([codes % 16, codes // 16], -1).flatten(1).long()
    e, m = (c // 2) % 4, (c % 2).double()
    mag = torch.where(e == 0, m / 2.0, (1.0 + m / 2.0) * 2.0 ** (e - 1).double())
    scale = torch.ldexp(torch.ones_like(exponents, dtype=torch.float64), exponents.int() - 127)
    return torch.where(c >= 8, -mag, mag) * scale.repeat_interleave(GROUP, 1)


def _exact_matmul(s):
    off = s["offsets"].tolist()
    out = torch.zeros(s["out_rows"].shape, dtype=torch.float64, device="cuda")
    for e in range(s["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        if s["op"] == "wgrad":
            torch.mm(s["dy"][lo:hi].double().t(), s["a"][lo:hi].double(), out=out[e])
        elif s["op"] == "dgrad":
            out[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
        elif s["op"] == "matmul":
            out[lo:hi] = s["a"][lo:hi].double() @ s["w"][e].double().t()
        else:
            out[lo:hi] = s["a"][lo:hi].double() @ _exact_fp4(s["w"][e], s["w_scales"][e]).t()
    return out


def exact(case, seed):
    op = case["op"]
    if op not in ("swiglu", "swiglu_bwd"):
        if 2 * case["rows"] * case["N"] * case["K"] > EXACT_FLOPS:
            return None
        return _exact_matmul(prepare(case, seed))
    s = prepare(case, seed)
    g, u = s["gate_up"].double().split(case["I"], -1)
    w = (s["row_weights"].double() if s["row_weights"] is not None
         else torch.ones(case["rows"], dtype=torch.float64, device="cuda"))[:, None]
    if op == "swiglu":
        return torch.sigmoid(g) * g * u * w
    d, sig = s["d_out"].double(), torch.sigmoid(g)
    dz = torch.cat([d * w * u * (sig + g * sig * torch.sigmoid(-g)), d * w * g * sig], -1)
    return dz if s["row_weights"] is None else (dz, (d * g * sig * u).sum(-1))
