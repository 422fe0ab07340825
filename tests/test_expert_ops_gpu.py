"""The expert layer's operators (router with balance loss, block-scaled e4m3 products,
gated activation, and their gradients) against plain implementations in 64 bits.

Tolerances (u = 2^-24, the unit roundoff of fp32; bf16 rounds by at most 2^-8 of a value,
e4m3 by at most 2^-4 of a normal value and 2^-10 of its scale below):
  * products: one bf16 rounding, plus fp32 sums of n terms: n * 2 u times the sum of the
    terms' magnitudes (2 u per step: the tensor core may cut instead of round).  Over many
    outputs the bf16 rounding is about uniform, so its 2-norm is at most 2^-8 / sqrt(3).
    Small whole codes with power-of-two scales make every sum exact: bit-equal there.
  * weight gradients: both factors held in f16, scale and product rounded by 2^-11 each:
    2^-9 of each term, and next to that the bf16 rounding of the result.
  * router: exp, sums over E <= 8192 scores and divisions: 1e-5 of a score covers
    |l - max| u (at most 40 u) for the exponential and log2(E) + V steps of summation.
  * activation: the fast exponential and reciprocal, 1e-5 of a value.
"""
import math

import numpy as np
import pytest
import torch

from combine_mp_layout_gb300 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def zeros(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


# ------------------------------------------------------------------ router

def route_ref(logits, K, scoring, bias, active, normalize, scale, coef):
    """(ids, weights, counts, routed, loss, keys) in float64; logits [R][N][E]."""
    x = logits.double()
    R, N, E = x.shape
    ok = ~(torch.isnan(x) | (x == math.inf)).any(-1)
    if active is not None:
        ok &= active.bool()
    x = torch.where(ok[..., None], x, -math.inf)
    allowed = x > -math.inf
    s = scores_ref(x, scoring)
    share = s / s.sum(-1, keepdim=True).clamp(min=1e-300)
    key = x if scoring == B.MP_SOFTMAX else s + (bias.double() if bias is not None else 0.0)
    key = torch.where(allowed, key, -math.inf)
    val, order = torch.sort(key, dim=-1, descending=True, stable=True)
    chosen = val[..., :K] > -math.inf
    ids = torch.where(chosen, order[..., :K], -1)
    return ids, allowed, s, share, key, chosen


def scores_ref(x, scoring):
    allowed = x > -math.inf
    if scoring == B.MP_SOFTMAX:
        m = x.amax(-1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        e = torch.where(allowed, torch.exp(x - m), 0.0)
        return e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    return torch.where(allowed, torch.sigmoid(x), 0.0)


def objective_ref(x, ids, counts, routed, scoring, normalize, scale, coef, dw, dl, K):
    """sum(weights * dw) + sum(loss * dl) for fixed ids and counts, float64, differentiable."""
    E = x.shape[-1]
    s = scores_ref(x, scoring)
    share = s / s.sum(-1, keepdim=True).clamp(min=1e-300)
    chosen = ids >= 0
    w = torch.where(chosen, s.gather(-1, ids.clamp(min=0).long()), 0.0)
    if normalize:
        tot = w.sum(-1, keepdim=True)
        w = torch.where(tot > 0, w / tot.clamp(min=1e-300), 0.0)
    w = w * scale
    token = chosen.any(-1, keepdim=True)
    mass = torch.where(token, share, 0.0).sum(1)
    t = routed.double().clamp(min=1)
    loss = coef * E / (K * t * t) * (counts.double() * mass).sum(-1)
    return (w * dw.double()).sum() + (loss * dl.double()).sum(), w, loss


def run_route(logits, K, scoring, bias=None, active=None, normalize=True, scale=1.0, coef=0.01,
              ws=None):
    R, N, E = logits.shape
    out = dict(ids=torch.full((R, N, K), -7, dtype=torch.int32, device=DEV),
               w=zeros((R, N, K)) - 7, counts=zeros((R, E), torch.int32) - 7,
               routed=zeros(R, torch.int32) - 7, loss=zeros(R) - 7, err=zeros(1, torch.int32))
    ws = zeros(B.mp_route_workspace_size(R, N, E), torch.uint8) if ws is None else ws
    B.check(B.mp_route(R, N, K, E, scoring, logits, bias, active, normalize, scale, coef,
                       out["ids"], out["w"], out["counts"], out["routed"], out["loss"],
                       out["err"], ws), "mp_route")
    torch.cuda.synchronize()
    assert int(ws.count_nonzero()) == 0
    return out


ROUTES = [  # R, N, E, K, scoring, dtype, masked, normalize
    (1, 1, 1, 1, 0, torch.float32, False, True),
    (1, 8, 64, 6, 0, torch.float32, False, True),
    (2, 64, 8, 2, 0, torch.bfloat16, True, True),
    (3, 77, 33, 8, 1, torch.float32, True, False),
    (8, 257, 256, 8, 1, torch.float32, False, True),
    (4, 130, 500, 5, 0, torch.bfloat16, False, False),
    (2, 65, 1000, 32, 1, torch.bfloat16, True, True),
    (2, 19, 1025, 8, 0, torch.float32, True, True),
    (1, 7, 4099, 7, 1, torch.float32, False, True),
    (1, 5, 8192, 32, 0, torch.float32, False, True),
    (32, 3, 96, 4, 1, torch.float32, False, True),
    (1, 20011, 64, 6, 0, torch.float32, True, True),
]


def route_inputs(R, N, E, scoring, dtype, masked, seed):
    g = gen(seed)
    logits = (torch.randn((R, N, E), generator=g, device=DEV) * 2).to(dtype)
    logits[torch.rand((R, N, E), generator=g, device=DEV) < 0.1] = -math.inf
    bias = torch.randn(E, generator=g, device=DEV) * 0.1 if scoring == B.MP_SIGMOID else None
    active = ((torch.rand((R, N), generator=g, device=DEV) < 0.8).to(torch.uint8)
              if masked else None)
    return logits, bias, active


@pytest.mark.parametrize("R,N,E,K,scoring,dtype,masked,normalize", ROUTES)
def test_route(R, N, E, K, scoring, dtype, masked, normalize):
    logits, bias, active = route_inputs(R, N, E, scoring, dtype, masked, 1)
    scale, coef = 2.5, 0.03
    got = run_route(logits, K, scoring, bias, active, normalize, scale, coef)
    assert int(got["err"]) == 0
    ids, allowed, s, share, key, chosen = route_ref(logits, K, scoring, bias, active, normalize,
                                                    scale, coef)
    gi = got["ids"].long()
    if scoring == B.MP_SOFTMAX:
        assert torch.equal(gi, ids)
    else:  # keys are rounded to fp32 before they are compared: 4 u of a key of at most 2
        assert torch.equal(gi >= 0, chosen)
        gk = torch.where(gi >= 0, key.gather(-1, gi.clamp(min=0)), 0.0)
        rk = torch.where(chosen, key.gather(-1, ids.clamp(min=0)), 0.0)
        assert float((gk - rk).abs().max()) <= 8 * U
        hit = torch.zeros_like(key).scatter_add_(-1, gi.clamp(min=0), (gi >= 0).double())
        assert float(hit.max()) <= 1
    counts = torch.zeros((R, E), dtype=torch.int64, device=DEV)
    counts.scatter_add_(1, gi.clamp(min=0).view(R, -1), (gi >= 0).long().view(R, -1))
    assert torch.equal(got["counts"].long(), counts)
    routed = (gi >= 0).any(-1).sum(1)
    assert torch.equal(got["routed"].long(), routed)
    ok = (torch.ones((R, N), dtype=torch.bool, device=DEV) if active is None else active.bool())
    x = torch.where(ok[..., None], logits.double(), -math.inf)
    _, w, loss = objective_ref(x, gi, counts, routed, scoring, normalize, scale, coef,
                               zeros((R, N, K)), zeros(R), K)
    assert float(((got["w"].double() - w).abs() - 1e-5 * w).max()) <= 1e-30
    assert float(((got["loss"].double() - loss).abs() - 2e-5 * loss).max()) <= 1e-30
    again = run_route(logits, K, scoring, bias, active, normalize, scale, coef)
    for k in ("ids", "w", "counts", "routed", "loss"):
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("E,K", [(33, 1), (64, 6), (64, 20), (64, 21), (100, 20), (256, 8),
                                 (256, 16), (256, 20), (256, 32), (500, 8), (1024, 8), (1000, 20),
                                 (1024, 32)])
def test_route_selection_with_many_equal_keys(E, K):
    """Rows of few distinct values, from all equal to nearly all different, and rows with their
    largest keys all in a few lanes: the choices are a stable sort's."""
    g = gen(5)
    rows = []
    for levels in (1, 2, 3, 5, 9, 17, 33, 65, 129, 4097):
        x = torch.randint(0, levels, (40, E), generator=g, device=DEV).float() - levels // 2
        rows.append(x * 0.0 if levels == 2 else x / 8)     # (-0 and +0 among them)
    x = torch.randn((120, E), generator=g, device=DEV)
    e = torch.arange(E, device=DEV)
    for i in range(120):                                   # experts e % 32 in one to eight lanes
        x[i, e % 32 < 1 + i % 8] += 20.0 if i < 60 else 0.5
    x[torch.rand(x.shape, generator=g, device=DEV) < 0.3] = -math.inf
    rows.append(x)
    few = torch.full((40, E), -math.inf, device=DEV)       # fewer experts than choices
    for i in range(40):
        few[i, torch.randperm(E, generator=g, device=DEV)[:i % (K + 2)]] = float(i % 3)
    rows.append(few)
    x = torch.cat(rows)[None].contiguous()
    key = torch.where(torch.isnan(x), -math.inf, x)
    val, order = torch.sort(key + 0.0, dim=-1, descending=True, stable=True)
    want = torch.where(val[..., :K] > -math.inf, order[..., :K], -1)
    got = run_route(x, K, B.MP_SOFTMAX)
    assert torch.equal(got["ids"].long(), want)
    # sigmoid of 0 everywhere: the bias alone decides, and -inf in it forbids an expert
    bias = torch.randint(-2, 3, (E,), generator=g, device=DEV).float()
    bias[torch.rand(E, generator=g, device=DEV) < 0.2] = -math.inf
    y = torch.where(x > -math.inf, 0.0, x)
    key = torch.where(y > -math.inf, 0.5 + bias, -math.inf)
    val, order = torch.sort(key, dim=-1, descending=True, stable=True)
    want = torch.where(val[..., :K] > -math.inf, order[..., :K], -1)
    got = run_route(y, K, B.MP_SIGMOID, bias=bias)
    assert torch.equal(got["ids"].long(), want)


def test_route_ties_extremes_and_dead_rows():
    """Equal logits go to the lower expert; the type's lowest value is an ordinary logit, -inf
    never chosen; rows of nothing, of NaN and of +inf are routed nowhere."""
    lowest = torch.finfo(torch.float32).min
    E, K = 70, 4
    x = torch.full((1, 8, E), -1.0, device=DEV)
    x[0, 0] = 3.0                                   # all equal
    x[0, 1] = lowest                                # all lowest
    x[0, 2] = -math.inf                             # nothing left
    x[0, 3] = -math.inf
    x[0, 3, 66] = lowest                            # one expert left
    x[0, 4, 5] = math.nan
    x[0, 5, 69] = math.inf
    x[0, 6, 1::2] = 0.0
    x[0, 6, 0::2] = -0.0                            # -0 equals +0
    x[0, 7, 40:] = -math.inf                        # masked tail, tie among the rest
    for scoring in (B.MP_SOFTMAX, B.MP_SIGMOID):
        got = run_route(x, K, scoring)
        ids = got["ids"][0].cpu().tolist()
        first = [0, 1, 2, 3]
        assert ids == [first, first, [-1] * 4, [66, -1, -1, -1], [-1] * 4, [-1] * 4, first, first]
        assert int(got["err"]) == B.MP_ERR_BAD_VALUE
        assert int(got["routed"]) == 5
        w = got["w"][0].cpu()
        live = [0, 1, 3, 6, 7] if scoring == B.MP_SOFTMAX else [0, 6, 7]
        for r in live:  # (sigmoid of the lowest value is 0: weights 0 there)
            assert float(w[r].sum()) == pytest.approx(1.0, abs=1e-6)
        assert torch.isfinite(w).all() and torch.isfinite(got["loss"]).all()
        assert float(w[[2, 4, 5]].abs().max()) == 0.0
        d = torch.full_like(x, 9.0)
        dw = torch.ones((1, 8, K), device=DEV)
        B.check(B.mp_route_backward(1, 8, K, E, scoring, x, None, True, 1.0, 0.01, got["ids"], dw,
                                    got["counts"], got["routed"], zeros(1) + 1, d))
        torch.cuda.synchronize()
        assert torch.isfinite(d).all()
        assert float(d[0, [2, 4, 5]].abs().max()) == 0.0
        assert float(d[0, 7, 40:].abs().max()) == 0.0


def test_route_bias_only_moves_the_choice_and_may_forbid():
    x = torch.zeros((1, 1, 8), device=DEV)
    bias = torch.tensor([0.0, -math.inf, 0.5, math.nan, 0.25, 0.0, 0.0, 0.0], device=DEV)
    got = run_route(x, 8, B.MP_SIGMOID, bias, None, False)
    assert got["ids"][0, 0].cpu().tolist() == [2, 4, 0, 5, 6, 7, -1, -1]
    assert got["w"][0, 0].cpu().tolist() == [0.5] * 6 + [0.0] * 2


def test_route_without_tokens():
    got = run_route(zeros((2, 0, 16)), 2, B.MP_SOFTMAX)
    assert int(got["counts"].abs().sum()) == 0 and int(got["routed"].abs().sum()) == 0
    assert float(got["loss"].abs().sum()) == 0.0


def test_route_counts_are_the_layouts():
    """num_tokens_per_expert is what mp_layout counts from the same ids."""
    from combine_mp_layout_gb300.pipeline import EPPlan
    R, N, E, K = 4, 300, 32, 4
    logits, _, active = route_inputs(R, N, E, B.MP_SOFTMAX, torch.float32, True, 5)
    got = run_route(logits, K, B.MP_SOFTMAX, None, active)
    plan = EPPlan(R, N, K, E, 64)
    plan.topk_idx.copy_(got["ids"])
    B.check(plan.layout())
    torch.cuda.synchronize()
    assert torch.equal(plan.num_tokens_per_expert, got["counts"])


@pytest.mark.parametrize("R,N,E,K,scoring,dtype,masked,normalize", ROUTES)
def test_route_backward(R, N, E, K, scoring, dtype, masked, normalize):
    logits, bias, active = route_inputs(R, N, E, scoring, dtype, masked, 2)
    scale, coef = 2.5, 0.5
    fwd = run_route(logits, K, scoring, bias, active, normalize, scale, coef)
    g = gen(3)
    dw = torch.randn((R, N, K), generator=g, device=DEV)
    dl = torch.randn(R, generator=g, device=DEV)
    d = torch.full_like(logits, 5.0)
    B.check(B.mp_route_backward(R, N, K, E, scoring, logits, active, normalize, scale, coef,
                                fwd["ids"], dw, fwd["counts"], fwd["routed"], dl, d))
    ok = (torch.ones((R, N), dtype=torch.bool, device=DEV) if active is None else active.bool())
    low = torch.where(ok[..., None], logits.double(), -math.inf)
    finite = low > -math.inf
    x = torch.where(finite, low, 0.0).requires_grad_(True)

    def objective(x):
        return objective_ref(torch.where(finite, x, -math.inf), fwd["ids"], fwd["counts"],
                             fwd["routed"], scoring, normalize, scale, coef, dw, dl, K)[0]
    want = torch.autograd.grad(objective(x), x)[0]
    want = torch.where(finite, want, 0.0)
    # magnitude of what is added up for an entry: score times the size of its own and the
    # averaged gradients; 1e-5 of it as for the forward pass, and one rounding for bf16
    s = scores_ref(low, scoring)
    share = s / s.sum(-1, keepdim=True).clamp(min=1e-300)
    chosen = fwd["ids"] >= 0
    sel = torch.where(chosen, s.gather(-1, fwd["ids"].clamp(min=0).long()), 0.0)
    per = scale / sel.sum(-1, keepdim=True).clamp(min=1e-300) if normalize else scale
    gk = torch.where(chosen, (dw.double().abs() + dw.double().abs().amax(-1, keepdim=True)) * per,
                     0.0)
    gs = torch.zeros_like(s).scatter_add_(-1, fwd["ids"].clamp(min=0).long(), gk)
    t = fwd["routed"].double().clamp(min=1)
    gp = (dl.double().abs() * coef * E / (K * t * t))[:, None, None] * fwd["counts"][:, None, :]
    if scoring == B.MP_SOFTMAX:
        h = gs + gp
        size = s * (h + (s * h).sum(-1, keepdim=True))
    else:
        size = s * (gs + (gp + (share * gp).sum(-1, keepdim=True))
                    / s.sum(-1, keepdim=True).clamp(min=1e-300))
    tol = 2e-5 * size + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0) + 1e-30
    assert float(((d.double() - want).abs() - tol).max()) <= 0.0
    # and against differences of the 64-bit objective along random directions
    if dtype == torch.float32:
        for k in range(3):
            v = torch.randn(logits.shape, generator=g, device=DEV, dtype=torch.float64) * finite
            h = 1e-5
            with torch.no_grad():
                diff = (objective(x + h * v) - objective(x - h * v)) / (2 * h)
            slope = (d.double() * v).sum()
            bound = (tol * v.abs()).sum() + 1e-6 * (size * v.abs()).sum()
            assert abs(float(diff - slope)) <= float(bound) + 1e-8


def test_route_backward_parts_and_bad_ids():
    """Either gradient alone; ids outside [0, E) count as not chosen."""
    R, N, E, K = 2, 40, 48, 4
    logits, _, _ = route_inputs(R, N, E, B.MP_SOFTMAX, torch.float32, False, 7)
    fwd = run_route(logits, K, B.MP_SOFTMAX)
    dw, dl = torch.randn((R, N, K), device=DEV), torch.randn(R, device=DEV)

    def back(ids, a, b):
        d = torch.full_like(logits, 5.0)
        B.check(B.mp_route_backward(R, N, K, E, B.MP_SOFTMAX, logits, None, True, 1.0, 0.01, ids,
                                    a, fwd["counts"], fwd["routed"], b, d))
        torch.cuda.synchronize()
        return d
    both = back(fwd["ids"], dw, dl)
    parts = back(fwd["ids"], dw, None) + back(fwd["ids"], None, dl)
    assert float((both - parts).abs().max()) <= 1e-5
    bad = fwd["ids"].clone()
    none = bad.clone()
    bad[0, 3, 1], bad[1, 5, 0], bad[1, 6, 2] = E, 2 ** 31 - 1, -5
    none[0, 3, 1], none[1, 5, 0], none[1, 6, 2] = -1, -1, -1
    assert torch.equal(back(bad, dw, dl), back(none, dw, dl))


# ------------------------------------------------------------------ products

def rows_ref(codes, scales):
    return codes.double() * scales.double().repeat_interleave(128, 1)


def weights_ref(w, scales):
    E, N, K = w.shape
    s = scales.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
    return w.double() * s


def codes(shape, g, exact):
    x = torch.randn(shape, generator=g, device=DEV)
    x = (x * 1.2).round().clamp(-2, 2) if exact else (x * 100).clamp(-448, 448)
    return x.to(torch.float8_e4m3fn)


def scales(shape, g, exact):
    x = torch.rand(shape, generator=g, device=DEV)
    return torch.exp2((x * 3).floor() - 1) if exact else x * 0.02 + 0.001


def offsets(counts, first=0):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
                            + first).to(torch.int32).to(DEV)


MM = [  # counts, N, K, slack rows at the end
    ([1], 16, 128, 0),
    ([3], 48, 256, 2),
    ([0, 1, 127, 129, 0], 144, 384, 7),
    ([128, 256, 5], 272, 128, 0),
    ([31, 33, 64, 65], 512, 1024, 3),
    ([1, 1, 0, 1, 1, 0, 1], 1024, 512, 0),
    ([700], 640, 384, 0),
    ([300, 0, 411], 256, 7168, 1),
    ([1], 4096, 2048, 0),
    ([2500], 384, 256, 0),
]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("counts,N,K,slack", MM)
def test_matmul(kind, counts, N, K, slack, exact):
    if kind == "dgrad":
        N = -(-N // 128) * 128
    g = gen(11)
    E, rows = len(counts), sum(counts) + slack
    src, dst = (K, N) if kind == "fwd" else (N, K)
    a, sa = codes((rows, src), g, exact), scales((rows, src // 128), g, exact)
    w, sw = codes((E, N, K), g, exact), scales((E, -(-N // 128), K // 128), g, exact)
    off = offsets(counts)
    out = torch.full((rows, dst), 7.0, dtype=torch.bfloat16, device=DEV)
    err = zeros(1, torch.int32)
    f = B.mp_expert_matmul_e4m3 if kind == "fwd" else B.mp_expert_matmul_dgrad_e4m3
    B.check(f(E, rows, N, K, a, sa, w, sw, off, out, err))
    torch.cuda.synchronize()
    assert int(err) == 0
    ad, wd = rows_ref(a, sa), weights_ref(w, sw)
    lo, se, sy = 0, 0.0, 0.0
    for e, n in enumerate(counts):
        we = wd[e].t() if kind == "fwd" else wd[e]
        y = ad[lo:lo + n] @ we
        got = out[lo:lo + n].double()
        if exact:
            assert torch.equal(got, y.to(torch.float32).to(torch.bfloat16).double())
        else:
            size = ad[lo:lo + n].abs() @ we.abs()
            tol = 2.0 ** -8 * y.abs() + (src + src // 128) * 2 * U * size
            assert float(((got - y).abs() - tol).max() if n else 0.0) <= 0.0
            se += float((got - y).square().sum())
            sy += float(y.square().sum())
        lo += n
    if not exact and sum(counts) * dst >= 4096:
        assert math.sqrt(se / sy) <= 2.0 ** -8 / math.sqrt(3) + 1e-4
    assert bool((out[lo:] == 7.0).all())


WG = [([1], 128, 128, 0), ([0, 1, 63, 65, 0], 128, 384, 7), ([64, 128, 5], 256, 256, 0),
      ([300, 0, 411], 384, 640, 1), ([5, 70, 0, 0, 130, 64, 1, 2], 256, 1024, 0),
      ([1500], 512, 1152, 0)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("counts,N,K,slack", WG)
def test_wgrad(counts, N, K, slack, exact):
    g = gen(12)
    E, rows = len(counts), sum(counts) + slack
    dy, sd = codes((rows, N), g, exact), scales((rows, N // 128), g, exact)
    a, sa = codes((rows, K), g, exact), scales((rows, K // 128), g, exact)
    dw = torch.full((E, N, K), 7.0, dtype=torch.bfloat16, device=DEV)
    err = zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_wgrad_e4m3(E, rows, N, K, dy, sd, a, sa, offsets(counts), dw, err))
    torch.cuda.synchronize()
    assert int(err) == 0
    dd, ad = rows_ref(dy, sd), rows_ref(a, sa)
    lo = 0
    for e, n in enumerate(counts):
        y = dd[lo:lo + n].t() @ ad[lo:lo + n]
        got = dw[e].double()
        if exact:
            assert torch.equal(got, y.to(torch.float32).to(torch.bfloat16).double())
        else:
            size = dd[lo:lo + n].abs().t() @ ad[lo:lo + n].abs()
            tol = (2.0 ** -9 + 2.0 ** -18 + n * 2 * U) * size + 2.0 ** -8 * y.abs()
            assert float(((got - y).abs() - tol).max()) <= 0.0
            if n >= 32:  # independent roundings of about uniform error
                assert float((got - y).norm() / y.norm()) <= 2.0 ** -8 / math.sqrt(3) + 2e-4
        lo += n


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("counts,N,K,slack", [
    ([2, 0, 3, 1, 0, 2], 272, 384, 0), ([0, 8], 16, 2048, 1), ([9], 512, 1152, 0),
    ([4, 60, 2], 256, 640, 0), ([130], 128, 2176, 0)])
def test_matmul_few_rows(kind, counts, N, K, slack):
    """The forms for few rows: row products, and reductions split over blocks."""
    test_matmul(kind, counts, N, K, slack, True)
    test_matmul(kind, counts, N, K, slack, False)


@pytest.mark.parametrize("rows", [1, 8, 9, 40, 300])
def test_matmul_block_sums_are_fp32(rows):
    """Within one scale block 448 * 448 cancels and 2^-5 stays: every partial sum has at most
    23 significant bits, so fp32 sums in any order give it exactly; sums kept in fewer bits
    would not."""
    N, K = 256, 256
    a = torch.zeros((rows, K), device=DEV)
    w = torch.zeros((1, N, K), device=DEV)
    a[:, 3], a[:, 77], a[:, 40] = 448.0, 448.0, 0.125
    w[:, :, 3], w[:, :, 77], w[:, :, 40] = 448.0, -448.0, 0.25
    a[:, 128 + 5], w[:, :, 128 + 5] = 1.0, 2.0
    out = zeros((rows, N), torch.bfloat16)
    err = zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_e4m3(1, rows, N, K, a.to(torch.float8_e4m3fn),
                                    torch.ones((rows, 2), device=DEV),
                                    w.to(torch.float8_e4m3fn), torch.ones((1, 2, 2), device=DEV),
                                    None, out, err))
    torch.cuda.synchronize()
    assert bool((out == 2.03125).all())


def test_wgrad_scales_of_any_size():
    """Scales far outside f16, different in every block and expert, rows of one block spread
    over 2^24: the rows below 2^-19 of a block's largest scale may lose bits, but no more than
    2^-11 of a code at 2^-19 of the largest scale."""
    g = gen(19)
    counts, N, K = [70, 0, 33], 256, 384
    E, rows = len(counts), sum(counts)
    dy, a = codes((rows, N), g, False), codes((rows, K), g, False)
    sd = torch.exp2(torch.rand((rows, N // 128), generator=g, device=DEV) * 24 - 70)
    sa = torch.exp2(torch.rand((rows, K // 128), generator=g, device=DEV) * 24 + 40)
    sd[:, 1] *= 2.0 ** 60
    dw, err = zeros((E, N, K), torch.bfloat16), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_wgrad_e4m3(E, rows, N, K, dy, sd, a, sa, offsets(counts), dw, err))
    torch.cuda.synchronize()
    assert int(err) == 0
    lo = 0
    for e, n in enumerate(counts):
        r = slice(lo, lo + n)
        lo += n
        if n == 0:
            assert float(dw[e].abs().max()) == 0.0
            continue
        d, x = rows_ref(dy[r], sd[r]), rows_ref(a[r], sa[r])
        # absolute floors of the two factors' errors, per channel block
        fd = 448 * 2.0 ** -30 * sd[r].double().amax(0).repeat_interleave(128)
        fa = 448 * 2.0 ** -30 * sa[r].double().amax(0).repeat_interleave(128)
        y = d.t() @ x
        ed, ex = 2.0 ** -10 * d.abs() + fd, 2.0 ** -10 * x.abs() + fa
        tol = (ed.t() @ (x.abs() + ex) + d.abs().t() @ ex + n * 2 * U * (d.abs().t() @ x.abs())
               + 2.0 ** -8 * y.abs())
        assert bool(((dw[e].double() - y).abs() <= tol).all())


def test_matmul_dense_without_offsets_and_gradient_identity():
    """E = 1 without offsets is the dense product; <dy, a w^T> = <dy w, a> = <dy^T a, w>."""
    g = gen(13)
    rows, N, K = 200, 256, 384
    a, sa = codes((rows, K), g, True), scales((rows, K // 128), g, True)
    dy, sd = codes((rows, N), g, True), scales((rows, N // 128), g, True)
    w, sw = codes((1, N, K), g, True), scales((1, N // 128, K // 128), g, True)
    y = zeros((rows, N), torch.bfloat16)
    dx = zeros((rows, K), torch.bfloat16)
    dw = zeros((1, N, K), torch.bfloat16)
    err = zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_e4m3(1, rows, N, K, a, sa, w, sw, None, y, err))
    B.check(B.mp_expert_matmul_dgrad_e4m3(1, rows, N, K, dy, sd, w, sw, None, dx, err))
    B.check(B.mp_expert_matmul_wgrad_e4m3(1, rows, N, K, dy, sd, a, sa, None, dw, err))
    torch.cuda.synchronize()
    assert int(err) == 0
    p = [(y.double() * rows_ref(dy, sd)), (dx.double() * rows_ref(a, sa)),
         (dw.double() * weights_ref(w, sw))]
    size = min(float(t.abs().sum()) for t in p)
    v = [float(t.sum()) for t in p]
    assert max(v) - min(v) <= 2 * 2.0 ** -8 * size


def test_matmul_reports_bad_offsets_and_stays_in_bounds():
    g = gen(14)
    rows, N, K, E = 100, 128, 128, 3
    a, sa = codes((rows, K), g, True), scales((rows, 1), g, True)
    w, sw = codes((E, N, K), g, True), scales((E, 1, 1), g, True)
    ref = rows_ref(a, sa) @ weights_ref(w, sw)[0].t()
    for off, bits in (([0, 50, 90, 130], B.MP_ERR_CAPACITY), ([0, 50, 40, 100], B.MP_ERR_INVALID_ARG),
                      ([-5, 50, 60, 100], B.MP_ERR_INVALID_ARG)):
        out = torch.full((rows + 64, N), 7.0, dtype=torch.bfloat16, device=DEV)
        err = zeros(1, torch.int32)
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        B.check(B.mp_expert_matmul_e4m3(E, rows, N, K, a, sa, w, sw, o, out, err))
        dw = zeros((E, N, K), torch.bfloat16)
        e2 = zeros(1, torch.int32)
        B.check(B.mp_expert_matmul_wgrad_e4m3(E, rows, N, K, a, sa, a, sa, o, dw, e2))
        torch.cuda.synchronize()
        assert int(err) & bits and int(e2) & bits
        assert bool((out[rows:] == 7.0).all())
        if bits == B.MP_ERR_CAPACITY:
            assert torch.equal(out[:50].double(), ref[:50].float().bfloat16().double())
        else:  # nothing is written
            assert bool((out == 7.0).all())


def test_matmul_nan_stays_in_its_row():
    g = gen(15)
    rows, N, K = 140, 256, 256
    a, sa = codes((rows, K), g, True), scales((rows, 2), g, True)
    w, sw = codes((2, N, K), g, True), scales((2, 2, 2), g, True)
    off = offsets([70, 70])
    clean, dirty = zeros((rows, N), torch.bfloat16), zeros((rows, N), torch.bfloat16)
    err = zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_e4m3(2, rows, N, K, a, sa, w, sw, off, clean, err))
    a[69] = math.nan
    sa[70, 1] = math.inf
    B.check(B.mp_expert_matmul_e4m3(2, rows, N, K, a, sa, w, sw, off, dirty, err))
    torch.cuda.synchronize()
    assert bool(dirty[69].isnan().all()) and not bool(dirty[70].isfinite().any())
    keep = [r for r in range(rows) if r not in (69, 70)]
    assert torch.equal(clean[keep], dirty[keep])


def test_matmul_rows_past_32_bit_offsets():
    """Elements past 2^31 in the rows, and in the output."""
    g = gen(16)
    err = zeros(1, torch.int32)
    for N, K in ((128, 7168), (7168, 128)):
        rows = 300_000
        off = torch.tensor([rows - 130, rows - 5, rows], dtype=torch.int32, device=DEV)
        a = zeros((rows, K), torch.float8_e4m3fn)
        sa = zeros((rows, K // 128))
        a[-130:], sa[-130:] = codes((130, K), g, True), scales((130, K // 128), g, True)
        w, sw = codes((2, N, K), g, True), scales((2, N // 128, K // 128), g, True)
        out = zeros((rows, N), torch.bfloat16)
        B.check(B.mp_expert_matmul_e4m3(2, rows, N, K, a, sa, w, sw, off, out, err))
        torch.cuda.synchronize()
        ad, wd = rows_ref(a[-130:], sa[-130:]), weights_ref(w, sw)
        y = torch.cat([ad[:125] @ wd[0].t(), ad[125:] @ wd[1].t()])
        assert torch.equal(out[-130:].double(), y.float().bfloat16().double())
        assert float(out[:-130].abs().max()) == 0.0
        del a, out
    assert int(err) == 0


def test_matmul_without_rows_and_many_experts():
    g = gen(17)
    err = zeros(1, torch.int32)
    dw = torch.full((2, 128, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    off = zeros(3, torch.int32)
    none8, none = zeros((0, 128), torch.float8_e4m3fn), zeros((0, 1))
    B.check(B.mp_expert_matmul_wgrad_e4m3(2, 0, 128, 128, none8, none, none8, none, off, dw, err))
    E, N, K = 8192, 16, 128
    counts = np.zeros(E, np.int64)
    counts[[3, 4000, 8191]] = [2, 1, 130]
    rows = int(counts.sum())
    a, sa = codes((rows, K), g, True), scales((rows, 1), g, True)
    w, sw = codes((E, N, K), g, True), scales((E, 1, 1), g, True)
    out = zeros((rows, N), torch.bfloat16)
    B.check(B.mp_expert_matmul_e4m3(E, rows, N, K, a, sa, w, sw, offsets(counts), out, err))
    torch.cuda.synchronize()
    assert int(err) == 0 and float(dw.abs().max()) == 0.0
    expert = torch.from_numpy(np.repeat(np.arange(E), counts)).to(DEV)
    y = torch.einsum("rk,rnk->rn", rows_ref(a, sa), weights_ref(w, sw)[expert])
    assert torch.equal(out.double(), y.float().bfloat16().double())


def test_matmul_on_another_stream():
    g = gen(18)
    rows, N, K = 64, 256, 512
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a, sa = codes((rows, K), g, True), scales((rows, K // 128), g, True)
        w, sw = codes((1, N, K), g, True), scales((1, N // 128, K // 128), g, True)
        out = zeros((rows, N), torch.bfloat16)
        err = zeros(1, torch.int32)
        B.check(B.mp_expert_matmul_e4m3(1, rows, N, K, a, sa, w, sw, None, out, err))
    side.synchronize()
    y = rows_ref(a, sa) @ weights_ref(w, sw)[0].t()
    assert torch.equal(out.double(), y.float().bfloat16().double())


# ------------------------------------------------------------------ activation

def swiglu_ref(x, I, w):
    g, u = x.double().split(I, -1)
    s = torch.sigmoid(g)
    return g, u, s, (torch.ones(x.shape[0], device=DEV).double() if w is None else w.double())[:, None]


def check_quantised(codes, scale, z):
    rows, C = z.shape
    if rows == 0:
        return
    amax = z.abs().view(rows, C // 128, 128).amax(-1)
    want = torch.where(amax / 448 >= 2.0 ** -126, amax / 448, 1.0)
    assert float(((scale.double() - want).abs() - 1e-5 * want).max()) <= 0.0
    wide = scale.double().repeat_interleave(128, 1)
    tol = (2.0 ** -4 + 1e-5) * z.abs() + wide * 2.0 ** -10
    assert float(((codes.double() * wide - z).abs() - tol).max()) <= 0.0


@pytest.mark.parametrize("shift", [0, 8])  # 8 elements: 16-byte but not 32-byte aligned
@pytest.mark.parametrize("rows,I,weighted,used", [
    (1, 128, False, None), (3, 640, True, None), (64, 2048, False, 40), (130, 512, True, 129),
    (5, 1152, True, 0), (257, 4096, True, None), (4, 4224, False, 9)])
def test_swiglu_and_backward(rows, I, weighted, used, shift):
    g = gen(21)

    def bf16(n, size):
        flat = zeros(n + shift, torch.bfloat16)
        flat[shift:] = (torch.randn(n, generator=g, device=DEV) * size).bfloat16()
        return flat[shift:]
    x = bf16(rows * 2 * I, 3.0).view(rows, 2 * I)
    d = bf16(rows * I, 0.5).view(rows, I)
    if rows > 2:
        x[1, :128] = 0          # a block of zeros: scale 1
        x[2, I:I + 128] = 0
    w = torch.randn(rows, generator=g, device=DEV) if weighted else None
    num = None if used is None else torch.tensor([used], dtype=torch.int32, device=DEV)
    n = rows if used is None else min(used, rows)
    out, sc = zeros((rows, I), torch.float8_e4m3fn), zeros((rows, I // 128)) - 7
    dg, dsc = zeros((rows, 2 * I), torch.float8_e4m3fn), zeros((rows, 2 * I // 128)) - 7
    dw = zeros(rows) - 7
    B.check(B.mp_swiglu_e4m3(rows, I, x, w, num, out, sc))
    B.check(B.mp_swiglu_backward_e4m3(rows, I, x, w, d, num, dg, dsc, dw))
    torch.cuda.synchronize()
    gg, u, s, ww = swiglu_ref(x, I, w)
    dd = d.double()
    check_quantised(out[:n], sc[:n], (gg * s * u * ww)[:n])
    dz = torch.cat([dd * ww * u * s * (1 + gg * (1 - s)), dd * ww * gg * s], -1)
    check_quantised(dg[:n], dsc[:n], dz[:n])
    terms = dd * gg * s * u
    assert bool(((dw.double() - terms.sum(-1)).abs() <= 1e-5 * terms.abs().sum(-1))[:n].all())
    for t in (sc[n:], dsc[n:], dw[n:]):
        assert bool((t == -7).all())
    assert int(out[n:].view(torch.uint8).count_nonzero()) == 0
    again, sc2 = torch.zeros_like(out), torch.zeros_like(sc)
    dw2 = torch.zeros_like(dw)
    B.check(B.mp_swiglu_e4m3(rows, I, x, w, num, again, sc2))
    B.check(B.mp_swiglu_backward_e4m3(rows, I, x, w, d, num, dg, dsc, dw2))
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))
    assert torch.equal(dw[:n], dw2[:n])


def test_swiglu_backward_against_differences():
    """The decoded gradient is within the code's rounding of central differences of the 64-bit
    activation."""
    g = gen(22)
    rows, I = 6, 256
    x = (torch.randn((rows, 2 * I), generator=g, device=DEV) * 2).bfloat16()
    d = torch.randn((rows, I), generator=g, device=DEV).bfloat16()
    w = torch.rand(rows, generator=g, device=DEV) + 0.5
    dg, dsc, dw = zeros((rows, 2 * I), torch.float8_e4m3fn), zeros((rows, 4)), zeros(rows)
    B.check(B.mp_swiglu_backward_e4m3(rows, I, x, w, d, None, dg, dsc, dw))
    torch.cuda.synchronize()

    def f(x, w):
        a, u = x.split(I, -1)
        return (a * torch.sigmoid(a) * u * w[:, None] * d.double()).sum(-1)
    h = 1e-5
    xd, wd = x.double(), w.double()
    for c in (0, 1, 127, 128, 255, 256, 300, 511):
        v = torch.zeros_like(xd)
        v[:, c] = h
        diff = (f(xd + v, wd) - f(xd - v, wd)) / (2 * h)
        wide = dsc.double()[:, c // 128]
        tol = (2.0 ** -4 + 1e-4) * diff.abs() + wide * 2.0 ** -10 + 1e-7
        assert bool(((dg.double()[:, c] * wide - diff).abs() <= tol).all())
    diff = (f(xd, wd + h) - f(xd, wd - h)) / (2 * h)
    size = (d.double() * f(xd, wd)[:, None]).abs().sum(-1)
    assert bool(((dw.double() - diff).abs() <= 1e-4 * diff.abs() + 1e-6 * size + 1e-4).all())


def test_swiglu_extremes():
    """Gates far out on both sides, values that overflow a product, NaN kept to its place."""
    x = zeros((3, 512), torch.bfloat16)
    x[0, :256] = torch.linspace(-120, 120, 256, device=DEV).bfloat16()
    x[0, 256:] = 1.5
    x[1, :256], x[1, 256:] = 2.0, 1.0
    x[1, 7] = math.nan
    x[2, :256], x[2, 256:] = 1e-30, 1e-20   # z about 5e-51: below fp32, scale 1
    out, sc = zeros((3, 256), torch.float8_e4m3fn), zeros((3, 2))
    B.check(B.mp_swiglu_e4m3(3, 256, x, None, None, out, sc))
    torch.cuda.synchronize()
    g, u, s, _ = swiglu_ref(x, 256, None)
    check_quantised(out[:1], sc[:1], (g * s * u)[:1])
    z = out[1].float() * sc[1].repeat_interleave(128)
    assert bool(z[7].isnan()) and int(z.isnan().sum()) == 1
    assert torch.allclose(z[8:], torch.full_like(z[8:], 2 / (1 + math.exp(-2))), rtol=0.07)
    assert sc[2].cpu().tolist() == [1.0, 1.0] and int(out[2].view(torch.uint8).count_nonzero()) == 0


def test_swiglu_rows_past_32_bit_offsets():
    rows, I = 66_000, 16_384   # 2 * rows * I is past 2^31
    x = zeros((rows, 2 * I), torch.bfloat16)
    x[-1] = torch.randn(2 * I, generator=gen(23), device=DEV).bfloat16()
    out, sc = zeros((rows, I), torch.float8_e4m3fn), zeros((rows, I // 128))
    B.check(B.mp_swiglu_e4m3(rows, I, x, None, None, out, sc))
    torch.cuda.synchronize()
    g, u, s, _ = swiglu_ref(x[-1:], I, None)
    check_quantised(out[-1:], sc[-1:], g * s * u)
    assert bool((sc[:-1] == 1.0).all())


# ------------------------------------------------------------------ the layer

@pytest.mark.parametrize("scoring,N", [("softmax", 64), ("sigmoid", 37)])
def test_moe_layer_forward_and_backward(scoring, N):
    """The whole layer against 64 bits on unquantised rows.  e4m3 rounds each value of a row
    with a relative error of at most 2^-4, about uniform: 2^-4 / sqrt(3) in the 2-norm, once
    for the tokens and once for the activation (forward), and for the gradients once more for
    each quantised factor: within 2^-4 * sqrt(2), and 2^-4 * sqrt(4)."""
    from combine_mp_layout_gb300.moe_layer import quantise_weights
    from combine_mp_layout_gb300.pipeline import MoELayerPlan
    R, K, E, H, I = 2, 2, 8, 256, 384
    g = gen(31)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)
    x, d_out = rand(R, N, H).bfloat16(), rand(R, N, H).bfloat16()
    logits, d_loss = rand(R, N, E) * 1.5, rand(R)
    active = (torch.rand((R, N), generator=g, device=DEV) < 0.9).to(torch.uint8)
    bias = rand(E) * 0.1 if scoring == "sigmoid" else None
    wg, wd = quantise_weights(rand(E, 2 * I, H) / 16), quantise_weights(rand(E, H, I) / 16)
    plan = MoELayerPlan(R, N, K, E, H, I, scoring=scoring, scale=1.5, loss_coef=0.1)
    plan.forward(x, logits, *wg, *wd, bias=bias, active=active)
    plan.backward(d_out, logits, *wg, *wd, d_balance_loss=d_loss, active=active)
    torch.cuda.synchronize()
    assert plan.device_error() == 0
    # the same layer in 64 bits, with the kernel's choice of experts
    xd = x.double().requires_grad_(True)
    ld = logits.double().requires_grad_(True)
    wgd = weights_ref(*wg).requires_grad_(True)
    wdd = weights_ref(*wd).requires_grad_(True)
    mode = B.MP_SOFTMAX if scoring == "softmax" else B.MP_SIGMOID
    lost = ~active.bool()[..., None]
    masked = torch.where(lost, torch.full_like(ld, -math.inf), ld)
    _, w, loss = objective_ref(masked, plan.topk_idx, plan.num_tokens_per_expert, plan.num_routed,
                               mode, True, 1.5, 0.1, zeros((R, N, K)), zeros(R), K)
    out = torch.zeros((R, N, H), dtype=torch.float64, device=DEV)
    for k in range(K):
        e = plan.topk_idx[..., k].long()
        on = (e >= 0)[..., None]
        ec = e.clamp(min=0)
        gu = torch.einsum("rnh,rnih->rni", xd, wgd[ec])
        a, u = gu.split(I, -1)
        z = a * torch.sigmoid(a) * u * w[..., k:k + 1]
        out = out + torch.where(on, torch.einsum("rni,rnhi->rnh", z, wdd[ec]), 0.0)
    assert torch.allclose(plan.balance_loss.double(), loss, rtol=1e-4)

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())
    assert off(plan.out, out.detach()) <= 2.0 ** -4 * math.sqrt(2)
    total = (out * d_out.double()).sum() + (loss * d_loss.double()).sum()
    dx, dlog, dwg, dwd = torch.autograd.grad(total, (xd, ld, wgd, wdd))
    for got, want in ((plan.d_x, dx), (plan.d_w_gate_up, dwg), (plan.d_w_down, dwd)):
        assert off(got, want) <= 2.0 ** -3
    live = active.bool()
    assert float(plan.d_logits[~live].abs().max()) == 0.0
    assert off(plan.d_logits[live], dlog[live]) <= 2.0 ** -3


def test_row_weights_and_back():
    R, N, K, cap = 2, 50, 3, 200
    g = gen(32)
    w = torch.rand((R, N, K), generator=g, device=DEV)
    slots = torch.randperm(R * N * K, generator=g, device=DEV).to(torch.int32).view(R, N, K)
    slots[0, 3, 1] = -1
    rows, back = zeros(cap) - 7, zeros((R, N, K)) - 7
    B.check(B.mp_ll_row_weights(R, N, K, w, slots, cap, rows))
    B.check(B.mp_ll_row_weights_backward(R, N, K, rows, cap, slots, back))
    torch.cuda.synchronize()
    placed = (slots >= 0) & (slots < cap)
    want = zeros(cap) - 7
    want[slots[placed].long()] = w[placed]
    assert torch.equal(rows, want)
    assert torch.equal(back, torch.where(placed, w, 0.0))


# ------------------------------------------------------------------ guard regions

class Guarded:
    """A buffer between two guard regions of 4 KB; `intact` after the calls."""

    def __init__(self, shape, dtype):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((4096 + n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        self.n = n
        self.t = self.raw[4096:4096 + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:4096] == 0x5A).all()) and bool((self.raw[4096 + self.n:] == 0x5A).all())


@pytest.mark.parametrize("counts,N,K", [([1], 144, 384), ([5, 0, 130], 272, 128), ([40], 16, 640),
                                        ([129, 3], 400, 256)])
def test_products_write_only_their_outputs(counts, N, K):
    g = gen(41)
    E, rows = len(counts), sum(counts)
    n128 = -(-N // 128) * 128
    a, sa = codes((rows, K), g, False), scales((rows, K // 128), g, False)
    dy, sd = codes((rows, n128), g, False), scales((rows, n128 // 128), g, False)
    w, sw = codes((E, N, K), g, False), scales((E, n128 // 128, K // 128), g, False)
    w2 = codes((E, n128, K), g, False)
    out, dx = Guarded((rows, N), torch.bfloat16), Guarded((rows, K), torch.bfloat16)
    dw, err = Guarded((E, n128, K), torch.bfloat16), Guarded((1,), torch.int32)
    err.t.zero_()
    off = offsets(counts)
    B.check(B.mp_expert_matmul_e4m3(E, rows, N, K, a, sa, w, sw, off, out.t, err.t))
    B.check(B.mp_expert_matmul_dgrad_e4m3(E, rows, n128, K, dy, sd, w2, sw, off, dx.t, err.t))
    B.check(B.mp_expert_matmul_wgrad_e4m3(E, rows, n128, K, dy, sd, a, sa, off, dw.t, err.t))
    torch.cuda.synchronize()
    assert int(err.t) == 0
    assert all(b.intact() for b in (out, dx, dw, err))


@pytest.mark.parametrize("R,N,E,K", [(1, 1, 1, 1), (3, 29, 70, 5), (2, 11, 1500, 32)])
def test_router_and_activation_write_only_their_outputs(R, N, E, K):
    g = gen(42)
    logits = torch.randn((R, N, E), generator=g, device=DEV)
    f32, i32 = torch.float32, torch.int32
    ids, w, counts = Guarded((R, N, K), i32), Guarded((R, N, K), f32), Guarded((R, E), i32)
    routed, loss, err = Guarded((R,), i32), Guarded((R,), f32), Guarded((1,), i32)
    ws, d = Guarded((B.mp_route_workspace_size(R, N, E),), torch.uint8), Guarded((R, N, E), f32)
    ws.t.zero_()
    err.t.zero_()
    B.check(B.mp_route(R, N, K, E, B.MP_SIGMOID, logits, None, None, True, 1.0, 0.1, ids.t, w.t,
                       counts.t, routed.t, loss.t, err.t, ws.t))
    B.check(B.mp_route_backward(R, N, K, E, B.MP_SIGMOID, logits, None, True, 1.0, 0.1, ids.t,
                                torch.ones_like(w.t), counts.t, routed.t, torch.ones_like(loss.t),
                                d.t))
    rows, I = 3 * R, 128 * (1 + N % 7)
    x = torch.randn((rows, 2 * I), generator=g, device=DEV).bfloat16()
    f8 = torch.float8_e4m3fn
    out, sc = Guarded((rows, I), f8), Guarded((rows, I // 128), f32)
    dg, dsc = Guarded((rows, 2 * I), f8), Guarded((rows, 2 * I // 128), f32)
    dw = Guarded((rows,), f32)
    B.check(B.mp_swiglu_e4m3(rows, I, x, None, None, out.t, sc.t))
    B.check(B.mp_swiglu_backward_e4m3(rows, I, x, None, x[:, :I].contiguous(), None, dg.t, dsc.t,
                                      dw.t))
    torch.cuda.synchronize()
    assert all(b.intact() for b in (ids, w, counts, routed, loss, err, ws, d, out, sc, dg, dsc, dw))


def test_products_repeat_bit_for_bit_and_in_a_graph():
    """No order of blocks changes a bit, and the calls can be captured."""
    g = gen(43)
    E, rows, N, K = 3, 333, 512, 1024
    a, sa = codes((rows, K), g, False), scales((rows, K // 128), g, False)
    dy, sd = codes((rows, N), g, False), scales((rows, N // 128), g, False)
    w, sw = codes((E, N, K), g, False), scales((E, N // 128, K // 128), g, False)
    off, err = offsets([100, 33, 200]), zeros(1, torch.int32)
    outs = [zeros((rows, N), torch.bfloat16), zeros((rows, K), torch.bfloat16),
            zeros((E, N, K), torch.bfloat16)]

    def calls():
        B.check(B.mp_expert_matmul_e4m3(E, rows, N, K, a, sa, w, sw, off, outs[0], err))
        B.check(B.mp_expert_matmul_dgrad_e4m3(E, rows, N, K, dy, sd, w, sw, off, outs[1], err))
        B.check(B.mp_expert_matmul_wgrad_e4m3(E, rows, N, K, dy, sd, a, sa, off, outs[2], err))
    calls()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(5):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, f) for o, f in zip(outs, first))
    assert int(err) == 0
