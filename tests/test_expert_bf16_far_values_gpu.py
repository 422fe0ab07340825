"""The operators on bf16 rows where values lie far apart: weight scales of every size side by
side, rows whose values differ by many powers of two, gates far below zero.

Every product below has one term that is not zero, so it is that term rounded to bf16: bit-equal.
The activation's tolerance stands at its test.
"""
import math

import pytest
import torch

from combine_mp_layout_gb300 import binding as B
from tests.test_expert_bf16_gpu import BF, DEV, fp4_ref, gate_ref, rounded, zeros

pytestmark = pytest.mark.gpu


def packed(codes):
    """e2m1 codes [..., K], two a byte."""
    c = codes.to(torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


@pytest.mark.parametrize("rows", [4, 8, 128, 300])  # the row form with room for 4 and 8, tiles
@pytest.mark.parametrize("K", [128, 512])           # scales that TMA cannot load, and can
def test_mxfp4_scales_side_by_side(rows, K):
    """Scale bytes 0 to 252 in neighbouring channels and in both groups of every 64 steps: what a
    weight is does not depend on its neighbours' scales.  Row r reads reduction step r alone."""
    N, groups = 520, K // 32
    n, j = torch.arange(N, device=DEV)[:, None], torch.arange(groups, device=DEV)[None]
    s = ((n * 37 + j * 101) % 253).to(torch.uint8)[None].contiguous()
    assert all(int((s[0, :, 0] == v).sum()) >= 2 for v in (0, 1, 128, 129, 191, 192, 252))
    k = torch.arange(K, device=DEV)[None]
    w = packed((n * 5 + k) % 16)[None]
    ref = fp4_ref(w, s)[0]
    err = zeros(1, torch.int32)
    for factor, seen in ((2.0 ** 100, s < 200), (2.0 ** -100, s > 101)):
        # (what is left out would leave fp32's normal numbers, on either side)
        seen = seen[0].repeat_interleave(32, -1).t()
        for r0 in range(0, K, rows):
            a, out = zeros((rows, K), BF), zeros((rows, N), BF)
            m = min(rows, K - r0)
            at = torch.arange(m, device=DEV)
            a[at, r0 + at] = factor
            B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, w, s, None, out, err))
            torch.cuda.synchronize()
            want = rounded(ref.t()[r0:r0 + m] * factor)
            differ = (out[:m].double() != want) & seen[r0:r0 + m]
            assert int(differ.sum()) == 0, (factor, r0, differ.nonzero()[:5])
    assert int(err) == 0


# ------------------------------------------------------------------ gates far below zero
# A gate's e^g is the square of a number whose exponent, |g| log2(e) / 2 <= 128, is off by 2^-24 of
# itself for the product and 2^-25 for the constant: 128 * 1.5 * 2^-24 * ln 2 = 8e-6 of its value,
# twice that for the square, and the exponential's, reciprocal's and products' few 2^-23: below
# 3e-5.  Gates below -177 count as minus infinity in the exponential: e^g is below 2^-255 there, so
# |g e^g| and |(1 + g) e^g| are below 2^-247.
FAR = 3e-5


def far_off(got, want, size):
    """The largest excess over the tolerance: the above, a rounding to bf16 (2^-8 of a normal
    number, 2^-134 below), and 2^-247 of what e^g is multiplied by."""
    tol = (2.0 ** -8 + FAR) * want.abs() + 2.0 ** -134 + 2.0 ** -247 * size
    bad = (got.double() - want).abs() > tol
    return [(t.item(), w.item()) for t, w in zip(got[bad][:4], want[bad][:4])]


@pytest.mark.parametrize("I", [256, 264])  # 16 and 8 channels a lane
@pytest.mark.parametrize("weighted", [True, False])
def test_swiglu_gates_far_below_zero(I, weighted):
    """Gates from -60 to -220 with up values and output gradients that bring the results back into
    bf16's range; plain forms that form exp(-g) in fp32 have zeros from -88.8 on."""
    ups = [1.5, -3.0, 2.0 ** 30, -2.0 ** 60, 1.25 * 2.0 ** 90, 2.0 ** 110, 1.0]
    rows = len(ups)
    x, d = zeros((rows, 2 * I), BF), torch.ones((rows, I), dtype=BF, device=DEV)
    x[:, :I] = torch.linspace(-60, -220, I, device=DEV).to(BF)
    x[:, I:] = torch.tensor(ups, device=DEV)[:, None].to(BF)
    d[1], d[6] = -0.75, 2.0 ** 115
    w = torch.linspace(0.25, 1.5, rows, device=DEV) if weighted else None
    out, dg, dw = zeros((rows, I), BF), zeros((rows, 2 * I), BF), zeros(rows)
    B.check(B.mp_swiglu_bf16(rows, I, x, w, None, out))
    B.check(B.mp_swiglu_backward_bf16(rows, I, x, w, d, None, dg, dw))
    torch.cuda.synchronize()
    g, u, s, ww = gate_ref(x, I, w)
    dd = d.double()
    want = g * s * u * ww
    assert far_off(out, want, (u * ww).abs().expand_as(want)) == []
    slope = s * (1 + g * (1 - s))
    assert far_off(dg[:, :I], dd * ww * u * slope, (dd * ww * u).abs()) == []
    assert far_off(dg[:, I:], dd * ww * g * s, (dd * ww).abs().expand_as(want)) == []
    terms = dd * g * s * u
    # (fp32 sums: 2^-24 a step, far below FAR; its smallest step is 2^-149)
    tol = 2 * FAR * terms.abs().sum(-1) + 2.0 ** -140 + 2.0 ** -247 * (dd * u).abs().sum(-1)
    assert bool(((dw.double() - terms.sum(-1)).abs() <= tol).all())
    assert float(out[3, I // 5].abs()) > 0  # (a gate past -88.8)


@pytest.mark.parametrize("I", [256, 264])
def test_swiglu_far_gates_leave_their_neighbours_alone(I):
    """The other channels of a row with far gates, minus infinity and NaN among them, keep their
    bits; so do the row weights' gradients where the far channels' terms are nothing."""
    g = torch.Generator(device=DEV)
    g.manual_seed(51)
    rows = 40
    x = (torch.randn((rows, 2 * I), generator=g, device=DEV) * 2).to(BF)
    d = torch.randn((rows, I), generator=g, device=DEV).to(BF)
    w = torch.rand(rows, generator=g, device=DEV) + 0.5
    far = torch.rand((rows, I), generator=g, device=DEV) < 0.2
    near, there = x.clone(), x.clone()
    near[:, :I][far], there[:, :I][far] = 0.0, -150.0
    there[3, 5], there[4, 6] = -math.inf, math.nan
    far[3, 5] = far[4, 6] = True
    near[3, 5] = near[4, 6] = 0.0
    results = []
    for t in (near, there):
        out, dg, dw = zeros((rows, I), BF), zeros((rows, 2 * I), BF), zeros(rows)
        B.check(B.mp_swiglu_bf16(rows, I, t, w, None, out))
        B.check(B.mp_swiglu_backward_bf16(rows, I, t, w, d, None, dg, dw))
        torch.cuda.synchronize()
        results.append((out, dg[:, :I], dg[:, I:], dw))
    (a, b) = results
    for p, q in zip(a[:3], b[:3]):
        assert torch.equal(p[~far], q[~far])
    keep = [r for r in range(rows) if r not in (3, 4)]
    assert torch.equal(a[3][keep], b[3][keep])
    assert bool(b[0][3, 5].isnan()) and bool(b[0][4, 6].isnan())  # -inf * 0, as the formula has it
    rest = far.clone()
    rest[3, 5] = rest[4, 6] = False
    assert float(b[0][rest].abs().max()) == 0.0
