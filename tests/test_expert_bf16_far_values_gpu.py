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


# ------------------------------------------------------------------ rows whose values lie far apart


@pytest.mark.parametrize("rows", [1, 3, 7, 16, 128])  # the row form, tiles
@pytest.mark.parametrize("K,scale", [(224, 127), (512, 127), (512, 60), (512, 200), (736, 252)])
@pytest.mark.parametrize("largest", [127, 60, 0, -60])
def test_mxfp4_small_values_beside_large_ones(rows, K, scale, largest):
    """The first of every 32 values of a row is the largest, and its weights are 0; the others are
    2^-1 to 2^-220 of it with all of bf16's bits, and each is what one channel reads: it comes out
    as if it stood alone, whatever the number of rows.  (Where that is below bf16's normal numbers
    it may be off by bf16's smallest step: fp32 has few bits there too.)"""
    N = K
    k = torch.arange(K, device=DEV)
    away = 1 + (k * 7) % 220
    value = torch.ldexp(1 + ((k * 37) % 128).double() / 128, largest - away)
    value[::32] = 1.5 * 2.0 ** (largest - 1)
    a = value.to(BF)[None].expand(rows, K).contiguous()
    a[1::2] *= -1
    codes = torch.zeros((1, N, K), dtype=torch.int64, device=DEV)
    codes[0, k, k] = torch.where(k % 32 == 0, 0, 1 + k % 7) + 8 * (k % 2)
    w, s = packed(codes), torch.full((1, N, K // 32), scale, dtype=torch.uint8, device=DEV)
    out, err = zeros((rows, N), BF), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, w, s, None, out, err))
    torch.cuda.synchronize()
    want = rounded(a.double() * fp4_ref(w, s)[0].diagonal())
    differ = (out.double() != want) & ((want.abs() >= 2.0 ** -126)
                                       | ((out.double() - want).abs() > 2.0 ** -133))
    assert int(differ.sum()) == 0, [(int(c), float(a[0, c]), float(out[r, c]), float(want[r, c]))
                                    for r, c in differ.nonzero()[:6].tolist()]
    assert int(err) == 0


@pytest.mark.parametrize("rows", [2, 6, 140])
def test_mxfp4_far_values_of_one_row_and_the_rest(rows):
    """Row 0 has values far apart, infinity and NaN where channels 1 and 2 alone have weights that
    are not 0; the other rows keep their bits, and an infinite weight makes the smallest value
    infinite."""
    g = torch.Generator(device=DEV)
    g.manual_seed(52)
    N, K = 264, 512
    codes = torch.randint(0, 16, (1, N, K), generator=g, device=DEV)
    a = torch.randn((rows, K), generator=g, device=DEV).round().clamp(-2, 2).to(BF)
    s = torch.full((1, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    codes[0, 3], codes[0, 3, 40] = 0, 7
    s[0, 3, 1] = 254                     # 6 * 2^127, of channel 3 alone
    w, err = packed(codes), zeros(1, torch.int32)
    clean, dirty = zeros((rows, N), BF), zeros((rows, N), BF)
    B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, w, s, None, clean, err))
    b = a.clone()
    b[0] = 0
    b[0, 32], b[0, 40], b[0, 41] = 2.0 ** 60, -2.0 ** -100, 1.0
    B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, b, w, s, None, dirty, err))
    torch.cuda.synchronize()
    assert torch.equal(clean[1:, :3], dirty[1:, :3]) and torch.equal(clean[1:, 4:], dirty[1:, 4:])
    assert float(dirty[0, 3]) == -math.inf
    ref = fp4_ref(w, s)[0]
    y, size = b[0].double() @ ref.t(), b[0].double().abs() @ ref.abs().t()
    rest = torch.arange(N, device=DEV) != 3
    # (three terms: 2^-23 a step of their sum, and the rounding to bf16)
    tol = 2.0 ** -8 * y.abs() + 3 * 2.0 ** -23 * size
    assert bool(((dirty[0].double() - y).abs() <= tol)[rest].all())
    b[0, 300], b[0, 41] = math.nan, math.inf
    B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, b, w, s, None, dirty, err))
    torch.cuda.synchronize()
    assert bool(dirty[0].isnan().all()) and torch.equal(clean[1:, 4:], dirty[1:, 4:])
    assert int(err) == 0


def test_mxfp4_rows_of_both_kinds_in_turn():
    """Many experts of a few rows each, every other expert's with values far apart: a block that
    takes several experts one after the other takes each one's rows as they want it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(53)
    E, N, K, each = 40, 1160, 736, 3
    rows = E * each
    codes = torch.randint(0, 16, (E, N, K), generator=g, device=DEV)
    codes[..., 0::32] = 0
    w = packed(codes)
    s = torch.randint(126, 129, (E, N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    a = torch.randint(-2, 3, (rows, K), generator=g, device=DEV).to(BF)
    expert = torch.arange(rows, device=DEV) // each
    far = expert % 2 == 1
    a[far] *= 2.0 ** -50                 # all but the first of 32 values, whose weights are 0
    a[far, 0::32] = 3.0
    off = (torch.arange(E + 1, device=DEV) * each).to(torch.int32)
    out, err = zeros((rows, N), BF), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a, w, s, off, out, err))
    torch.cuda.synchronize()
    want = torch.cat([a[e * each:(e + 1) * each].double() @ fp4_ref(w[e], s[e]).t()
                      for e in range(E)])
    assert torch.equal(out.double(), rounded(want)) and int(err) == 0


@pytest.mark.parametrize("rows", [2, 8, 128])
@pytest.mark.parametrize("far", [False, True])  # values far apart in the row
@pytest.mark.parametrize("scale", [245, 252, 253, 254, 255])
def test_mxfp4_largest_scales(rows, far, scale):
    """Every code at the largest scales: what passes bf16's largest number is infinite, 255 is
    NaN."""
    N, K, at = 32, 512, 103
    n = torch.arange(N, device=DEV)
    codes = torch.zeros((1, N, K), dtype=torch.int64, device=DEV)
    codes[0, :, at] = n % 16
    s = torch.full((1, N, K // 32), 127, dtype=torch.uint8, device=DEV)
    s[0, :, at // 32] = scale
    s[0, 16:, at // 32] = 127            # (neighbours in the warp)
    w = packed(codes)
    a = zeros((rows, K), BF)
    a[:, at] = 2.0 ** -100
    if far:
        a[:, at + 1] = 2.0 ** 20         # (its weights are 0, but not of scale 255)
    ref = fp4_ref(w, torch.clamp(s, max=254))[0, :, at]
    want = ref * 2.0 ** -100
    want = torch.where(ref.abs() >= 2.0 ** 128, torch.copysign(torch.full_like(ref, math.inf), ref),
                       want)
    if scale == 255:
        want[:16] = math.nan
    out, err = zeros((rows, N), BF), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, w, s, None, out, err))
    torch.cuda.synchronize()
    got = out.double()
    same = (got == rounded(want)) | (got.isnan() & want.isnan())
    assert bool(same.all()), (got[0] - want).nonzero()
    assert int(err) == 0
