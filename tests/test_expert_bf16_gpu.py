"""The expert layer's operators on bf16 rows (products with bf16 weights, their gradients, gated
activation) against plain implementations in 64 bits.

Tolerances (U = 2^-24, the unit roundoff of fp32; bf16 rounds by at most 2^-8 of a value):
  * products: one bf16 rounding, plus fp32 sums of n terms: n * 2 U times the sum of the terms'
    magnitudes (2 U per step: the tensor core may cut instead of round).  Over many outputs the
    bf16 rounding is about uniform, so its 2-norm is at most 2^-8 / sqrt(3).  Small whole numbers
    make every sum exact: bit-equal there.
  * activation: the fast exponential and reciprocal and four products, 1e-5 of a value, and the
    bf16 rounding (of a subnormal result: half of bf16's smallest step, 2^-134).
"""
import math
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from combine_mp_layout_gb300 import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda"
BF = torch.bfloat16


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def zeros(shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def values(shape, g, exact):
    x = torch.randn(shape, generator=g, device=DEV)
    return ((x * 1.2).round().clamp(-2, 2) if exact else x).to(BF)


def offsets(counts, first=0):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
                            + first).to(torch.int32).to(DEV)


def rounded(y, dtype=BF):
    """64-bit values that fp32 holds exactly, in the output's type."""
    return y.to(torch.float32).to(dtype).double()


class Guarded:
    """A buffer between two guard regions of 4 KB; `intact` after the calls."""

    def __init__(self, shape, dtype, fill=7.0):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((4096 + n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        self.n = n
        self.t = self.raw[4096:4096 + n].view(dtype).view(shape)
        self.t.fill_(fill)

    def intact(self):
        return bool((self.raw[:4096] == 0x5A).all()) and bool((self.raw[4096 + self.n:] == 0x5A).all())


# ------------------------------------------------------------------ products

MM = [  # counts, N, K, slack rows at the end
    ([1], 8, 8, 0),
    ([1], 16, 72, 1),
    ([3], 48, 256, 2),
    ([0, 1, 127, 129, 0], 136, 392, 7),
    ([128, 256, 5], 264, 64, 0),
    ([31, 33, 64, 65], 512, 1024, 3),
    ([1, 1, 0, 1, 1, 0, 1], 1024, 512, 0),
    ([700], 640, 384, 0),
    ([257, 0, 513], 256, 7168, 1),
    ([1], 4096, 2048, 0),
    ([2500], 384, 264, 0),
    ([40] * 90, 520, 200, 0),
    ([2, 0, 3, 1], 4104, 64, 0),
    ([2, 1, 2], 16392, 200, 1),
    ([8], 776, 7168, 0),
]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("counts,N,K,slack", MM)
def test_matmul(kind, counts, N, K, slack, exact):
    g = gen(11)
    E, rows = len(counts), sum(counts) + slack
    src, dst = (K, N) if kind == "fwd" else (N, K)
    a, w = values((rows, src), g, exact), values((E, N, K), g, exact)
    off, err = offsets(counts), zeros(1, torch.int32)
    buf = Guarded((rows, dst), BF)
    f = B.mp_expert_matmul_bf16 if kind == "fwd" else B.mp_expert_matmul_dgrad_bf16
    B.check(f(E, rows, N, K, a, w, off, buf.t, err))
    torch.cuda.synchronize()
    assert int(err) == 0 and buf.intact()
    out = buf.t
    lo, se, sy = 0, 0.0, 0.0
    for e, n in enumerate(counts):
        x = a[lo:lo + n].double()
        we = w[e].double().t() if kind == "fwd" else w[e].double()
        y, got = x @ we, out[lo:lo + n].double()
        if exact:
            assert torch.equal(got, rounded(y))
        else:
            tol = 2.0 ** -8 * y.abs() + src * 2 * U * (x.abs() @ we.abs())
            assert float(((got - y).abs() - tol).max() if n else 0.0) <= 0.0
            se += float((got - y).square().sum())
            sy += float(y.square().sum())
        lo += n
    if not exact and sum(counts) * dst >= 4096:
        assert math.sqrt(se / sy) <= 2.0 ** -8 / math.sqrt(3) + 1e-4
    assert bool((out[lo:] == 7.0).all())


WG = [([1], 8, 8, 0), ([0, 1, 63, 65, 0], 136, 392, 7), ([64, 128, 5], 256, 264, 0),
      ([300, 0, 411], 384, 640, 1), ([5, 70, 0, 0, 130, 64, 1, 2], 248, 1024, 0),
      ([1500], 520, 1160, 0), ([7] * 300, 256, 296, 0), ([3001], 264, 392, 2),
      ([700, 0, 1, 1900], 256, 248, 0), ([40, 2000], 8, 520, 1)]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("out", ["bf16", "fp32", "add"])
@pytest.mark.parametrize("counts,N,K,slack", WG)
def test_wgrad(counts, N, K, slack, out, exact):
    g = gen(12)
    E, rows = len(counts), sum(counts) + slack
    dy, a = values((rows, N), g, exact), values((rows, K), g, exact)
    before = values((E, N, K), g, exact).float()
    buf, err = Guarded((E, N, K), BF if out == "bf16" else torch.float32), zeros(1, torch.int32)
    if out == "add":
        buf.t.copy_(before)
    B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, dy, a, offsets(counts), out == "add",
                                          buf.t, err))
    torch.cuda.synchronize()
    assert int(err) == 0 and buf.intact()
    lo = 0
    for e, n in enumerate(counts):
        x, d = a[lo:lo + n].double(), dy[lo:lo + n].double()
        y, got = d.t() @ x, buf.t[e].double()
        size = d.abs().t() @ x.abs()
        if out == "add":
            y = y + before[e].double()
        if exact:
            assert torch.equal(got, rounded(y, buf.t.dtype))
        else:
            last = 2.0 ** -8 if out == "bf16" else U
            tol = n * 2 * U * size + last * y.abs()
            if out == "add":  # the sum is rounded, and then it plus what was there
                tol = tol + U * size
            assert float(((got - y).abs() - tol).max()) <= 0.0
        lo += n


@pytest.mark.parametrize("counts", [[63, 65], [1, 1, 130], [33, 0, 64, 96]])
def test_wgrad_takes_no_row_of_another_expert(counts):
    """Rows of NaN and infinity (in other experts, and past the last one) do not count."""
    g = gen(13)
    N, K, E = 264, 136, len(counts)
    rows = sum(counts) + 3
    dy, a = values((rows, N), g, True), values((rows, K), g, True)
    off, err = offsets(counts), zeros(1, torch.int32)
    lo = 0
    for e, n in enumerate(counts):
        d, x = torch.full_like(dy, math.nan), torch.full_like(a, math.inf)
        d[lo:lo + n], x[lo:lo + n] = dy[lo:lo + n], a[lo:lo + n]
        dw = zeros((E, N, K), BF)
        B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, d, x, off, False, dw, err))
        torch.cuda.synchronize()
        assert torch.equal(dw[e].double(), rounded(d[lo:lo + n].double().t() @ x[lo:lo + n].double()))
        lo += n
    assert int(err) == 0


def test_dense_without_offsets_and_gradient_identity():
    """E = 1 without offsets is the dense product; <dy, a w^T> = <dy w, a> = <dy^T a, w>."""
    g = gen(14)
    rows, N, K = 200, 248, 384
    a, dy, w = values((rows, K), g, True), values((rows, N), g, True), values((1, N, K), g, True)
    y, dx, dw = zeros((rows, N), BF), zeros((rows, K), BF), zeros((1, N, K))
    err = zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_bf16(1, rows, N, K, a, w, None, y, err))
    B.check(B.mp_expert_matmul_dgrad_bf16(1, rows, N, K, dy, w, None, dx, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(1, rows, N, K, dy, a, None, False, dw, err))
    torch.cuda.synchronize()
    assert int(err) == 0
    p = [y.double() * dy.double(), dx.double() * a.double(), dw.double() * w.double()]
    v = [float(t.sum()) for t in p]
    assert max(v) - min(v) <= 2 * 2.0 ** -8 * min(float(t.abs().sum()) for t in p)


def test_gradients_against_differences():
    """Whole numbers: moving one factor by h moves the product's sum by h times the gradient."""
    g = gen(15)
    counts, N, K = [5, 0, 9], 24, 40
    rows, E = sum(counts), 3
    a, dy, w = values((rows, K), g, True), values((rows, N), g, True), values((E, N, K), g, True)
    off, err = offsets(counts), zeros(1, torch.int32)
    dx, dw = zeros((rows, K), BF), zeros((E, N, K))
    B.check(B.mp_expert_matmul_dgrad_bf16(E, rows, N, K, dy, w, off, dx, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, dy, a, off, False, dw, err))

    def objective(a, w):
        y = zeros((rows, N), BF)
        B.check(B.mp_expert_matmul_bf16(E, rows, N, K, a, w, off, y, err))
        return float((y.double() * dy.double()).sum())
    for r, k in ((0, 0), (4, 39), (5, 7), (13, 20)):
        up, down = a.clone(), a.clone()
        up[r, k] += 1
        down[r, k] -= 1
        assert (objective(up, w) - objective(down, w)) / 2 == float(dx[r, k])
    for e, n, k in ((0, 0, 0), (0, 23, 39), (1, 3, 3), (2, 11, 17)):
        up, down = w.clone(), w.clone()
        up[e, n, k] += 1
        down[e, n, k] -= 1
        assert (objective(a, up) - objective(a, down)) / 2 == float(dw[e, n, k])
    assert int(err) == 0


def test_sums_are_fp32():
    """Sums that cancel at 2^15 and leave 2^-8: no step of the sum has less than 24 bits."""
    rows, N, K = 40, 256, 512
    a, w = zeros((rows, K), BF), zeros((1, N, K), BF)
    a[:, 0], a[:, 511], a[:, 100] = 256.0, -256.0, 2.0 ** -8
    w[:] = 128.0
    w[..., 100] = 1.0
    y, err = zeros((rows, N), BF), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_bf16(1, rows, N, K, a, w, None, y, err))
    torch.cuda.synchronize()
    assert bool((y == 2.0 ** -8).all())


def test_reports_bad_offsets_and_stays_in_bounds():
    g = gen(16)
    rows, N, K, E = 100, 128, 128, 3
    a, w = values((rows, K), g, True), values((E, N, K), g, True)
    ref = a.double() @ w[0].double().t()
    for off, bits in (([0, 50, 90, 130], B.MP_ERR_CAPACITY), ([0, 50, 40, 100], B.MP_ERR_INVALID_ARG),
                      ([-5, 50, 60, 100], B.MP_ERR_INVALID_ARG)):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        out, dx, dw = (Guarded((rows, N), BF), Guarded((rows, K), BF), Guarded((E, N, K), BF))
        errs = [zeros(1, torch.int32) for _ in range(3)]
        B.check(B.mp_expert_matmul_bf16(E, rows, N, K, a, w, o, out.t, errs[0]))
        B.check(B.mp_expert_matmul_dgrad_bf16(E, rows, N, K, a, w, o, dx.t, errs[1]))
        B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, a, a, o, False, dw.t, errs[2]))
        torch.cuda.synchronize()
        assert all(int(e) & bits for e in errs)
        assert out.intact() and dx.intact() and dw.intact()
        if bits == B.MP_ERR_CAPACITY:
            assert torch.equal(out.t[:50].double(), rounded(ref[:50]))
        else:  # nothing is written
            assert bool((out.t == 7.0).all()) and bool((dx.t == 7.0).all())


def test_nan_and_infinity_stay_in_their_row():
    g = gen(17)
    rows, N, K = 140, 256, 256
    a, w = values((rows, K), g, True), values((2, N, K), g, True)
    off, err = offsets([70, 70]), zeros(1, torch.int32)
    clean, dirty = zeros((rows, N), BF), zeros((rows, N), BF)
    B.check(B.mp_expert_matmul_bf16(2, rows, N, K, a, w, off, clean, err))
    a[69], a[70, 3] = math.nan, math.inf
    B.check(B.mp_expert_matmul_bf16(2, rows, N, K, a, w, off, dirty, err))
    torch.cuda.synchronize()
    assert bool(dirty[69].isnan().all()) and not bool(dirty[70].isfinite().any())
    keep = [r for r in range(rows) if r not in (69, 70)]
    assert torch.equal(clean[keep], dirty[keep])
    # weights of another expert do not reach a row either, at the end of an odd reduction
    w2 = values((2, 40, K), g, True)
    w2[1] = math.nan
    dy, dx = values((rows, 40), g, True), zeros((rows, K), BF)
    B.check(B.mp_expert_matmul_dgrad_bf16(2, rows, 40, K, dy, w2, off, dx, err))
    torch.cuda.synchronize()
    assert torch.equal(dx[:70].double(), rounded(dy[:70].double() @ w2[0].double()))
    assert bool(dx[70:].isnan().all()) and int(err) == 0


def test_rows_past_32_bit_offsets():
    """Elements past 2^31 in the rows, in the output and in the weights."""
    g = gen(18)
    err = zeros(1, torch.int32)
    for N, K in ((128, 7168), (7168, 128)):
        rows = 300_000
        off = torch.tensor([rows - 130, rows - 5, rows], dtype=torch.int32, device=DEV)
        a = zeros((rows, K), BF)
        a[-130:] = values((130, K), g, True)
        w = values((2, N, K), g, True)
        out = zeros((rows, N), BF)
        B.check(B.mp_expert_matmul_bf16(2, rows, N, K, a, w, off, out, err))
        ad, wd = a[-130:].double(), w.double()
        y = torch.cat([ad[:125] @ wd[0].t(), ad[125:] @ wd[1].t()])
        torch.cuda.synchronize()
        assert torch.equal(out[-130:].double(), rounded(y))
        assert float(out[:-130].abs().max()) == 0.0
        if N == 128:
            dy, dw = zeros((rows, N), BF), zeros((2, N, K))
            dy[-130:] = values((130, N), g, True)
            B.check(B.mp_expert_matmul_wgrad_bf16(2, rows, N, K, dy, a, off, False, dw, err))
            torch.cuda.synchronize()
            dd = dy[-130:].double()
            assert torch.equal(dw[0].double(), dd[:125].t() @ ad[:125])
            assert torch.equal(dw[1].double(), dd[125:].t() @ ad[125:])
        del a, out
    E, N, K = 600, 2048, 2048  # 2.5e9 weights
    w = zeros((E, N, K), BF)
    w[-1] = values((N, K), g, True)
    a = values((3, K), g, True)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = 3
    for rows in (3, 3000):  # the rows that there is room for choose the form
        room, out = zeros((rows, K), BF), zeros((rows, N), BF)
        room[:3] = a
        B.check(B.mp_expert_matmul_bf16(E, rows, N, K, room, w, off, out, err))
        torch.cuda.synchronize()
        assert torch.equal(out[:3].double(), rounded(a.double() @ w[-1].double().t()))
    del w
    dw = torch.full((E, N, K), 7.0, dtype=BF, device=DEV)
    dy = values((3, N), g, True)
    B.check(B.mp_expert_matmul_wgrad_bf16(E, 3, N, K, dy, a, off, False, dw, err))
    torch.cuda.synchronize()
    assert torch.equal(dw[-1].double(), rounded(dy.double().t() @ a.double()))
    assert all(float(dw[e].abs().max()) == 0.0 for e in (0, 299, 598))
    assert int(err) == 0


@pytest.mark.parametrize("form", ["bf16", "mxfp4", "dgrad", "wgrad"])
def test_longest_reductions(form):
    """Nearly 2^31 steps, few of them not zero, at both ends."""
    err = zeros(1, torch.int32)
    if form == "wgrad":  # its reduction is over the rows
        rows = 2 ** 31 - 1025
        dy, a = zeros((rows, 8), BF), zeros((rows, 8), BF)
        dy[0], dy[-1], a[0], a[-1] = 1.0, 2.0, 3.0, 5.0
        dw = zeros((1, 8, 8)) + 7
        B.check(B.mp_expert_matmul_wgrad_bf16(1, rows, 8, 8, dy, a, None, False, dw, err))
        torch.cuda.synchronize()
        assert bool((dw == 13.0).all()) and int(err) == 0
        return
    K = 2 ** 31 - 1056
    a, out = zeros((1, K), BF), zeros((1, 8), BF)
    a[0, 0], a[0, 1], a[0, -1] = 1.0, 3.0, 2.0
    if form == "mxfp4":
        w = zeros((1, 8, K // 2), torch.uint8)
        s = torch.full((1, 8, K // 32), 127, dtype=torch.uint8, device=DEV)
        w[..., 0], w[..., -1] = 0x24, 0x40  # codes 4 (2) and 2 (1); 0 and 4 (2)
        B.check(B.mp_expert_matmul_mxfp4(1, 1, 8, K, a, w, s, None, out, err))
    elif form == "bf16":
        w = zeros((1, 8, K), BF)
        w[..., 0], w[..., 1], w[..., -1] = 2.0, 1.0, 2.0
        B.check(B.mp_expert_matmul_bf16(1, 1, 8, K, a, w, None, out, err))
    else:  # the same sums, over the weights' other axis
        w = zeros((1, K, 8), BF)
        w[0, 0], w[0, 1], w[0, -1] = 2.0, 1.0, 2.0
        B.check(B.mp_expert_matmul_dgrad_bf16(1, 1, K, 8, a, w, None, out, err))
    torch.cuda.synchronize()
    assert bool((out == 9.0).all()) and int(err) == 0


def test_without_rows_and_many_experts():
    g = gen(19)
    err = zeros(1, torch.int32)
    none, off = zeros((0, 128), BF), zeros(3, torch.int32)
    dw, kept = torch.full((2, 128, 128), 7.0, dtype=BF, device=DEV), zeros((2, 128, 128)) + 7
    B.check(B.mp_expert_matmul_wgrad_bf16(2, 0, 128, 128, none, none, off, False, dw, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(2, 0, 128, 128, none, none, off, True, kept, err))
    w = values((2, 128, 128), g, True)
    B.check(B.mp_expert_matmul_bf16(2, 0, 128, 128, none, w, off, none, err))
    B.check(B.mp_expert_matmul_dgrad_bf16(2, 0, 128, 128, none, w, off, none, err))
    E, N, K = 8192, 16, 136
    counts = np.zeros(E, np.int64)
    counts[[3, 4000, 8191]] = [2, 1, 130]
    rows = int(counts.sum())
    a, w = values((rows, K), g, True), values((E, N, K), g, True)
    out = zeros((rows, N), BF)
    B.check(B.mp_expert_matmul_bf16(E, rows, N, K, a, w, offsets(counts), out, err))
    torch.cuda.synchronize()
    assert int(err) == 0 and float(dw.abs().max()) == 0.0 and bool((kept == 7).all())
    expert = torch.from_numpy(np.repeat(np.arange(E), counts)).to(DEV)
    y = torch.einsum("rk,rnk->rn", a.double(), w[expert].double())
    assert torch.equal(out.double(), rounded(y))


def test_on_another_stream():
    g = gen(20)
    rows, N, K = 64, 256, 512
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a, w = values((rows, K), g, True), values((1, N, K), g, True)
        out, err = zeros((rows, N), BF), zeros(1, torch.int32)
        B.check(B.mp_expert_matmul_bf16(1, rows, N, K, a, w, None, out, err))
    side.synchronize()
    assert torch.equal(out.double(), rounded(a.double() @ w[0].double().t()))


@pytest.mark.parametrize("shift", [8, 16])  # elements: 16- and 32-byte aligned
def test_other_alignments(shift):
    g = gen(21)
    counts, N, K = [3, 90], 272, 320
    rows = sum(counts)

    def moved(t):
        flat = zeros(t.numel() + shift, t.dtype)
        flat[shift:] = t.flatten()
        return flat[shift:].view(t.shape)
    a, w = moved(values((rows, K), g, True)), moved(values((2, N, K), g, True))
    dy = moved(values((rows, N), g, True))
    y, dx, dw = moved(zeros((rows, N), BF)), moved(zeros((rows, K), BF)), moved(zeros((2, N, K), BF))
    dw32 = zeros(2 * N * K + 4)[4:].view(2, N, K)
    off, err = offsets(counts), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_bf16(2, rows, N, K, a, w, off, y, err))
    B.check(B.mp_expert_matmul_dgrad_bf16(2, rows, N, K, dy, w, off, dx, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(2, rows, N, K, dy, a, off, False, dw, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(2, rows, N, K, dy, a, off, True, dw32, err))
    torch.cuda.synchronize()
    for e, s in enumerate((slice(0, 3), slice(3, 93))):
        x, d, we = a[s].double(), dy[s].double(), w[e].double()
        assert torch.equal(y[s].double(), rounded(x @ we.t()))
        assert torch.equal(dx[s].double(), rounded(d @ we))
        assert torch.equal(dw[e].double(), rounded(d.t() @ x))
        assert torch.equal(dw32[e].double(), d.t() @ x)
    assert int(err) == 0


@pytest.mark.parametrize("rows", [64, 8192])  # split reductions, whole tiles
def test_many_and_few_experts_from_two_threads(rows):
    """The shared memory of a call grows with its experts; threads whose calls alternate do not
    take it from each other."""
    N, K = 512, 1024
    err = zeros(1, torch.int32)

    def prepared(E):
        g = gen(22)
        counts = np.zeros(E, np.int64)
        counts[[0, E - 1]] = [rows - 3, 3]
        a = values((rows, K), g, True)
        w = zeros((E, N, K), BF)
        w[[0, E - 1]] = values((2, N, K), g, True)
        ad, off = a.double(), offsets(counts)
        want = torch.cat([ad[:-3] @ w[0].double().t(), ad[-3:] @ w[E - 1].double().t()])
        want = want.float().to(BF)
        torch.cuda.synchronize()

        def call():
            out = zeros((rows, N), BF)
            status = B.mp_expert_matmul_bf16(E, rows, N, K, a, w, off, out, err)
            torch.cuda.synchronize()
            return status, torch.equal(out, want)
        return call
    many, few = prepared(4000), prepared(2)
    with ThreadPoolExecutor(1) as one, ThreadPoolExecutor(1) as other:
        for _ in range(3):
            assert one.submit(many).result() == (B.MP_OK, True)
            assert other.submit(few).result() == (B.MP_OK, True)
    assert int(err) == 0


def test_products_repeat_bit_for_bit_and_in_a_graph():
    """No order of blocks changes a bit, and the calls can be captured."""
    g = gen(23)
    E, rows, N, K = 3, 333, 512, 1024
    a, dy, w = values((rows, K), g, False), values((rows, N), g, False), values((E, N, K), g, False)
    off, err = offsets([100, 33, 200]), zeros(1, torch.int32)
    outs = [zeros((rows, N), BF), zeros((rows, K), BF), zeros((E, N, K), BF), zeros((E, N, K)),
            zeros((2, N), BF)]

    def calls():
        B.check(B.mp_expert_matmul_bf16(E, rows, N, K, a, w, off, outs[0], err))
        B.check(B.mp_expert_matmul_dgrad_bf16(E, rows, N, K, dy, w, off, outs[1], err))
        B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, dy, a, off, False, outs[2], err))
        B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, dy, a, off, True, outs[3], err))
        B.check(B.mp_expert_matmul_bf16(1, 2, N, K, a, w, None, outs[4], err))
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


# ------------------------------------------------------------------ activation

def gate_ref(x, I, w):
    g, u = x.double().split(I, -1)
    s = torch.sigmoid(g)
    return g, u, s, (torch.ones(x.shape[0], device=DEV).double() if w is None else w.double())[:, None]


def near(got, want):
    tol = (2.0 ** -8 + 1e-5) * want.abs() + 2.0 ** -134
    return float(((got.double() - want).abs() - tol).max() if want.numel() else 0.0) <= 0.0


@pytest.mark.parametrize("shift", [0, 8])  # 8 elements: 16-byte but not 32-byte aligned
@pytest.mark.parametrize("rows,I,weighted,used", [
    (1, 8, False, None), (3, 640, True, None), (64, 2048, False, 40), (130, 520, True, 129),
    (5, 136, True, 0), (257, 4096, True, None), (4, 4224, False, 9), (1001, 48, True, 900),
    (9, 64, True, None), (300, 264, False, -3)])
def test_swiglu_and_backward(rows, I, weighted, used, shift):
    g = gen(31)

    def bf16(n, size):
        flat = zeros(n + shift, BF)
        flat[shift:] = (torch.randn(n, generator=g, device=DEV) * size).to(BF)
        return flat[shift:]
    x, d = bf16(rows * 2 * I, 3.0).view(rows, 2 * I), bf16(rows * I, 0.5).view(rows, I)
    w = torch.randn(rows, generator=g, device=DEV) if weighted else None
    num = None if used is None else torch.tensor([used], dtype=torch.int32, device=DEV)
    n = rows if used is None else min(max(used, 0), rows)
    out, dg, dw = Guarded((rows, I), BF), Guarded((rows, 2 * I), BF), Guarded((rows,), torch.float32)
    B.check(B.mp_swiglu_bf16(rows, I, x, w, num, out.t))
    B.check(B.mp_swiglu_backward_bf16(rows, I, x, w, d, num, dg.t, dw.t))
    torch.cuda.synchronize()
    gg, u, s, ww = gate_ref(x, I, w)
    dd = d.double()
    assert near(out.t[:n], (gg * s * u * ww)[:n])
    assert near(dg.t[:n], torch.cat([dd * ww * u * s * (1 + gg * (1 - s)), dd * ww * gg * s], -1)[:n])
    terms = dd * gg * s * u
    assert bool(((dw.t.double() - terms.sum(-1)).abs() <= 1e-5 * terms.abs().sum(-1))[:n].all())
    for b in (out, dg, dw):
        assert b.intact() and bool((b.t[n:] == 7.0).all())
    first = [b.t.clone() for b in (out, dg, dw)]
    B.check(B.mp_swiglu_bf16(rows, I, x, w, num, out.t))
    B.check(B.mp_swiglu_backward_bf16(rows, I, x, w, d, num, dg.t, dw.t))
    torch.cuda.synchronize()
    assert all(torch.equal(b.t, f) for b, f in zip((out, dg, dw), first))
    B.check(B.mp_swiglu_backward_bf16(rows, I, x, w, d, num, dg.t, None))
    torch.cuda.synchronize()
    assert torch.equal(dg.t, first[1])


def test_swiglu_backward_against_differences():
    g = gen(32)
    rows, I = 6, 256
    x = (torch.randn((rows, 2 * I), generator=g, device=DEV) * 2).to(BF)
    d = torch.randn((rows, I), generator=g, device=DEV).to(BF)
    w = torch.rand(rows, generator=g, device=DEV) + 0.5
    dg, dw = zeros((rows, 2 * I), BF), zeros(rows)
    B.check(B.mp_swiglu_backward_bf16(rows, I, x, w, d, None, dg, dw))
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
        # a difference of sums: 2^-52 of them over h, 1e-7 with room
        assert bool(((dg.double()[:, c] - diff).abs() <= (2.0 ** -8 + 1e-5) * diff.abs() + 1e-7).all())
    diff = (f(xd, wd + h) - f(xd, wd - h)) / (2 * h)
    assert bool(((dw.double() - diff).abs() <= 1e-4 * diff.abs() + 1e-4).all())


def test_swiglu_extremes():
    """Gates far out on both sides, infinities, NaN kept to its place."""
    x = zeros((2, 512), BF)
    x[0, :256] = torch.linspace(-80, 120, 256, device=DEV).to(BF)
    x[0, 256:] = 1.5
    x[1, :256], x[1, 256:] = 2.0, 1.0
    x[1, 7], x[1, 8], x[1, 300] = math.nan, math.inf, -math.inf
    out = zeros((2, 256), BF)
    B.check(B.mp_swiglu_bf16(2, 256, x, None, None, out))
    torch.cuda.synchronize()
    g, u, s, _ = gate_ref(x, 256, None)
    assert near(out[:1], (g * s * u)[:1])
    assert bool(out[1, 7].isnan()) and int(out[1].isnan().sum()) == 1
    assert float(out[1, 8]) == math.inf and float(out[1, 44]) == -math.inf


def test_swiglu_past_32_bit_offsets():
    rows, I = 66_000, 16_392   # 2 * rows * I is past 2^31; I not a multiple of 16
    x = zeros((rows, 2 * I), BF)
    x[-1] = torch.randn(2 * I, generator=gen(33), device=DEV).to(BF)
    out, dg = zeros((rows, I), BF), zeros((rows, 2 * I), BF)
    B.check(B.mp_swiglu_bf16(rows, I, x, None, None, out))
    B.check(B.mp_swiglu_backward_bf16(rows, I, x, None, x[:, :I].contiguous(), None, dg, None))
    torch.cuda.synchronize()
    g, u, s, _ = gate_ref(x[-1:], I, None)
    assert near(out[-1:], g * s * u) and float(out[:-1].abs().max()) == 0.0
    assert near(dg[-1:], torch.cat([g * u * s * (1 + g * (1 - s)), g * g * s], -1))
    assert float(dg[:-1].abs().max()) == 0.0


# ------------------------------------------------------------------ 4-bit weights

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def fp4_weights(shape, g, low=126, high=128):
    """Random codes and scale bytes (low to high), and the weights in 64 bits."""
    E, N, K = shape
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(low, high + 1, (E, N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return w, s


def fp4_ref(w, s):
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    codes = torch.stack([w & 15, w >> 4], -1).flatten(-2).long()
    return table[codes] * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


MX = [  # counts, N, K, slack rows at the end
    ([1], 8, 32, 0),
    ([1], 16, 96, 1),
    ([3], 48, 256, 2),
    ([0, 1, 127, 129, 0], 136, 416, 7),
    ([128, 256, 5], 264, 64, 0),
    ([31, 33, 64, 65], 512, 1024, 3),
    ([1, 1, 0, 1, 1, 0, 1], 1024, 512, 0),
    ([5, 0, 2, 8, 1], 520, 736, 0),
    ([700], 640, 384, 0),
    ([257, 0, 513], 256, 7168, 1),
    ([1], 4096, 2048, 0),
    ([4], 4096, 7168, 0),
    ([40] * 90, 520, 224, 0),
    ([2, 0, 3, 1, 9] * 30, 392, 256, 0),   # one piece of the reduction, several units a block
    ([3, 1, 6, 2] * 20, 1160, 736, 5),     # three pieces, several units a block
    ([1, 2, 3] * 9, 4104, 2048, 0),
    ([285], 264, 544, 0),
    ([300, 0, 270, 288, 577, 100], 520, 736, 1),
    ([256, 257, 288, 289] * 12, 776, 352, 0),
    ([900, 650], 264, 352, 0),
]


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("counts,N,K,slack", MX)
def test_mxfp4(counts, N, K, slack, exact):
    g = gen(41)
    E, rows = len(counts), sum(counts) + slack
    a = values((rows, K), g, exact)
    w, s = fp4_weights((E, N, K), g) if exact else fp4_weights((E, N, K), g, 110, 140)
    ref = fp4_ref(w, s)
    err, buf = zeros(1, torch.int32), Guarded((rows, N), BF)
    B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a, w, s, offsets(counts), buf.t, err))
    torch.cuda.synchronize()
    assert int(err) == 0 and buf.intact()
    lo = 0
    for e, n in enumerate(counts):
        x, we = a[lo:lo + n].double(), ref[e].t()
        y, got = x @ we, buf.t[lo:lo + n].double()
        if exact:
            assert torch.equal(got, rounded(y))
        else:
            tol = 2.0 ** -8 * y.abs() + K * 2 * U * (x.abs() @ we.abs())
            assert float(((got - y).abs() - tol).max() if n else 0.0) <= 0.0
        lo += n
    assert bool((buf.t[lo:] == 7.0).all())


@pytest.mark.parametrize("groups", [253, 256])  # scales that TMA cannot load, and can
@pytest.mark.parametrize("rows", [1, 5, 300])
def test_mxfp4_scales_of_any_size(rows, groups):
    """One term per output: the weight itself, through all codes and scales that leave it finite
    (6 * 2^125 is the largest), with a token that brings the product into range."""
    N, K = 16, 32 * groups
    w = torch.arange(16, dtype=torch.uint8, device=DEV)  # channel n: code n everywhere
    w = (w | (w << 4))[:, None].expand(N, K // 2).contiguous()[None]
    s = torch.arange(groups, device=DEV).clamp(max=252).to(torch.uint8)
    s = s[None].expand(N, groups).contiguous()[None]
    err = zeros(1, torch.int32)
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    for scale in (0, 1, 3, 60, 126, 127, 128, 129, 130, 200, 251, 252):
        for factor in (2.0 ** (100 if scale < 127 else -100), 1.0):
            a, out = zeros((rows, K), BF), zeros((rows, N), BF)
            a[:, scale * 32 + 7] = factor
            B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, w, s, None, out, err))
            torch.cuda.synchronize()
            want = rounded(table * 2.0 ** (scale - 127) * factor)[None].expand(rows, N)
            assert torch.equal(out.double(), want), (scale, factor)
    a = torch.full((rows, K), 2.0 ** -100, dtype=BF, device=DEV)
    out = zeros((rows, N), BF)
    s[0, 3, 17] = 255   # of channel 3 alone
    s[0, 7, 100] = 254  # 6 * 2^127, of channel 7 alone
    B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, w, s, None, out, err))
    torch.cuda.synchronize()
    assert bool(out[:, 3].isnan().all()) and int(out.isnan().sum()) == rows
    assert bool((out[:, 7] == math.inf).all()) and int(out.isinf().sum()) == rows
    assert int(err) == 0


def test_mxfp4_of_the_librarys_own_quantiser():
    """Weights as the quantising all-gather leaves them with one rank."""
    g = gen(42)
    E, N, K, counts = 3, 136, 256, [4, 0, 70]
    full = torch.randn((E, N, K), generator=g, device=DEV).to(BF)
    w, s = zeros((E, N, K // 2), torch.uint8), zeros((E, N, K // 32), torch.uint8)
    B.check(B.mp_allgatherv_mxfp4(1, K, [E * N], full, w, s))
    a, err = values((74, K), g, False), zeros(1, torch.int32)
    out = zeros((74, N), BF)
    B.check(B.mp_expert_matmul_mxfp4(E, 74, N, K, a, w, s, offsets(counts), out, err))
    torch.cuda.synchronize()
    ref = fp4_ref(w, s)
    # e2m1 rounds by at most a quarter of a value of its block's size
    assert float((ref - full.double()).norm() / full.double().norm()) < 0.25
    for sl, e in ((slice(0, 4), 0), (slice(4, 74), 2)):
        y, size = a[sl].double() @ ref[e].t(), a[sl].double().abs() @ ref[e].abs().t()
        assert bool(((out[sl].double() - y).abs() <= 2.0 ** -8 * y.abs() + K * 2 * U * size).all())
    assert int(err) == 0


@pytest.mark.parametrize("rows,shift", [(2, 1), (2, 8), (140, 1), (140, 4)])
def test_mxfp4_alignments_infinities_and_bad_offsets(rows, shift):
    """Scales at any address; infinity and NaN stay in their row; offsets out of order."""
    g = gen(43)
    N, K, E = 264, 512, 2
    w, s0 = fp4_weights((E, N, K), g)
    flat = zeros(s0.numel() + shift, torch.uint8)
    flat[shift:] = s0.flatten()
    s = flat[shift:].view(s0.shape)
    a, err = values((rows, K), g, True), zeros(1, torch.int32)
    ref = fp4_ref(w, s)
    half = rows // 2
    off = offsets([half, rows - half])
    clean, dirty = Guarded((rows, N), BF), Guarded((rows, N), BF)
    B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a, w, s, off, clean.t, err))
    a2 = a.clone()
    a2[half - 1, 3], a2[half, 4] = math.nan, math.inf
    B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a2, w, s, off, dirty.t, err))
    torch.cuda.synchronize()
    y = torch.cat([a[:half].double() @ ref[0].t(), a[half:].double() @ ref[1].t()])
    assert torch.equal(clean.t.double(), rounded(y)) and int(err) == 0
    assert bool(dirty.t[half - 1].isnan().all()) and not bool(dirty.t[half].isfinite().any())
    keep = [r for r in range(rows) if r not in (half - 1, half)]
    assert torch.equal(clean.t[keep], dirty.t[keep])
    for o, bits in (([0, half, rows + 30], B.MP_ERR_CAPACITY), ([0, rows, half], B.MP_ERR_INVALID_ARG),
                    ([-1, half, rows], B.MP_ERR_INVALID_ARG)):
        out, e2 = Guarded((rows, N), BF), zeros(1, torch.int32)
        o = torch.tensor(o, dtype=torch.int32, device=DEV)
        B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a, w, s, o, out.t, e2))
        torch.cuda.synchronize()
        assert int(e2) & bits and out.intact()
        want = rounded(y) if bits == B.MP_ERR_CAPACITY else torch.full_like(y, 7.0)
        assert torch.equal(out.t.double(), want)


def test_mxfp4_many_experts_far_offsets_and_a_graph():
    g = gen(44)
    err = zeros(1, torch.int32)
    E, N, K = 8192, 16, 96
    counts = np.zeros(E, np.int64)
    counts[[3, 4000, 8191]] = [2, 1, 130]
    rows = int(counts.sum())
    a = values((rows, K), g, True)
    w, s = fp4_weights((E, N, K), g)
    out = zeros((rows, N), BF)
    B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a, w, s, offsets(counts), out, err))
    expert = torch.from_numpy(np.repeat(np.arange(E), counts)).to(DEV)
    y = torch.einsum("rk,rnk->rn", a.double(), fp4_ref(w[expert], s[expert]))
    torch.cuda.synchronize()
    assert torch.equal(out.double(), rounded(y))
    E, N, K = 1200, 2048, 2048  # 5e9 codes in 2.5e9 bytes
    w, s = zeros((E, N, K // 2), torch.uint8), zeros((E, N, K // 32), torch.uint8) + 127
    w[-1], s[-1] = (t[0] for t in fp4_weights((1, N, K), g))
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[-1] = 3
    for rows in (3, 3000):  # the rows that there is room for choose the form
        room, out = values((rows, K), g, True), zeros((rows, N), BF)

        def call():
            B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, room, w, s, off, out, err))
        call()
        torch.cuda.synchronize()
        first = out.clone()
        assert torch.equal(out[:3].double(), rounded(room[:3].double() @ fp4_ref(w[-1], s[-1]).t()))
        assert float(out[3:].abs().max() if rows > 3 else 0.0) == 0.0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)
    assert int(err) == 0


@pytest.mark.parametrize("rows", [3, 200])
def test_mxfp4_rows_of_any_size(rows):
    """Values of a row far apart: each group of 32 channels has its own largest, from 2^-133 to
    2^127, and one term of it counts (the others' codes are 0), so that nothing is rounded away."""
    N, groups = 24, 256
    K = 32 * groups
    g = gen(45)
    w = torch.zeros((1, N, K), dtype=torch.uint8, device=DEV)
    pick = torch.randint(0, 32, (groups,), generator=g, device=DEV)
    at = torch.arange(groups, device=DEV) * 32 + pick
    s = torch.full((1, N, groups), 127, dtype=torch.uint8, device=DEV)
    packed = None
    for group in (0, 1, 130, 255):
        # channel n reads group `group` alone, with code n & 7 and the sign of n >= 8
        w.zero_()
        w[0, :, at[group]] = (torch.arange(N, device=DEV) % 16).to(torch.uint8)
        packed = (w[..., 0::2] | (w[..., 1::2] << 4)).contiguous()
        a = zeros((rows, K), BF)
        a[:, at] = torch.exp2(torch.arange(groups, device=DEV).double() - 133).clamp(
            max=2.0 ** 120).to(BF) * 1.0
        a[1::2] *= -1
        out, err = zeros((rows, N), BF), zeros(1, torch.int32)
        B.check(B.mp_expert_matmul_mxfp4(1, rows, N, K, a, packed, s, None, out, err))
        torch.cuda.synchronize()
        want = a.double() @ fp4_ref(packed, s)[0].t()
        assert torch.equal(out.double(), rounded(want)), group
        assert int(err) == 0


# ------------------------------------------------------------------ many sizes

@pytest.mark.parametrize("seed", range(40))
def test_random_problems(seed):
    """Sizes drawn over the forms that the launchers choose among (rows, split reductions, tiles of
    each size), whole numbers throughout: bit-equal."""
    r = np.random.default_rng(1000 + seed)
    E = int(r.choice([1, 1, 2, 3, 5, 8, 20, 64]))
    rows = int(np.exp(r.uniform(0, np.log(3000))))
    N, K = 8 * int(np.exp(r.uniform(0, np.log(160)))), 32 * int(np.exp(r.uniform(0, np.log(50))))
    p = r.dirichlet(np.full(E, r.choice([0.2, 1.0, 20.0])))
    counts = r.multinomial(rows, p)
    g = gen(seed)
    a, dy, w = values((rows, K), g, True), values((rows, N), g, True), values((E, N, K), g, True)
    codes, s = fp4_weights((E, N, K), g)
    ref = fp4_ref(codes, s)
    off, err = offsets(counts), zeros(1, torch.int32)
    y, y4, dx = Guarded((rows, N), BF), Guarded((rows, N), BF), Guarded((rows, K), BF)
    dw, dw32 = Guarded((E, N, K), BF), Guarded((E, N, K), torch.float32)
    B.check(B.mp_expert_matmul_bf16(E, rows, N, K, a, w, off, y.t, err))
    B.check(B.mp_expert_matmul_mxfp4(E, rows, N, K, a, codes, s, off, y4.t, err))
    B.check(B.mp_expert_matmul_dgrad_bf16(E, rows, N, K, dy, w, off, dx.t, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, dy, a, off, False, dw.t, err))
    B.check(B.mp_expert_matmul_wgrad_bf16(E, rows, N, K, dy, a, off, True, dw32.t, err))
    torch.cuda.synchronize()
    assert int(err) == 0 and all(b.intact() for b in (y, y4, dx, dw, dw32))
    lo = 0
    for e, n in enumerate(counts):
        x, d = a[lo:lo + n].double(), dy[lo:lo + n].double()
        assert torch.equal(y.t[lo:lo + n].double(), rounded(x @ w[e].double().t()))
        assert torch.equal(y4.t[lo:lo + n].double(), rounded(x @ ref[e].t()))
        assert torch.equal(dx.t[lo:lo + n].double(), rounded(d @ w[e].double()))
        assert torch.equal(dw.t[e].double(), rounded(d.t() @ x))
        assert torch.equal(dw32.t[e].double(), d.t() @ x + 7.0)
        lo += n


def test_first_calls_in_a_capture():
    """A process whose first calls are captured (limits are raised and asked for there)."""
    import subprocess
    import sys
    code = """
import torch
from combine_mp_layout_gb300 import binding as B
dev = dict(device="cuda")
E, N, K = 2, 64, 512
off = {n: torch.tensor([0, n // 2, n], dtype=torch.int32, **dev) for n in (2, 60, 600)}
a = {n: torch.ones((n, K), dtype=torch.bfloat16, **dev) for n in off}
w = torch.ones((E, N, K), dtype=torch.bfloat16, **dev)
w4 = torch.full((E, N, K // 2), 0x22, dtype=torch.uint8, **dev)
s = torch.full((E, N, K // 32), 127, dtype=torch.uint8, **dev)
out = {(n, k): torch.zeros((n, N), dtype=torch.bfloat16, **dev) for n in off for k in (0, 1)}
dw, err = torch.zeros((E, N, K), **dev), torch.zeros(1, dtype=torch.int32, **dev)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for n in off:
        B.check(B.mp_expert_matmul_bf16(E, n, N, K, a[n], w, off[n], out[n, 0], err))
        B.check(B.mp_expert_matmul_mxfp4(E, n, N, K, a[n], w4, s, off[n], out[n, 1], err))
    B.check(B.mp_expert_matmul_wgrad_bf16(E, 60, N, K, out[60, 0], a[60], off[60], False, dw, err))
graph.replay()
torch.cuda.synchronize()
assert int(err) == 0 and all(bool((t == K).all()) for t in out.values())
assert bool((dw == 30 * K).all())
print("fine")
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "fine" in done.stdout, done.stderr[-2000:]
