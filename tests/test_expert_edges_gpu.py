"""The expert layer's operators at the edges of what they accept, against 64-bit forms."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from combine_mp_layout_gb300 import binding as B
from tests.test_expert_ops_gpu import DEV, codes, gen, offsets, rows_ref, scales, zeros

pytestmark = pytest.mark.gpu


def wgrad(counts, dy, sd, a, sa):
    E, (rows, N), K = len(counts), dy.shape, a.shape[1]
    dw, err = zeros((E, N, K), torch.bfloat16), zeros(1, torch.int32)
    B.check(B.mp_expert_matmul_wgrad_e4m3(E, rows, N, K, dy, sd, a, sa, offsets(counts), dw, err))
    torch.cuda.synchronize()
    assert int(err) == 0
    return dw


def wgrad_ref(counts, dy, sd, a, sa):
    dd, ad = rows_ref(dy, sd), rows_ref(a, sa)
    ends = np.cumsum(counts)
    return torch.stack([dd[e - n:e].t() @ ad[e - n:e] for n, e in zip(counts, ends)])


def test_wgrad_many_tiles_of_one_stage():
    """Experts of at most 64 rows, many tiles per pair of blocks: the two groups of converting
    warps take every other tile.  Whole codes and power-of-two scales: exact sums."""
    g = gen(51)
    counts = [int(n) for n in np.random.default_rng(51).integers(0, 65, 400)]
    rows, N, K = sum(counts), 256, 512
    dy, sd = codes((rows, N), g, True), scales((rows, N // 128), g, True)
    a, sa = codes((rows, K), g, True), scales((rows, K // 128), g, True)
    want = wgrad_ref(counts, dy, sd, a, sa).float().bfloat16()
    for _ in range(3):
        assert torch.equal(wgrad(counts, dy, sd, a, sa), want)


def wgrad_tolerance(counts, dy, sd, a, sa, want):
    """Both factors in f16 with a relative error of at most 2^-10, fp32 sums, one rounding to
    bf16 (as in test_wgrad of the operators' tests)."""
    size = wgrad_ref(counts, dy.float().abs(), sd, a.float().abs(), sa)
    n = torch.tensor(counts, device=DEV, dtype=torch.float64)[:, None, None]
    return (2.0 ** -9 + 2.0 ** -18 + n * 2 * 2.0 ** -24) * size + 2.0 ** -8 * want.abs()


@pytest.mark.parametrize("N,K", [(256, 384), (512, 1024)])  # scales by loads, and by TMA
@pytest.mark.parametrize("dy_exp,a_exp", [(-28, 0), (-45, 3), (0, -30), (-60, -40), (20, 0)])
@pytest.mark.parametrize("share", [0.02, 0.6])
def test_wgrad_blocks_of_zeros_cost_the_others_nothing(N, K, dy_exp, a_exp, share):
    """Quantisers give a block of zeros scale 1, whatever the scales beside it are; a row of a
    token without a gradient (padding, a masked loss) is all such blocks.  The other rows' scales
    here lie within 2^5 of one another, so their factors keep their relative error."""
    g = gen(52)
    counts = [300, 0, 40, 1, 700, 33]
    rows = sum(counts)
    dy, sd = codes((rows, N), g, False), scales((rows, N // 128), g, False) * 2.0 ** dy_exp
    a, sa = codes((rows, K), g, False), scales((rows, K // 128), g, False) * 2.0 ** a_exp

    def clear(c, s):  # a share of the blocks, at least one per column, -0 codes among them
        z = torch.rand(s.shape, generator=g, device=DEV) < share
        z[7] = True
        z[301] = z[310:330] = True
        c = c.float().view(rows, -1, 128)
        sign = torch.randint(0, 2, c.shape, generator=g, device=DEV) * -0.0
        return (torch.where(z[..., None], sign, c).view(rows, -1).to(torch.float8_e4m3fn),
                torch.where(z, 1.0, s))
    dy, sd = clear(dy, sd)
    a, sa = clear(a, sa)
    want = wgrad_ref(counts, dy, sd, a, sa)
    got = wgrad(counts, dy, sd, a, sa).double()
    assert bool(((got - want).abs() <= wgrad_tolerance(counts, dy, sd, a, sa, want)).all())


def test_wgrad_all_zero_rows_and_scales_without_bound():
    """Blocks of zeros only, with the largest finite scale and with scale 0."""
    N, K, rows = 256, 256, 80
    zero = zeros((rows, N), torch.float8_e4m3fn)
    one = torch.full((rows, K), 1.5, device=DEV).to(torch.float8_e4m3fn)
    for s in (0.0, 1e-30, 1.0, torch.finfo(torch.float32).max):
        sd = torch.full((rows, 2), s, device=DEV)
        assert float(wgrad([rows], zero, sd, one, torch.ones_like(sd)).abs().max()) == 0.0
    sd[3], dy = 2.0 ** -120, zero.clone()
    dy[3] = 2.0
    got = wgrad([rows], dy, sd, one, torch.ones_like(sd))
    assert bool((got == 3.0 * 2.0 ** -120).all())


def test_wgrad_infinite_and_nan_scales_stay_in_their_channel_block():
    g = gen(53)
    counts, N, K = [90, 70], 512, 512
    rows = sum(counts)
    dy, sd = codes((rows, N), g, True), scales((rows, N // 128), g, True) * 2.0 ** -40
    a, sa = codes((rows, K), g, True), scales((rows, K // 128), g, True)
    dy[5], sd[5] = 0.0, 1.0
    dy[120], sd[120] = 0.0, 1.0
    clean = wgrad(counts, dy, sd, a, sa)
    sd[11, 1], sa[20, 2], sd[130, 3] = torch.inf, torch.nan, -torch.inf
    got = wgrad(counts, dy, sd, a, sa)
    hit = torch.zeros((2, N, K), dtype=torch.bool, device=DEV)
    hit[0, 128:256] = hit[0, :, 256:384] = hit[1, 384:] = True
    assert not bool(got[hit].isfinite().any())
    assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("dy_exp,a_exp", [(120, -120), (-120, 120), (100, -90), (-124, 60),
                                          (60, -124), (126, -126)])
def test_wgrad_products_of_far_scales(dy_exp, a_exp):
    """Scales whose products are ordinary numbers, each one near an end of fp32's range: small
    whole codes, so every sum is exact."""
    g = gen(54)
    counts, N, K = [70, 33], 256, 256
    rows = sum(counts)
    dy, a = codes((rows, N), g, True), codes((rows, K), g, True)
    sd = torch.full((rows, 2), 2.0 ** dy_exp, device=DEV)
    sa = torch.full((rows, 2), 2.0 ** a_exp, device=DEV)
    want = wgrad_ref(counts, dy, sd, a, sa).float().bfloat16()
    assert torch.equal(wgrad(counts, dy, sd, a, sa), want)


@pytest.mark.parametrize("rows,dy_exp", [(400_000_000, 0), (60_000_000, -30)])
def test_wgrad_of_one_expert_with_very_many_rows(rows, dy_exp):
    """Seconds of work in one tile: no wait for it gives up.  All rows are zeros but for three
    (scale 1 for the others: with small scales beside it each row's codes have to be looked at)."""
    need = rows * 2 * (128 + 4) + (2 << 30)
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs %d GB of free device memory" % (need >> 30))
    g = gen(55)
    at = torch.tensor([0, rows // 3, rows - 1], device=DEV)
    dy, a = (torch.zeros((rows, 128), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
             for _ in range(2))
    sd, sa = (torch.ones((rows, 1), device=DEV) for _ in range(2))
    few = [codes((3, 128), g, True), codes((3, 128), g, True)]
    dy.view(torch.uint8)[at], a.view(torch.uint8)[at] = (t.view(torch.uint8) for t in few)
    sd[at] = 2.0 ** dy_exp
    got = wgrad([rows], dy, sd, a, sa)[0]
    want = (few[0].double() * 2.0 ** dy_exp).t() @ few[1].double()
    assert torch.equal(got, want.float().bfloat16())


def test_wgrad_small_codes_at_small_scales():
    """A factor is off by at most 2^-10 of its value (two roundings of 2^-11, and 2^-22 for
    their product), 2^-30 of the largest scale for its product, and as much times the code
    where the scale is below 2^-19 of the largest: both only below f16's normal range.  Each
    expert has one row that sets the largest scale (its other factor is zero) and one to look at."""
    U11 = 2.0 ** -11
    code = torch.tensor([2.0 ** -9, 2.0 ** -6, 9 * 2.0 ** -9, 0.125, 1.0, 1.875, 13.0, 448.0],
                        device=DEV)
    ratio = [1.99, 1.37, 1.0, 0.7] + [f * 2.0 ** -k for k in (9, 10, 14, 18, 19, 22, 27, 31)
                                      for f in (1.0, 1.1, 1.37, 1.93)]
    E, N, K = len(ratio), 128, 128
    dy = torch.zeros((E, 2, N), device=DEV)
    dy[:, 0, 5] = 448.0
    dy[:, 1] = code.repeat(N // 8)
    s = torch.ones((E, 2, 1), device=DEV)
    s[:, 1, 0] = torch.tensor(ratio, device=DEV)
    a = torch.zeros((E, 2, K), device=DEV)
    a[:, 1] = 1.0
    f8 = torch.float8_e4m3fn
    got = wgrad([2] * E, dy.view(-1, N).to(f8), s.view(-1, 1), a.view(-1, K).to(f8),
                torch.ones((2 * E, 1), device=DEV)).double()
    scale, c = s[:, 1].double(), dy[:, 1].to(f8).double()
    top = s.double().amax(1)
    want = scale * c
    err = want * (2 * U11 + U11 * U11)
    err = torch.where(scale * c < 2.0 ** -18 * top, err + 2.0 ** -30 * top, err)
    err = torch.where(scale < 2.0 ** -18 * top, err + 2.0 ** -30 * top * c * (1 + U11), err)
    # one term, so the sum is exact, and rounding to bf16 keeps the order
    low, high = ((want + d).float().bfloat16().double()[..., None] for d in (-err, err))
    assert bool(((low <= got) & (got <= high)).all())


@pytest.mark.parametrize("kind", ["fwd", "dgrad"])
@pytest.mark.parametrize("rows,N", [(64, 128), (8192, 512)])  # split reductions, whole tiles
def test_products_of_many_and_few_experts_from_two_threads(kind, rows, N):
    """The shared memory of a call grows with its experts; threads whose calls alternate do not
    take it from each other."""
    K = 2048
    err = zeros(1, torch.int32)
    f = B.mp_expert_matmul_e4m3 if kind == "fwd" else B.mp_expert_matmul_dgrad_e4m3
    src, dst = (K, N) if kind == "fwd" else (N, K)

    def prepared(E):
        g = gen(56)
        counts = np.zeros(E, np.int64)
        counts[[0, E - 1]] = [rows - 3, 3]
        a, sa = codes((rows, src), g, True), scales((rows, src // 128), g, True)
        w = torch.zeros((E, N, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        w[[0, E - 1]] = codes((2, N, K), g, True)
        sw = scales((E, N // 128, K // 128), g, True)
        ws = w[[0, E - 1]].double() * sw[[0, E - 1]].double().repeat_interleave(
            128, 1).repeat_interleave(128, 2)
        if kind == "fwd":
            ws = ws.transpose(1, 2)
        ad, off = rows_ref(a, sa), offsets(counts)
        want = torch.cat([ad[:-3] @ ws[0], ad[-3:] @ ws[1]]).float().bfloat16()
        torch.cuda.synchronize()

        def call():
            out = zeros((rows, dst), torch.bfloat16)
            status = f(E, rows, N, K, a, sa, w, sw, off, out, err)
            torch.cuda.synchronize()
            return status, torch.equal(out, want)
        return call
    many, few = prepared(4000), prepared(2)
    with ThreadPoolExecutor(1) as one, ThreadPoolExecutor(1) as other:
        for _ in range(3):
            assert one.submit(many).result() == (B.MP_OK, True)
            assert other.submit(few).result() == (B.MP_OK, True)
    assert int(err) == 0


def test_layouts_of_many_and_fewer_experts_from_two_threads():
    """The same for the layout kernels that the layer stands on: more than 48 KB of shared
    memory in both threads, more of it in one."""
    R, N, K = 2, 300, 32

    def prepared(E):
        g = gen(58)
        idx = torch.randint(0, E, (R, N, K), generator=g, device=DEV, dtype=torch.int32)
        want = torch.stack([torch.bincount(idx[r].flatten().long(), minlength=E) for r in range(R)])
        i32 = torch.int32
        per_rank, per_expert = zeros((R, R), i32), zeros((R, E), i32)
        mask, err = zeros((R, N), i32), zeros(1, i32)
        ws = zeros(B.mp_workspace_size(R, N, E), torch.uint8)
        off, src = zeros(E + 1, i32), zeros((E, R), i32)
        token, slot = zeros(R * N * K, i32), zeros((R, N, K), i32)
        torch.cuda.synchronize()

        def call():
            status = [B.mp_layout(R, N, K, E, idx, per_rank, per_expert, mask, err, ws),
                      B.mp_dispatch_ll_offsets(R, N, K, E, idx, per_expert, R * N * K, off, src,
                                               token, slot, err)]
            torch.cuda.synchronize()
            assert int(err) == 0 and torch.equal(per_expert.long(), want)
            assert torch.equal(off[1:].long(), want.sum(0).cumsum(0))
            return status
        return call
    for fewer in (4200, 6000):
        many, few = prepared(8192), prepared(fewer)
        with ThreadPoolExecutor(1) as one, ThreadPoolExecutor(1) as other:
            for _ in range(3):
                assert one.submit(many).result() == [B.MP_OK] * 2
                assert other.submit(few).result() == [B.MP_OK] * 2


def test_activation_scales_and_codes_are_as_near_as_stated():
    """With gates of 32 the sigmoid is 1 in fp32 and z = 32 u w is rounded once, so z is known:
    scales within one ulp (2^-23) of amax / 448, and each code that of a value within 1.5 ulp (at
    most 1.5 * 2^-23 of it) of z / scale."""
    g = gen(57)
    rows, I = 600, 512
    x = zeros((rows, 2 * I), torch.bfloat16)
    x[:, :I] = 32.0
    u = torch.randn((rows, I), generator=g, device=DEV).bfloat16()
    x[:, I:] = u
    w = torch.rand(rows, generator=g, device=DEV) * torch.exp2(
        torch.randint(-100, 100, (rows,), generator=g, device=DEV).float())
    f8 = torch.float8_e4m3fn
    out, sc = zeros((rows, I), f8), zeros((rows, I // 128))
    B.check(B.mp_swiglu_e4m3(rows, I, x, w, None, out, sc))
    z = ((u.float() * 32) * w[:, None]).double().view(rows, -1, 128)
    want = z.abs().amax(-1) / 448
    assert bool(((sc.double() - want).abs() <= 2.0 ** -23 * want).all())
    q = (z / sc.double()[..., None]).view(rows, I).abs()
    low, high = ((q * (1 + d * 1.5 * 2.0 ** -23)).clamp(max=448.0).float().to(f8).double()
                 for d in (-1, 1))
    got = out.double().abs()
    assert bool(((low <= got) & (got <= high)).all())
    assert bool((out.double().sign() * z.view(rows, I).sign() >= 0).all())
