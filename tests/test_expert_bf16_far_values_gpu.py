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
