"""The expert layer's operators at the edges of what they accept, against 64-bit forms."""
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
