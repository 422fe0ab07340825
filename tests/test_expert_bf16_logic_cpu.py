"""Logic of the operators on bf16 rows that can be followed without a GPU, taken from their
source, and refusals."""
import re

import pytest
import torch

from combine_mp_layout_gb300 import binding as B
from tests.test_expert_bf16_cpu import BAD, L, MM, _p, no_gpu  # noqa: F401 (L: a fixture)
from tests.test_expert_kernel_logic_cpu import run_c, source


def bf16(bits):
    return (torch.tensor(bits, dtype=torch.int64) << 16).to(torch.int32).view(torch.float32).double()


def returned(text, name):
    """What a one-line function returns."""
    return re.search(r"uint32_t %s\(uint32_t s\) \{\s*return ([^;]*);" % name, text).group(1)


def test_mxfp4_scales_of_both_conversions(tmp_path):
    """The multipliers of the tiles' weights, as their source computes them: codes are held as
    2^-126 of their value, so those for scales up to 128 are 2^126 * 2^(s - 127), and the careful
    conversion's, which can meet any scale, 2^126 and then 2^(s - 127)."""
    text = source("mp_expert_matmul_mxfp4.cu")
    out = run_c(tmp_path, """
  for (uint32_t s = 0; s < 256; ++s)
    std::printf("%%u %%u\\n", uint32_t(%s), uint32_t(%s));""" % (
        returned(text, "multiplier"), returned(text, "large_multiplier")))
    plain, careful = zip(*(map(int, line.split()) for line in out.split("\n") if line))
    first = int(re.search(r"LARGE \? (0x[0-9a-f]+)u : multiplier", text).group(1), 16)
    for v in plain[:129] + careful + (first,):
        assert v >> 16 == v & 0xffff  # both channels of a pair alike
    exact = [2.0 ** (s - 127) for s in range(255)]
    assert bf16([v & 0xffff for v in plain[:129]]).tolist() == [v * 2.0 ** 126 for v in exact[:129]]
    assert float(bf16([first & 0xffff])[0]) == 2.0 ** 126
    assert bf16([v & 0xffff for v in careful[:255]]).tolist() == exact
    assert bool(bf16([careful[255] & 0xffff]).isnan().all())


@no_gpu
@pytest.mark.parametrize("bad", [b for b in BAD if b.get("K") != 2 ** 26])
def test_mxfp4_rejects_all_that_the_products_do(L, bad):
    """Every refusal of the bf16 product (but of as many column tiles as only its gradient has),
    rows that are missing among them."""
    a = dict(MM, **bad)
    assert L.mp_expert_matmul_mxfp4(a["E"], a["rows"], a["N"], a["K"], a["a"], a["w"], _p(),
                                    a["off"], a["out"], a["err"], _p(0)) == B.MP_ERR_INVALID_ARG
