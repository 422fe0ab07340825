"""The operators on bf16 rows without a GPU: host-side refusals (every call below fails a host
check, so nothing is launched)."""
import ctypes

import pytest
import torch

from combine_mp_layout_gb300 import _build, binding as B

FAKE = 0x10000  # never dereferenced

no_gpu = pytest.mark.skipif(
    torch.cuda.is_available(),
    reason="fake-pointer argument checks run only on a host without a visible GPU")


def _p(v=FAKE):
    return ctypes.c_void_p(v)


@pytest.fixture(scope="module")
def L():
    _build.build()
    return B.lib()


MM = dict(E=2, rows=8, N=64, K=64, a=_p(), w=_p(), off=_p(), out=_p(), err=_p(), dtype=0, add=0)
BAD = [
    dict(E=0), dict(E=8193), dict(rows=-1), dict(rows=2 ** 31 - 1024), dict(N=0), dict(N=12),
    dict(K=0), dict(K=60), dict(N=2 ** 31 - 1016), dict(K=2 ** 31 - 1016),
    dict(N=2 ** 20, K=2 ** 19), dict(E=8192, N=2 ** 26, K=2 ** 11, rows=0),
    dict(E=8192, N=2 ** 11, K=2 ** 26, rows=0), dict(a=_p(0)), dict(w=_p(0)), dict(off=_p(0)),
    dict(out=_p(0)), dict(err=_p(0)), dict(a=_p(FAKE + 8)), dict(w=_p(FAKE + 4)),
    dict(out=_p(FAKE + 8)), dict(off=_p(FAKE + 1)), dict(err=_p(FAKE + 2)),
]


@no_gpu
@pytest.mark.parametrize("bad", BAD)
def test_matmul_rejects(L, bad):
    a = dict(MM, **bad)
    for call, tiles in (("mp_expert_matmul_bf16", a["N"]), ("mp_expert_matmul_dgrad_bf16", a["K"])):
        if a["E"] == 8192 and tiles < 2 ** 20:
            continue  # (this side's tiles are few enough)
        assert getattr(L, call)(a["E"], a["rows"], a["N"], a["K"], a["a"], a["w"], a["off"],
                                a["out"], a["err"], _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("bad", BAD + [
    dict(dtype=1), dict(dtype=3), dict(dtype=-1), dict(add=1), dict(rows=0, out=_p(0)),
    dict(E=8192, N=2 ** 17, K=2 ** 17, rows=0)])
def test_wgrad_rejects(L, bad):
    a = dict(MM, **bad)
    assert L.mp_expert_matmul_wgrad_bf16(a["E"], a["rows"], a["N"], a["K"], a["a"], a["w"],
                                         a["off"], a["dtype"], a["add"], a["out"], a["err"],
                                         _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("bad", BAD[:-11] + BAD[-9:] + [
    dict(K=48), dict(K=72), dict(s=_p(0)), dict(rows=2 ** 31 - 1025, N=160 * 256)])
def test_mxfp4_rejects(L, bad):
    a = dict(MM, s=_p(FAKE + 1), **bad) if "s" not in bad else dict(MM, **bad)
    assert L.mp_expert_matmul_mxfp4(a["E"], a["rows"], a["N"], a["K"], a["a"], a["w"], a["s"],
                                    a["off"], a["out"], a["err"], _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(I=0), dict(I=4), dict(I=20), dict(I=2 ** 31 - 4088), dict(x=_p(0)),
    dict(out=_p(0)), dict(x=_p(FAKE + 8)), dict(out=_p(FAKE + 8)), dict(w=_p(FAKE + 2)),
    dict(num=_p(FAKE + 1)), dict(d=_p(0)), dict(d=_p(FAKE + 2)), dict(dw=_p(FAKE + 2))])
def test_swiglu_rejects(L, bad):
    a = dict(rows=4, I=64, x=_p(), w=_p(0), num=_p(0), out=_p(), d=_p(), dw=_p(0))
    a.update(bad)
    if "d" not in bad and "dw" not in bad:
        assert L.mp_swiglu_bf16(a["rows"], a["I"], a["x"], a["w"], a["num"], a["out"],
                                _p(0)) == B.MP_ERR_INVALID_ARG
    assert L.mp_swiglu_backward_bf16(a["rows"], a["I"], a["x"], a["w"], a["d"], a["num"], a["out"],
                                     a["dw"], _p(0)) == B.MP_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors_and_other_types(L):
    t = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        B.mp_swiglu_bf16(1, 8, t, None, None, t)
    with pytest.raises(TypeError):
        B.mp_expert_matmul_bf16(1, 1, 8, 8, t, t, None, t, t)
    with pytest.raises(TypeError):
        B.mp_expert_matmul_wgrad_bf16(1, 1, 8, 8, t, t, None, False, t.half(), t)
