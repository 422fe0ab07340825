"""The expert layer's entry points without a GPU: workspace sizing and host-side refusals
(every call below fails a host check, so nothing is launched)."""
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


def test_route_workspace_size(L):
    assert B.mp_route_workspace_size(8, 4096, 256) == 32 * 8 + 8 * 256 * 12
    assert B.mp_route_workspace_size(1, 0, 1) > 0
    assert B.mp_route_workspace_size(0, 1, 8) == 0
    assert B.mp_route_workspace_size(33, 1, 8) == 0
    assert B.mp_route_workspace_size(1, 1, 8193) == 0
    assert B.mp_route_workspace_size(1, -1, 8) == 0


def test_new_status_string(L):
    assert "logit" in B.mp_status_string(B.MP_ERR_BAD_VALUE)


ROUTE = dict(R=2, N=8, K=2, E=8, scoring=0, dtype=2, logits=_p(), bias=_p(0), active=_p(0), idx=_p(),
             w=_p(), counts=_p(), routed=_p(), loss=_p(), err=_p(), ws=_p())


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(R=0), dict(R=33), dict(N=-1), dict(K=0), dict(K=9), dict(K=33, E=64), dict(E=8193),
    dict(scoring=2), dict(dtype=1), dict(dtype=3), dict(bias=_p()), dict(logits=_p(0)),
    dict(logits=_p(FAKE + 2)), dict(scoring=1, bias=_p(FAKE + 2)), dict(idx=_p(0)), dict(w=_p(0)),
    dict(counts=_p(0)), dict(routed=_p(0)), dict(loss=_p(0)), dict(err=_p(0)), dict(ws=_p(0)),
    dict(ws=_p(FAKE + 8)), dict(R=32, N=2 ** 26, K=2, E=64),
])
def test_route_rejects(L, bad):
    a = dict(ROUTE, **bad)
    assert L.mp_route(a["R"], a["N"], a["K"], a["E"], a["scoring"], a["dtype"], a["logits"],
                      a["bias"], a["active"], 1, 1.0, 0.01, a["idx"], a["w"], a["counts"],
                      a["routed"], a["loss"], a["err"], a["ws"], _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(R=0), dict(K=9), dict(scoring=-1), dict(dtype=1), dict(logits=_p(0)), dict(idx=_p(0)),
    dict(counts=_p(0)), dict(routed=_p(0)), dict(dl=_p(0)), dict(dl=_p(FAKE + 2)),
    dict(dw=_p(FAKE + 1)), dict(dloss=_p(FAKE + 2)),
])
def test_route_backward_rejects(L, bad):
    a = dict(ROUTE, dl=_p(), dw=_p(0), dloss=_p(0), **{k: v for k, v in bad.items() if k in ROUTE})
    a.update(bad)
    assert L.mp_route_backward(a["R"], a["N"], a["K"], a["E"], a["scoring"], a["dtype"],
                               a["logits"], a["active"], 1, 1.0, 0.01, a["idx"], a["dw"],
                               a["counts"], a["routed"], a["dloss"], a["dl"],
                               _p(0)) == B.MP_ERR_INVALID_ARG


MM = dict(E=2, rows=8, N=128, K=128, a=_p(), sa=_p(), w=_p(), sw=_p(), off=_p(), out=_p(), err=_p())


@no_gpu
@pytest.mark.parametrize("call", ["mp_expert_matmul_e4m3", "mp_expert_matmul_dgrad_e4m3",
                                  "mp_expert_matmul_wgrad_e4m3"])
@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=8193), dict(rows=-1), dict(N=0), dict(N=24), dict(K=0), dict(K=64),
    dict(K=192), dict(E=8192, N=2 ** 19), dict(a=_p(0)), dict(sa=_p(0)), dict(w=_p(0)),
    dict(sw=_p(0)), dict(off=_p(0)), dict(out=_p(0)), dict(err=_p(0)), dict(a=_p(FAKE + 8)),
    dict(w=_p(FAKE + 4)), dict(out=_p(FAKE + 8)), dict(sa=_p(FAKE + 2)), dict(off=_p(FAKE + 1)),
])
def test_matmul_rejects(L, call, bad):
    a = dict(MM, **bad)
    assert getattr(L, call)(a["E"], a["rows"], a["N"], a["K"], a["a"], a["sa"], a["w"], a["sw"],
                            a["off"], a["out"], a["err"], _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
def test_gradient_products_reject_partial_blocks(L):
    """The gradients reduce over (or scale) the N axis in whole blocks of 128."""
    for call in (L.mp_expert_matmul_dgrad_e4m3, L.mp_expert_matmul_wgrad_e4m3):
        assert call(1, 8, 144, 128, _p(), _p(), _p(), _p(), _p(0), _p(), _p(),
                    _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(I=0), dict(I=64), dict(I=192), dict(x=_p(0)), dict(out=_p(0)),
    dict(sc=_p(0)), dict(x=_p(FAKE + 8)), dict(out=_p(FAKE + 8)), dict(sc=_p(FAKE + 2)),
    dict(w=_p(FAKE + 2)), dict(num=_p(FAKE + 1)), dict(d=_p(0)), dict(d=_p(FAKE + 2)),
    dict(dw=_p(FAKE + 2)),
])
def test_swiglu_rejects(L, bad):
    a = dict(rows=4, I=128, x=_p(), w=_p(0), num=_p(0), out=_p(), sc=_p(), d=_p(), dw=_p(0))
    a.update(bad)
    if "d" not in bad and "dw" not in bad:
        assert L.mp_swiglu_e4m3(a["rows"], a["I"], a["x"], a["w"], a["num"], a["out"], a["sc"],
                                _p(0)) == B.MP_ERR_INVALID_ARG
    assert L.mp_swiglu_backward_e4m3(a["rows"], a["I"], a["x"], a["w"], a["d"], a["num"], a["out"],
                                     a["sc"], a["dw"], _p(0)) == B.MP_ERR_INVALID_ARG


@no_gpu
@pytest.mark.parametrize("bad", [dict(R=0), dict(R=33), dict(N=-1), dict(K=0), dict(K=33),
                                 dict(cap=-1), dict(w=_p(0)), dict(slots=_p(0)), dict(rows=_p(0)),
                                 dict(w=_p(FAKE + 2)), dict(slots=_p(FAKE + 1)),
                                 dict(R=32, N=2 ** 25, K=2)])
def test_row_weights_reject(L, bad):
    a = dict(dict(R=2, N=8, K=2, cap=16, w=_p(), slots=_p(), rows=_p()), **bad)
    assert L.mp_ll_row_weights(a["R"], a["N"], a["K"], a["w"], a["slots"], a["cap"], a["rows"],
                               _p(0)) == B.MP_ERR_INVALID_ARG
    assert L.mp_ll_row_weights_backward(a["R"], a["N"], a["K"], a["rows"], a["cap"], a["slots"],
                                        a["w"], _p(0)) == B.MP_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors(L):
    t = torch.zeros(8)
    with pytest.raises(TypeError):
        B.mp_swiglu_e4m3(1, 128, t, None, None, t, t)
