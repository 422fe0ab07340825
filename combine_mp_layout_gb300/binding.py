"""Thin ctypes binding of ``libmp_layout.so`` (the C ABI in include/mp_layout.h).

Argument marshalling only: every function takes torch CUDA tensors (device
memory), passes their device pointers and the current CUDA stream to the C
entry point of the same name and returns its status.  Every step of the path
runs in the library's CUDA kernels; there is no CPU fallback, and a missing
library or a CPU tensor raises at once.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import _build

MP_OK = 0
MP_ERR_INVALID_ARG = 1
MP_ERR_CUDA = 2
MP_ERR_CAPACITY = 4
MP_ERR_BAD_EXPERT = 8
MP_ERR_TIMEOUT = 16
MP_ERR_BAD_VALUE = 32
MP_BF16 = 0
MP_E4M3 = 1
MP_FP32 = 2
# score functions of the router
MP_SOFTMAX = 0
MP_SIGMOID = 1
SCALE_BLOCK = 128
# formats of the low-latency dispatch's in-kernel quantisation
MP_Q_E4M3 = 0
MP_Q_MXFP8 = 1
MP_Q_MXFP4 = 2

_lib = None


class MPError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s: status %d (%s)" % (what or "mp_layout", status,
                                                 mp_status_string(status)))


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise RuntimeError("libmp_layout.so is not built (run __graft_entry__.build() or "
                               "python -m combine_mp_layout_gb300._build): the CUDA path is "
                               "required, there is no fallback")
        L = ctypes.CDLL(_build.LIB)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.mp_status_string.argtypes = [i32]
        L.mp_status_string.restype = ctypes.c_char_p
        L.mp_workspace_size.argtypes = [i32, i32, i32]
        L.mp_workspace_size.restype = ctypes.c_size_t
        L.mp_layout.argtypes = [i32, i32, i32, i32, P, P, P, P, P, P, P]
        L.mp_dispatch.argtypes = [i32, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, i64,
                                  P, P, P, P, P, P, P, P, P, P, P, P, P]
        L.mp_dispatch_offsets.argtypes = [i32, i32, i32, i32, P, P, P, P, P, i64,
                                          P, P, P, P, P, P, P, P, P, P, P]
        L.mp_dispatch_rows.argtypes = [i32, i32, i32, i32, P, P, P, i64, P, P, P]
        L.mp_dispatch_rows_e4m3.argtypes = [i32, i32, i32, P, P, i64, P, P, P]
        L.mp_dispatch_rows_mxfp8.argtypes = [i32, i32, i32, P, P, i64, P, P, P]
        L.mp_dispatch_offsets_global.argtypes = [i32, i32, i32, i32, P, P, P, P, P, i64,
                                                 ctypes.c_int32, P, P, P, P, P, P, P, P, P, P, P]
        L.mp_combine_weights.argtypes = [i32, i32, i32, P, i64, P, P, P, P]
        L.mp_dispatch_ll_offsets.argtypes = [i32, i32, i32, i32, P, P, i64, P, P, P, P, P, P]
        L.mp_dispatch_ll_offsets_rank_major.argtypes = L.mp_dispatch_ll_offsets.argtypes
        L.mp_dispatch_ll_rows.argtypes = [i32, i32, i32, i32, i32, P, P, P, i64, P, P, P]
        L.mp_combine_ll.argtypes = [i32, i32, i32, i32, P, i64, P, P, P, P, P]
        L.mp_combine.argtypes = [i32, i32, i32, P, i64, P, P, P, P]
        L.mp_reducescatterv.argtypes = [i32, i32, P, P, P, P]
        L.mp_allgatherv.argtypes = [i32, i64, P, P, P, P]
        L.mp_allgatherv_e4m3.argtypes = [i32, i32, P, P, P, P, P]
        L.mp_allgatherv_mxfp8.argtypes = [i32, i32, P, P, P, P, P]
        L.mp_allgatherv_mxfp4.argtypes = [i32, i32, P, P, P, P, P]
        L.mp_dispatch_rows_mxfp4.argtypes = [i32, i32, i32, P, P, i64, P, P, P]
        L.mp_dispatch_rows_bulk.argtypes = [i32, i32, i32, i32, P, P, P, i64, P, P, P, P]
        L.mp_layout_and_offsets.argtypes = [i32, i32, i32, i32, P, P, i64] + [P] * 14
        L.mp_dispatch_noalloc.argtypes = [i32] * 6 + [P] * 7 + [i64] + [P] * 12
        L.mp_layout_dispatch.argtypes = [i32] * 6 + [P] * 4 + [i64] + [P] * 16
        L.mp_dispatch_ll_rows_quant.argtypes = [i32] * 5 + [P, P, i64, P, P, P]
        L.mp_dispatch_ll_quant.argtypes = [i32] * 7 + [P] * 3 + [i64] + [P] * 8
        L.mp_allgatherv_multi.argtypes = [i32, i32, P, P, P, P, P]
        f32 = ctypes.c_float
        L.mp_route_workspace_size.argtypes = [i32, i32, i32]
        L.mp_route_workspace_size.restype = ctypes.c_size_t
        L.mp_route.argtypes = [i32] * 6 + [P] * 3 + [i32, f32, f32] + [P] * 8
        L.mp_route_backward.argtypes = [i32] * 6 + [P] * 2 + [i32, f32, f32] + [P] * 7
        L.mp_expert_matmul_e4m3.argtypes = [i32] * 4 + [P] * 8
        L.mp_expert_matmul_dgrad_e4m3.argtypes = [i32] * 4 + [P] * 8
        L.mp_expert_matmul_wgrad_e4m3.argtypes = [i32] * 4 + [P] * 8
        L.mp_swiglu_e4m3.argtypes = [i32] * 2 + [P] * 6
        L.mp_swiglu_backward_e4m3.argtypes = [i32] * 2 + [P] * 8
        L.mp_ll_row_weights.argtypes = [i32] * 3 + [P, P, i64, P, P]
        L.mp_ll_row_weights_backward.argtypes = [i32] * 3 + [P, i64, P, P, P]
        L.mp_dispatch_ll.argtypes = [i32] * 7 + [P] * 4 + [i64] + [P] * 8
        for f in ("mp_layout", "mp_dispatch", "mp_dispatch_offsets", "mp_dispatch_rows",
                  "mp_dispatch_rows_e4m3", "mp_dispatch_rows_mxfp8", "mp_dispatch_offsets_global",
                  "mp_combine_weights",
                  "mp_dispatch_ll_offsets", "mp_dispatch_ll_offsets_rank_major",
                  "mp_dispatch_ll_rows", "mp_combine_ll",
                  "mp_combine", "mp_reducescatterv", "mp_allgatherv",
                  "mp_allgatherv_e4m3", "mp_allgatherv_mxfp8", "mp_allgatherv_mxfp4",
                  "mp_dispatch_rows_mxfp4", "mp_dispatch_rows_bulk",
                  "mp_layout_and_offsets", "mp_dispatch_noalloc", "mp_allgatherv_multi",
                  "mp_dispatch_ll", "mp_layout_dispatch", "mp_dispatch_ll_rows_quant",
                  "mp_dispatch_ll_quant", "mp_route", "mp_route_backward",
                  "mp_expert_matmul_e4m3", "mp_expert_matmul_dgrad_e4m3",
                  "mp_expert_matmul_wgrad_e4m3", "mp_swiglu_e4m3", "mp_swiglu_backward_e4m3",
                  "mp_ll_row_weights", "mp_ll_row_weights_backward"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _dev(t: torch.Tensor | None, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor (the library runs on the GPU only)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def check(status: int, what: str = "") -> int:
    if status != MP_OK:
        raise MPError(status, what)
    return status


def mp_status_string(status: int) -> str:
    return lib().mp_status_string(status).decode()


def mp_workspace_size(R: int, N: int, E: int) -> int:
    return int(lib().mp_workspace_size(R, N, E))


def mp_layout(R, N, K, E, topk_idx, num_tokens_per_rank, num_tokens_per_expert,
              is_token_in_rank, dev_err, workspace, stream=None) -> int:
    return lib().mp_layout(R, N, K, E, _dev(topk_idx, "topk_idx"),
                           _dev(num_tokens_per_rank, "num_tokens_per_rank"),
                           _dev(num_tokens_per_expert, "num_tokens_per_expert"),
                           _dev(is_token_in_rank, "is_token_in_rank"),
                           _dev(dev_err, "dev_err"), _dev(workspace, "workspace"),
                           _stream(stream))


def mp_dispatch(R, N, K, E, H, dtype, x, x_scales, topk_idx, topk_weights, is_token_in_rank,
                num_tokens_per_rank, num_tokens_per_expert, recv_capacity, recv_x,
                recv_scales, recv_src_rank, recv_src_idx, recv_topk_idx, recv_topk_weights,
                dest_offsets, rank_prefix, num_recv_tokens_per_expert, send_row, dev_err,
                workspace, stream=None) -> int:
    return lib().mp_dispatch(
        R, N, K, E, H, dtype, _dev(x, "x"), _dev(x_scales, "x_scales"),
        _dev(topk_idx, "topk_idx"), _dev(topk_weights, "topk_weights"),
        _dev(is_token_in_rank, "is_token_in_rank"),
        _dev(num_tokens_per_rank, "num_tokens_per_rank"),
        _dev(num_tokens_per_expert, "num_tokens_per_expert"), int(recv_capacity),
        _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"),
        _dev(recv_src_rank, "recv_src_rank"), _dev(recv_src_idx, "recv_src_idx"),
        _dev(recv_topk_idx, "recv_topk_idx"), _dev(recv_topk_weights, "recv_topk_weights"),
        _dev(dest_offsets, "dest_offsets"), _dev(rank_prefix, "rank_prefix"),
        _dev(num_recv_tokens_per_expert, "num_recv_tokens_per_expert"),
        _dev(send_row, "send_row"), _dev(dev_err, "dev_err"), _dev(workspace, "workspace"),
        _stream(stream))


def mp_dispatch_offsets(R, N, K, E, topk_idx, topk_weights, is_token_in_rank,
                        num_tokens_per_rank, num_tokens_per_expert, recv_capacity,
                        recv_src_rank, recv_src_idx, recv_topk_idx, recv_topk_weights,
                        dest_offsets, rank_prefix, num_recv_tokens_per_expert, send_row, dev_err,
                        workspace, stream=None) -> int:
    return lib().mp_dispatch_offsets(
        R, N, K, E, _dev(topk_idx, "topk_idx"), _dev(topk_weights, "topk_weights"),
        _dev(is_token_in_rank, "is_token_in_rank"),
        _dev(num_tokens_per_rank, "num_tokens_per_rank"),
        _dev(num_tokens_per_expert, "num_tokens_per_expert"), int(recv_capacity),
        _dev(recv_src_rank, "recv_src_rank"), _dev(recv_src_idx, "recv_src_idx"),
        _dev(recv_topk_idx, "recv_topk_idx"), _dev(recv_topk_weights, "recv_topk_weights"),
        _dev(dest_offsets, "dest_offsets"), _dev(rank_prefix, "rank_prefix"),
        _dev(num_recv_tokens_per_expert, "num_recv_tokens_per_expert"),
        _dev(send_row, "send_row"), _dev(dev_err, "dev_err"), _dev(workspace, "workspace"),
        _stream(stream))


def mp_dispatch_rows(R, N, H, dtype, x, x_scales, send_row, recv_capacity, recv_x, recv_scales,
                     stream=None) -> int:
    return lib().mp_dispatch_rows(R, N, H, dtype, _dev(x, "x"), _dev(x_scales, "x_scales"),
                                  _dev(send_row, "send_row"), int(recv_capacity),
                                  _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"),
                                  _stream(stream))


def mp_layout_and_offsets(R, N, K, E, topk_idx, topk_weights, recv_capacity,
                          num_tokens_per_rank, num_tokens_per_expert, is_token_in_rank,
                          recv_src_rank, recv_src_idx, recv_topk_idx, recv_topk_weights,
                          dest_offsets, rank_prefix, num_recv_tokens_per_expert, send_row,
                          dev_err, workspace, stream=None) -> int:
    return lib().mp_layout_and_offsets(
        R, N, K, E, _dev(topk_idx, "topk_idx"), _dev(topk_weights, "topk_weights"),
        int(recv_capacity), _dev(num_tokens_per_rank, "num_tokens_per_rank"),
        _dev(num_tokens_per_expert, "num_tokens_per_expert"),
        _dev(is_token_in_rank, "is_token_in_rank"), _dev(recv_src_rank, "recv_src_rank"),
        _dev(recv_src_idx, "recv_src_idx"), _dev(recv_topk_idx, "recv_topk_idx"),
        _dev(recv_topk_weights, "recv_topk_weights"), _dev(dest_offsets, "dest_offsets"),
        _dev(rank_prefix, "rank_prefix"),
        _dev(num_recv_tokens_per_expert, "num_recv_tokens_per_expert"),
        _dev(send_row, "send_row"), _dev(dev_err, "dev_err"), _dev(workspace, "workspace"),
        _stream(stream))


def mp_layout_dispatch(R, N, K, E, H, dtype, x, x_scales, topk_idx, topk_weights, recv_capacity,
                       num_tokens_per_rank, num_tokens_per_expert, is_token_in_rank, recv_x,
                       recv_scales, recv_src_rank, recv_src_idx, recv_topk_idx, recv_topk_weights,
                       dest_offsets, rank_prefix, num_recv_tokens_per_expert, send_row, dev_err,
                       workspace, stream=None) -> int:
    return lib().mp_layout_dispatch(
        R, N, K, E, H, dtype, _dev(x, "x"), _dev(x_scales, "x_scales"),
        _dev(topk_idx, "topk_idx"), _dev(topk_weights, "topk_weights"), int(recv_capacity),
        _dev(num_tokens_per_rank, "num_tokens_per_rank"),
        _dev(num_tokens_per_expert, "num_tokens_per_expert"),
        _dev(is_token_in_rank, "is_token_in_rank"), _dev(recv_x, "recv_x"),
        _dev(recv_scales, "recv_scales"), _dev(recv_src_rank, "recv_src_rank"),
        _dev(recv_src_idx, "recv_src_idx"), _dev(recv_topk_idx, "recv_topk_idx"),
        _dev(recv_topk_weights, "recv_topk_weights"), _dev(dest_offsets, "dest_offsets"),
        _dev(rank_prefix, "rank_prefix"),
        _dev(num_recv_tokens_per_expert, "num_recv_tokens_per_expert"),
        _dev(send_row, "send_row"), _dev(dev_err, "dev_err"), _dev(workspace, "workspace"),
        _stream(stream))


def mp_dispatch_offsets_global(R, N, K, E, topk_idx, topk_weights, is_token_in_rank,
                               num_tokens_per_rank, num_tokens_per_expert, recv_capacity, sentinel,
                               recv_src_rank, recv_src_idx, recv_topk_idx, recv_topk_weights,
                               dest_offsets, rank_prefix, num_recv_tokens_per_expert, send_row,
                               dev_err, workspace, stream=None) -> int:
    return lib().mp_dispatch_offsets_global(
        R, N, K, E, _dev(topk_idx, "topk_idx"), _dev(topk_weights, "topk_weights"),
        _dev(is_token_in_rank, "is_token_in_rank"),
        _dev(num_tokens_per_rank, "num_tokens_per_rank"),
        _dev(num_tokens_per_expert, "num_tokens_per_expert"), int(recv_capacity), int(sentinel),
        _dev(recv_src_rank, "recv_src_rank"), _dev(recv_src_idx, "recv_src_idx"),
        _dev(recv_topk_idx, "recv_topk_idx"), _dev(recv_topk_weights, "recv_topk_weights"),
        _dev(dest_offsets, "dest_offsets"), _dev(rank_prefix, "rank_prefix"),
        _dev(num_recv_tokens_per_expert, "num_recv_tokens_per_expert"),
        _dev(send_row, "send_row"), _dev(dev_err, "dev_err"), _dev(workspace, "workspace"),
        _stream(stream))


def mp_combine_weights(R, N, K, recv_topk_weights, recv_rows, send_row, combined, dev_err,
                       stream=None) -> int:
    return lib().mp_combine_weights(R, N, K, _dev(recv_topk_weights, "recv_topk_weights"),
                                    int(recv_rows), _dev(send_row, "send_row"),
                                    _dev(combined, "combined_topk_weights"),
                                    _dev(dev_err, "dev_err"), _stream(stream))


def mp_dispatch_rows_bulk(R, N, H, dtype, x, x_scales, send_row, recv_capacity, recv_x,
                          recv_scales, dev_err, stream=None) -> int:
    return lib().mp_dispatch_rows_bulk(R, N, H, dtype, _dev(x, "x"), _dev(x_scales, "x_scales"),
                                       _dev(send_row, "send_row"), int(recv_capacity),
                                       _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"),
                                       _dev(dev_err, "dev_err"), _stream(stream))


def mp_dispatch_rows_e4m3(R, N, H, x, send_row, recv_capacity, recv_x, recv_scales,
                          stream=None) -> int:
    return lib().mp_dispatch_rows_e4m3(R, N, H, _dev(x, "x"), _dev(send_row, "send_row"),
                                       int(recv_capacity), _dev(recv_x, "recv_x"),
                                       _dev(recv_scales, "recv_scales"), _stream(stream))


def mp_dispatch_rows_mxfp8(R, N, H, x, send_row, recv_capacity, recv_x, recv_scales,
                           stream=None) -> int:
    return lib().mp_dispatch_rows_mxfp8(R, N, H, _dev(x, "x"), _dev(send_row, "send_row"),
                                        int(recv_capacity), _dev(recv_x, "recv_x"),
                                        _dev(recv_scales, "recv_scales"), _stream(stream))


def mp_dispatch_rows_mxfp4(R, N, H, x, send_row, recv_capacity, recv_x, recv_scales,
                           stream=None) -> int:
    return lib().mp_dispatch_rows_mxfp4(R, N, H, _dev(x, "x"), _dev(send_row, "send_row"),
                                        int(recv_capacity), _dev(recv_x, "recv_x"),
                                        _dev(recv_scales, "recv_scales"), _stream(stream))


def mp_combine(R, N, H, y, y_rows, send_row, out, dev_err, stream=None) -> int:
    return lib().mp_combine(R, N, H, _dev(y, "y"), int(y_rows), _dev(send_row, "send_row"),
                            _dev(out, "out"), _dev(dev_err, "dev_err"), _stream(stream))


def _host_sizes(sizes):
    arr = (ctypes.c_int64 * len(sizes))(*[int(s) for s in sizes])
    return arr


def mp_reducescatterv(R, H, sizes, inp, out, stream=None) -> int:
    return lib().mp_reducescatterv(R, H, _host_sizes(sizes), _dev(inp, "in"), _dev(out, "out"),
                                   _stream(stream))


def mp_allgatherv(R, row_bytes, sizes, inp, out, stream=None) -> int:
    return lib().mp_allgatherv(R, int(row_bytes), _host_sizes(sizes), _dev(inp, "in"),
                               _dev(out, "out"), _stream(stream))


def mp_allgatherv_e4m3(R, H, sizes, inp, out, out_scales, stream=None) -> int:
    return lib().mp_allgatherv_e4m3(R, H, _host_sizes(sizes), _dev(inp, "in"), _dev(out, "out"),
                                    _dev(out_scales, "out_scales"), _stream(stream))


def mp_allgatherv_mxfp8(R, H, sizes, inp, out, out_scales, stream=None) -> int:
    return lib().mp_allgatherv_mxfp8(R, H, _host_sizes(sizes), _dev(inp, "in"), _dev(out, "out"),
                                     _dev(out_scales, "out_scales"), _stream(stream))


def mp_allgatherv_mxfp4(R, H, sizes, inp, out, out_scales, stream=None) -> int:
    return lib().mp_allgatherv_mxfp4(R, H, _host_sizes(sizes), _dev(inp, "in"), _dev(out, "out"),
                                     _dev(out_scales, "out_scales"), _stream(stream))


def mp_dispatch_noalloc(R, N, K, E, H, dtype, x, x_scales, topk_idx, topk_weights,
                        is_token_in_rank, num_tokens_per_rank, num_tokens_per_expert,
                        recv_capacity, recv_x, recv_scales, recv_src_rank, recv_src_idx,
                        recv_topk_idx, recv_topk_weights, dest_offsets, rank_prefix,
                        num_recv_tokens_per_expert, send_row, dev_err, stream=None) -> int:
    """mp_dispatch without a workspace, for callers that cannot allocate device memory
    (the scan's scratch is a fixed array inside the library; see the C header)."""
    f = lib().mp_dispatch_noalloc
    return f(R, N, K, E, H, dtype, _dev(x, "x"), _dev(x_scales, "x_scales"),
             _dev(topk_idx, "topk_idx"), _dev(topk_weights, "topk_weights"),
             _dev(is_token_in_rank, "is_token_in_rank"),
             _dev(num_tokens_per_rank, "num_tokens_per_rank"),
             _dev(num_tokens_per_expert, "num_tokens_per_expert"), int(recv_capacity),
             _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"),
             _dev(recv_src_rank, "recv_src_rank"), _dev(recv_src_idx, "recv_src_idx"),
             _dev(recv_topk_idx, "recv_topk_idx"), _dev(recv_topk_weights, "recv_topk_weights"),
             _dev(dest_offsets, "dest_offsets"), _dev(rank_prefix, "rank_prefix"),
             _dev(num_recv_tokens_per_expert, "num_recv_tokens_per_expert"),
             _dev(send_row, "send_row"), _dev(dev_err, "dev_err"), _stream(stream))


def mp_allgatherv_multi(R, row_bytes, sizes, inputs, outputs, stream=None) -> int:
    """All-gatherv of several tensors with the same per-rank row counts, one launch."""
    f = lib().mp_allgatherv_multi
    n = len(inputs)
    if len(outputs) != n or len(row_bytes) != n:
        raise ValueError("one row size and one output per input")
    rb = (ctypes.c_int64 * n)(*[int(b) for b in row_bytes])
    ins = (ctypes.c_void_p * n)(*[_dev(t, "in").value for t in inputs])
    outs = (ctypes.c_void_p * n)(*[_dev(t, "out").value for t in outputs])
    return f(R, n, rb, _host_sizes(sizes), ins, outs, _stream(stream))


def mp_dispatch_ll_offsets(R, N, K, E, topk_idx, num_tokens_per_expert, recv_capacity,
                           expert_offsets, expert_src_offsets, recv_src_token, slot_row, dev_err,
                           stream=None) -> int:
    return lib().mp_dispatch_ll_offsets(
        R, N, K, E, _dev(topk_idx, "topk_idx"), _dev(num_tokens_per_expert, "num_tokens_per_expert"),
        int(recv_capacity), _dev(expert_offsets, "expert_offsets"),
        _dev(expert_src_offsets, "expert_src_offsets"), _dev(recv_src_token, "recv_src_token"),
        _dev(slot_row, "slot_row"), _dev(dev_err, "dev_err"), _stream(stream))


def mp_dispatch_ll_offsets_rank_major(R, N, K, E, topk_idx, num_tokens_per_expert,
                                      recv_capacity, dest_offsets, dest_src_offsets,
                                      recv_src_token, slot_row, dev_err, stream=None) -> int:
    return lib().mp_dispatch_ll_offsets_rank_major(
        R, N, K, E, _dev(topk_idx, "topk_idx"), _dev(num_tokens_per_expert, "num_tokens_per_expert"),
        int(recv_capacity), _dev(dest_offsets, "dest_offsets"),
        _dev(dest_src_offsets, "dest_src_offsets"), _dev(recv_src_token, "recv_src_token"),
        _dev(slot_row, "slot_row"), _dev(dev_err, "dev_err"), _stream(stream))


def mp_dispatch_ll_rows(R, N, K, H, dtype, x, x_scales, slot_row, recv_capacity, recv_x,
                        recv_scales, stream=None) -> int:
    return lib().mp_dispatch_ll_rows(R, N, K, H, dtype, _dev(x, "x"), _dev(x_scales, "x_scales"),
                                     _dev(slot_row, "slot_row"), int(recv_capacity),
                                     _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"),
                                     _stream(stream))


def mp_dispatch_ll(R, N, K, E, H, dtype, rank_major, x, x_scales, topk_idx,
                   num_tokens_per_expert, recv_capacity, bin_offsets, bin_src_offsets,
                   recv_src_token, slot_row, recv_x, recv_scales, dev_err,
                   stream=None) -> int:
    return lib().mp_dispatch_ll(
        R, N, K, E, H, dtype, int(rank_major), _dev(x, "x"), _dev(x_scales, "x_scales"),
        _dev(topk_idx, "topk_idx"), _dev(num_tokens_per_expert, "num_tokens_per_expert"),
        int(recv_capacity), _dev(bin_offsets, "bin_offsets"),
        _dev(bin_src_offsets, "bin_src_offsets"), _dev(recv_src_token, "recv_src_token"),
        _dev(slot_row, "slot_row"), _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"),
        _dev(dev_err, "dev_err"), _stream(stream))


def mp_combine_ll(R, N, K, H, y, y_rows, slot_row, topk_weights, out, dev_err, stream=None) -> int:
    return lib().mp_combine_ll(R, N, K, H, _dev(y, "y"), int(y_rows), _dev(slot_row, "slot_row"),
                               _dev(topk_weights, "topk_weights"), _dev(out, "out"),
                               _dev(dev_err, "dev_err"), _stream(stream))


def mp_dispatch_ll_rows_quant(R, N, K, H, qformat, x, slot_row, recv_capacity, recv_x,
                              recv_scales, stream=None) -> int:
    """LL row copy with the quantisation in the kernel (qformat MP_Q_E4M3 / _MXFP8 /
    _MXFP4): bf16 token rows in, codes and scales at every slot row."""
    return lib().mp_dispatch_ll_rows_quant(R, N, K, H, int(qformat), _dev(x, "x"),
                                           _dev(slot_row, "slot_row"), int(recv_capacity),
                                           _dev(recv_x, "recv_x"),
                                           _dev(recv_scales, "recv_scales"), _stream(stream))


def mp_dispatch_ll_quant(R, N, K, E, H, qformat, rank_major, x, topk_idx, num_tokens_per_expert,
                         recv_capacity, bin_offsets, bin_src_offsets, recv_src_token, slot_row,
                         recv_x, recv_scales, dev_err, stream=None) -> int:
    """mp_dispatch_ll with the quantisation in the row copy."""
    return lib().mp_dispatch_ll_quant(
        R, N, K, E, H, int(qformat), int(rank_major), _dev(x, "x"), _dev(topk_idx, "topk_idx"),
        _dev(num_tokens_per_expert, "num_tokens_per_expert"), int(recv_capacity),
        _dev(bin_offsets, "bin_offsets"), _dev(bin_src_offsets, "bin_src_offsets"),
        _dev(recv_src_token, "recv_src_token"), _dev(slot_row, "slot_row"),
        _dev(recv_x, "recv_x"), _dev(recv_scales, "recv_scales"), _dev(dev_err, "dev_err"),
        _stream(stream))


def _arr(t, name, dtype, numel):
    """The device address of a dense CUDA tensor of this type with room for `numel` elements."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() < numel:
        _dev(t, name)
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
        raise ValueError("%s holds %d elements, %d are needed" % (name, t.numel(), numel))
    return t.data_ptr()


def _raw_stream(stream):
    """The stream's handle; the current device's current one costs no stream object."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


@functools.lru_cache(maxsize=None)
def mp_route_workspace_size(R: int, N: int, E: int) -> int:
    return int(lib().mp_route_workspace_size(R, N, E))


def _logits(t, name, numel):
    if t is not None and t.dtype is torch.bfloat16:
        return MP_BF16, _arr(t, name, torch.bfloat16, numel)
    return MP_FP32, _arr(t, name, torch.float32, numel)


def mp_route(R, N, K, E, scoring, logits, bias, active, normalize, scale, loss_coef, topk_idx,
             topk_weights, num_tokens_per_expert, num_routed, balance_loss, dev_err, workspace,
             stream=None) -> int:
    """The router: top-K experts, weights, per-expert counts and balance loss of the fp32 or
    bf16 logits [R][N][E] (see the C header)."""
    dtype, lp = _logits(logits, "logits", R * N * E)
    return lib().mp_route(
        R, N, K, E, int(scoring), dtype, lp, _arr(bias, "bias", torch.float32, E),
        _arr(active, "active", torch.uint8, R * N), int(bool(normalize)), float(scale),
        float(loss_coef), _arr(topk_idx, "topk_idx", torch.int32, R * N * K),
        _arr(topk_weights, "topk_weights", torch.float32, R * N * K),
        _arr(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, R * E),
        _arr(num_routed, "num_routed", torch.int32, R),
        _arr(balance_loss, "balance_loss", torch.float32, R),
        _arr(dev_err, "dev_err", torch.int32, 1),
        _arr(workspace, "workspace", torch.uint8, mp_route_workspace_size(R, N, E)),
        _raw_stream(stream))


def mp_route_backward(R, N, K, E, scoring, logits, active, normalize, scale, loss_coef, topk_idx,
                      d_topk_weights, num_tokens_per_expert, num_routed, d_balance_loss, d_logits,
                      stream=None) -> int:
    """The gradient of mp_route's weights and loss with respect to the logits."""
    dtype, lp = _logits(logits, "logits", R * N * E)
    return lib().mp_route_backward(
        R, N, K, E, int(scoring), dtype, lp, _arr(active, "active", torch.uint8, R * N),
        int(bool(normalize)), float(scale), float(loss_coef),
        _arr(topk_idx, "topk_idx", torch.int32, R * N * K),
        _arr(d_topk_weights, "d_topk_weights", torch.float32, R * N * K),
        _arr(num_tokens_per_expert, "num_tokens_per_expert", torch.int32, R * E),
        _arr(num_routed, "num_routed", torch.int32, R),
        _arr(d_balance_loss, "d_balance_loss", torch.float32, R),
        _arr(d_logits, "d_logits", torch.bfloat16 if dtype == MP_BF16 else torch.float32,
             R * N * E), _raw_stream(stream))


_F8 = torch.float8_e4m3fn


def mp_expert_matmul_e4m3(E, rows, N, K, a, a_scales, w, w_scales, expert_offsets, out, dev_err,
                          stream=None) -> int:
    """out[r] = a[r] w[e]^T for the rows of every expert: e4m3 with one fp32 scale per 128
    channels of a row and per 128 x 128 block of a weight, bf16 out."""
    return lib().mp_expert_matmul_e4m3(
        E, rows, N, K, _arr(a, "a", _F8, rows * K),
        _arr(a_scales, "a_scales", torch.float32, rows * (K // SCALE_BLOCK)),
        _arr(w, "w", _F8, E * N * K),
        _arr(w_scales, "w_scales", torch.float32, E * -(-N // SCALE_BLOCK) * (K // SCALE_BLOCK)),
        _arr(expert_offsets, "expert_offsets", torch.int32, E + 1),
        _arr(out, "out", torch.bfloat16, rows * N), _arr(dev_err, "dev_err", torch.int32, 1),
        _raw_stream(stream))


def mp_expert_matmul_dgrad_e4m3(E, rows, N, K, dy, dy_scales, w, w_scales, expert_offsets, dx,
                                dev_err, stream=None) -> int:
    """dx[r] = dy[r] w[e]: the gradient of the rows, with the weights as they are stored."""
    return lib().mp_expert_matmul_dgrad_e4m3(
        E, rows, N, K, _arr(dy, "dy", _F8, rows * N),
        _arr(dy_scales, "dy_scales", torch.float32, rows * (N // SCALE_BLOCK)),
        _arr(w, "w", _F8, E * N * K),
        _arr(w_scales, "w_scales", torch.float32, E * -(-N // SCALE_BLOCK) * (K // SCALE_BLOCK)),
        _arr(expert_offsets, "expert_offsets", torch.int32, E + 1),
        _arr(dx, "dx", torch.bfloat16, rows * K), _arr(dev_err, "dev_err", torch.int32, 1),
        _raw_stream(stream))


def mp_expert_matmul_wgrad_e4m3(E, rows, N, K, dy, dy_scales, a, a_scales, expert_offsets, dw,
                                dev_err, stream=None) -> int:
    """dw[e] = dy^T a over the rows of every expert, bf16 (zeros for an expert without rows)."""
    return lib().mp_expert_matmul_wgrad_e4m3(
        E, rows, N, K, _arr(dy, "dy", _F8, rows * N),
        _arr(dy_scales, "dy_scales", torch.float32, rows * (N // SCALE_BLOCK)),
        _arr(a, "a", _F8, rows * K),
        _arr(a_scales, "a_scales", torch.float32, rows * (K // SCALE_BLOCK)),
        _arr(expert_offsets, "expert_offsets", torch.int32, E + 1),
        _arr(dw, "dw", torch.bfloat16, E * N * K), _arr(dev_err, "dev_err", torch.int32, 1),
        _raw_stream(stream))


def mp_swiglu_e4m3(rows, I, gate_up, row_weights, num_rows, out, out_scales, stream=None) -> int:
    """row_weights * silu(gate) * up of bf16 [rows][2I], quantised to e4m3 with one fp32 scale
    per 128 channels."""
    return lib().mp_swiglu_e4m3(
        rows, I, _arr(gate_up, "gate_up", torch.bfloat16, rows * 2 * I),
        _arr(row_weights, "row_weights", torch.float32, rows),
        _arr(num_rows, "num_rows", torch.int32, 1), _arr(out, "out", _F8, rows * I),
        _arr(out_scales, "out_scales", torch.float32, rows * (I // SCALE_BLOCK)),
        _raw_stream(stream))


def mp_swiglu_backward_e4m3(rows, I, gate_up, row_weights, d_out, num_rows, d_gate_up,
                            d_gate_up_scales, d_row_weights, stream=None) -> int:
    """The gradient of mp_swiglu_e4m3: d_gate_up quantised the same way, d_row_weights fp32."""
    return lib().mp_swiglu_backward_e4m3(
        rows, I, _arr(gate_up, "gate_up", torch.bfloat16, rows * 2 * I),
        _arr(row_weights, "row_weights", torch.float32, rows),
        _arr(d_out, "d_out", torch.bfloat16, rows * I), _arr(num_rows, "num_rows", torch.int32, 1),
        _arr(d_gate_up, "d_gate_up", _F8, rows * 2 * I),
        _arr(d_gate_up_scales, "d_gate_up_scales", torch.float32, rows * (2 * I // SCALE_BLOCK)),
        _arr(d_row_weights, "d_row_weights", torch.float32, rows), _raw_stream(stream))


def mp_ll_row_weights(R, N, K, topk_weights, slot_row, recv_capacity, row_weights,
                      stream=None) -> int:
    """Routing weights of the low-latency slots at their receive rows."""
    return lib().mp_ll_row_weights(
        R, N, K, _arr(topk_weights, "topk_weights", torch.float32, R * N * K),
        _arr(slot_row, "slot_row", torch.int32, R * N * K), int(recv_capacity),
        _arr(row_weights, "row_weights", torch.float32, int(recv_capacity)),
        _raw_stream(stream))


def mp_ll_row_weights_backward(R, N, K, d_row_weights, rows, slot_row, d_topk_weights,
                               stream=None) -> int:
    """Gradients of the rows' weights back at their slots."""
    return lib().mp_ll_row_weights_backward(
        R, N, K, _arr(d_row_weights, "d_row_weights", torch.float32, int(rows)), int(rows),
        _arr(slot_row, "slot_row", torch.int32, R * N * K),
        _arr(d_topk_weights, "d_topk_weights", torch.float32, R * N * K), _raw_stream(stream))
