"""Python binding of libmla_decode.so: MLA decode attention in the ETAP form on B200.

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  torch tensors provide device memory and the current stream.
The names mirror the C ABI in ``include/mla_decode.h``.
"""

from __future__ import annotations

import ctypes
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_decode.so")

D_QK = 576
D_V = 512
PAGE_SIZE = 64
FLAG_SKIP_COMBINE = 1
FLAG_TEST_EXPIRE_WAITS = 0x40000000

STATUS = {0: "MLA_OK", -1: "MLA_ERR_INVALID_ARG", -2: "MLA_ERR_UNSUPPORTED", -3: "MLA_ERR_ALIGNMENT",
          -4: "MLA_ERR_WORKSPACE", -5: "MLA_ERR_CUDA", -6: "MLA_ERR_TIMEOUT", -7: "MLA_ERR_BLOCK_TABLE",
          -8: "MLA_ERR_PAGES"}

EXPORTS = ("mla_decode_workspace_size", "mla_decode_plan", "mla_decode_fwd", "mla_combine",
           "mla_decode_read_status", "mla_decode_plan_host", "mla_status_string", "mla_last_cuda_error",
           "mla_decode_fwd_static_ws", "mla_decode_static_ws_status", "mla_decode_fwd_ragged", "mla_stream_probe", "mla_decode_fwd_fp8", "mla_form_ablation",
           "mla_decode_fwd_trace", "mla_decode_fwd_untransposed", "mla_decode_fwd_tree", "mla_decode_fwd_tree_fp8",
           "mla_cache_extend", "mla_cache_append", "mla_cache_append_fp8", "mla_cache_accept")
STATIC_WORKSPACE_BYTES = 16777216


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if it was not built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m mla_decode_attention_etap_b200.build` "
                              "(or __graft_entry__.build()) first; there is no non-CUDA fallback")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.mla_decode_workspace_size.argtypes = [i32, i32, i32, i32]
        L.mla_decode_workspace_size.restype = sz
        L.mla_decode_plan.argtypes = [vp, i32, i32, i32, i32, vp, sz, vp]
        L.mla_decode_plan.restype = i32
        L.mla_decode_fwd.argtypes = [vp, vp, vp, vp, i32, i32, i32, i64, i32, ctypes.c_float, i32, vp, vp, vp, sz,
                                     i32, ctypes.c_uint, vp]
        L.mla_decode_fwd.restype = i32
        L.mla_decode_fwd_ragged.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i64, i32, ctypes.c_float, i32, vp, vp,
                                            vp, sz, i32, ctypes.c_uint, vp]
        L.mla_decode_fwd_ragged.restype = i32
        L.mla_decode_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, i32, ctypes.c_float, i32, vp,
                                         vp, vp, sz, i32, ctypes.c_uint, vp]
        L.mla_decode_fwd_fp8.restype = i32
        L.mla_decode_fwd_untransposed.argtypes = [vp, vp, vp, vp, i32, i32, i32, i64, i32, ctypes.c_float, i32, vp,
                                                  vp, vp, sz, i32, ctypes.c_uint, vp]
        L.mla_decode_fwd_untransposed.restype = i32
        L.mla_combine.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
        L.mla_combine.restype = i32
        L.mla_decode_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_int), vp]
        L.mla_decode_read_status.restype = i32
        ip = ctypes.POINTER(ctypes.c_int)
        L.mla_decode_plan_host.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, ip, ip, ip, ip]
        L.mla_decode_plan_host.restype = i32
        L.mla_status_string.argtypes = [i32]
        L.mla_status_string.restype = ctypes.c_char_p
        L.mla_decode_fwd_static_ws.argtypes = [vp, vp, vp, vp, i32, i32, i32, i64, i32, ctypes.c_float, i32, vp,
                                               vp, i32, vp]
        L.mla_decode_fwd_static_ws.restype = i32
        L.mla_decode_static_ws_status.argtypes = [ctypes.POINTER(ctypes.c_int), vp]
        L.mla_decode_static_ws_status.restype = i32
        L.mla_form_ablation.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp]
        L.mla_form_ablation.restype = i32
        L.mla_decode_fwd_trace.argtypes = [vp, vp, vp, vp, i32, i32, i32, i64, i32, ctypes.c_float, i32, vp, vp, vp,
                                           sz, i32, vp, i32, vp]
        L.mla_decode_fwd_trace.restype = i32
        L.mla_stream_probe.argtypes = [vp, i64, i32, vp, vp]
        L.mla_stream_probe.restype = i32
        f32, u32 = ctypes.c_float, ctypes.c_uint
        L.mla_decode_fwd_tree.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, vp, sz, i32,
                                          u32, vp]
        L.mla_decode_fwd_tree.restype = i32
        L.mla_decode_fwd_tree_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i64, i32, f32, vp, vp, vp,
                                              sz, i32, u32, vp]
        L.mla_decode_fwd_tree_fp8.restype = i32
        L.mla_cache_extend.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, i64, vp, vp, vp, vp, vp, vp, vp]
        L.mla_cache_extend.restype = i32
        L.mla_cache_append.argtypes = [vp, i64, vp, f32, vp, i32, i32, vp, vp, i32, vp, i64, vp, i64, i64, i32, vp,
                                       vp, vp]
        L.mla_cache_append.restype = i32
        L.mla_cache_append_fp8.argtypes = [vp, i64, vp, f32, vp, i32, i32, vp, vp, i32, vp, vp, i64, vp, i64, i64,
                                           i32, vp, vp, vp]
        L.mla_cache_append_fp8.restype = i32
        L.mla_cache_accept.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp, i32, vp, i64, vp, vp, vp,
                                       vp]
        L.mla_cache_accept.restype = i32
        L.mla_last_cuda_error.argtypes = []
        L.mla_last_cuda_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(code: int, what: str):
    if code != 0:
        if code == -5:
            what = f"{what} ({lib().mla_last_cuda_error().decode()})"
        raise MlaError(code, what)


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, name: str, dtype, device, min_numel: int = 0, dim: Optional[int] = None,
             last: Optional[int] = None, min_rows: int = 0) -> None:
    """Reject a tensor whose raw pointer the library could not use safely: the C ABI sees only the
    pointer, so dtype, device, layout and size are checked here (TypeError / ValueError)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device} (all tensors on the device of q)")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name}: {t.dim()}-D, expected {dim}-D")
    if last is not None and (t.dim() == 0 or t.shape[-1] != last):
        raise ValueError(f"{name}: last dimension must be {last}, got shape {tuple(t.shape)}")
    if min_rows and (t.dim() == 0 or t.shape[0] < min_rows):
        raise ValueError(f"{name}: needs at least {min_rows} rows in dimension 0, got shape {tuple(t.shape)}")
    if t.numel() < min_numel:
        raise ValueError(f"{name}: {t.numel()} elements, needs at least {min_numel}")


def check_decode_args(q, kv, seqlens, block_table, o, lse, workspace, q_lens=None, kv_scale=None) -> None:
    """Shapes, dtypes and devices of a decode call (``kv_scale`` given: the FP8 cache, ``kv`` uint8)."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q: expected a torch.Tensor")
    dev = q.device
    _require(q, "q", torch.bfloat16, dev, dim=4, last=D_QK)
    B, q_len, h, _ = q.shape
    fp8 = kv_scale is not None
    _require(kv, "kv8" if fp8 else "kv", torch.uint8 if fp8 else torch.bfloat16, dev, dim=3, last=D_QK,
             min_rows=0 if block_table is not None else B)
    _require(seqlens, "seqlens", torch.int32, dev, min_numel=B, dim=1)
    if block_table is not None:
        _require(block_table, "block_table", torch.int32, dev, dim=2, min_rows=B)
    if q_lens is not None:
        _require(q_lens, "q_lens", torch.int32, dev, min_numel=B, dim=1)
    if fp8:
        _require(kv_scale, "kv_scale", torch.float32, dev, min_numel=kv.shape[0] * kv.shape[1])
    _require(o, "o", torch.bfloat16, dev, min_numel=B * q_len * h * D_V)
    _require(lse, "lse", torch.float32, dev, min_numel=B * q_len * h)
    _require(workspace, "workspace", None, dev)


def _require_cuda(t, name: str) -> None:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name}: must be a CUDA tensor")


def _raw_stream(index: int) -> int:
    """The device's current stream as an address, without building a Stream object (2 us a call)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _launch(device, stream, call, what: str) -> None:
    """``call(stream pointer)`` with ``device`` current, on ``stream`` or that device's current stream."""
    if stream is None:
        s = _raw_stream(device.index)
    elif getattr(stream, "device", device) != device:  # (a stream object may name no device)
        raise ValueError(f"{what}: stream on {stream.device}, tensors on {device}")
    else:
        s = stream.cuda_stream
    if device.index == torch._C._cuda_getDevice():
        code = call(s)
    else:
        with torch.cuda.device(device):
            code = call(s)
    if code != 0:
        _check(code, what)


def num_sms(device=None) -> int:
    return torch.cuda.get_device_properties(device if device is not None else torch.cuda.current_device()
                                            ).multi_processor_count


def mla_decode_workspace_size(batch: int, q_len: int, num_heads: int, n_sms: int) -> int:
    n = lib().mla_decode_workspace_size(batch, q_len, num_heads, n_sms)
    if n == 0:
        raise MlaError(-1, "mla_decode_workspace_size")
    return int(n)


def mla_decode_plan(seqlens: torch.Tensor, q_len: int, num_heads: int, workspace: torch.Tensor, n_sms: int,
                    stream=None) -> None:
    _require_cuda(seqlens, "seqlens")
    home = seqlens.device
    _require(seqlens, "seqlens", torch.int32, home, dim=1)
    _require(workspace, "workspace", None, home)
    a = (seqlens.data_ptr(), seqlens.numel(), q_len, num_heads, n_sms, workspace.data_ptr(), _nbytes(workspace))
    _launch(home, stream, lambda s: lib().mla_decode_plan(*a, s), "mla_decode_plan")


def mla_decode_fwd(q, kv, seqlens, block_table, softmax_scale, causal, o, lse, workspace, n_sms, flags=0,
                   stream=None, q_lens=None) -> None:
    """``q_lens`` (optional int32 device tensor [B]): ragged batch, q_lens[b] real query tokens of the
    q_len rows of sequence b (``mla_decode_fwd_ragged``)."""
    _require_cuda(q, "q")
    check_decode_args(q, kv, seqlens, block_table, o, lse, workspace, q_lens)
    B, q_len, h, _ = q.shape
    if block_table is not None:
        kv_rows, max_blocks = kv.shape[0] * kv.shape[1], block_table.shape[1]
    else:
        kv_rows, max_blocks = kv.shape[1], 0
    if q_lens is None:
        _launch(q.device, stream,
                lambda s: lib().mla_decode_fwd(_ptr(q), _ptr(kv), _ptr(seqlens), _ptr(block_table), B, q_len, h,
                                               kv_rows, max_blocks, float(softmax_scale), int(bool(causal)), _ptr(o),
                                               _ptr(lse), _ptr(workspace), _nbytes(workspace), n_sms, flags, s),
                "mla_decode_fwd")
    else:
        _launch(q.device, stream,
                lambda s: lib().mla_decode_fwd_ragged(_ptr(q), _ptr(kv), _ptr(seqlens), _ptr(q_lens),
                                                      _ptr(block_table), B, q_len, h, kv_rows, max_blocks,
                                                      float(softmax_scale), int(bool(causal)), _ptr(o), _ptr(lse),
                                                      _ptr(workspace), _nbytes(workspace), n_sms, flags, s),
                "mla_decode_fwd_ragged")


def mla_decode_fwd_untransposed(q, kv, seqlens, block_table, softmax_scale, causal, o, lse, workspace, n_sms,
                                flags=0, stream=None) -> None:
    """The same decode in the untransposed form, S = Q K^T with the query columns on M (padded to 64
    or 128): the form the pages set ETAP against, for the A/B comparison (``mla_decode_fwd_untransposed``;
    bf16 cache, one q_len for every sequence)."""
    _require_cuda(q, "q")
    check_decode_args(q, kv, seqlens, block_table, o, lse, workspace)
    B, q_len, h, _ = q.shape
    if block_table is not None:
        kv_rows, max_blocks = kv.shape[0] * kv.shape[1], block_table.shape[1]
    else:
        kv_rows, max_blocks = kv.shape[1], 0
    _launch(q.device, stream,
            lambda s: lib().mla_decode_fwd_untransposed(_ptr(q), _ptr(kv), _ptr(seqlens), _ptr(block_table), B, q_len,
                                                        h, kv_rows, max_blocks, float(softmax_scale),
                                                        int(bool(causal)), _ptr(o), _ptr(lse), _ptr(workspace),
                                                        _nbytes(workspace), n_sms, flags, s),
            "mla_decode_fwd_untransposed")


def mla_decode_fwd_fp8(q, kv8, kv_scale, seqlens, block_table, softmax_scale, causal, o, lse, workspace, n_sms,
                       flags=0, stream=None, q_lens=None) -> None:
    """Decode over an FP8 cache: ``kv8`` uint8 E4M3 codes laid out like the bf16 cache, ``kv_scale``
    fp32 with one scale per cache row (``mla_decode_fwd_fp8``; up to MLA_MAX_COLUMNS query columns)."""
    _require_cuda(q, "q")
    check_decode_args(q, kv8, seqlens, block_table, o, lse, workspace, q_lens, kv_scale=kv_scale)
    B, q_len, h, _ = q.shape
    if block_table is not None:
        kv_rows, max_blocks = kv8.shape[0] * kv8.shape[1], block_table.shape[1]
    else:
        kv_rows, max_blocks = kv8.shape[1], 0
    _launch(q.device, stream,
            lambda s: lib().mla_decode_fwd_fp8(_ptr(q), _ptr(kv8), _ptr(kv_scale), _ptr(seqlens), _ptr(q_lens),
                                               _ptr(block_table), B, q_len, h, kv_rows, max_blocks,
                                               float(softmax_scale), int(bool(causal)), _ptr(o), _ptr(lse),
                                               _ptr(workspace), _nbytes(workspace), n_sms, flags, s),
            "mla_decode_fwd_fp8")


def _tree_words(q_len: int) -> int:
    return (q_len + 31) // 32


def check_tree_args(q, kv, seqlens, block_table, tree_mask, o, lse, workspace, q_lens=None, kv_scale=None) -> tuple:
    """check_decode_args, the page size and the mask words of every query token -> the addresses and sizes
    that mla_decode_fwd_tree(_fp8) passes on, up to the softmax scale and from the outputs on.

    The conditions are tested in one go (4 us less than one by one); only where one fails does each check run
    by itself, for its message."""
    good = False
    try:
        index, fp8 = q.get_device(), kv_scale is not None
        B, q_len, h, width = q.shape
        rows, per, kv_width = kv.shape
        columns = B * q_len * h
        bf16 = torch.bfloat16
        good = (q.dtype is bf16 and width == D_QK and q.is_contiguous()
                and kv.dtype is (torch.uint8 if fp8 else bf16) and kv_width == D_QK and kv.get_device() == index
                and kv.is_contiguous() and _is(seqlens, _INT32, index, B) and seqlens.dim() == 1
                and (rows >= B if block_table is None else per == PAGE_SIZE and _is(block_table, _INT32, index, 0)
                     and block_table.dim() == 2 and block_table.shape[0] >= B)
                and (q_lens is None or _is(q_lens, _INT32, index, B) and q_lens.dim() == 1)
                and (not fp8 or _is(kv_scale, torch.float32, index, rows * per))
                and tree_mask.shape == (B, q_len, _tree_words(q_len)) and _is(tree_mask, _INT32, index, 0)
                and _is(o, bf16, index, columns * D_V) and _is(lse, torch.float32, index, columns)
                and workspace.get_device() == index and workspace.is_contiguous())
    except (AttributeError, TypeError, ValueError):
        pass
    if not good:
        check_decode_args(q, kv, seqlens, block_table, o, lse, workspace, q_lens, kv_scale)
        if block_table is not None and kv.shape[1] != PAGE_SIZE:
            raise ValueError(f"kv: pages of {kv.shape[1]} rows, expected {PAGE_SIZE}")
        _require(tree_mask, "tree_mask", torch.int32, q.device)
        want = (B, q_len, _tree_words(q_len))
        raise ValueError(f"tree_mask: shape {tuple(tree_mask.shape)}, expected {want}")
    table, max_blocks = (0, 0) if block_table is None else (block_table.data_ptr(), block_table.shape[1])
    return [q.data_ptr(), kv.data_ptr()] + ([kv_scale.data_ptr()] if fp8 else []) + [
        seqlens.data_ptr(), 0 if q_lens is None else q_lens.data_ptr(), tree_mask.data_ptr(), table, B, q_len, h,
        per if block_table is None else rows * per, max_blocks], [
        o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size()]


def _is(t, dtype, index: int, min_numel: int) -> bool:
    """A contiguous tensor of this dtype on this device, with so many elements."""
    return t.dtype is dtype and t.get_device() == index and t.is_contiguous() and t.numel() >= min_numel


def mla_decode_fwd_tree(q, kv, seqlens, block_table, softmax_scale, tree_mask, o, lse, workspace, n_sms, flags=0,
                        stream=None, q_lens=None) -> None:
    """Decode of drafts that form a tree: token t sees the rows ahead of the q_lens[b] (or q_len) new
    ones and the new tokens u whose bit is set in ``tree_mask`` (int32 [B, q_len, ceil(q_len / 32)])."""
    _require_cuda(q, "q")
    ahead, behind = check_tree_args(q, kv, seqlens, block_table, tree_mask, o, lse, workspace, q_lens)
    scale = float(softmax_scale)
    _launch(q.device, stream, lambda s: lib().mla_decode_fwd_tree(*ahead, scale, *behind, n_sms, flags, s),
            "mla_decode_fwd_tree")


def mla_decode_fwd_tree_fp8(q, kv8, kv_scale, seqlens, block_table, softmax_scale, tree_mask, o, lse, workspace,
                            n_sms, flags=0, stream=None, q_lens=None) -> None:
    """mla_decode_fwd_tree over an FP8 cache (E4M3 codes and one fp32 scale per cache row)."""
    _require_cuda(q, "q")
    if kv_scale is None:
        raise TypeError("kv_scale: expected a torch.Tensor, got NoneType")
    ahead, behind = check_tree_args(q, kv8, seqlens, block_table, tree_mask, o, lse, workspace, q_lens, kv_scale)
    scale = float(softmax_scale)
    _launch(q.device, stream, lambda s: lib().mla_decode_fwd_tree_fp8(*ahead, scale, *behind, n_sms, flags, s),
            "mla_decode_fwd_tree_fp8")


TRACE_ROLES = ("K-tile producer", "step-1 issuer", "value producer", "softmax", "step-3 issuer")


def mla_decode_fwd_trace(q, kv, seqlens, block_table, softmax_scale, causal, o, lse, workspace, n_sms, trace,
                         stream=None) -> None:
    """mla_decode_fwd that also records the event stamps of cluster 0's roles into ``trace`` (int64 device
    tensor of 2 * 5 * cap + 4 * n_sms elements, zeroed by the caller, made by trace_buffer()); see
    decode_trace_events() and decode_trace_spans()."""
    _require_cuda(q, "q")
    check_decode_args(q, kv, seqlens, block_table, o, lse, workspace)
    _require(trace, "trace", torch.int64, q.device, dim=1)
    cap = (trace.numel() - 4 * n_sms) // (2 * len(TRACE_ROLES))
    if cap < 1 or trace.numel() != 2 * len(TRACE_ROLES) * cap + 4 * n_sms:
        raise ValueError("trace: use trace_buffer(cap, n_sms)")
    B, q_len, h, _ = q.shape
    if block_table is not None:
        kv_rows, max_blocks = kv.shape[0] * kv.shape[1], block_table.shape[1]
    else:
        kv_rows, max_blocks = kv.shape[1], 0
    _launch(q.device, stream,
            lambda s: lib().mla_decode_fwd_trace(_ptr(q), _ptr(kv), _ptr(seqlens), _ptr(block_table), B, q_len, h,
                                                 kv_rows, max_blocks, float(softmax_scale), int(bool(causal)), _ptr(o),
                                                 _ptr(lse), _ptr(workspace), _nbytes(workspace), n_sms, _ptr(trace),
                                                 cap, s), "mla_decode_fwd_trace")


def trace_buffer(cap: int, n_sms: int, device=None):
    """A zeroed trace buffer for mla_decode_fwd_trace: [2 CTAs][5 roles][cap] stamps, then [n_sms][4]."""
    return torch.zeros(2 * len(TRACE_ROLES) * cap + 4 * n_sms, dtype=torch.int64, device=device)


def decode_trace_spans(trace, n_sms: int):
    """Trace buffer -> [n_sms, 4] (entry, start of work, end of work, exit) ns of every CTA, relative to the
    earliest entry (rows of CTAs that did not run stay 0)."""
    import numpy as np
    t = np.asarray(trace.cpu() if isinstance(trace, torch.Tensor) else trace).astype(np.int64)
    sp = t[len(t) - 4 * n_sms:].reshape(n_sms, 4).copy()
    live = sp[:, 0] > 0
    if live.any():
        sp[live] -= sp[live, 0].min()
    return sp


def decode_trace_events(trace, n_sms: int = None):
    """Trace buffer -> list of (cta, role, code, index, t_ns) sorted by time (t relative to the first stamp)."""
    import numpy as np
    t = np.asarray(trace.cpu() if isinstance(trace, torch.Tensor) else trace).astype(np.uint64)
    if n_sms is not None:
        t = t[:len(t) - 4 * n_sms]
    t = t.reshape(2, len(TRACE_ROLES), -1)
    out = []
    for cta in range(t.shape[0]):
        for role in range(t.shape[1]):
            for w in t[cta, role]:
                w = int(w)
                if w == 0:
                    break
                out.append((cta, role, w >> 56, (w >> 40) & 0xFFFF, w & 0xFFFFFFFFFF))
    if not out:
        return out
    t0 = min(e[4] for e in out)
    out = [(c, r, k, i, ts - t0) for c, r, k, i, ts in out]
    return sorted(out, key=lambda e: e[4])


def mla_stream_probe(kv, units: int, err, stream=None) -> None:
    """Stream ``kv`` ([..., 576] bf16, rows a multiple of 128) with the decode's TMA read pattern and
    no computation (a bandwidth probe).  ``err``: int32 device tensor [1], zeroed by the caller."""
    _require_cuda(kv, "kv")
    _require(kv, "kv", torch.bfloat16, kv.device, last=D_QK)
    _require(err, "err", torch.int32, kv.device, min_numel=1)
    rows = kv.numel() // 576
    _launch(kv.device, stream,
            lambda s: lib().mla_stream_probe(_ptr(kv), rows, units, _ptr(err), s), "mla_stream_probe")


def mla_form_ablation(form: int, heads: int, streams: int, tiles: int, cycles, err, stream=None) -> None:
    """Tensor-core instructions of ``tiles`` KV tiles per CTA in the transposed (form 0) or untransposed
    (form 1) layout; ``cycles``: uint64-compatible int64 device tensor [ctas], ``err``: int32 [1] zeroed."""
    _require_cuda(cycles, "cycles")
    _require(cycles, "cycles", torch.int64, cycles.device, min_numel=1)
    _require(err, "err", torch.int32, cycles.device, min_numel=1)
    _launch(cycles.device, stream,
            lambda s: lib().mla_form_ablation(form, heads, streams, tiles, cycles.numel(), _ptr(cycles), _ptr(err), s),
            "mla_form_ablation")


def mla_combine(workspace, batch, q_len, num_heads, n_sms, o, lse, stream=None) -> None:
    _require_cuda(o, "o")
    _require(o, "o", torch.bfloat16, o.device, min_numel=batch * q_len * num_heads * D_V)
    _require(lse, "lse", torch.float32, o.device, min_numel=batch * q_len * num_heads)
    _require(workspace, "workspace", None, o.device)
    _launch(o.device, stream,
            lambda s: lib().mla_combine(_ptr(workspace), batch, q_len, num_heads, n_sms, _ptr(o), _ptr(lse), s),
            "mla_combine")


# The checks of the cache operators.  These calls are made for every token, so the accepted case is kept
# short: `home` is (device, its index as Tensor.get_device() gives it), since comparing indices takes half
# the time of comparing devices, and the errors are worked out apart.
def _home(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    return t.device, t.get_device()


def _dense(t, name: str, dtype, home, shape) -> int:
    """Address of a contiguous tensor of exactly this dtype and shape (None: 0), or TypeError / ValueError."""
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == home[1] and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _require(t, name, dtype, home[0])
    raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


_INT32 = torch.int32


def _int32(t, name: str, home, shape) -> int:
    """_dense of an int32 tensor (a call checks up to twelve: its own copy of the test takes 0.1 us off each)."""
    if t is None:
        return 0
    try:
        if t.dtype is _INT32 and t.shape == shape and t.get_device() == home[1] and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _dense(t, name, _INT32, home, shape)


def _status_word(status, home) -> int:
    try:
        if status.dtype is torch.int32 and status.get_device() == home[1] and status.is_contiguous() and status.numel():
            return status.data_ptr()
    except AttributeError:
        pass
    _require(status, "status", torch.int32, home[0], min_numel=1)
    return status.data_ptr()


def _cache_rows(kv, kv_scale, home) -> tuple:
    """A cache of 576-wide rows -> (shape, its addresses), codes and scales for the FP8 cache."""
    fp8 = kv_scale is not None
    dtype = torch.uint8 if fp8 else torch.bfloat16
    try:
        shape = kv.shape
        good = kv.dtype is dtype and kv.get_device() == home[1] and kv.is_contiguous() and shape[-1] == D_QK
    except (AttributeError, IndexError):
        good = False
    if not good:
        _require(kv, "kv8" if fp8 else "kv", dtype, home[0], last=D_QK)
    if not fp8:
        return shape, [kv.data_ptr()]
    _require(kv_scale, "kv_scale", torch.float32, home[0], min_numel=math.prod(shape[:-1]))
    return shape, [kv.data_ptr(), kv_scale.data_ptr()]


def _page_stack(block_table, free_pages, num_free, num_free_out, B: int, home):
    """Table and stack of a paged cache -> (table, max_blocks, stack, capacity, count, count out)."""
    if block_table is None:
        return 0, 0, 0, 0, 0, 0
    if num_free is None or num_free_out is None:
        raise ValueError("num_free and num_free_out: a paged cache needs both")
    if not (isinstance(block_table, torch.Tensor) and isinstance(free_pages, torch.Tensor)):
        _home(block_table, "block_table"), _home(free_pages, "free_pages")
    if block_table.dim() != 2:
        raise ValueError(f"block_table: {block_table.dim()}-D, expected 2-D")
    blocks, pages = block_table.shape[1], free_pages.numel()
    return (_int32(block_table, "block_table", home, (B, blocks)), blocks,
            _int32(free_pages, "free_pages", home, (pages,)), pages, _int32(num_free, "num_free", home, (1,)),
            _int32(num_free_out, "num_free_out", home, (1,)))


def check_extend_args(seqlens, new_lens, block_table, free_pages, num_free, slots, positions, seqlens_out,
                      num_free_out, status, parents=None, tree_mask=None) -> list:
    """Shapes, dtypes and devices of mla_cache_extend -> the addresses and sizes it passes on."""
    home = _home(slots, "slots")
    if slots.dim() != 2:
        raise ValueError(f"slots: {slots.dim()}-D, expected 2-D")
    shape = slots.shape
    B, q_len = shape
    if (parents is None) != (tree_mask is None):
        raise ValueError("parents and tree_mask: give both or neither")
    if seqlens is None or positions is None or seqlens_out is None:
        raise ValueError("seqlens, positions and seqlens_out are not optional")
    per_seq = (B,)
    table, max_blocks, stack, capacity, nfree, nfree_out = _page_stack(block_table, free_pages, num_free,
                                                                       num_free_out, B, home)
    return [_int32(seqlens, "seqlens", home, per_seq), _int32(new_lens, "new_lens", home, per_seq),
            _int32(parents, "parents", home, shape), B, q_len, table, max_blocks, stack, capacity, nfree,
            _int32(slots, "slots", home, shape), _int32(positions, "positions", home, shape),
            _int32(tree_mask, "tree_mask", home, (B, q_len, _tree_words(q_len))),
            _int32(seqlens_out, "seqlens_out", home, per_seq), nfree_out, _status_word(status, home)]


def mla_cache_extend(seqlens, new_lens, block_table, free_pages, num_free, kv_rows: int, slots, positions,
                     seqlens_out, num_free_out, status, parents=None, tree_mask=None, stream=None) -> None:
    """Pages, cache rows, positions and ancestor masks of new tokens, from the request lengths.

    ``slots`` and ``positions`` (int32 [B, q_len]) are written, ``block_table`` is extended with pages from
    the end of ``free_pages``, ``seqlens_out`` and ``num_free_out`` (they may be the inputs themselves)
    receive the new lengths and the pages left.  ``new_lens`` None: q_len for every sequence;
    ``block_table`` None: a contiguous cache of ``kv_rows`` rows per sequence, no pages.  ``parents``
    (int32 [B, q_len], -1 behind the context) makes the tokens a tree and fills ``tree_mask``."""
    a = check_extend_args(seqlens, new_lens, block_table, free_pages, num_free, slots, positions, seqlens_out,
                          num_free_out, status, parents, tree_mask)
    _require_cuda(slots, "slots")
    _launch(slots.device, stream, lambda s: lib().mla_cache_extend(*a[:10], kv_rows, *a[10:], s), "mla_cache_extend")


def check_append_args(latent, norm_weight, rope_table, positions, slots, kv, status, q_rope=None, q=None,
                      kv_scale=None) -> tuple:
    """Shapes, dtypes and devices of mla_cache_append(_fp8) -> (arguments ahead of the cache, the cache's,
    those behind it)."""
    home = _home(latent, "latent")
    if latent.dtype is not torch.bfloat16:
        raise TypeError(f"latent: dtype {latent.dtype}, expected torch.bfloat16")
    shape = latent.shape
    if len(shape) != 2 or shape[1] != D_QK or (shape[0] > 0 and latent.stride(1) != 1):
        raise ValueError(f"latent: shape {tuple(shape)}, expected [tokens, {D_QK}] with dense rows")
    T = shape[0]
    if positions is None or slots is None:
        raise ValueError("positions and slots are not optional")
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q: give both or neither")
    max_pos = rope_table.shape[0] if isinstance(rope_table, torch.Tensor) and rope_table.dim() else 0
    per_token = (T,)
    weight = _dense(norm_weight, "norm_weight", torch.bfloat16, home, (D_V,))
    table = _dense(rope_table, "rope_table", torch.float32, home, (max_pos, 64))
    if not table:
        raise ValueError("rope_table: not optional, and needs a row")
    where = [_int32(positions, "positions", home, per_token), _int32(slots, "slots", home, per_token), T]
    cache_shape, cache = _cache_rows(kv, kv_scale, home)
    queries = [0, 0, 0, 0, 0]
    if q is not None:
        if _home(q_rope, "q_rope") != home:
            raise ValueError(f"q_rope: on {q_rope.device}, expected {home[0]} (all tensors on one device)")
        if q_rope.dtype is not torch.bfloat16:
            raise TypeError(f"q_rope: dtype {q_rope.dtype}, expected torch.bfloat16")
        rs = q_rope.shape
        if len(rs) != 3 or rs[0] != T or rs[2] != 64 or q_rope.stride(2) != 1:
            raise ValueError(f"q_rope: shape {tuple(rs)}, expected [{T}, heads, 64] with dense rows")
        h = rs[1]
        _home(q, "q")
        qs = q.shape
        if math.prod(qs) != T * h * D_QK or len(qs) < 2 or qs[-2] != h or qs[-1] != D_QK:
            raise ValueError(f"q: shape {tuple(qs)}, expected [{T}, {h}, {D_QK}] or its tokens as [B, q_len]")
        stride = q_rope.stride()  # (that of a dimension of one entry may be anything)
        queries = [q_rope.data_ptr(), stride[0] if T > 1 else 0, stride[1] if h > 1 else 0, h,
                   _dense(q, "q", torch.bfloat16, home, qs)]
    return ([latent.data_ptr(), latent.stride(0) if T > 1 else D_QK, weight], [table, max_pos], where,
            cache + [math.prod(cache_shape[:-1])], queries + [_status_word(status, home)])


def mla_cache_append(latent, norm_weight, eps, rope_table, interleaved, positions, slots, kv, status, q_rope=None,
                     q=None, stream=None) -> None:
    """Norm the 512 latent columns, rotate the 64 rope columns of each row of ``latent`` ([tokens, 576] bf16,
    rows may be strided) and store the row at ``slots`` of the bf16 cache; with ``q_rope`` ([tokens, heads,
    64], may be strided) also rotate the queries' rope columns into ``q[..., 512:]``."""
    ahead, table, where, cache, behind = check_append_args(latent, norm_weight, rope_table, positions, slots, kv,
                                                           status, q_rope, q)
    _require_cuda(latent, "latent")
    _launch(latent.device, stream,
            lambda s: lib().mla_cache_append(*ahead, eps, *table, int(bool(interleaved)), *where, *cache, *behind, s),
            "mla_cache_append")


def mla_cache_append_fp8(latent, norm_weight, eps, rope_table, interleaved, positions, slots, kv8, kv_scale, status,
                         q_rope=None, q=None, stream=None) -> None:
    """mla_cache_append into an FP8 cache: E4M3 codes and one fp32 scale per row, max|row| / 448."""
    if kv_scale is None:
        raise TypeError("kv_scale: expected a torch.Tensor, got NoneType")
    ahead, table, where, cache, behind = check_append_args(latent, norm_weight, rope_table, positions, slots, kv8,
                                                           status, q_rope, q, kv_scale)
    _require_cuda(latent, "latent")
    _launch(latent.device, stream,
            lambda s: lib().mla_cache_append_fp8(*ahead, eps, *table, int(bool(interleaved)), *where, *cache, *behind,
                                                 s),
            "mla_cache_append_fp8")


def check_accept_args(kv, seqlens, new_lens, path, path_lens, block_table, free_pages, num_free, seqlens_out,
                      num_free_out, status, kv_scale=None) -> tuple:
    """Shapes, dtypes and devices of mla_cache_accept -> (arguments ahead of kv_rows, kv_rows, those behind)."""
    home = _home(path, "path")
    if path.dim() != 2:
        raise ValueError(f"path: {path.dim()}-D, expected 2-D")
    B, P = path.shape
    shape, cache = _cache_rows(kv, kv_scale, home)
    if len(shape) != 3:
        raise ValueError(f"kv: {len(shape)}-D, expected 3-D")
    if block_table is not None:
        if shape[1] != PAGE_SIZE:
            raise ValueError(f"kv: pages of {shape[1]} rows, expected {PAGE_SIZE}")
    elif shape[0] < B:
        raise ValueError(f"kv: {shape[0]} sequences, needs at least {B}")
    if seqlens is None or new_lens is None or path_lens is None or seqlens_out is None:
        raise ValueError("seqlens, new_lens, path_lens and seqlens_out are not optional")
    table, max_blocks, stack, capacity, nfree, nfree_out = _page_stack(block_table, free_pages, num_free,
                                                                       num_free_out, B, home)
    per_seq = (B,)
    ahead = cache + ([] if kv_scale is not None else [0]) + [
        _int32(seqlens, "seqlens", home, per_seq), _int32(new_lens, "new_lens", home, per_seq),
        _int32(path, "path", home, (B, P)), _int32(path_lens, "path_lens", home, per_seq), B, 2 ** 31 - 1, P, table,
        max_blocks, stack, capacity, nfree]
    return (ahead, shape[0] * shape[1] if block_table is not None else shape[1],
            [_int32(seqlens_out, "seqlens_out", home, per_seq), nfree_out, _status_word(status, home)])


def mla_cache_accept(kv, seqlens, new_lens, path, path_lens, block_table, free_pages, num_free, seqlens_out,
                     num_free_out, status, kv_scale=None, stream=None) -> None:
    """Keep the accepted path of each sequence's new_lens[b] last rows: row path[b, i] of them becomes row i
    (i < path_lens[b]; -1: the sequence has ended), the rest is dropped and the pages past the new length
    are pushed on ``free_pages``.  ``seqlens_out`` and ``num_free_out`` may be the inputs themselves;
    ``kv_scale`` given: the FP8 cache."""
    ahead, kv_rows, behind = check_accept_args(kv, seqlens, new_lens, path, path_lens, block_table, free_pages,
                                               num_free, seqlens_out, num_free_out, status, kv_scale)
    _require_cuda(kv, "kv")
    _launch(kv.device, stream, lambda s: lib().mla_cache_accept(*ahead, kv_rows, *behind, s), "mla_cache_accept")


def mla_decode_read_status(workspace, stream=None) -> int:
    _require_cuda(workspace, "workspace")
    out = ctypes.c_int(0)
    _launch(workspace.device, stream, lambda s: lib().mla_decode_read_status(_ptr(workspace), ctypes.byref(out), s),
            "mla_decode_read_status")
    return int(out.value)


def mla_decode_plan_host(seqlens, q_len: int, num_heads: int, n_sms: int, schedule: int = 1):
    """Host mirror of a schedule -> (cta_ranges [ctas, 2], seq_info [B, 4], num_ctas, num_groups, unit_rows,
    group_cols).  schedule 1: the one mla_decode_fwd (bf16 cache) uses; 0: the one mla_decode_fwd_fp8 uses;
    2: the one the tree decodes use."""
    import numpy as np
    sl = np.ascontiguousarray(np.asarray(seqlens, dtype=np.int32))
    nct, ngr, urows, gcols = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().mla_decode_plan_host(sl.ctypes.data_as(ctypes.c_void_p), sl.size, q_len, num_heads, n_sms, schedule,
                                      None, None, ctypes.byref(nct), ctypes.byref(ngr), ctypes.byref(urows),
                                      ctypes.byref(gcols)), "mla_decode_plan_host")
    ranges = np.zeros((nct.value, 2), np.int32)
    info = np.zeros((sl.size, 4), np.int32)
    _check(lib().mla_decode_plan_host(sl.ctypes.data_as(ctypes.c_void_p), sl.size, q_len, num_heads, n_sms, schedule,
                                      ranges.ctypes.data_as(ctypes.c_void_p), info.ctypes.data_as(ctypes.c_void_p),
                                      ctypes.byref(nct), ctypes.byref(ngr), ctypes.byref(urows), ctypes.byref(gcols)),
           "mla_decode_plan_host")
    return ranges, info, nct.value, ngr.value, urows.value, gcols.value


class MlaDecoder:
    """Owns the workspace for one (batch, q_len, num_heads) shape; plan() then fwd()."""

    def __init__(self, batch: int, q_len: int, num_heads: int, device=None, n_sms: Optional[int] = None):
        self.device = torch.device(device if device is not None else "cuda")
        self.batch, self.q_len, self.num_heads = batch, q_len, num_heads
        self.n_sms = n_sms if n_sms is not None else num_sms(self.device)
        nbytes = mla_decode_workspace_size(batch, q_len, num_heads, self.n_sms)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self._planned: Optional[int] = None  # sequences of the last plan

    def plan(self, seqlens: torch.Tensor, stream=None):
        mla_decode_plan(seqlens, self.q_len, self.num_heads, self.workspace, self.n_sms, stream)
        self._planned = seqlens.numel()

    def _tree_shape(self, q) -> tuple:
        """(batch, q_len, heads) of a tree decode's q, which have to be the planned ones."""
        B, q_len, h, _ = q.shape
        if q_len != self.q_len or h != self.num_heads or (self._planned is not None and B != self._planned):
            batch = self.batch if self._planned is None else self._planned
            raise ValueError(f"q: {B} sequences of {q_len} tokens and {h} heads, planned for {batch} of {self.q_len} "
                             f"and {self.num_heads}")
        return B, q_len, h

    def fwd(self, q, kv, seqlens, block_table=None, softmax_scale=None, causal=False, o=None, lse=None,
            flags=0, stream=None, q_lens=None):
        B, q_len, h, _ = q.shape
        if o is None:
            o = torch.empty(B, q_len, h, D_V, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(B, q_len, h, dtype=torch.float32, device=q.device)
        scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(D_QK)
        mla_decode_fwd(q, kv, seqlens, block_table, scale, causal, o, lse, self.workspace, self.n_sms, flags,
                       stream, q_lens=q_lens)
        return o, lse

    def fwd_fp8(self, q, kv8, kv_scale, seqlens, block_table=None, softmax_scale=None, causal=False, o=None,
                lse=None, flags=0, stream=None, q_lens=None):
        """fwd over an FP8 cache (E4M3 codes + one fp32 scale per cache row)."""
        B, q_len, h, _ = q.shape
        if o is None:
            o = torch.empty(B, q_len, h, D_V, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(B, q_len, h, dtype=torch.float32, device=q.device)
        scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(D_QK)
        mla_decode_fwd_fp8(q, kv8, kv_scale, seqlens, block_table, scale, causal, o, lse, self.workspace, self.n_sms,
                           flags, stream, q_lens=q_lens)
        return o, lse

    def fwd_tree(self, q, kv, seqlens, tree_mask, block_table=None, softmax_scale=None, o=None, lse=None, flags=0,
                 stream=None, q_lens=None):
        """fwd for drafts that form a tree (mask words from mla_cache_extend, or the caller's own)."""
        B, q_len, h = self._tree_shape(q)
        if o is None:
            o = torch.empty(B, q_len, h, D_V, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(B, q_len, h, dtype=torch.float32, device=q.device)
        scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(D_QK)
        mla_decode_fwd_tree(q, kv, seqlens, block_table, scale, tree_mask, o, lse, self.workspace, self.n_sms, flags,
                            stream, q_lens=q_lens)
        return o, lse

    def fwd_tree_fp8(self, q, kv8, kv_scale, seqlens, tree_mask, block_table=None, softmax_scale=None, o=None,
                     lse=None, flags=0, stream=None, q_lens=None):
        """fwd_tree over an FP8 cache (E4M3 codes + one fp32 scale per cache row)."""
        B, q_len, h = self._tree_shape(q)
        if o is None:
            o = torch.empty(B, q_len, h, D_V, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(B, q_len, h, dtype=torch.float32, device=q.device)
        scale = softmax_scale if softmax_scale is not None else 1.0 / math.sqrt(D_QK)
        mla_decode_fwd_tree_fp8(q, kv8, kv_scale, seqlens, block_table, scale, tree_mask, o, lse, self.workspace,
                                self.n_sms, flags, stream, q_lens=q_lens)
        return o, lse

    def status(self, stream=None) -> int:
        return mla_decode_read_status(self.workspace, stream)


def mla_decode(q, kv, seqlens, block_table=None, softmax_scale=None, causal=False, q_lens=None):
    """One-shot convenience: plan + decode (+ combine).  Returns (O bf16, LSE fp32)."""
    dec = MlaDecoder(q.shape[0], q.shape[1], q.shape[2], device=q.device)
    dec.plan(seqlens)
    return dec.fwd(q, kv, seqlens, block_table, softmax_scale, causal, q_lens=q_lens)
