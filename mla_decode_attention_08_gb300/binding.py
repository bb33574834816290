"""ctypes binding of libmla_decode (argument marshalling only).

Every function here forwards to the C ABI declared in ``include/mla_decode.h``
under the same name.  Tensors must already live on a CUDA device: there is no
CPU path, and a missing library raises instead of falling back.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import LIB as LIB_PATH

NUM_HEADS, QK_HEAD_DIM, V_HEAD_DIM, TILE_TOKENS = 16, 576, 512, 128

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported device", 3: "workspace too small",
          4: "CUDA call failed"}
DERR = {1: "qo_indptr", 2: "kv_indptr", 4: "kv_index", 8: "timeout", 16: "mx_scale",
        64: "seq_len", 128: "free_pages", 256: "capacity", 512: "position"}
STEP_WORKSPACE_BYTES = 256
PREFILL_QK_DIM, PREFILL_NOPE_DIM, PREFILL_V_DIM = 192, 128, 128
ROPE_DIM = QK_HEAD_DIM - V_HEAD_DIM


class MlaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class mla_plan_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("max_kv_len", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("abi_version", ctypes.c_int32),
                ("qo_len", ctypes.c_int32), ("cluster", ctypes.c_int32),
                ("ws_bytes", ctypes.c_uint64), ("ws_prefix_offset", ctypes.c_uint64),
                ("ws_workers_offset", ctypes.c_uint64), ("ws_lse_offset", ctypes.c_uint64),
                ("ws_partial_offset", ctypes.c_uint64)]


class mla_prefill_plan_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("max_kv_len", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("tiles", ctypes.c_int32), ("abi_version", ctypes.c_int32),
                ("ws_bytes", ctypes.c_uint64), ("ws_lse_offset", ctypes.c_uint64),
                ("ws_partial_offset", ctypes.c_uint64)]


class mla_shared_plan_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_q", ctypes.c_int32),
                ("max_kv_len", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("workers", ctypes.c_int32), ("split", ctypes.c_int32),
                ("start", ctypes.c_int32), ("abi_version", ctypes.c_int32),
                ("ws_bytes", ctypes.c_uint64), ("ws_lse_offset", ctypes.c_uint64),
                ("ws_partial_offset", ctypes.c_uint64)]


_VP, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_PLANP = ctypes.POINTER(mla_plan_t)
_FWD_ARGS = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _PLANP, _VP, _I64, _I64, _VP, _SZ]
_FWD_BF16KV_ARGS = _FWD_ARGS[:2] + _FWD_ARGS[3:]  # no kv_scale
# q, kv_fp4, kv_scales, scale_bias, qo_indptr, kv_indptr, out, stream, plan, kv_rows, ws, ws_bytes
_FWD_MXFP4_ARGS = [_VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _PLANP, _I64, _VP, _SZ]
_F32 = ctypes.c_float
_SHARED_PLANP = ctypes.POINTER(mla_shared_plan_t)
# q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, lse, stream, plan, kv_indices + len, kv_rows, ws, ws_bytes
_SHARED_ARGS = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _SHARED_PLANP, _VP, _I64, _I64, _VP, _SZ]
# kv, kv_scale, kv_rows, slots, num_tokens, means, num_pages, page_size, ws, ws_bytes, stream
_MEANS_ARGS = [_VP, _VP, _I64, _VP, _I64, _VP, _I32, _I32, _VP, _SZ, _VP]
_PREFILL_PLANP = ctypes.POINTER(mla_prefill_plan_t)
# kv, kv_stride, weight, eps, rope_table, max_positions, interleaved, positions, slots, num_tokens,
# cache, kv_scale, kv_rows, latent_out, q_pe + strides, q_out + strides, heads, ws, ws_bytes, stream
_APPEND_ARGS = [_VP, _I64, _VP, _F32, _VP, _I32, _I32, _VP, _VP, _I32, _VP, _VP, _I64, _VP,
                _VP, _I64, _I64, _VP, _I64, _I64, _I32, _VP, _SZ, _VP]
# q, k_nope, k_rope, v with their strides, total_kv, indptrs, scale, causal, out, lse, stream, plan, ws
_PREFILL_ARGS = [_VP, _I64, _I64, _VP, _I64, _I64, _VP, _I64, _VP, _I64, _I64, _I64, _VP, _VP, _F32,
                 _I32, _VP, _VP, _VP, _PREFILL_PLANP, _VP, _SZ]
SIGNATURES = {
    "mla_page_map": (ctypes.c_int, [_VP, _VP, _I32, _VP, _I64, _I32, _I32, _I32, _VP, _I32, _VP, _VP,
                                    _VP, _I64, _VP, _VP, _I64, _VP, _VP, _SZ, _VP]),
    "mla_kv_append": (ctypes.c_int, _APPEND_ARGS),
    "mla_kv_append_bf16kv": (ctypes.c_int, _APPEND_ARGS[:11] + _APPEND_ARGS[12:]),  # no kv_scale
    "mla_prefill_plan": (ctypes.c_int, [_I32, _I32, _I32, _I32, _I32, _PREFILL_PLANP]),
    "mla_prefill_fwd": (ctypes.c_int, _PREFILL_ARGS),
    "mla_prefill_fwd_stall_stream": (ctypes.c_int, _PREFILL_ARGS),
    "mla_attn_merge": (ctypes.c_int, [_VP, _VP, _I32, _I64, _I32, _VP, _VP, _VP]),
    "mla_shared_plan": (ctypes.c_int, [_I32, _I32, _I32, _I32, _SHARED_PLANP]),
    "mla_shared_fwd": (ctypes.c_int, _SHARED_ARGS),
    "mla_shared_fwd_stall_stream": (ctypes.c_int, _SHARED_ARGS),
    "mla_block_means": (ctypes.c_int, _MEANS_ARGS),
    "mla_block_means_bf16kv": (ctypes.c_int, _MEANS_ARGS[:1] + _MEANS_ARGS[2:]),  # no kv_scale
    "mla_block_scores": (ctypes.c_int, [_VP, _I32, _VP, _I32, _VP, _I64, _I32, _VP, _VP, _I32, _I32, _VP, _I64,
                                        _VP, _SZ, _VP]),
    "mla_block_select": (ctypes.c_int, [_VP, _I64, _VP, _I64, _I32, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _VP,
                                        _VP, _I64, _VP, _VP, _SZ, _VP]),
    "mla_decode_fwd_lse": (ctypes.c_int, _FWD_ARGS[:6] + [_VP] + _FWD_ARGS[6:]),
    "mla_decode_fwd_bf16kv_lse": (ctypes.c_int, _FWD_BF16KV_ARGS[:5] + [_VP] + _FWD_BF16KV_ARGS[5:]),
    "mla_decode_fwd_mxfp4_lse": (ctypes.c_int, _FWD_MXFP4_ARGS[:7] + [_VP] + _FWD_MXFP4_ARGS[7:]),
    "mla_decode_plan": (ctypes.c_int, [_I32, _I32, _I32, _PLANP]),
    "mla_decode_plan_mtp": (ctypes.c_int, [_I32, _I32, _I32, _I32, _PLANP]),
    "mla_decode_fwd": (ctypes.c_int, _FWD_ARGS),
    "mla_decode_fwd_stall_stream": (ctypes.c_int, _FWD_ARGS),
    "mla_decode_stage1": (ctypes.c_int, _FWD_ARGS),
    "mla_decode_fwd_bf16kv": (ctypes.c_int, _FWD_BF16KV_ARGS),
    "mla_decode_stage1_bf16kv": (ctypes.c_int, _FWD_BF16KV_ARGS),
    "mla_decode_fwd_static_scratch": (ctypes.c_int, _FWD_ARGS[:-2]),
    "mla_decode_static_scratch_read_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32), _I32, _VP]),
    "mla_decode_fwd_mxfp4": (ctypes.c_int, _FWD_MXFP4_ARGS),
    "mla_decode_stage1_mxfp4": (ctypes.c_int, _FWD_MXFP4_ARGS),
    "mla_decode_fwd_mxfp4_stall_stream": (ctypes.c_int, _FWD_MXFP4_ARGS),
    "mla_mxfp4_quantize": (ctypes.c_int, [_VP, _I64, _VP, _VP, _VP]),
    "mla_debug_q_operand": (ctypes.c_int, [_VP, _I32, _I32, _VP, _VP, _VP, _VP]),
    "mla_decode_trace_read": (ctypes.c_int, [_VP, _VP, _I32]),
    "mla_debug_p_split": (ctypes.c_int, [_VP, _I64, _VP, _VP, _VP]),
    "mla_decode_stage2": (ctypes.c_int, [_VP, _VP, _VP, _PLANP, _VP, _SZ]),
    "mla_fp8_quantize_per_tensor": (ctypes.c_int, [_VP, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "mla_decode_workspace_init": (ctypes.c_int, [_VP, _SZ, _VP]),
    "mla_decode_read_error": (ctypes.c_int, [_VP, ctypes.POINTER(ctypes.c_int32), _I32, _VP]),
    "mla_decode_schedule_host": (ctypes.c_int, [_VP, _I32, _I32, _VP, _VP]),
    "mla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mla_decode_abi_version": (ctypes.c_int32, []),
}

_lib: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmla_decode.so (raises when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                               "(python -m mla_decode_attention_08_gb300.build)")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name, None)
            if fn is None:  # a library from before this entry point; calling it raises
                continue
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MlaError(fn, status)


def _dev_ptr(t: Optional[torch.Tensor], name: str, dtype=None) -> Optional[int]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def mla_decode_plan(batch: int, max_kv_len: int, num_sms: int = 0, qo_len: int = 1,
                    persistent: bool = False) -> mla_plan_t:
    """Plan for ``batch`` rows of ``qo_len`` query tokens (1 to 4; 2-4 for multi-token decode).

    ``persistent=True`` forces the persistent split (``plan.cluster = 0``) where
    the plan would take the cluster split of small batches."""
    plan = mla_plan_t()
    _check("mla_decode_plan_mtp", load_library().mla_decode_plan_mtp(batch, qo_len, max_kv_len,
                                                                    num_sms, ctypes.byref(plan)))
    if persistent:
        plan.cluster = 0
    return plan


def _e4m3_cache(kv_fp8) -> torch.Tensor:
    """The e4m3 cache as [rows, 576] bytes; anything else is refused (a bf16 or
    MXFP4 cache passed here would otherwise be read as e4m3 codes)."""
    if not isinstance(kv_fp8, torch.Tensor):
        raise TypeError("kv_fp8 must be a CUDA tensor")
    if kv_fp8.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"kv_fp8 must hold e4m3fn codes (uint8 or float8_e4m3fn), got {kv_fp8.dtype}")
    if kv_fp8.dim() not in (2, 3) or kv_fp8.numel() != kv_fp8.shape[0] * QK_HEAD_DIM:
        raise ValueError(f"kv_fp8 must be [rows, 576] or [rows, 1, 576], got {tuple(kv_fp8.shape)}")
    return kv_fp8 if kv_fp8.dim() == 2 else kv_fp8.reshape(kv_fp8.shape[0], QK_HEAD_DIM)


def _fwd_args(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan, kv_indices,
              workspace):
    kv_fp8 = _e4m3_cache(kv_fp8)
    kv_rows = int(kv_fp8.shape[0])
    return (_dev_ptr(q, "q", torch.bfloat16), _dev_ptr(kv_fp8, "kv_fp8"),
            _dev_ptr(kv_scale, "kv_scale", torch.float32),
            _dev_ptr(qo_indptr, "qo_indptr", torch.int32),
            _dev_ptr(kv_indptr, "kv_indptr", torch.int32), _dev_ptr(out, "out", torch.bfloat16),
            _stream(stream), ctypes.byref(plan),
            _dev_ptr(kv_indices, "kv_indices", torch.int32),
            0 if kv_indices is None else int(kv_indices.numel()), kv_rows,
            _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size())


def _fwd_bf16kv_args(q, kv_bf16, qo_indptr, kv_indptr, out, stream, plan, kv_indices, workspace):
    if kv_bf16.dim() == 3:
        kv_bf16 = kv_bf16.reshape(kv_bf16.shape[0], -1)
    return (_dev_ptr(q, "q", torch.bfloat16), _dev_ptr(kv_bf16, "kv_bf16", torch.bfloat16),
            _dev_ptr(qo_indptr, "qo_indptr", torch.int32),
            _dev_ptr(kv_indptr, "kv_indptr", torch.int32), _dev_ptr(out, "out", torch.bfloat16),
            _stream(stream), ctypes.byref(plan),
            _dev_ptr(kv_indices, "kv_indices", torch.int32),
            0 if kv_indices is None else int(kv_indices.numel()), int(kv_bf16.shape[0]),
            _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size())


def _fwd_mxfp4_args(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out, stream, plan, workspace,
                    scale_bias):
    kv_fp4 = kv_fp4.reshape(kv_fp4.shape[0], -1)
    if kv_fp4.shape[1] != QK_HEAD_DIM // 2 or kv_scales.numel() != kv_fp4.shape[0] * 18:
        raise ValueError("kv_fp4 must be [N, 288] uint8 and kv_scales [N, 18] uint8")
    return (_dev_ptr(q, "q", torch.bfloat16), _dev_ptr(kv_fp4, "kv_fp4", torch.uint8),
            _dev_ptr(kv_scales, "kv_scales", torch.uint8), int(scale_bias),
            _dev_ptr(qo_indptr, "qo_indptr", torch.int32),
            _dev_ptr(kv_indptr, "kv_indptr", torch.int32), _dev_ptr(out, "out", torch.bfloat16),
            _stream(stream), ctypes.byref(plan), int(kv_fp4.shape[0]),
            _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size())


def _fwd(fn: str, args: tuple, q, lse, at: int) -> None:
    """Call decode step ``fn``, or where a tensor for the log-sum-exps is given the form of
    it that reports them, whose argument it is in place ``at``."""
    if lse is not None:
        p_lse = _dev_ptr(lse, "lse", torch.float32)
        if lse.shape != q.shape[:2] or lse.device != q.device:
            raise ValueError(f"lse must be {list(q.shape[:2])} on {q.device}, got {list(lse.shape)} on {lse.device}")
        fn, args = fn + "_lse", (*args[:at], p_lse, *args[at:])
    _check(fn, getattr(load_library(), fn)(*args))


def mla_decode_fwd_mxfp4(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out, stream=None, *, plan,
                         workspace, scale_bias: int = 0, lse=None) -> torch.Tensor:
    """Decode step over an MXFP4 cache (elements ``[N, 288]``, scales ``[N, 18]``); returns ``out``.

    ``lse`` float32 [T, 16] or None, as in mla_decode_fwd."""
    _fwd("mla_decode_fwd_mxfp4", _fwd_mxfp4_args(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out, stream,
                                                 plan, workspace, scale_bias), q, lse, 7)
    return out


def mla_decode_stage1_mxfp4(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out, stream=None, *,
                            plan, workspace, scale_bias: int = 0) -> None:
    _check("mla_decode_stage1_mxfp4", load_library().mla_decode_stage1_mxfp4(
        *_fwd_mxfp4_args(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out, stream, plan, workspace,
                         scale_bias)))


def mla_decode_fwd_mxfp4_stall_stream(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out,
                                      stream=None, *, plan, workspace, scale_bias: int = 0) -> None:
    """Test hook: the MXFP4 step with a cache stream that never arrives."""
    _check("mla_decode_fwd_mxfp4_stall_stream", load_library().mla_decode_fwd_mxfp4_stall_stream(
        *_fwd_mxfp4_args(q, kv_fp4, kv_scales, qo_indptr, kv_indptr, out, stream, plan, workspace,
                         scale_bias)))


def mla_mxfp4_quantize(src_bf16, dst_fp4, dst_scales, stream=None) -> None:
    """MXFP4 of bf16 rows ``[N, 576]`` into ``dst_fp4 [N, 288]`` and ``dst_scales [N, 18]``."""
    src = src_bf16.reshape(-1, QK_HEAD_DIM)
    rows = int(src.shape[0])
    if dst_fp4.numel() != rows * 288 or dst_scales.numel() != rows * 18:
        raise ValueError("dst_fp4 must hold [N, 288] and dst_scales [N, 18] bytes")
    _check("mla_mxfp4_quantize", load_library().mla_mxfp4_quantize(
        _dev_ptr(src, "src_bf16", torch.bfloat16), rows, _dev_ptr(dst_fp4, "dst_fp4", torch.uint8),
        _dev_ptr(dst_scales, "dst_scales", torch.uint8), _stream(stream)))


def mla_decode_fwd_bf16kv(q, kv_bf16, qo_indptr, kv_indptr, out, stream=None, *, plan,
                          workspace, kv_indices=None, lse=None) -> torch.Tensor:
    """Decode step over a bf16 cache ``[N, 576]`` (no scale); writes and returns ``out``.

    ``lse`` float32 [T, 16] or None, as in mla_decode_fwd."""
    _fwd("mla_decode_fwd_bf16kv", _fwd_bf16kv_args(q, kv_bf16, qo_indptr, kv_indptr, out, stream, plan,
                                                   kv_indices, workspace), q, lse, 5)
    return out


def mla_decode_stage1_bf16kv(q, kv_bf16, qo_indptr, kv_indptr, out, stream=None, *, plan,
                             workspace, kv_indices=None) -> None:
    _check("mla_decode_stage1_bf16kv", load_library().mla_decode_stage1_bf16kv(
        *_fwd_bf16kv_args(q, kv_bf16, qo_indptr, kv_indptr, out, stream, plan, kv_indices,
                          workspace)))


def mla_decode_fwd(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream=None, *, plan,
                   workspace, kv_indices=None, lse=None) -> torch.Tensor:
    """Decode step; writes ``out`` (bf16 [B, 16, 512]) and returns it.

    ``lse`` float32 [T, 16] takes each token's and head's natural log-sum-exp
    (mla_decode_fwd_lse), with which mla_attn_merge joins ``out`` to attention over other keys."""
    _fwd("mla_decode_fwd", _fwd_args(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan, kv_indices,
                                     workspace), q, lse, 6)
    return out


def mla_decode_fwd_stall_stream(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream=None, *,
                                plan, workspace, kv_indices=None) -> None:
    """Test hook: the decode launches with a cache stream that never arrives,
    so the bounded waits run out and the call reports MLA_DERR_TIMEOUT."""
    _check("mla_decode_fwd_stall_stream", load_library().mla_decode_fwd_stall_stream(
        *_fwd_args(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan, kv_indices,
                   workspace)))


def mla_decode_fwd_static_scratch(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream=None, *,
                                  plan, kv_indices=None) -> torch.Tensor:
    """Decode step with the library's own static scratch instead of a workspace,
    for callers that may not allocate device memory (see the C header)."""
    kv_fp8 = _e4m3_cache(kv_fp8)
    _check("mla_decode_fwd_static_scratch", load_library().mla_decode_fwd_static_scratch(
        _dev_ptr(q, "q", torch.bfloat16), _dev_ptr(kv_fp8, "kv_fp8"),
        _dev_ptr(kv_scale, "kv_scale", torch.float32), _dev_ptr(qo_indptr, "qo_indptr", torch.int32),
        _dev_ptr(kv_indptr, "kv_indptr", torch.int32), _dev_ptr(out, "out", torch.bfloat16),
        _stream(stream), ctypes.byref(plan), _dev_ptr(kv_indices, "kv_indices", torch.int32),
        0 if kv_indices is None else int(kv_indices.numel()), int(kv_fp8.shape[0])))
    return out


def mla_decode_static_scratch_read_error(clear: bool = True, stream=None) -> int:
    """Error word of the current device's static scratch (MLA_DERR_* bits)."""
    v = ctypes.c_int32(0)
    _check("mla_decode_static_scratch_read_error",
           load_library().mla_decode_static_scratch_read_error(ctypes.byref(v), int(clear),
                                                               _stream(stream)))
    return int(v.value)


def mla_decode_stage1(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream=None, *, plan,
                      workspace, kv_indices=None) -> None:
    _check("mla_decode_stage1", load_library().mla_decode_stage1(
        *_fwd_args(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan, kv_indices,
                   workspace)))


def mla_decode_stage2(qo_indptr, out, stream=None, *, plan, workspace) -> None:
    _check("mla_decode_stage2", load_library().mla_decode_stage2(
        _dev_ptr(qo_indptr, "qo_indptr", torch.int32), _dev_ptr(out, "out", torch.bfloat16),
        _stream(stream), ctypes.byref(plan), _dev_ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size()))


def mla_fp8_quantize_per_tensor(src_bf16, dst_fp8, scale_out, tmp, stream=None) -> None:
    """e4m3fn codes of a bf16 tensor with a per-tensor absmax scale (float32 [1])."""
    _check("mla_fp8_quantize_per_tensor", load_library().mla_fp8_quantize_per_tensor(
        _dev_ptr(src_bf16, "src", torch.bfloat16), src_bf16.numel(), _dev_ptr(dst_fp8, "dst"),
        _dev_ptr(scale_out, "scale_out", torch.float32), _dev_ptr(tmp, "tmp"),
        tmp.numel() * tmp.element_size(), _stream(stream)))


# ---------------------------------------------------------------- around the decode step
# A step makes several of these small calls, so their host time counts: operands
# are checked in one pass each, by the tensors' cheap accessors.
_Tensor, _BF16, _F32T, _I32T = torch.Tensor, torch.bfloat16, torch.float32, torch.int32
_E4M3_CODES = (torch.uint8, torch.float8_e4m3fn)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _refuse(t, name: str, dtype, dev) -> None:
    """Raise what is wrong with an operand that failed its checks."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the first operand on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _device_of(t, name: str) -> int:
    """Index of the CUDA device that a call's first operand, and so every other one, is on."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        _refuse(t, name, None, None)
    return t.get_device()


def _view_ptr(t, name: str, dtype, dev: int) -> int:
    """Address of an operand on device ``dev`` that may be strided."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(t, name, dtype, dev)
    return t.data_ptr()


def _ptr(t, name: str, dtype, dev: int) -> int:
    """Address of a contiguous operand on device ``dev``."""
    if (not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, name, dtype, dev)
    return t.data_ptr()


def _workspace(t, dev: int) -> int:
    if not isinstance(t, _Tensor) or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, "workspace", None, dev)
    return t.data_ptr()


def _expect(name: str, t, shape) -> None:
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _strides2(name: str, t):
    """(token, head) strides of a [tokens, heads, dim] operand; a dimension of size one has
    no stride of its own (torch may report any value)."""
    a, b, c = t.stride()
    n, h, d = t.shape
    if c != 1 and d > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return (a if n > 1 else d), (b if h > 1 else d)


def _stride1(name: str, t) -> int:
    """Row stride of a [tokens, dim] operand."""
    a, c = t.stride()
    n, d = t.shape
    if c != 1 and d > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return a if n > 1 else d


def _on(fn: str, stream, dev: int) -> Optional[int]:
    """The stream's handle: ``stream``, or device ``dev``'s current one."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on cuda:{dev}")
        return stream.cuda_stream
    return int(stream)


def _call(fn: str, dev: int, *args) -> None:
    """Call entry point ``fn`` with device ``dev`` current."""
    entry = getattr(_lib or load_library(), fn)
    if _current_device() == dev:
        status = entry(*args)
    else:
        with torch.cuda.device(dev):
            status = entry(*args)
    if status != 0:
        raise MlaError(fn, status)


def mla_page_map(kv_lens, new_lens, block_table, free_pages, qo_indptr, kv_indptr, kv_indices, slots,
                 positions, pages_used, stream=None, *, page_size: int, num_pages: int,
                 workspace) -> None:
    """Tables and maps of one step from the rows' lengths (see the C header).

    ``kv_lens``/``new_lens`` int32 [B] (cached tokens, and tokens this step adds),
    ``block_table`` int32 [B, max_pages] (rows may be strided; new pages are filled
    in from ``free_pages`` int32 [F] or None), then the outputs: ``qo_indptr``,
    ``kv_indptr`` int32 [B + 1], ``kv_indices`` int32, ``slots`` and ``positions``
    int32 of one length (or both None), ``pages_used`` int32 [1].  ``workspace``:
    STEP_WORKSPACE_BYTES, zeroed once; errors are read by mla_decode_read_error."""
    dev = _device_of(kv_lens, "kv_lens")
    p_len = _ptr(kv_lens, "kv_lens", _I32T, dev)
    p_new = _ptr(new_lens, "new_lens", _I32T, dev)
    p_table = _view_ptr(block_table, "block_table", _I32T, dev)
    p_free = None if free_pages is None else _ptr(free_pages, "free_pages", _I32T, dev)
    p_qo = _ptr(qo_indptr, "qo_indptr", _I32T, dev)
    p_kv = _ptr(kv_indptr, "kv_indptr", _I32T, dev)
    p_idx = _ptr(kv_indices, "kv_indices", _I32T, dev)
    p_slots = None if slots is None else _ptr(slots, "slots", _I32T, dev)
    p_pos = None if positions is None else _ptr(positions, "positions", _I32T, dev)
    p_used = _ptr(pages_used, "pages_used", _I32T, dev)
    p_ws = _workspace(workspace, dev)
    b = kv_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != b:
        raise ValueError(f"block_table must be [{b}, max_pages], got {list(block_table.shape)}")
    if (new_lens.numel() != b or qo_indptr.numel() != b + 1 or kv_indptr.numel() != b + 1
            or pages_used.numel() != 1):
        raise ValueError("new_lens must hold B entries, the indptrs B + 1, pages_used one")
    n_slots = 0 if slots is None else slots.numel()
    if n_slots != (0 if positions is None else positions.numel()):
        raise ValueError("slots and positions must have one length")
    width = block_table.shape[1]
    row = _stride1("block_table", block_table)
    if row < width:
        raise ValueError("block_table's rows must not overlap")
    _call("mla_page_map", dev, p_len, p_new, b, p_table, row, width, page_size, num_pages, p_free,
          0 if free_pages is None else free_pages.numel(), p_qo, p_kv, p_idx, kv_indices.numel(),
          p_slots, p_pos, n_slots, p_used, p_ws, workspace.nbytes, _on("mla_page_map", stream, dev))


def _append(fn, kv, norm_weight, rope_table, positions, slots, cache, kv_scale, stream, workspace,
            eps, interleaved, q_pe, q_out, latent_out):
    dev = _device_of(kv, "kv")
    rows = cache.shape
    if len(rows) not in (2, 3) or rows[-1] != QK_HEAD_DIM or len(rows) == 3 and rows[1] != 1:
        raise ValueError(f"the cache must be [rows, 576] or [rows, 1, 576], got {list(rows)}")
    p_kv = _view_ptr(kv, "kv", _BF16, dev)
    p_weight = _ptr(norm_weight, "norm_weight", _BF16, dev)
    p_table = _ptr(rope_table, "rope_table", _F32T, dev)
    p_pos = _ptr(positions, "positions", _I32T, dev)
    p_slots = _ptr(slots, "slots", _I32T, dev)
    p_cache = _ptr(cache, "cache", cache.dtype, dev)
    scale = () if kv_scale is None else (_ptr(kv_scale, "kv_scale", _F32T, dev),)
    p_dense = None if latent_out is None else _ptr(latent_out, "latent_out", _BF16, dev)
    p_ws = _workspace(workspace, dev)
    shape, table = kv.shape, rope_table.shape
    if len(shape) != 2 or shape[1] != QK_HEAD_DIM:
        raise ValueError(f"kv must be [tokens, {QK_HEAD_DIM}], got {list(shape)}")
    if len(table) != 2 or table[1] != ROPE_DIM:
        raise ValueError(f"rope_table must be [positions, {ROPE_DIM}], got {list(table)}")
    t = shape[0]
    if norm_weight.numel() != V_HEAD_DIM or positions.numel() != t or slots.numel() != t:
        raise ValueError("norm_weight must hold 512 values, positions and slots one entry a token")
    if latent_out is not None:
        _expect("latent_out", latent_out, (t, QK_HEAD_DIM))
    if (q_pe is None) != (q_out is None):
        raise ValueError("q_pe and q_out come together")
    if q_pe is None:
        queries = (None, 0, 0, None, 0, 0, 0)
    else:
        p_q, p_out = _view_ptr(q_pe, "q_pe", _BF16, dev), _view_ptr(q_out, "q_out", _BF16, dev)
        shape = q_pe.shape
        if len(shape) != 3 or shape[0] != t or shape[2] != ROPE_DIM:
            raise ValueError(f"q_pe must be [{t}, heads, {ROPE_DIM}], got {list(shape)}")
        _expect("q_out", q_out, shape)
        queries = (p_q, *_strides2("q_pe", q_pe), p_out, *_strides2("q_out", q_out), shape[1])
    _call(fn, dev, p_kv, _stride1("kv", kv), p_weight, eps, p_table, table[0],
          1 if interleaved else 0, p_pos, p_slots, t, p_cache, *scale, rows[0], p_dense,
          *queries, p_ws, workspace.nbytes, _on(fn, stream, dev))


def mla_kv_append(kv, norm_weight, rope_table, positions, slots, kv_fp8, kv_scale, stream=None, *,
                  workspace, eps: float = 1e-6, interleaved: bool = True, q_pe=None, q_out=None,
                  latent_out=None) -> None:
    """New tokens into an e4m3 cache: norm of the latent, rotation of the key (and of
    the queries), quantisation, scatter (see the C header).

    ``kv`` bf16 [T, 576] (rows may be strided), ``norm_weight`` bf16 [512], ``rope_table``
    float32 [positions, 64] (cos | sin of 32 pairs), ``positions``/``slots`` int32 [T]
    (a negative slot skips the token), ``kv_fp8`` [rows, 576], ``kv_scale`` float32 [1];
    ``q_pe`` -> ``q_out`` bf16 [T, H, 64] (strided; may be one tensor), ``latent_out``
    bf16 [T, 576].  ``workspace``: STEP_WORKSPACE_BYTES, zeroed once."""
    if kv_scale is not None and not isinstance(kv_scale, _Tensor):
        _refuse(kv_scale, "kv_scale", _F32T, None)
    if kv_scale is None or kv_scale.numel() != 1:
        raise ValueError("kv_scale must be one float32")
    if not isinstance(kv_fp8, _Tensor) or kv_fp8.dtype not in _E4M3_CODES:
        _e4m3_cache(kv_fp8)  # says what is wrong
    _append("mla_kv_append", kv, norm_weight, rope_table, positions, slots, kv_fp8,
            kv_scale, stream, workspace, eps, interleaved, q_pe, q_out, latent_out)


def mla_kv_append_bf16kv(kv, norm_weight, rope_table, positions, slots, kv_bf16, stream=None, *,
                         workspace, eps: float = 1e-6, interleaved: bool = True, q_pe=None,
                         q_out=None, latent_out=None) -> None:
    """mla_kv_append into a bf16 cache ``[rows, 576]`` (no scale)."""
    if not isinstance(kv_bf16, _Tensor) or kv_bf16.dtype is not _BF16:
        raise TypeError("kv_bf16 must be a bfloat16 CUDA tensor")
    _append("mla_kv_append_bf16kv", kv, norm_weight, rope_table, positions, slots, kv_bf16, None,
            stream, workspace, eps, interleaved, q_pe, q_out, latent_out)


def mla_prefill_plan(batch: int, total_q: int, max_kv_len: int, num_heads: int = NUM_HEADS,
                     num_sms: int = 0) -> mla_prefill_plan_t:
    """Plan of mla_prefill_fwd for ``batch`` rows with ``total_q`` query tokens in all."""
    plan = mla_prefill_plan_t()
    _check("mla_prefill_plan", load_library().mla_prefill_plan(batch, total_q, max_kv_len, num_heads,
                                                              num_sms, ctypes.byref(plan)))
    return plan


def _prefill(fn, q, k_nope, k_rope, v, qo_indptr, kv_indptr, out, stream, plan, workspace, scale,
             causal, lse):
    dev = _device_of(q, "q")
    p_q, p_kn = _view_ptr(q, "q", _BF16, dev), _view_ptr(k_nope, "k_nope", _BF16, dev)
    p_kr, p_v = _view_ptr(k_rope, "k_rope", _BF16, dev), _view_ptr(v, "v", _BF16, dev)
    p_qo = _ptr(qo_indptr, "qo_indptr", _I32T, dev)
    p_kv = _ptr(kv_indptr, "kv_indptr", _I32T, dev)
    p_out = _ptr(out, "out", _BF16, dev)
    p_lse = None if lse is None else _ptr(lse, "lse", _F32T, dev)
    p_ws = _workspace(workspace, dev)
    t, h, b = plan.total_q, plan.num_heads, plan.batch
    n = k_nope.shape[0] if k_nope.shape else 0
    _expect("q", q, (t, h, PREFILL_QK_DIM))
    _expect("k_nope", k_nope, (n, h, PREFILL_NOPE_DIM))
    _expect("k_rope", k_rope, (n, PREFILL_QK_DIM - PREFILL_NOPE_DIM))
    _expect("v", v, (n, h, PREFILL_V_DIM))
    _expect("out", out, (t, h, PREFILL_V_DIM))
    if lse is not None:
        _expect("lse", lse, (t, h))
    if qo_indptr.numel() != b + 1 or kv_indptr.numel() != b + 1:
        raise ValueError("qo_indptr and kv_indptr must hold plan.batch + 1 entries")
    _call(fn, dev, p_q, *_strides2("q", q), p_kn, *_strides2("k_nope", k_nope), p_kr,
          _stride1("k_rope", k_rope), p_v, *_strides2("v", v), n, p_qo, p_kv,
          PREFILL_QK_DIM ** -0.5 if scale is None else scale, 1 if causal else 0, p_out, p_lse,
          _on(fn, stream, dev), ctypes.byref(plan), p_ws, workspace.nbytes)


def mla_prefill_fwd(q, k_nope, k_rope, v, qo_indptr, kv_indptr, out, stream=None, *, plan, workspace,
                    scale: Optional[float] = None, causal: bool = True, lse=None) -> torch.Tensor:
    """Attention of prompts in the expanded form (see the C header); writes and returns ``out``.

    ``q`` bf16 [total_q, H, 192], ``k_nope`` and ``v`` bf16 [tokens, H, 128], ``k_rope`` bf16
    [tokens, 64] (all may be strided views with a dense last dimension), ``out`` bf16
    [total_q, H, 128], ``lse`` float32 [total_q, H] or None; ``scale`` defaults to 192 ** -0.5."""
    _prefill("mla_prefill_fwd", q, k_nope, k_rope, v, qo_indptr, kv_indptr, out, stream, plan,
             workspace, scale, causal, lse)
    return out


def mla_prefill_fwd_stall_stream(q, k_nope, k_rope, v, qo_indptr, kv_indptr, out, stream=None, *,
                                 plan, workspace, scale: Optional[float] = None,
                                 causal: bool = True, lse=None) -> None:
    """Test hook: the launch of mla_prefill_fwd with copies that never arrive, so that the
    bounded waits run out and the call reports MLA_DERR_TIMEOUT."""
    _prefill("mla_prefill_fwd_stall_stream", q, k_nope, k_rope, v, qo_indptr, kv_indptr, out, stream,
             plan, workspace, scale, causal, lse)


def mla_attn_merge(parts, lses, out, stream=None, *, lse_out=None) -> torch.Tensor:
    """Join attention over disjoint keys: ``parts`` bf16 [S, ..., dim] with natural
    log-sum-exps ``lses`` float32 [S, ...] into ``out`` bf16 [..., dim] (and ``lse_out``
    float32 [...]); returns ``out`` (see the C header)."""
    dev = _device_of(parts, "parts")
    p_parts, p_lses = _ptr(parts, "parts", _BF16, dev), _ptr(lses, "lses", _F32T, dev)
    p_out = _ptr(out, "out", _BF16, dev)
    p_lse = None if lse_out is None else _ptr(lse_out, "lse_out", _F32T, dev)
    shape = parts.shape
    if len(shape) < 2 or lses.shape != shape[:-1] or out.shape != shape[1:]:
        raise ValueError("parts must be [S, ..., dim], lses [S, ...], out [..., dim]")
    if lse_out is not None and lse_out.shape != shape[1:-1]:
        raise ValueError("lse_out must have one entry a row")
    _call("mla_attn_merge", dev, p_parts, p_lses, shape[0], shape[1:-1].numel(), shape[-1], p_out, p_lse,
          _on("mla_attn_merge", stream, dev))
    return out


# ---------------------------------------------------------------- decode steps over long contexts
def mla_shared_plan(batch: int, total_q: int, max_kv_len: int, num_sms: int = 0) -> mla_shared_plan_t:
    """Plan of mla_shared_fwd for ``batch`` groups with ``total_q`` query tokens in all."""
    plan = mla_shared_plan_t()
    _check("mla_shared_plan", load_library().mla_shared_plan(batch, total_q, max_kv_len, num_sms,
                                                            ctypes.byref(plan)))
    return plan


def _cache_rows(cache, name: str, dtypes) -> int:
    """Rows of a cache [rows, 576] or [rows, 1, 576] of one of ``dtypes``."""
    if not isinstance(cache, _Tensor) or cache.dtype not in dtypes:
        raise TypeError(f"{name} must be a CUDA tensor of {' or '.join(map(str, dtypes))}")
    shape = cache.shape
    if len(shape) not in (2, 3) or shape[-1] != QK_HEAD_DIM or len(shape) == 3 and shape[1] != 1:
        raise ValueError(f"{name} must be [rows, 576] or [rows, 1, 576], got {list(shape)}")
    return shape[0]


def _scale_ptr(kv_scale, dev: int) -> int:
    p = _ptr(kv_scale, "kv_scale", _F32T, dev)
    if kv_scale.numel() != 1:
        raise ValueError("kv_scale must be one float32")
    return p


def _shared(fn, q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan, workspace, kv_indices, lse):
    dev = _device_of(q, "q")
    rows = _cache_rows(kv_fp8, "kv_fp8", _E4M3_CODES)
    p_q, p_kv = _ptr(q, "q", _BF16, dev), _ptr(kv_fp8, "kv_fp8", kv_fp8.dtype, dev)
    p_scale = _scale_ptr(kv_scale, dev)
    p_qo, p_ki = _ptr(qo_indptr, "qo_indptr", _I32T, dev), _ptr(kv_indptr, "kv_indptr", _I32T, dev)
    p_out = _ptr(out, "out", _BF16, dev)
    p_idx = None if kv_indices is None else _ptr(kv_indices, "kv_indices", _I32T, dev)
    p_lse = None if lse is None else _ptr(lse, "lse", _F32T, dev)
    p_ws = _workspace(workspace, dev)
    t, b = plan.total_q, plan.batch
    _expect("q", q, (t, NUM_HEADS, QK_HEAD_DIM))
    _expect("out", out, (t, NUM_HEADS, V_HEAD_DIM))
    if lse is not None:
        _expect("lse", lse, (t, NUM_HEADS))
    if qo_indptr.numel() != b + 1 or kv_indptr.numel() != b + 1:
        raise ValueError("qo_indptr and kv_indptr must hold plan.batch + 1 entries")
    _call(fn, dev, p_q, p_kv, p_scale, p_qo, p_ki, p_out, p_lse, _on(fn, stream, dev), ctypes.byref(plan),
          p_idx, 0 if kv_indices is None else kv_indices.numel(), rows, p_ws, workspace.nbytes)


def mla_shared_fwd(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream=None, *, plan, workspace,
                   kv_indices=None, lse=None) -> torch.Tensor:
    """Attention of groups of decode queries over keys that their whole group sees, for
    instance a prefix that a batch shares (see the C header); writes and returns ``out``.

    ``q`` bf16 [total_q, 16, 576], ``kv_fp8`` [rows, 576], ``qo_indptr``/``kv_indptr`` int32
    [groups + 1], ``out`` bf16 [total_q, 16, 512], ``lse`` float32 [total_q, 16] or None,
    ``kv_indices`` int32 cache rows of the groups' keys, or None where they are the rows
    themselves."""
    _shared("mla_shared_fwd", q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan, workspace,
            kv_indices, lse)
    return out


def mla_shared_fwd_stall_stream(q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream=None, *, plan,
                                workspace, kv_indices=None, lse=None) -> None:
    """Test hook: the launch of mla_shared_fwd with copies that never arrive, so that the
    bounded waits run out and the call reports MLA_DERR_TIMEOUT."""
    _shared("mla_shared_fwd_stall_stream", q, kv_fp8, kv_scale, qo_indptr, kv_indptr, out, stream, plan,
            workspace, kv_indices, lse)


def _pages_of(means, dev: int):
    p, shape = _ptr(means, "means", _BF16, dev), means.shape
    if len(shape) != 2 or shape[1] != QK_HEAD_DIM:
        raise ValueError(f"means must be [pages, {QK_HEAD_DIM}], got {list(shape)}")
    return p, shape[0]


def _means(fn, cache, rows, scale, slots, means, stream, page_size, workspace, dev):
    p_cache = _ptr(cache, "the cache", cache.dtype, dev)
    p_slots, p_ws = _ptr(slots, "slots", _I32T, dev), _workspace(workspace, dev)
    p_means, pages = _pages_of(means, dev)
    _call(fn, dev, p_cache, *scale, rows, p_slots, slots.numel(), p_means, pages, page_size, p_ws,
          workspace.nbytes, _on(fn, stream, dev))


def mla_block_means(kv_fp8, kv_scale, slots, means, stream=None, *, page_size: int, workspace) -> None:
    """The mean cache row of every page that ``slots`` (int32 [T], as mla_kv_append took them)
    wrote to, into ``means`` bf16 [pages, 576]; other pages' means are left alone (see the C
    header).  ``workspace``: STEP_WORKSPACE_BYTES, zeroed once."""
    rows = _cache_rows(kv_fp8, "kv_fp8", _E4M3_CODES)
    dev = _device_of(kv_fp8, "kv_fp8")
    _means("mla_block_means", kv_fp8, rows, (_scale_ptr(kv_scale, dev),), slots, means, stream, page_size,
           workspace, dev)


def mla_block_means_bf16kv(kv_bf16, slots, means, stream=None, *, page_size: int, workspace) -> None:
    """mla_block_means of a bf16 cache ``[rows, 576]`` (no scale)."""
    rows = _cache_rows(kv_bf16, "kv_bf16", (_BF16,))
    _means("mla_block_means_bf16kv", kv_bf16, rows, (), slots, means, stream, page_size, workspace,
           _device_of(kv_bf16, "kv_bf16"))


def _rows_of(name: str, t, dtype, dev: int, batch: int):
    """Address, row stride and width of a [batch, width] operand with dense rows."""
    p, shape = _view_ptr(t, name, dtype, dev), t.shape
    if len(shape) != 2 or shape[0] != batch:
        raise ValueError(f"{name} must be [{batch}, max_pages], got {list(shape)}")
    width = shape[1]
    row, col = t.stride()
    if col != 1 and width > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    if batch == 1:  # (a dimension of size one has no stride of its own)
        row = width
    if row < width:
        raise ValueError(f"{name}'s rows must not overlap")
    return p, row, width


def mla_block_scores(q, means, block_table, qo_indptr, kv_indptr, scores, stream=None, *, page_size: int,
                     workspace) -> torch.Tensor:
    """The highest product of a row's queries with each of its pages' means, over 24 (see the
    C header); writes and returns ``scores``.

    ``q`` bf16 [T, 16, 576], ``means`` bf16 [pages, 576], ``block_table`` int32 [B, max_pages] and
    ``scores`` float32 [B, max_pages] (rows may be strided), ``qo_indptr``/``kv_indptr`` int32
    [B + 1]; scores behind a row's pages are -inf."""
    dev = _device_of(q, "q")
    p_q, (p_means, pages), shape = _ptr(q, "q", _BF16, dev), _pages_of(means, dev), q.shape
    if len(shape) != 3 or shape[1] != NUM_HEADS or shape[2] != QK_HEAD_DIM:
        raise ValueError(f"q must be [tokens, {NUM_HEADS}, {QK_HEAD_DIM}], got {list(shape)}")
    p_qo, p_kv = _ptr(qo_indptr, "qo_indptr", _I32T, dev), _ptr(kv_indptr, "kv_indptr", _I32T, dev)
    b = kv_indptr.numel() - 1
    if qo_indptr.numel() != b + 1:
        raise ValueError("qo_indptr and kv_indptr must have one length")
    p_table, table_row, width = _rows_of("block_table", block_table, _I32T, dev, b)
    p_scores, scores_row, scores_width = _rows_of("scores", scores, _F32T, dev, b)
    if scores_width != width:
        raise ValueError("block_table and scores must have one width")
    p_ws = _workspace(workspace, dev)
    _call("mla_block_scores", dev, p_q, shape[0], p_means, pages, p_table, table_row, width, p_qo, p_kv, b,
          page_size, p_scores, scores_row, p_ws, workspace.nbytes, _on("mla_block_scores", stream, dev))
    return scores


def mla_block_select(scores, block_table, kv_indptr, sel_indptr, sel_indices, stream=None, *, page_size: int,
                     num_pages: int, blocks: int, sink: int, recent: int, workspace, chosen=None) -> None:
    """The pages that each row attends, as mla_decode_fwd's page table (see the C header): all of
    up to ``blocks`` pages, else the first ``sink``, the last ``recent`` and the highest scores.

    ``scores`` float32 and ``block_table`` int32 [B, max_pages] (rows may be strided), ``kv_indptr``
    int32 [B + 1] of the whole rows, then the outputs: ``sel_indptr`` int32 [B + 1],
    ``sel_indices`` int32, ``chosen`` int32 [B, blocks] or None."""
    dev = _device_of(scores, "scores")
    p_kv = _ptr(kv_indptr, "kv_indptr", _I32T, dev)
    b = kv_indptr.numel() - 1
    p_scores, scores_row, scores_width = _rows_of("scores", scores, _F32T, dev, b)
    p_table, table_row, width = _rows_of("block_table", block_table, _I32T, dev, b)
    if scores_width != width:
        raise ValueError("block_table and scores must have one width")
    p_ptr, p_idx = _ptr(sel_indptr, "sel_indptr", _I32T, dev), _ptr(sel_indices, "sel_indices", _I32T, dev)
    if sel_indptr.numel() != b + 1:
        raise ValueError("sel_indptr must hold one entry a row and one more")
    p_chosen = None if chosen is None else _ptr(chosen, "chosen", _I32T, dev)
    if chosen is not None:
        _expect("chosen", chosen, (b, blocks))
    p_ws = _workspace(workspace, dev)
    _call("mla_block_select", dev, p_scores, scores_row, p_table, table_row, width, p_kv, b, page_size, num_pages,
          blocks, sink, recent, p_ptr, p_idx, sel_indices.numel(), p_chosen, p_ws, workspace.nbytes,
          _on("mla_block_select", stream, dev))


def mla_debug_q_operand(q, kv_scale, tokens_per_cta: int = 1, stream=None):
    """Test hook: stage 1's query operand of an e4m3 cache for every token of
    ``q`` [T, 16, 576]: (codes uint8 [T, 2, 16, 576] = hi then lo, qk_scale float [T])."""
    t = int(q.shape[0])
    codes = torch.empty((t, 2, NUM_HEADS, QK_HEAD_DIM), dtype=torch.uint8, device=q.device)
    qk_scale = torch.empty(t, dtype=torch.float32, device=q.device)
    _check("mla_debug_q_operand", load_library().mla_debug_q_operand(
        _dev_ptr(q, "q", torch.bfloat16), t, int(tokens_per_cta),
        _dev_ptr(kv_scale, "kv_scale", torch.float32), _dev_ptr(codes, "codes"),
        _dev_ptr(qk_scale, "qk_scale"), _stream(stream)))
    return codes, qk_scale


def mla_debug_p_split(p, stream=None):
    """Test hook: stage 1's two-term e4m3 split of float probabilities ``p``
    (numel a multiple of 16): (hi uint8, lo uint8), shaped like ``p``."""
    hi = torch.empty(p.shape, dtype=torch.uint8, device=p.device)
    lo = torch.empty(p.shape, dtype=torch.uint8, device=p.device)
    _check("mla_debug_p_split", load_library().mla_debug_p_split(
        _dev_ptr(p, "p", torch.float32), p.numel(), _dev_ptr(hi, "hi"), _dev_ptr(lo, "lo"),
        _stream(stream)))
    return hi, lo


TRACE_CTAS, TRACE_EVENTS, TRACE2_BLOCKS = 320, 40, 4096


def mla_decode_trace_read(clear: bool = True):
    """Trace builds only: (stage-1 stamps uint64 [TRACE_CTAS, TRACE_EVENTS], stage-2 stamps uint64 [TRACE2_BLOCKS, 3])."""
    import numpy as np
    s1 = np.zeros((TRACE_CTAS, TRACE_EVENTS), dtype=np.uint64)
    s2 = np.zeros((TRACE2_BLOCKS, 3), dtype=np.uint64)
    _check("mla_decode_trace_read", load_library().mla_decode_trace_read(
        s1.ctypes.data, s2.ctypes.data, int(clear)))
    return s1, s2


def mla_decode_workspace_init(workspace, stream=None) -> None:
    _check("mla_decode_workspace_init", load_library().mla_decode_workspace_init(
        _dev_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def mla_decode_read_error(workspace, clear: bool = True, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check("mla_decode_read_error", load_library().mla_decode_read_error(
        _dev_ptr(workspace, "workspace"), ctypes.byref(v), int(clear), _stream(stream)))
    return int(v.value)


def mla_decode_schedule_host(kv_indptr, grid: int):
    """(workers int32 [grid, 4], prefix int32 [B + 1]) from a host kv_indptr."""
    import numpy as np
    ind = np.ascontiguousarray(np.asarray(kv_indptr, dtype=np.int32))
    batch = ind.shape[0] - 1
    workers = np.zeros((grid, 4), dtype=np.int32)
    prefix = np.zeros(batch + 1, dtype=np.int32)
    _check("mla_decode_schedule_host", load_library().mla_decode_schedule_host(
        ind.ctypes.data, batch, grid, workers.ctypes.data, prefix.ctypes.data))
    return workers, prefix


def new_workspace(plan: mla_plan_t, device=None) -> torch.Tensor:
    """A zeroed uint8 workspace of plan.ws_bytes on ``device`` (256-byte aligned)."""
    ws = torch.zeros(int(plan.ws_bytes), dtype=torch.uint8, device=device or "cuda")
    assert ws.data_ptr() % 256 == 0
    return ws


def workspace_views(plan: mla_plan_t, ws: torch.Tensor) -> dict:
    """Typed views of the workspace regions (for tests and tools)."""
    g, b, nq = int(plan.grid), int(plan.batch), int(plan.qo_len)

    def view(off, n, dtype):
        size = torch.tensor([], dtype=dtype).element_size()
        return ws[off:off + n * size].view(dtype)

    return {"err": view(0, 1, torch.int32),
            "prefix": view(plan.ws_prefix_offset, b + 1, torch.int32),
            "workers": view(plan.ws_workers_offset, 8 * g, torch.int32).view(g, 8)[:, :4],
            "jobs": view(plan.ws_workers_offset, 8 * g, torch.int32).view(g, 8)[:, 4:],
            "lse": view(plan.ws_lse_offset, 2 * g * nq * 16, torch.float32).view(2 * g, nq, 16),
            # bf16, stored [slot][token][dim / 128][head / 8][dim % 128][head % 8];
            # viewed as [slot][token][head][dim]
            "partial": view(plan.ws_partial_offset, 2 * g * nq * 16 * 512, torch.bfloat16)
                       .view(2 * g, nq, 4, 2, 128, 8).permute(0, 1, 3, 5, 2, 4)
                       .reshape(2 * g, nq, 16, 512)}
