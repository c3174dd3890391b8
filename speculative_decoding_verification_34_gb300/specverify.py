"""Python binding of libspecverify (argument marshalling only).

Every function here has the name of the C entry point it calls and does nothing but check
tensor types, shapes and devices, take raw device pointers and the current CUDA stream from
PyTorch, and forward them.  All of the verification runs in the library's CUDA kernels; if
the shared library is missing this module raises instead of computing anything itself.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

from . import build as _build

SPEC_BF16 = 0
SPEC_F32 = 1
SPEC_MAX_GAMMA = 32
ST_BAD_DRAFT, ST_R_ZERO, ST_CLAMPED_GAMMA, ST_HISTORY_FULL = 1, 2, 4, 8
ST_TIMEOUT, ST_STOPPED, ST_BAD_TREE, ST_BAD_ROW = 16, 32, 64, 128
ST_BAD_PAGE, ST_BAD_KV = 256, 512

_lib = None


class SpecVerifyError(RuntimeError):
    pass


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def library_path() -> str:
    return _build.LIB


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libspecverify.so (built in-tree by build.build()); raises if it is absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise SpecVerifyError(f"{p} is missing: build it with "
                              "speculative_decoding_verification_34_gb300.build.build()")
    lib = ctypes.CDLL(p)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int
    size_t = ctypes.c_size_t
    lib.spec_verify_greedy.argtypes = [vp, i32, vp, vp, sz, sz, sz, vp, vp, vp, vp, size_t, vp]
    lib.spec_verify_greedy.restype = i32
    lib.spec_verify_sample.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp, vp, size_t, vp]
    lib.spec_verify_sample.restype = i32
    lib.spec_verify_greedy_split.argtypes = [vp, vp, i32, vp, vp, sz, sz, sz, vp, vp, vp, vp, size_t, vp]
    lib.spec_verify_greedy_split.restype = i32
    lib.spec_verify_sample_split.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp, vp,
                                             size_t, vp]
    lib.spec_verify_sample_split.restype = i32
    lib.spec_verify_tree_greedy.argtypes = [vp, i32, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp, vp, size_t, vp]
    lib.spec_verify_sample_truncated.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp,
                                                 vp, size_t, vp]
    lib.spec_verify_sample_truncated.restype = i32
    lib.spec_verify_sample_truncated_split.argtypes = [vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, sz, sz, vp,
                                                       vp, vp, vp, vp, size_t, vp]
    lib.spec_verify_sample_truncated_split.restype = i32
    lib.spec_verify_tree_greedy.restype = i32
    lib.spec_verify_tree_greedy_commit.argtypes = [vp, i32, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp, vp, size_t,
                                                   vp, vp, i32, vp, vp, sz, vp]
    lib.spec_verify_tree_greedy_commit.restype = i32
    lib.spec_verify_sample_static.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp, vp]
    lib.spec_verify_greedy_commit.argtypes = [vp, i32, vp, vp, sz, sz, sz, vp, vp, vp, vp, size_t,
                                              vp, vp, i32, vp, vp, sz, vp]
    lib.spec_verify_greedy_commit.restype = i32
    lib.spec_verify_sample_commit.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, sz, sz, sz, vp, vp, vp, vp, vp,
                                              size_t, vp, vp, i32, vp, vp, sz, vp]
    lib.spec_verify_sample_commit.restype = i32
    lib.spec_verify_sample_truncated_commit.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, sz, sz, vp, vp,
                                                        vp, vp, vp, size_t, vp, vp, i32, vp, vp, sz, vp]
    lib.spec_verify_sample_truncated_commit.restype = i32
    lib.spec_verify_sample_static.restype = i32
    lib.spec_verify_workspace_bytes.argtypes = [sz, sz, sz, i32]
    lib.spec_verify_workspace_bytes.restype = size_t
    lib.spec_commit_kv_lengths.argtypes = [vp, sz, vp, vp, i32, vp, sz, vp, vp, sz, vp, vp]
    lib.spec_commit_kv_lengths.restype = i32
    lib.spec_apply_stops.argtypes = [vp, vp, sz, sz, i32, vp, vp, vp]
    lib.spec_apply_stops.restype = i32
    cp = ctypes.POINTER(_CacheStruct)
    lib.spec_process_logits.argtypes = [vp, vp, i32, sz, sz, i32, sz, vp, vp, vp, sz, vp, vp, vp, sz, vp, vp, vp, vp, vp,
                                        sz, vp, sz, vp, vp]
    lib.spec_process_logits.restype = i32
    lib.spec_kv_append.argtypes = [cp, vp, vp, i32, vp, sz, sz, vp, sz, vp, vp, vp, vp]
    lib.spec_kv_append.restype = i32
    lib.spec_kv_read.argtypes = [cp, vp, sz, vp, vp, sz, sz, vp, vp, i32, vp, vp]
    lib.spec_kv_read.restype = i32
    lib.spec_kv_keep_path.argtypes = [cp, vp, sz, vp, vp, vp, sz, sz, i32, vp, vp]
    lib.spec_kv_keep_path.restype = i32
    lib.spec_verify_attention.argtypes = [cp, vp, i32, vp, sz, sz, i32, sz, vp, sz, vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                          size_t, vp]
    lib.spec_verify_attention.restype = i32
    lib.spec_attention_workspace_bytes.argtypes = [sz, sz, sz, sz, sz]
    lib.spec_attention_workspace_bytes.restype = size_t
    lib.spec_last_error.argtypes = []
    lib.spec_last_error.restype = ctypes.c_char_p
    lib.spec_launch_count.argtypes = []
    lib.spec_launch_count.restype = ctypes.c_uint64
    lib.spec_verify_plan.argtypes = [i32, i32, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    lib.spec_verify_plan.restype = i32
    if path is None:
        _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        msg = load_library().spec_last_error().decode(errors="replace")
        raise SpecVerifyError(f"specverify error {rc}: {msg}")


def _ptr(t: Optional[torch.Tensor], name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    if t.dtype == torch.float32:
        return SPEC_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Context in which the call's stream is the current one.  A workspace allocated in it is filled before the call's kernels
    run, and once dropped is not handed out again but to that stream, behind them."""
    handle = _stream(stream)
    if handle == torch.cuda.current_stream().cuda_stream:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):        # (0 and 1: the legacy default stream)
        stream = torch.cuda.default_stream() if handle in (None, 0, 1) else torch.cuda.ExternalStream(handle)
    return torch.cuda.stream(stream)


def spec_verify_workspace_bytes(B: int, gmax: int, V: int, dtype: int = SPEC_BF16) -> int:
    return int(load_library().spec_verify_workspace_bytes(B, gmax, V, dtype))


def alloc_workspace(B: int, gmax: int, V: int, dtype: int = SPEC_BF16, device=None) -> torch.Tensor:
    """A zero-filled device workspace for verify calls of these sizes (reusable: every call
    returns its counters to zero; one call at a time)."""
    n = spec_verify_workspace_bytes(B, gmax, V, dtype)
    return torch.zeros(max(n, 64), dtype=torch.uint8, device=device or "cuda")


def _ws(workspace, B, gmax, V, code, device, stream):
    if workspace is None:
        with _on(stream):
            workspace = alloc_workspace(B, gmax, V, code, device)
    if workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    return workspace, _ptr(workspace, "workspace"), workspace.numel()


def spec_verify_greedy(target_logits: torch.Tensor, draft_tokens: torch.Tensor,
                       num_draft: Optional[torch.Tensor], out_tokens: torch.Tensor,
                       num_accepted: torch.Tensor, status: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    lib = load_library()
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    _check(lib.spec_verify_greedy(
        _ptr(target_logits, "target_logits"), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def spec_verify_sample(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                       draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor],
                       temperature: torch.Tensor, u_accept: torch.Tensor, u_sample: torch.Tensor,
                       out_tokens: torch.Tensor, num_accepted: torch.Tensor,
                       diag: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    lib = load_library()
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    _check(lib.spec_verify_sample(
        _ptr(target_logits, "target_logits"),
        _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)),
        _ptr(temperature, "temperature", torch.float32, (B,)),
        _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
        _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def _commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len):
    cap = history.shape[1] if history is not None else 0
    return (_ptr(target_kv_len, "target_kv_len", torch.int32, (B,)),
            _ptr(draft_kv_len, "draft_kv_len", torch.int32, (B,)), int(bool(correction_processed)),
            _ptr(history, "history", torch.int32), _ptr(committed_len, "committed_len", torch.int32, (B,)), cap)


def spec_verify_greedy_commit(target_logits: torch.Tensor, draft_tokens: torch.Tensor,
                              num_draft: Optional[torch.Tensor], out_tokens: torch.Tensor,
                              num_accepted: torch.Tensor, target_kv_len: torch.Tensor,
                              draft_kv_len: Optional[torch.Tensor] = None, correction_processed: bool = True,
                              history: Optional[torch.Tensor] = None, committed_len: Optional[torch.Tensor] = None,
                              status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                              stream=None) -> None:
    """spec_verify_greedy and spec_commit_kv_lengths of the same round in one launch."""
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    lib = load_library()
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    _check(lib.spec_verify_greedy_commit(
        _ptr(target_logits, "target_logits"), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn,
        *_commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len),
        _stream(stream)))


def _sample_commit_args(target_logits, draft_logits, draft_tokens, num_draft, temperature, u_accept, u_sample,
                        out_tokens, num_accepted, diag, status, workspace, target_kv_len, draft_kv_len,
                        correction_processed, history, committed_len, stream):
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"),
            _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)),
            _ptr(temperature, "temperature", torch.float32, (B,)),
            _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
            _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn,
            *_commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len),
            _stream(stream))
    return args, ws


def spec_verify_sample_commit(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                              draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor],
                              temperature: torch.Tensor, u_accept: torch.Tensor, u_sample: torch.Tensor,
                              out_tokens: torch.Tensor, num_accepted: torch.Tensor, target_kv_len: torch.Tensor,
                              draft_kv_len: Optional[torch.Tensor] = None, correction_processed: bool = True,
                              history: Optional[torch.Tensor] = None, committed_len: Optional[torch.Tensor] = None,
                              diag: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_sample and spec_commit_kv_lengths of the same round in one launch."""
    args, _ = _sample_commit_args(target_logits, draft_logits, draft_tokens, num_draft, temperature, u_accept,
                                  u_sample, out_tokens, num_accepted, diag, status, workspace, target_kv_len,
                                  draft_kv_len, correction_processed, history, committed_len, stream)
    _check(load_library().spec_verify_sample_commit(*args))


def spec_verify_sample_truncated(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                                 draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor],
                                 temperature: torch.Tensor, top_k: Optional[torch.Tensor],
                                 top_p: Optional[torch.Tensor], u_accept: torch.Tensor, u_sample: torch.Tensor,
                                 out_tokens: torch.Tensor, num_accepted: torch.Tensor,
                                 diag: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_sample on top-k / top-p truncated distributions (top_k int32 [B], top_p
    float32 [B], either None); bf16 logits."""
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    lib = load_library()
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    _check(lib.spec_verify_sample_truncated(
        _ptr(target_logits, "target_logits"),
        _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)),
        _ptr(temperature, "temperature", torch.float32, (B,)),
        _ptr(top_k, "top_k", torch.int32, (B,)), _ptr(top_p, "top_p", torch.float32, (B,)),
        _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
        _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def _truncated_commit_args(target_logits, draft_logits, draft_tokens, num_draft, temperature, top_k, top_p,
                           u_accept, u_sample, out_tokens, num_accepted, diag, status, workspace, target_kv_len,
                           draft_kv_len, correction_processed, history, committed_len, stream):
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"),
            _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)),
            _ptr(temperature, "temperature", torch.float32, (B,)),
            _ptr(top_k, "top_k", torch.int32, (B,)), _ptr(top_p, "top_p", torch.float32, (B,)),
            _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
            _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn,
            *_commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len),
            _stream(stream))
    return args, ws


def spec_verify_sample_truncated_commit(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                                        draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor],
                                        temperature: torch.Tensor, top_k: Optional[torch.Tensor],
                                        top_p: Optional[torch.Tensor], u_accept: torch.Tensor,
                                        u_sample: torch.Tensor, out_tokens: torch.Tensor,
                                        num_accepted: torch.Tensor, target_kv_len: torch.Tensor,
                                        draft_kv_len: Optional[torch.Tensor] = None,
                                        correction_processed: bool = True, history: Optional[torch.Tensor] = None,
                                        committed_len: Optional[torch.Tensor] = None,
                                        diag: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_sample_truncated and spec_commit_kv_lengths of the same round, fused."""
    args, _ = _truncated_commit_args(target_logits, draft_logits, draft_tokens, num_draft, temperature, top_k,
                                     top_p, u_accept, u_sample, out_tokens, num_accepted, diag, status, workspace,
                                     target_kv_len, draft_kv_len, correction_processed, history, committed_len,
                                     stream)
    _check(load_library().spec_verify_sample_truncated_commit(*args))


def spec_verify_sample_truncated_split(saved_logits: torch.Tensor, block_logits: Optional[torch.Tensor],
                                       draft_logits: torch.Tensor, draft_tokens: torch.Tensor,
                                       num_draft: Optional[torch.Tensor], temperature: torch.Tensor,
                                       top_k: Optional[torch.Tensor], top_p: Optional[torch.Tensor],
                                       u_accept: torch.Tensor, u_sample: torch.Tensor, out_tokens: torch.Tensor,
                                       num_accepted: torch.Tensor, diag: Optional[torch.Tensor] = None,
                                       status: Optional[torch.Tensor] = None,
                                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_sample_truncated with target row 0 (saved_logits [B][V]) apart from rows
    1..gmax (block_logits [B][gmax][V])."""
    B, gmax, V = _split_shapes(saved_logits, block_logits)
    if draft_logits.dtype != saved_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    lib = load_library()
    code = _dtype_code(saved_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, saved_logits.device, stream)
    _check(lib.spec_verify_sample_truncated_split(
        _ptr(saved_logits, "saved_logits"), _ptr(block_logits, "block_logits"),
        _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)),
        _ptr(temperature, "temperature", torch.float32, (B,)),
        _ptr(top_k, "top_k", torch.int32, (B,)), _ptr(top_p, "top_p", torch.float32, (B,)),
        _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
        _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def spec_verify_tree_greedy(target_logits: torch.Tensor, node_tokens: torch.Tensor,
                            node_parents: torch.Tensor, num_nodes: Optional[torch.Tensor],
                            out_tokens: torch.Tensor, num_accepted: torch.Tensor,
                            path_nodes: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Greedy verification of draft trees: target_logits [B][nmax+1][V] (row j after node j),
    node_tokens and node_parents [B][nmax] (node j+1's token and parent, parent < j+1)."""
    B, np1, V = target_logits.shape
    nmax = np1 - 1
    lib = load_library()
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, nmax, V, code, target_logits.device, stream)
    _check(lib.spec_verify_tree_greedy(
        _ptr(target_logits, "target_logits"), code,
        _ptr(node_tokens, "node_tokens", torch.int32, (B, nmax)),
        _ptr(node_parents, "node_parents", torch.int32, (B, nmax)),
        _ptr(num_nodes, "num_nodes", torch.int32, (B,)), B, nmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, nmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(path_nodes, "path_nodes", torch.int32, (B, nmax)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def _tree_args(target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted, path_nodes, status,
               workspace, stream):
    B, np1, V = target_logits.shape
    nmax = np1 - 1
    ws, wsp, wsn = _ws(workspace, B, nmax, V, _dtype_code(target_logits), target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"), _dtype_code(target_logits),
            _ptr(node_tokens, "node_tokens", torch.int32, (B, nmax)),
            _ptr(node_parents, "node_parents", torch.int32, (B, nmax)),
            _ptr(num_nodes, "num_nodes", torch.int32, (B,)), B, nmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, nmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(path_nodes, "path_nodes", torch.int32, (B, nmax)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn)
    return args, ws


def spec_verify_tree_greedy_commit(target_logits: torch.Tensor, node_tokens: torch.Tensor,
                                   node_parents: torch.Tensor, num_nodes: Optional[torch.Tensor],
                                   out_tokens: torch.Tensor, num_accepted: torch.Tensor, target_kv_len: torch.Tensor,
                                   draft_kv_len: Optional[torch.Tensor] = None, correction_processed: bool = True,
                                   history: Optional[torch.Tensor] = None,
                                   committed_len: Optional[torch.Tensor] = None,
                                   path_nodes: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_tree_greedy and spec_commit_kv_lengths (gmax = nmax) of the same round, fused."""
    B = target_logits.shape[0]
    args, _ = _tree_args(target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted, path_nodes,
                         status, workspace, stream)
    _check(load_library().spec_verify_tree_greedy_commit(
        *args, *_commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len),
        _stream(stream)))


def prepare_verify_tree_greedy_commit(target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted,
                                      target_kv_len, draft_kv_len=None, correction_processed=True, history=None,
                                      committed_len=None, path_nodes=None, status=None, workspace=None,
                                      stream=None) -> "_Prepared":
    B = target_logits.shape[0]
    args, ws = _tree_args(target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted, path_nodes,
                          status, workspace, stream)
    args = args + _commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len) + \
        (_stream(stream),)
    keep = (target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted, path_nodes, status, ws,
            target_kv_len, draft_kv_len, history, committed_len)
    return _Prepared(load_library().spec_verify_tree_greedy_commit, args, keep)


def prepare_verify_tree_greedy(target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted,
                               path_nodes=None, status=None, workspace=None, stream=None) -> "_Prepared":
    B, np1, V = target_logits.shape
    nmax = np1 - 1
    lib = load_library()
    ws, wsp, wsn = _ws(workspace, B, nmax, V, _dtype_code(target_logits), target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"), _dtype_code(target_logits),
            _ptr(node_tokens, "node_tokens", torch.int32, (B, nmax)),
            _ptr(node_parents, "node_parents", torch.int32, (B, nmax)),
            _ptr(num_nodes, "num_nodes", torch.int32, (B,)), B, nmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, nmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(path_nodes, "path_nodes", torch.int32, (B, nmax)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream))
    keep = (target_logits, node_tokens, node_parents, num_nodes, out_tokens, num_accepted, path_nodes, status, ws)
    return _Prepared(lib.spec_verify_tree_greedy, args, keep)


def _split_shapes(saved_logits, block_logits):
    B, V = saved_logits.shape
    if block_logits is None:
        return B, 0, V
    Bb, gmax, Vb = block_logits.shape
    if (Bb, Vb) != (B, V) or block_logits.dtype != saved_logits.dtype:
        raise ValueError(f"block_logits {tuple(block_logits.shape)} does not match saved_logits {(B, V)}")
    return B, gmax, V


def spec_verify_greedy_split(saved_logits: torch.Tensor, block_logits: Optional[torch.Tensor],
                             draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor],
                             out_tokens: torch.Tensor, num_accepted: torch.Tensor,
                             status: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_greedy with target row 0 (saved_logits [B][V]) apart from rows 1..gmax
    (block_logits [B][gmax][V])."""
    B, gmax, V = _split_shapes(saved_logits, block_logits)
    lib = load_library()
    code = _dtype_code(saved_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, saved_logits.device, stream)
    _check(lib.spec_verify_greedy_split(
        _ptr(saved_logits, "saved_logits"), _ptr(block_logits, "block_logits"), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def spec_verify_sample_split(saved_logits: torch.Tensor, block_logits: Optional[torch.Tensor],
                             draft_logits: torch.Tensor, draft_tokens: torch.Tensor,
                             num_draft: Optional[torch.Tensor], temperature: torch.Tensor,
                             u_accept: torch.Tensor, u_sample: torch.Tensor, out_tokens: torch.Tensor,
                             num_accepted: torch.Tensor, diag: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_sample with target row 0 (saved_logits [B][V]) apart from rows 1..gmax
    (block_logits [B][gmax][V])."""
    B, gmax, V = _split_shapes(saved_logits, block_logits)
    if draft_logits.dtype != saved_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    lib = load_library()
    code = _dtype_code(saved_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, saved_logits.device, stream)
    _check(lib.spec_verify_sample_split(
        _ptr(saved_logits, "saved_logits"), _ptr(block_logits, "block_logits"),
        _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)),
        _ptr(temperature, "temperature", torch.float32, (B,)),
        _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
        _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
        _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream)))


def spec_verify_sample_static(target_logits: torch.Tensor, draft_logits: torch.Tensor,
                              draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor],
                              temperature: torch.Tensor, u_accept: torch.Tensor,
                              u_sample: torch.Tensor, out_tokens: torch.Tensor,
                              num_accepted: torch.Tensor, diag: Optional[torch.Tensor] = None,
                              status: Optional[torch.Tensor] = None, stream=None) -> None:
    """spec_verify_sample on the library's per-device static workspace: allocates nothing.
    Calls on one device share that workspace, so calls that may overlap must be serialised;
    the first call on a device clears it and should come before any stream capture."""
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    if draft_logits.dtype != target_logits.dtype:
        raise TypeError("target and draft logits must have the same dtype")
    lib = load_library()
    code = _dtype_code(target_logits)
    _check(lib.spec_verify_sample_static(
        _ptr(target_logits, "target_logits"),
        _ptr(draft_logits, "draft_logits", None, (B, gmax, V)), code,
        _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
        _ptr(num_draft, "num_draft", torch.int32, (B,)),
        _ptr(temperature, "temperature", torch.float32, (B,)),
        _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
        _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
        _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
        _ptr(status, "status", torch.int32, (B,)), _stream(stream)))


def spec_apply_stops(out_tokens: torch.Tensor, num_accepted: torch.Tensor, eos_id: int,
                     max_new: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Cut each round's emit at its first end token and to the remaining budget, in place."""
    B, gp1 = out_tokens.shape
    lib = load_library()
    _check(lib.spec_apply_stops(
        _ptr(out_tokens, "out_tokens", torch.int32, (B, gp1)),
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)), B, gp1 - 1, int(eos_id),
        _ptr(max_new, "max_new", torch.int32, (B,)),
        _ptr(status, "status", torch.int32, (B,)), _stream(stream)))


def _commit_gmax(out_tokens, gmax):
    if out_tokens is not None:
        g = out_tokens.shape[1] - 1
        if gmax is not None and gmax != g:
            raise ValueError(f"gmax={gmax} disagrees with out_tokens width {g + 1}")
        return g
    if gmax is None:
        raise ValueError("gmax is required when out_tokens is not given")
    return int(gmax)


def spec_commit_kv_lengths(num_accepted: torch.Tensor, target_kv_len: torch.Tensor,
                           draft_kv_len: Optional[torch.Tensor], correction_processed: bool,
                           out_tokens: Optional[torch.Tensor] = None,
                           history: Optional[torch.Tensor] = None,
                           committed_len: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None,
                           gmax: Optional[int] = None) -> None:
    B = num_accepted.shape[0]
    gmax = _commit_gmax(out_tokens, gmax)
    cap = history.shape[1] if history is not None else 0
    lib = load_library()
    _check(lib.spec_commit_kv_lengths(
        _ptr(num_accepted, "num_accepted", torch.int32, (B,)), B,
        _ptr(target_kv_len, "target_kv_len", torch.int32, (B,)),
        _ptr(draft_kv_len, "draft_kv_len", torch.int32, (B,)), int(bool(correction_processed)),
        _ptr(out_tokens, "out_tokens", torch.int32), gmax,
        _ptr(history, "history", torch.int32), _ptr(committed_len, "committed_len", torch.int32, (B,)),
        cap, _ptr(status, "status", torch.int32, (B,)), _stream(stream)))


def spec_launch_count() -> int:
    return int(load_library().spec_launch_count())


def spec_verify_plan(V: int, dtype: int = SPEC_BF16):
    """(blocks per sequence, vocabulary ids per block) a verify call uses for this V."""
    cl, ch = ctypes.c_int(), ctypes.c_int()
    _check(load_library().spec_verify_plan(V, dtype, ctypes.byref(cl), ctypes.byref(ch)))
    return cl.value, ch.value


class _Prepared:
    """A verify/commit call whose arguments were checked and marshalled once; calling it
    re-issues the same C call (same buffers, same stream) with no per-call Python checks."""

    def __init__(self, fn, args, keep):
        self._fn, self._args, self._keep = fn, args, keep

    def __call__(self):
        _check(self._fn(*self._args))


def prepare_verify_sample(target_logits, draft_logits, draft_tokens, num_draft, temperature,
                          u_accept, u_sample, out_tokens, num_accepted, diag=None, status=None,
                          workspace=None, stream=None) -> _Prepared:
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    lib = load_library()
    ws, wsp, wsn = _ws(workspace, B, gmax, V, _dtype_code(target_logits), target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"),
            _ptr(draft_logits, "draft_logits", target_logits.dtype, (B, gmax, V)),
            _dtype_code(target_logits),
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)),
            _ptr(temperature, "temperature", torch.float32, (B,)),
            _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
            _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream))
    keep = (target_logits, draft_logits, draft_tokens, num_draft, temperature, u_accept,
            u_sample, out_tokens, num_accepted, diag, status, ws)
    return _Prepared(lib.spec_verify_sample, args, keep)


def prepare_verify_greedy_commit(target_logits, draft_tokens, num_draft, out_tokens, num_accepted, target_kv_len,
                                 draft_kv_len=None, correction_processed=True, history=None, committed_len=None,
                                 status=None, workspace=None, stream=None) -> _Prepared:
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    code = _dtype_code(target_logits)
    ws, wsp, wsn = _ws(workspace, B, gmax, V, code, target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"), code,
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)), B, gmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn,
            *_commit_args(B, target_kv_len, draft_kv_len, correction_processed, history, committed_len),
            _stream(stream))
    keep = (target_logits, draft_tokens, num_draft, out_tokens, num_accepted, status, ws, target_kv_len,
            draft_kv_len, history, committed_len)
    return _Prepared(load_library().spec_verify_greedy_commit, args, keep)


def prepare_verify_sample_commit(target_logits, draft_logits, draft_tokens, num_draft, temperature, u_accept,
                                 u_sample, out_tokens, num_accepted, target_kv_len, draft_kv_len=None,
                                 correction_processed=True, history=None, committed_len=None, diag=None,
                                 status=None, workspace=None, stream=None) -> _Prepared:
    args, ws = _sample_commit_args(target_logits, draft_logits, draft_tokens, num_draft, temperature, u_accept,
                                   u_sample, out_tokens, num_accepted, diag, status, workspace, target_kv_len,
                                   draft_kv_len, correction_processed, history, committed_len, stream)
    keep = (target_logits, draft_logits, draft_tokens, num_draft, temperature, u_accept, u_sample, out_tokens,
            num_accepted, diag, status, ws, target_kv_len, draft_kv_len, history, committed_len)
    return _Prepared(load_library().spec_verify_sample_commit, args, keep)


def prepare_verify_sample_truncated(target_logits, draft_logits, draft_tokens, num_draft, temperature, top_k,
                                    top_p, u_accept, u_sample, out_tokens, num_accepted, diag=None, status=None,
                                    workspace=None, stream=None) -> _Prepared:
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    lib = load_library()
    ws, wsp, wsn = _ws(workspace, B, gmax, V, _dtype_code(target_logits), target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"),
            _ptr(draft_logits, "draft_logits", target_logits.dtype, (B, gmax, V)),
            _dtype_code(target_logits),
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)),
            _ptr(temperature, "temperature", torch.float32, (B,)),
            _ptr(top_k, "top_k", torch.int32, (B,)), _ptr(top_p, "top_p", torch.float32, (B,)),
            _ptr(u_accept, "u_accept", torch.float32, (B, gmax)),
            _ptr(u_sample, "u_sample", torch.float32, (B,)), B, gmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(diag, "diag", torch.float32, (B, 2 * gmax + 1)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream))
    keep = (target_logits, draft_logits, draft_tokens, num_draft, temperature, top_k, top_p, u_accept,
            u_sample, out_tokens, num_accepted, diag, status, ws)
    return _Prepared(lib.spec_verify_sample_truncated, args, keep)


def prepare_verify_sample_truncated_commit(target_logits, draft_logits, draft_tokens, num_draft, temperature,
                                           top_k, top_p, u_accept, u_sample, out_tokens, num_accepted,
                                           target_kv_len, draft_kv_len=None, correction_processed=True,
                                           history=None, committed_len=None, diag=None, status=None,
                                           workspace=None, stream=None) -> _Prepared:
    args, ws = _truncated_commit_args(target_logits, draft_logits, draft_tokens, num_draft, temperature, top_k,
                                      top_p, u_accept, u_sample, out_tokens, num_accepted, diag, status, workspace,
                                      target_kv_len, draft_kv_len, correction_processed, history, committed_len,
                                      stream)
    keep = (target_logits, draft_logits, draft_tokens, num_draft, temperature, top_k, top_p, u_accept, u_sample,
            out_tokens, num_accepted, diag, status, ws, target_kv_len, draft_kv_len, history, committed_len)
    return _Prepared(load_library().spec_verify_sample_truncated_commit, args, keep)


def prepare_verify_greedy(target_logits, draft_tokens, num_draft, out_tokens, num_accepted,
                          status=None, workspace=None, stream=None) -> _Prepared:
    B, gp1, V = target_logits.shape
    gmax = gp1 - 1
    lib = load_library()
    ws, wsp, wsn = _ws(workspace, B, gmax, V, _dtype_code(target_logits), target_logits.device, stream)
    args = (_ptr(target_logits, "target_logits"), _dtype_code(target_logits),
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)), B, gmax, V,
            _ptr(out_tokens, "out_tokens", torch.int32, (B, gmax + 1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)),
            _ptr(status, "status", torch.int32, (B,)), wsp, wsn, _stream(stream))
    keep = (target_logits, draft_tokens, num_draft, out_tokens, num_accepted, status, ws)
    return _Prepared(lib.spec_verify_greedy, args, keep)


def prepare_apply_stops(out_tokens, num_accepted, eos_id, max_new=None, status=None, stream=None) -> _Prepared:
    B, gp1 = out_tokens.shape
    lib = load_library()
    args = (_ptr(out_tokens, "out_tokens", torch.int32, (B, gp1)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)), B, gp1 - 1, int(eos_id),
            _ptr(max_new, "max_new", torch.int32, (B,)), _ptr(status, "status", torch.int32, (B,)),
            _stream(stream))
    return _Prepared(lib.spec_apply_stops, args, (out_tokens, num_accepted, max_new, status))


def prepare_commit_kv_lengths(num_accepted, target_kv_len, draft_kv_len, correction_processed,
                              out_tokens=None, history=None, committed_len=None, status=None,
                              stream=None, gmax=None) -> _Prepared:
    B = num_accepted.shape[0]
    gmax = _commit_gmax(out_tokens, gmax)
    cap = history.shape[1] if history is not None else 0
    lib = load_library()
    args = (_ptr(num_accepted, "num_accepted", torch.int32, (B,)), B,
            _ptr(target_kv_len, "target_kv_len", torch.int32, (B,)),
            _ptr(draft_kv_len, "draft_kv_len", torch.int32, (B,)), int(bool(correction_processed)),
            _ptr(out_tokens, "out_tokens", torch.int32), gmax, _ptr(history, "history", torch.int32),
            _ptr(committed_len, "committed_len", torch.int32, (B,)), cap,
            _ptr(status, "status", torch.int32, (B,)), _stream(stream))
    keep = (num_accepted, target_kv_len, draft_kv_len, out_tokens, history, committed_len, status)
    return _Prepared(lib.spec_commit_kv_lengths, args, keep)


def _one_device(*tensors):
    """The tensors of a call are on the current device: kernels run there, on its current stream."""
    for t in tensors:
        if t is not None and t.is_cuda and t.device.index != torch.cuda.current_device():
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _strided(t: torch.Tensor, name: str, shape, dtype=None):
    """Pointer and strides of a tensor whose last dimension is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    # a dimension of one entry has no stride of its own
    return t.data_ptr(), [st if n > 1 else 0 for st, n in zip(t.stride()[:-1], t.shape[:-1])]


def _process_logits_args(logits, out, history, committed_len, prompt_len, draft_tokens, num_draft, node_parents,
                         repetition, frequency, presence, bias_ids, bias_values, allowed, first_row, status, stream):
    B, rows, V = logits.shape
    gmax = draft_tokens.shape[1]
    cap = history.shape[1] if history is not None else 0
    nbias = bias_ids.shape[1] if bias_ids is not None else 0
    words = allowed.shape[-1] if allowed is not None else 0
    keep = (logits, out, history, committed_len, prompt_len, draft_tokens, num_draft, node_parents, repetition, frequency,
            presence, bias_ids, bias_values, allowed, status)
    _one_device(*keep)
    args = (_ptr(logits, "logits"), _ptr(out, "out", logits.dtype, (B, rows, V)), _dtype_code(logits), B, rows,
            int(first_row), V, _ptr(history, "history", torch.int32, (B, cap)),
            _ptr(committed_len, "committed_len", torch.int32, (B,)), _ptr(prompt_len, "prompt_len", torch.int32, (B,)), cap,
            _ptr(draft_tokens, "draft_tokens", torch.int32, (B, gmax)), _ptr(num_draft, "num_draft", torch.int32, (B,)),
            _ptr(node_parents, "node_parents", torch.int32, (B, gmax)), gmax,
            _ptr(repetition, "repetition", torch.float32, (B,)), _ptr(frequency, "frequency", torch.float32, (B,)),
            _ptr(presence, "presence", torch.float32, (B,)), _ptr(bias_ids, "bias_ids", torch.int32, (B, nbias)),
            _ptr(bias_values, "bias_values", torch.float32, (B, nbias)), nbias,
            _ptr(allowed, "allowed", torch.int32, (B, rows, words)), words,
            _ptr(status, "status", torch.int32, (B,)), _stream(stream))
    return args, keep


def spec_process_logits(logits: torch.Tensor, out: torch.Tensor, history: Optional[torch.Tensor],
                        committed_len: Optional[torch.Tensor], prompt_len: Optional[torch.Tensor],
                        draft_tokens: torch.Tensor, num_draft: Optional[torch.Tensor] = None,
                        node_parents: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                        frequency: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                        bias_ids: Optional[torch.Tensor] = None, bias_values: Optional[torch.Tensor] = None,
                        allowed: Optional[torch.Tensor] = None, first_row: int = 0,
                        status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Penalties, biases and grammar masks (int32 bit words [B, rows, words]) on a block's logits
    [B, rows, V], into `out` (which may be `logits`)."""
    args, _ = _process_logits_args(logits, out, history, committed_len, prompt_len, draft_tokens, num_draft, node_parents,
                                   repetition, frequency, presence, bias_ids, bias_values, allowed, first_row, status,
                                   stream)
    _check(load_library().spec_process_logits(*args))


def prepare_process_logits(logits, out, history, committed_len, prompt_len, draft_tokens, num_draft=None,
                           node_parents=None, repetition=None, frequency=None, presence=None, bias_ids=None,
                           bias_values=None, allowed=None, first_row=0, status=None, stream=None) -> _Prepared:
    args, keep = _process_logits_args(logits, out, history, committed_len, prompt_len, draft_tokens, num_draft,
                                      node_parents, repetition, frequency, presence, bias_ids, bias_values, allowed,
                                      first_row, status, stream)
    return _Prepared(load_library().spec_process_logits, args, keep)


class KVCache:
    """A paged 8-bit KV cache: codes [pages, kv_heads, page_size, head_dim] (uint8, e4m3) and exponents
    [pages, kv_heads] (int8) of K and of V; value = code * 2^exponent."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_exp: torch.Tensor, v_exp: torch.Tensor):
        if k_codes.dim() != 4:
            raise ValueError(f"codes must have shape [pages, kv_heads, page_size, head_dim], got {tuple(k_codes.shape)}")
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = shape = tuple(k_codes.shape)
        self.k_codes, self.v_codes, self.k_exp, self.v_exp = k_codes, v_codes, k_exp, v_exp
        self._struct = _CacheStruct(
            _ptr(k_codes, "k_codes", torch.uint8, shape), _ptr(v_codes, "v_codes", torch.uint8, shape),
            _ptr(k_exp, "k_exp", torch.int8, shape[:2]), _ptr(v_exp, "v_exp", torch.int8, shape[:2]), *shape)
        self.tensors = (k_codes, v_codes, k_exp, v_exp)
        if len({t.device for t in self.tensors}) > 1:
            raise ValueError("the cache's arrays must be on one device")


def alloc_kv_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device=None) -> KVCache:
    """An empty cache (its memory is not initialised: no call reads an entry before it is written)."""
    codes = [torch.empty(num_pages, kv_heads, page_size, head_dim, dtype=torch.uint8, device=device or "cuda")
             for _ in range(2)]
    exps = [torch.empty(num_pages, kv_heads, dtype=torch.int8, device=device or "cuda") for _ in range(2)]
    return KVCache(*codes, *exps)


def _table_args(cache, page_table, B):
    _one_device(*cache.tensors, page_table)
    return _ptr(page_table, "page_table", torch.int32, (B, page_table.shape[1])), page_table.shape[1]


def _kv_append_args(k, v, cache, page_table, kv_len, num_new, status, stream):
    B, n = k.shape[:2]
    shape = (B, n, cache.kv_heads, cache.head_dim)
    kp, ks = _strided(k, "k", shape)
    vp, vs = _strided(v, "v", shape, k.dtype)
    strides = (ctypes.c_int64 * 6)(*ks, *vs)
    keep = (k, v, cache, page_table, kv_len, num_new, status, strides)
    _one_device(k, v, kv_len, num_new, status)
    args = (ctypes.byref(cache._struct), kp, vp, _dtype_code(k), strides, B, n, *_table_args(cache, page_table, B),
            _ptr(kv_len, "kv_len", torch.int32, (B,)), _ptr(num_new, "num_new", torch.int32, (B,)),
            _ptr(status, "status", torch.int32, (B,)), _stream(stream))
    return args, keep


def spec_kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_len: torch.Tensor,
                   num_new: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise k, v [B, n, kv_heads, head_dim] (strided views allowed) into the cache from position kv_len on."""
    args, keep = _kv_append_args(k, v, cache, page_table, kv_len, num_new, status, stream)
    _check(load_library().spec_kv_append(*args))


def prepare_kv_append(k, v, cache, page_table, kv_len, num_new=None, status=None, stream=None) -> _Prepared:
    return _Prepared(load_library().spec_kv_append,
                     *_kv_append_args(k, v, cache, page_table, kv_len, num_new, status, stream))


def _kv_read_args(cache, page_table, start, num, k_out, v_out, status, stream):
    B, n = k_out.shape[:2]
    shape = (B, n, cache.kv_heads, cache.head_dim)
    keep = (cache, page_table, start, num, k_out, v_out, status)
    _one_device(start, num, k_out, v_out, status)
    args = (ctypes.byref(cache._struct), *_table_args(cache, page_table, B), _ptr(start, "start", torch.int32, (B,)),
            _ptr(num, "num", torch.int32, (B,)), B, n, _ptr(k_out, "k_out", None, shape),
            _ptr(v_out, "v_out", k_out.dtype, shape), _dtype_code(k_out), _ptr(status, "status", torch.int32, (B,)),
            _stream(stream))
    return args, keep


def spec_kv_read(cache: KVCache, page_table: torch.Tensor, start: Optional[torch.Tensor], num: Optional[torch.Tensor],
                 k_out: torch.Tensor, v_out: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Positions start .. start + num - 1 of each sequence as values, to the first rows of k_out, v_out."""
    args, keep = _kv_read_args(cache, page_table, start, num, k_out, v_out, status, stream)
    _check(load_library().spec_kv_read(*args))


def prepare_kv_read(cache, page_table, start, num, k_out, v_out, status=None, stream=None) -> _Prepared:
    return _Prepared(load_library().spec_kv_read, *_kv_read_args(cache, page_table, start, num, k_out, v_out, status,
                                                                 stream))


def _kv_keep_path_args(cache, page_table, kv_len, path_nodes, num_accepted, with_root, status, stream):
    B, nmax = path_nodes.shape
    keep = (cache, page_table, kv_len, path_nodes, num_accepted, status)
    _one_device(kv_len, path_nodes, num_accepted, status)
    args = (ctypes.byref(cache._struct), *_table_args(cache, page_table, B), _ptr(kv_len, "kv_len", torch.int32, (B,)),
            _ptr(path_nodes, "path_nodes", torch.int32, (B, nmax)),
            _ptr(num_accepted, "num_accepted", torch.int32, (B,)), B, nmax, int(bool(with_root)),
            _ptr(status, "status", torch.int32, (B,)), _stream(stream))
    return args, keep


def spec_kv_keep_path(cache: KVCache, page_table: torch.Tensor, kv_len: torch.Tensor, path_nodes: torch.Tensor,
                      num_accepted: torch.Tensor, with_root: bool = True, status: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """Move the cache entries of a verified tree's path to the front of their block (kv_len: before the commit)."""
    args, keep = _kv_keep_path_args(cache, page_table, kv_len, path_nodes, num_accepted, with_root, status, stream)
    _check(load_library().spec_kv_keep_path(*args))


def prepare_kv_keep_path(cache, page_table, kv_len, path_nodes, num_accepted, with_root=True, status=None,
                         stream=None) -> _Prepared:
    return _Prepared(load_library().spec_kv_keep_path,
                     *_kv_keep_path_args(cache, page_table, kv_len, path_nodes, num_accepted, with_root, status, stream))


def spec_attention_workspace_bytes(B: int, gmax: int, Hq: int, Hkv: int, D: int) -> int:
    return int(load_library().spec_attention_workspace_bytes(B, gmax, Hq, Hkv, D))


def alloc_attention_workspace(B: int, gmax: int, Hq: int, Hkv: int, D: int, device=None) -> torch.Tensor:
    """A device workspace for attention calls of these sizes (one call at a time)."""
    n = spec_attention_workspace_bytes(B, gmax, Hq, Hkv, D)
    return torch.empty(max(n, 64), dtype=torch.uint8, device=device or "cuda")


def _attention_args(q, cache, page_table, kv_len, out, num_draft, node_parents, with_root, scale, status, workspace,
                    stream):
    B, rows, Hq, D = q.shape
    gmax = rows - 1 if with_root else rows
    if D != cache.head_dim:
        raise ValueError(f"q has head_dim {D}, the cache {cache.head_dim}")
    if workspace is None:
        with _on(stream):
            workspace = alloc_attention_workspace(B, gmax, Hq, cache.kv_heads, D, q.device)
    if workspace.dtype != torch.uint8:
        raise TypeError("workspace must be a uint8 tensor")
    qp, qs = _strided(q, "q", (B, rows, Hq, D))
    strides = (ctypes.c_int64 * 3)(*qs)
    keep = (q, cache, page_table, kv_len, out, num_draft, node_parents, status, workspace, strides)
    _one_device(q, kv_len, out, num_draft, node_parents, status, workspace)
    args = (ctypes.byref(cache._struct), qp, _dtype_code(q), strides, B, gmax, int(bool(with_root)), Hq,
            *_table_args(cache, page_table, B), _ptr(kv_len, "kv_len", torch.int32, (B,)),
            _ptr(num_draft, "num_draft", torch.int32, (B,)), _ptr(node_parents, "node_parents", torch.int32, (B, gmax)),
            D ** -0.5 if scale is None else float(scale), _ptr(out, "out", q.dtype, (B, rows, Hq, D)),
            _ptr(status, "status", torch.int32, (B,)), _ptr(workspace, "workspace"), workspace.numel(), _stream(stream))
    return args, keep


def spec_verify_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_len: torch.Tensor,
                          out: torch.Tensor, num_draft: Optional[torch.Tensor] = None,
                          node_parents: Optional[torch.Tensor] = None, with_root: bool = True,
                          scale: Optional[float] = None, status: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention of a block's rows q [B, rows, Hq, head_dim] (bf16, strided views allowed) over the cache, which holds the
    block's own entries from position kv_len on; scale None: head_dim ** -0.5."""
    args, keep = _attention_args(q, cache, page_table, kv_len, out, num_draft, node_parents, with_root, scale, status,
                                 workspace, stream)
    _check(load_library().spec_verify_attention(*args))


def prepare_verify_attention(q, cache, page_table, kv_len, out, num_draft=None, node_parents=None, with_root=True,
                             scale=None, status=None, workspace=None, stream=None) -> _Prepared:
    return _Prepared(load_library().spec_verify_attention,
                     *_attention_args(q, cache, page_table, kv_len, out, num_draft, node_parents, with_root, scale, status,
                                      workspace, stream))
