"""Q4_0 dequantize-and-multiply on MI355X (gfx950): Python binding of libq4gemv.so.

Argument marshalling only.  Every function checks dtypes, shapes, devices and
contiguity of torch tensors, then calls the C ABI declared in
``include/q4gemv.h`` with raw device pointers and torch's current HIP stream.
All arithmetic happens in the HIP kernels; there is no CPU fallback, and the
import fails loudly when the library has not been built
(``python -m q4_dequant_gemv_block_amd.build``).

Weight tensors are uint8 of shape [N, K/32*18] (packed Q4_0 rows, the block
format the pages call "GGUF Q4_0": f16 scale then 16 bytes of nibble codes,
weight = (code - 8) * scale); activations are float16; outputs float32.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4gemv.so")

Q4_OK = 0
Q4_ERR_INVALID_ARG = -1
Q4_ERR_MISALIGNED = -2
Q4_ERR_WORKSPACE = -3
Q4_ERR_HIP = -4

Q4_OP_GEMV = 0
Q4_OP_GEMM_SMALLM = 1
Q4_OP_GEMM_PREFILL = 2
Q4_OP_LM_HEAD_ARGMAX = 3
Q4_OP_LM_HEAD_VERIFY = 4
Q4_OP_LM_HEAD_NORM_ARGMAX = 5

# Every symbol include/q4gemv.h declares.
EXPORTS = (
    "q4_abi_version", "q4_last_error", "q4_workspace_bytes", "q4_0_gemv", "q4_0_gemm_smallm",
    "q4_0_gemm_prefill", "lm_head_argmax", "lm_head_argmax_noalloc", "lm_head_norm_argmax", "lm_head_verify",
    "q4_0_gemv_handoff", "q8_0_gemv", "q8_0_gemv_batch_plan_bytes",
    "q8_0_gemv_batch_plan", "q8_0_gemv_batch",
    "q4_0_gemv_batch_plan_bytes", "q4_0_gemv_batch_plan",
    "q4_0_gemm_smallm_batch_plan_bytes", "q4_0_gemm_smallm_batch_plan", "q4_0_gemm_smallm_batch",
    "q4_0_gemm_prefill_batch_plan_bytes", "q4_0_gemm_prefill_batch_plan", "q4_0_gemm_prefill_batch",
    "q4_0_gemv_batch", "q4_0_gemv_batch_handoff",
    "q4_rope", "q4_kv_append", "q4_attention_paged_workspace_bytes", "q4_attention_paged",
    "q4_kv_assign", "q4_norm_rope", "q4_kv_append_norm", "q4_attention_tree_workspace_bytes", "q4_attention_tree",
    "q4_attention_workspace_most",
    "q4_logits_argmax_workspace_bytes", "q4_logits_argmax", "q4_tree_accept", "q4_tree_accept_stored", "q4_kv_move",
)

Q4_TYPE_F16 = 0
Q4_TYPE_BF16 = 1
Q4_TYPE_F32 = 2
Q4_ROPE_HALF = 0
Q4_ROPE_INTERLEAVED = 1
_TYPES = {torch.float16: Q4_TYPE_F16, torch.bfloat16: Q4_TYPE_BF16, torch.float32: Q4_TYPE_F32}
_LAYOUTS = {"half": Q4_ROPE_HALF, "interleaved": Q4_ROPE_INTERLEAVED}


class Q4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("q4 status %d: %s" % (status, message))
        self.status = status


class GemvDesc(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class GemvPlan(ctypes.Structure):
    _fields_ = [("device", ctypes.c_void_p), ("count", ctypes.c_int), ("max_k", ctypes.c_int),
                ("grid", ctypes.c_int), ("nchunks", ctypes.c_int), ("flags", ctypes.c_int)]


class Q8Plan(ctypes.Structure):
    _fields_ = [("device", ctypes.c_void_p), ("count", ctypes.c_int), ("n_slab", ctypes.c_int),
                ("grid_slab", ctypes.c_int), ("nchunks_slab", ctypes.c_int), ("max_k", ctypes.c_int),
                ("grid", ctypes.c_int), ("offset_other", ctypes.c_size_t)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("type", ctypes.c_int)]


class CacheDesc(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_page_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64), ("k_slot_stride", ctypes.c_int64),
                ("v_page_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64), ("v_slot_stride", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("type", ctypes.c_int)]


class BatchDesc(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_pages", ctypes.c_int),
                ("seqs", ctypes.c_int), ("query_start", ctypes.c_void_p), ("context_len", ctypes.c_void_p),
                ("max_query", ctypes.c_int), ("max_context", ctypes.c_int)]


class StepDesc(ctypes.Structure):
    _fields_ = [("table_in", ctypes.c_void_p), ("table_in_stride", ctypes.c_int64), ("held_in", ctypes.c_void_p),
                ("past_len", ctypes.c_void_p), ("new_len", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("free_capacity", ctypes.c_int64), ("free_count", ctypes.c_void_p), ("parents", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("held", ctypes.c_void_p),
                ("query_start", ctypes.c_void_p), ("context_len", ctypes.c_void_p), ("missing", ctypes.c_void_p),
                ("free_left", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("mask_words", ctypes.c_int), ("seqs", ctypes.c_int),
                ("table_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("tokens", ctypes.c_int64)]


class RulesDesc(ctypes.Structure):
    _fields_ = [("seqs", ctypes.c_int), ("query_start", ctypes.c_void_p), ("history", ctypes.c_void_p),
                ("history_stride", ctypes.c_int64), ("history_tokens", ctypes.c_int), ("history_len", ctypes.c_void_p),
                ("prompt_len", ctypes.c_void_p), ("draft", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("mask_words", ctypes.c_int), ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("bias_start", ctypes.c_void_p), ("bias_tokens", ctypes.c_void_p),
                ("bias_values", ctypes.c_void_p), ("biases", ctypes.c_int64), ("allowed", ctypes.c_void_p),
                ("allowed_stride", ctypes.c_int64), ("allowed_rows", ctypes.c_int64), ("allowed_row", ctypes.c_void_p)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libq4gemv.so and declare its signatures (raises if it is not built)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libq4gemv.so is not built (%s); run python -m q4_dequant_gemv_block_amd.build" % path)
    lib = ctypes.CDLL(path)
    vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.q4_abi_version.restype = ctypes.c_int
    lib.q4_abi_version.argtypes = []
    lib.q4_last_error.restype = ctypes.c_char_p
    lib.q4_last_error.argtypes = []
    lib.q4_workspace_bytes.restype = ctypes.c_size_t
    lib.q4_workspace_bytes.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.q4_0_gemv.restype = st
    lib.q4_0_gemv.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.q4_0_gemm_smallm.restype = st
    lib.q4_0_gemm_smallm.argtypes = [vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4_0_gemm_prefill.restype = st
    lib.q4_0_gemm_prefill.argtypes = [vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.lm_head_argmax.restype = st
    lib.lm_head_argmax.argtypes = [vp, vp, vp, vp, i64, i64, vp, ctypes.c_size_t, vp]
    lib.lm_head_argmax_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, vp]
    lib.lm_head_argmax_noalloc.restype = st
    lib.lm_head_verify.restype = st
    lib.q8_0_gemv.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.q8_0_gemv.restype = ctypes.c_int
    lib.q4_0_gemv_batch_handoff.argtypes = [ctypes.POINTER(GemvPlan), vp, vp, vp, vp]
    lib.q4_0_gemv_batch_handoff.restype = ctypes.c_int
    lib.q8_0_gemv_batch_plan_bytes.argtypes = [ctypes.POINTER(GemvDesc), ctypes.c_int]
    lib.q8_0_gemv_batch_plan_bytes.restype = ctypes.c_size_t
    lib.q8_0_gemv_batch_plan.argtypes = [ctypes.POINTER(GemvDesc), ctypes.c_int, vp, ctypes.c_size_t,
                                         ctypes.POINTER(Q8Plan), vp]
    lib.q8_0_gemv_batch_plan.restype = ctypes.c_int
    lib.q8_0_gemv_batch.argtypes = [ctypes.POINTER(Q8Plan), vp]
    lib.q8_0_gemv_batch.restype = ctypes.c_int
    lib.q4_0_gemv_handoff.argtypes = [vp, vp, vp, vp, i64, i64, vp]
    lib.q4_0_gemv_handoff.restype = ctypes.c_int
    lib.lm_head_norm_argmax.argtypes = [vp, vp, vp, ctypes.c_float, vp, vp, vp, i64, i64, vp, ctypes.c_size_t, vp]
    lib.lm_head_norm_argmax.restype = ctypes.c_int
    lib.lm_head_verify.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, ctypes.c_size_t, vp]
    lib.q4_0_gemv_batch_plan_bytes.restype = ctypes.c_size_t
    lib.q4_0_gemv_batch_plan_bytes.argtypes = [ctypes.POINTER(GemvDesc), ctypes.c_int]
    lib.q4_0_gemv_batch_plan.restype = st
    lib.q4_0_gemv_batch_plan.argtypes = [ctypes.POINTER(GemvDesc), ctypes.c_int, vp, ctypes.c_size_t,
                                         ctypes.POINTER(GemvPlan), vp]
    lib.q4_0_gemv_batch.restype = st
    lib.q4_0_gemv_batch.argtypes = [ctypes.POINTER(GemvPlan), vp]
    lib.q4_0_gemm_smallm_batch_plan_bytes.restype = ctypes.c_size_t
    lib.q4_0_gemm_smallm_batch_plan_bytes.argtypes = [ctypes.c_int]
    lib.q4_0_gemm_smallm_batch_plan.restype = st
    lib.q4_0_gemm_smallm_batch_plan.argtypes = [ctypes.POINTER(GemvDesc), ctypes.c_int, i64, vp, ctypes.c_size_t,
                                                ctypes.POINTER(GemmPlan), vp]
    lib.q4_0_gemm_smallm_batch.restype = st
    lib.q4_0_gemm_smallm_batch.argtypes = [ctypes.POINTER(GemmPlan), vp, ctypes.c_size_t, vp]
    lib.q4_0_gemm_prefill_batch_plan_bytes.restype = ctypes.c_size_t
    lib.q4_0_gemm_prefill_batch_plan_bytes.argtypes = [ctypes.c_int]
    lib.q4_0_gemm_prefill_batch_plan.restype = st
    lib.q4_0_gemm_prefill_batch_plan.argtypes = [ctypes.POINTER(GemvDesc), ctypes.c_int, i64, vp, ctypes.c_size_t,
                                                 ctypes.POINTER(PrefillPlan), vp]
    lib.q4_0_gemm_prefill_batch.restype = st
    lib.q4_0_gemm_prefill_batch.argtypes = [ctypes.POINTER(PrefillPlan), vp]
    # descriptors by address (byref): no pointer type to convert to on each call
    i32, f32 = ctypes.c_int, ctypes.c_float
    lib.q4_rope.restype = st
    lib.q4_rope.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, i32, f32, vp]
    lib.q4_kv_append.restype = st
    lib.q4_kv_append.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, i32, i32, f32, vp]
    lib.q4_attention_paged_workspace_bytes.restype = ctypes.c_size_t
    lib.q4_attention_paged_workspace_bytes.argtypes = [vp, vp, i32, i64, i64]
    lib.q4_attention_paged.restype = st
    lib.q4_attention_paged.argtypes = [vp, vp, vp, vp, vp, i32, i64, f32, i64, vp, ctypes.c_size_t, vp]
    size = ctypes.c_size_t
    lib.q4_kv_assign.restype = st
    lib.q4_kv_assign.argtypes = [vp, vp]
    lib.q4_norm_rope.restype = st
    lib.q4_norm_rope.argtypes = [vp, vp, vp, i32, f32, vp, vp, i64, i32, i32, i32, i32, f32, vp]
    lib.q4_kv_append_norm.restype = st
    lib.q4_kv_append_norm.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, vp, vp, i32, f32, vp, vp, i32, i32, f32, vp]
    lib.q4_attention_tree_workspace_bytes.restype = size
    lib.q4_attention_tree_workspace_bytes.argtypes = [vp, vp, i32, i64, i64]
    lib.q4_attention_workspace_most.restype = size
    lib.q4_attention_workspace_most.argtypes = [vp, i32, i64]
    lib.q4_attention_tree.restype = st
    lib.q4_attention_tree.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i64, f32, i64, vp, size, vp]
    lib.q4_logits_argmax_workspace_bytes.restype = size
    lib.q4_logits_argmax_workspace_bytes.argtypes = [i64, i64]
    lib.q4_logits_argmax.restype = st
    lib.q4_logits_argmax.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, vp, vp, size, vp]
    lib.q4_tree_accept.restype = st
    lib.q4_tree_accept.argtypes = [vp, vp, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, i64, i32, vp]
    lib.q4_tree_accept_stored.restype = st
    lib.q4_tree_accept_stored.argtypes = [vp, vp, i32, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i64, i32, vp]
    lib.q4_kv_move.restype = st
    lib.q4_kv_move.argtypes = [vp, i32, vp, vp, vp, i64, vp]
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(status: int):
    if status != Q4_OK:
        raise Q4Error(status, load_library().q4_last_error().decode())


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be on a GPU" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def row_bytes(k: int) -> int:
    return k // 32 * 18


def _weights(w: torch.Tensor, k: int) -> int:
    if w.dim() == 2:
        if w.shape[1] != row_bytes(k):
            raise ValueError("w has %d bytes per row, k=%d needs %d" % (w.shape[1], k, row_bytes(k)))
        return w.shape[0]
    if w.dim() == 1 and w.numel() % row_bytes(k) == 0:
        return w.numel() // row_bytes(k)
    raise ValueError("w must be uint8 [N, K/32*18]")


def abi_version() -> int:
    return load_library().q4_abi_version()


def last_error() -> str:
    return load_library().q4_last_error().decode()


def workspace_bytes(op: int, m: int, n: int, k: int) -> int:
    return int(load_library().q4_workspace_bytes(op, m, n, k))


def q4_0_gemv(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = W x for packed Q4_0 rows W (uint8 [N, K/32*18]) and x (float16 [K]); y float32 [N]."""
    if x.dim() != 1:
        raise ValueError("x must be float16 [K]")
    k = x.shape[0]
    n = _weights(w, k)
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=x.device)
    elif out.numel() != n:
        raise ValueError("out must hold N=%d floats" % n)
    _check(load_library().q4_0_gemv(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                    _ptr(out, torch.float32, "out"), n, k, _stream(stream)))
    return out


def q4_0_gemm_smallm(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W^T for X float16 [M, K] with 1 <= M <= 16; Y float32 [M, N]."""
    if x.dim() != 2:
        raise ValueError("x must be float16 [M, K]")
    m, k = x.shape
    n = _weights(w, k)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    elif out.numel() != m * n:
        raise ValueError("out must hold M*N floats")
    need = workspace_bytes(Q4_OP_GEMM_SMALLM, m, n, k)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wp = _ptr(workspace, torch.uint8, "workspace") if workspace is not None else None
    wb = workspace.numel() if workspace is not None else 0
    _check(load_library().q4_0_gemm_smallm(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                           _ptr(out, torch.float32, "out"), m, n, k, wp, wb, _stream(stream)))
    return out


def q4_0_gemm_prefill(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W^T for X float16 [M, K] (any M >= 1) on the matrix cores; Y float32 [M, N]."""
    if x.dim() != 2:
        raise ValueError("x must be float16 [M, K]")
    m, k = x.shape
    n = _weights(w, k)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    elif out.numel() != m * n:
        raise ValueError("out must hold M*N floats")
    need = workspace_bytes(Q4_OP_GEMM_PREFILL, m, n, k)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wp = _ptr(workspace, torch.uint8, "workspace") if workspace is not None else None
    wb = workspace.numel() if workspace is not None else 0
    _check(load_library().q4_0_gemm_prefill(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                            _ptr(out, torch.float32, "out"), m, n, k, wp, wb, _stream(stream)))
    return out


def lm_head_argmax(w: torch.Tensor, h: torch.Tensor, logits: torch.Tensor | None = None,
                   token: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(logits float32 [V], token int32 [1]) for the LM head W (uint8 [V, K/32*18]) and h (float16 [K])."""
    if h.dim() != 1:
        raise ValueError("h must be float16 [K]")
    k = h.shape[0]
    n = _weights(w, k)
    if logits is None:
        logits = torch.empty(n, dtype=torch.float32, device=h.device)
    if token is None:
        token = torch.empty(1, dtype=torch.int32, device=h.device)
    need = workspace_bytes(Q4_OP_LM_HEAD_ARGMAX, 1, n, k)
    if workspace is None:
        workspace = torch.empty(max(need, 8), dtype=torch.uint8, device=h.device)
    _check(load_library().lm_head_argmax(_ptr(w, torch.uint8, "w"), _ptr(h, torch.float16, "h"),
                                         _ptr(logits, torch.float32, "logits"), _ptr(token, torch.int32, "token"),
                                         n, k, _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                         _stream(stream)))
    return logits, token


def lm_head_argmax_noalloc(w: torch.Tensor, h: torch.Tensor, logits: torch.Tensor | None = None,
                           token: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """lm_head_argmax with the per-workgroup keys in the library's own per-device
    array: the C call allocates nothing (pass logits and token to allocate nothing here either)."""
    if h.dim() != 1:
        raise ValueError("h must be float16 [K]")
    k = h.shape[0]
    n = _weights(w, k)
    if logits is None:
        logits = torch.empty(n, dtype=torch.float32, device=h.device)
    if token is None:
        token = torch.empty(1, dtype=torch.int32, device=h.device)
    _check(load_library().lm_head_argmax_noalloc(_ptr(w, torch.uint8, "w"), _ptr(h, torch.float16, "h"),
                                                 _ptr(logits, torch.float32, "logits"),
                                                 _ptr(token, torch.int32, "token"), n, k, _stream(stream)))
    return logits, token


def q8_row_bytes(k: int) -> int:
    """Bytes of one Q8_0 row of K weights (K/32 blocks of 34 bytes)."""
    if k % 32:
        raise ValueError("K must be a multiple of 32")
    return k // 32 * 34


def q8_0_gemv(w: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y float32 [N] = W x for Q8_0 weights W (uint8 [N, K/32*34]) and x (float16 [K])."""
    if x.dim() != 1:
        raise ValueError("x must be float16 [K]")
    k = x.shape[0]
    if w.dim() != 2 or w.shape[1] != q8_row_bytes(k):
        raise ValueError("w must be uint8 [N, K/32*34]")
    n = w.shape[0]
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=x.device)
    _check(load_library().q8_0_gemv(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                    _ptr(out, torch.float32, "out"), n, k, _stream(stream)))
    return out


def q4_0_gemv_handoff(w: torch.Tensor, x: torch.Tensor, residual: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The stage hand-off: float16 [N] = binary16(residual + W x) for W (uint8 [N, K/32*18]),
    x (float16 [K]) and an optional float32 residual [N]."""
    if x.dim() != 1:
        raise ValueError("x must be float16 [K]")
    k = x.shape[0]
    n = _weights(w, k)
    if out is None:
        out = torch.empty(n, dtype=torch.float16, device=x.device)
    rp = 0
    if residual is not None:
        if residual.dim() != 1 or residual.shape[0] != n:
            raise ValueError("residual must be float32 [N]")
        rp = _ptr(residual, torch.float32, "residual")
    _check(load_library().q4_0_gemv_handoff(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"), rp,
                                            _ptr(out, torch.float16, "out"), n, k, _stream(stream)))
    return out


def lm_head_norm_argmax(w: torch.Tensor, h: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                        logits: torch.Tensor | None = None, token: torch.Tensor | None = None,
                        x_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Final norm of h, then the LM head: (logits float32 [V], token int32 [1]) for W
    (uint8 [V, K/32*18]), the hidden state h and the norm's gain gamma (float16 [K]).
    x_out (float16 [K], optional) receives the normed activation."""
    if h.dim() != 1 or gamma.dim() != 1 or gamma.shape[0] != h.shape[0]:
        raise ValueError("h and gamma must be float16 [K]")
    k = h.shape[0]
    n = _weights(w, k)
    if logits is None:
        logits = torch.empty(n, dtype=torch.float32, device=h.device)
    if token is None:
        token = torch.empty(1, dtype=torch.int32, device=h.device)
    need = workspace_bytes(Q4_OP_LM_HEAD_NORM_ARGMAX, 1, n, k)
    if workspace is None:
        workspace = torch.empty(max(need, 8), dtype=torch.uint8, device=h.device)
    xo = 0
    if x_out is not None:
        if x_out.dim() != 1 or x_out.shape[0] != k:
            raise ValueError("x_out must be float16 [K]")
        xo = _ptr(x_out, torch.float16, "x_out")
    _check(load_library().lm_head_norm_argmax(_ptr(w, torch.uint8, "w"), _ptr(h, torch.float16, "h"),
                                              _ptr(gamma, torch.float16, "gamma"), float(eps),
                                              _ptr(logits, torch.float32, "logits"),
                                              _ptr(token, torch.int32, "token"), xo, n, k,
                                              _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                              _stream(stream)))
    return logits, token


def lm_head_verify(w: torch.Tensor, h: torch.Tensor, draft: torch.Tensor, logits: torch.Tensor | None = None,
                   tokens: torch.Tensor | None = None, accepted: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """(logits float32 [M, V], tokens int32 [M], accepted int32 [1]) for the LM head W
    (uint8 [V, K/32*18]), the trunk's hidden states h (float16 [M, K], M <= 16) and the
    draft's tokens for the same positions (int32 [M])."""
    if h.dim() != 2:
        raise ValueError("h must be float16 [M, K]")
    m, k = h.shape
    n = _weights(w, k)
    if draft.dim() != 1 or draft.shape[0] != m:
        raise ValueError("draft must be int32 [M]")
    if logits is None:
        logits = torch.empty((m, n), dtype=torch.float32, device=h.device)
    if tokens is None:
        tokens = torch.empty(m, dtype=torch.int32, device=h.device)
    if accepted is None:
        accepted = torch.empty(1, dtype=torch.int32, device=h.device)
    need = workspace_bytes(Q4_OP_LM_HEAD_VERIFY, m, n, k)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=h.device)
    _check(load_library().lm_head_verify(_ptr(w, torch.uint8, "w"), _ptr(h, torch.float16, "h"),
                                         _ptr(logits, torch.float32, "logits"), _ptr(tokens, torch.int32, "tokens"),
                                         _ptr(draft, torch.int32, "draft"), _ptr(accepted, torch.int32, "accepted"),
                                         m, n, k, _ptr(workspace, torch.uint8, "workspace"), workspace.numel(),
                                         _stream(stream)))
    return logits, tokens, accepted


class GemmPlan(ctypes.Structure):
    _fields_ = [("device", ctypes.c_void_p), ("count", ctypes.c_int), ("m", ctypes.c_int),
                ("max_p", ctypes.c_int), ("flags", ctypes.c_int), ("total_cost", ctypes.c_int64),
                ("max_mn", ctypes.c_int64), ("workspace_bytes", ctypes.c_size_t)]


class PrefillPlan(ctypes.Structure):
    _fields_ = [("device", ctypes.c_void_p), ("count", ctypes.c_int), ("m", ctypes.c_int),
                ("tile_m", ctypes.c_int), ("count_chunked", ctypes.c_int), ("tiles_chunked", ctypes.c_int64),
                ("tiles_other", ctypes.c_int64)]


class GemvBatch:
    """A list of independent GEMVs (w, x, y) planned once and run as one launch per call."""

    def __init__(self, items, stream=None):
        items = list(items)
        descs = (GemvDesc * len(items))()
        self._keep = []
        for i, (w, x, y) in enumerate(items):
            k = x.shape[-1]
            n = _weights(w, k)
            if y.numel() != n:
                raise ValueError("descriptor %d: y must hold N=%d floats" % (i, n))
            descs[i] = GemvDesc(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                _ptr(y, torch.float32, "y"), n, k)
            self._keep.append((w, x, y))
        lib = load_library()
        dev = items[0][0].device if items else torch.device("cuda")
        self.plan = GemvPlan()
        with torch.cuda.device(dev):  # the schedule is cut for this device
            nbytes = int(lib.q4_0_gemv_batch_plan_bytes(descs, len(items)))
            if nbytes == 0:
                _check(Q4_ERR_INVALID_ARG)
            self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            _check(lib.q4_0_gemv_batch_plan(descs, len(items), self.buffer.data_ptr(), self.buffer.numel(),
                                            ctypes.byref(self.plan), _stream(stream)))

    def set_handoff(self, index: int, h16: torch.Tensor, residual: torch.Tensor | None = None, stream=None):
        """Make item `index` of the list the stage hand-off: it writes float16 h16 [N] =
        residual + W x (rounded once) instead of its float32 y."""
        n = self._keep[index][2].numel()
        if h16.numel() != n:
            raise ValueError("h16 must hold N=%d float16 values" % n)
        rp = 0
        if residual is not None:
            if residual.numel() != n:
                raise ValueError("residual must hold N=%d float32 values" % n)
            rp = _ptr(residual, torch.float32, "residual")
        y = self._keep[index][2]
        _check(load_library().q4_0_gemv_batch_handoff(ctypes.byref(self.plan), _ptr(y, torch.float32, "y"), rp,
                                                      _ptr(h16, torch.float16, "h16"), _stream(stream)))
        self._keep.append((h16, residual))

    def __call__(self, stream=None):
        _check(load_library().q4_0_gemv_batch(ctypes.byref(self.plan), _stream(stream)))


class Q8Batch:
    """A list of Q8_0 GEMVs (w, x, y), w uint8 [N, K/32*34], planned once and run as
    one launch per call."""

    def __init__(self, items, stream=None):
        items = list(items)
        descs = (GemvDesc * len(items))()
        self._keep = []
        for i, (w, x, y) in enumerate(items):
            k = x.shape[-1]
            if w.dim() != 2 or w.shape[1] != q8_row_bytes(k):
                raise ValueError("descriptor %d: w must be uint8 [N, K/32*34]" % i)
            n = w.shape[0]
            if y.numel() != n:
                raise ValueError("descriptor %d: y must hold N=%d floats" % (i, n))
            descs[i] = GemvDesc(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                _ptr(y, torch.float32, "y"), n, k)
            self._keep.append((w, x, y))
        lib = load_library()
        dev = items[0][0].device if items else torch.device("cuda")
        self.plan = Q8Plan()
        with torch.cuda.device(dev):  # the ranges are cut for this device's compute units
            nbytes = int(lib.q8_0_gemv_batch_plan_bytes(descs, len(items)))
            if nbytes == 0:
                _check(Q4_ERR_INVALID_ARG)
            self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=dev)
            _check(lib.q8_0_gemv_batch_plan(descs, len(items), self.buffer.data_ptr(), self.buffer.numel(),
                                            ctypes.byref(self.plan), _stream(stream)))

    def __call__(self, stream=None):
        _check(load_library().q8_0_gemv_batch(ctypes.byref(self.plan), _stream(stream)))


class SmallMBatch:
    """A list of small-M GEMMs (w, x, y) with x of shape (m, k) and y (m, n), the
    same m for all, planned once and run as one launch (plus one reduction of
    K-range partials when some GEMM splits K) per call."""

    def __init__(self, items, stream=None):
        items = list(items)
        if not items:
            raise ValueError("empty list")
        m = items[0][1].shape[0] if items[0][1].dim() == 2 else 1
        descs = (GemvDesc * len(items))()
        self._keep = []
        for i, (w, x, y) in enumerate(items):
            if x.dim() != 2 or x.shape[0] != m:
                raise ValueError("descriptor %d: x must be (m, k) with m = %d" % (i, m))
            k = x.shape[1]
            n = _weights(w, k)
            if y.numel() != m * n:
                raise ValueError("descriptor %d: y must hold m*N=%d floats" % (i, m * n))
            descs[i] = GemvDesc(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                _ptr(y, torch.float32, "y"), n, k)
            self._keep.append((w, x, y))
        lib = load_library()
        dev = items[0][0].device
        self.m = m
        self.plan = GemmPlan()
        with torch.cuda.device(dev):
            nbytes = int(lib.q4_0_gemm_smallm_batch_plan_bytes(len(items)))
            self.buffer = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
            _check(lib.q4_0_gemm_smallm_batch_plan(descs, len(items), m, self.buffer.data_ptr(),
                                                   self.buffer.numel(), ctypes.byref(self.plan),
                                                   _stream(stream)))
            self.workspace = torch.empty(max(int(self.plan.workspace_bytes), 16), dtype=torch.uint8, device=dev)

    def __call__(self, stream=None):
        _check(load_library().q4_0_gemm_smallm_batch(ctypes.byref(self.plan), self.workspace.data_ptr(),
                                                     self.workspace.numel(), _stream(stream)))


class PrefillBatch:
    """A list of prefill GEMMs (w, x, y) with x of shape (m, k) and y (m, n), the
    same m for all, planned once and run as one launch per call."""

    def __init__(self, items, stream=None):
        items = list(items)
        if not items:
            raise ValueError("empty list")
        m = items[0][1].shape[0]
        descs = (GemvDesc * len(items))()
        self._keep = []
        for i, (w, x, y) in enumerate(items):
            if x.dim() != 2 or x.shape[0] != m:
                raise ValueError("descriptor %d: x must be (m, k) with m = %d" % (i, m))
            k = x.shape[1]
            n = _weights(w, k)
            if y.numel() != m * n:
                raise ValueError("descriptor %d: y must hold m*N=%d floats" % (i, m * n))
            descs[i] = GemvDesc(_ptr(w, torch.uint8, "w"), _ptr(x, torch.float16, "x"),
                                _ptr(y, torch.float32, "y"), n, k)
            self._keep.append((w, x, y))
        lib = load_library()
        dev = items[0][0].device
        self.m = m
        self.plan = PrefillPlan()
        with torch.cuda.device(dev):
            nbytes = int(lib.q4_0_gemm_prefill_batch_plan_bytes(len(items)))
            self.buffer = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
            _check(lib.q4_0_gemm_prefill_batch_plan(descs, len(items), m, self.buffer.data_ptr(),
                                                    self.buffer.numel(), ctypes.byref(self.plan),
                                                    _stream(stream)))

    def __call__(self, stream=None):
        _check(load_library().q4_0_gemm_prefill_batch(ctypes.byref(self.plan), _stream(stream)))


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device="cuda") -> tuple[torch.Tensor, float]:
    """(inv_freq float64 [rot_dim / 2], mscale) for q4_rope and q4_kv_append, made once for a model.

    inv_freq[i] = base^(-2 i / rot_dim), scaled for contexts `factor` times as long as the trained ones:
      None      as it is;
      "linear"  positions divided by the factor;
      "ntk"     the base times factor^(rot_dim / (rot_dim - 2)), so that the slowest pair turns as with
                "linear" and the fastest as without;
      "yarn"    pairs that make beta_fast turns or more over `original_length` positions as without,
                those with beta_slow or fewer as with "linear", a ramp over the pair's index between,
                and mscale = 0.1 ln(factor) + 1 (on queries and keys alike).
    All of it in 64 bits on the host."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not base > 1.0 or not math.isfinite(base) or not factor >= 1.0 or not math.isfinite(factor):
        raise ValueError("base must be above 1 and factor at least 1")
    half, mscale = rot_dim // 2, 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim of at least 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * i / rot_dim) for i in range(half)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        if not original_length or original_length < 1:
            raise ValueError("yarn scaling needs original_length")
        if not beta_fast > beta_slow > 0:
            raise ValueError("beta_fast must be above beta_slow, and both above 0")

        def index(turns):  # the (fractional) pair that makes so many turns over the original length
            return rot_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low, high = max(math.floor(index(beta_fast)), 0), min(math.ceil(index(beta_slow)), rot_dim - 1)
        span = max(high - low, 1e-3)
        ramp = [min(max((i - low) / span, 0.0), 1.0) for i in range(half)]
        freq = [f * (1.0 - r) + f / factor * r for f, r in zip(freq, ramp)]
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    return torch.tensor(freq, dtype=torch.float64, device=device), mscale


def _heads(t: torch.Tensor, name: str, gpu: int) -> Heads:
    """Tokens x heads x head_dim on that GPU, the elements of a head side by side; other strides are free."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise TypeError("%s must be float16, bfloat16 or float32, got %s" % (name, t.dtype))
    if t.get_device() != gpu:
        raise ValueError("%s must be on GPU %d, is on %s" % (name, gpu, t.device))
    if t.dim() != 3:
        raise ValueError("%s must be [tokens, heads, head_dim]" % name)
    st, sh, sd = t.stride()
    if sd != 1 and t.shape[2] != 1:
        raise ValueError("the elements of a head of %s must be side by side" % name)
    return Heads(t.data_ptr(), st, sh, kind)


def _vector(t: torch.Tensor, dtype, name: str, n: int | None, gpu: int) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != gpu:
        raise ValueError("%s must be on GPU %d, is on %s" % (name, gpu, t.device))
    if t.dim() != 1 or (n is not None and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError("%s must be contiguous, %s" % (name, "[%d]" % n if n is not None else "of one dimension"))
    return t.data_ptr()


def _layout(layout: str) -> int:
    if layout not in _LAYOUTS:
        raise ValueError("layout must be 'half' or 'interleaved'")
    return _LAYOUTS[layout]


def _on(gpu: int, stream):
    """The context in which a call allocates and launches: the tensors' GPU and the given stream (so that what is
    allocated here belongs to the stream that uses it), or None where they are the current ones already."""
    if stream is not None:
        if stream.device.index != gpu:
            raise ValueError("stream is on %s, the tensors are on GPU %d" % (stream.device, gpu))
        return torch.cuda.stream(stream)
    if torch._C._cuda_getDevice() != gpu:
        return torch.cuda.device(gpu)
    return None


# The handle of a GPU's current stream (torch.cuda.current_stream makes an object of it, for 3 us a call).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (a torch built without GPUs has none)


def q4_rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, layout: str = "half",
            mscale: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x [T, H, D] (float16, bfloat16 or float32; the heads may lie apart, as in a part of packed projections)
    with the leading 2 * len(inv_freq) elements of each head turned by the angles positions[t] * inv_freq[i]
    (int32 [T], float64 [r / 2]; rope_frequencies makes them), the others as they are.  Pairs are elements i and
    i + r/2 ("half") or 2i and 2i + 1 ("interleaved"), results times mscale.  out: like x in shape, of any of the
    types, and may be x itself.  Turning by -positions undoes it and is its gradient.  No tokens: nothing to do."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be on a GPU")
    on = _on(dev, stream)
    if on is not None:
        with on:
            return q4_rope(x, positions, inv_freq, layout, mscale, out)
    hx = _heads(x, "x", dev)
    t, h, d = x.shape
    if out is None:
        out = x.new_empty((t, h, d))
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    ho = _heads(out, "out", dev)
    freq, pos, kind = _vector(inv_freq, torch.float64, "inv_freq", None, dev), _vector(positions, torch.int32, "positions", t, dev), _layout(layout)
    if t == 0:
        return out
    status = (_lib or load_library()).q4_rope(
        ctypes.byref(hx), ctypes.byref(ho), pos, freq, t, h, d, 2 * inv_freq.shape[0], kind, mscale, _current_stream(dev))
    if status:
        _check(status)
    return out


class KVCache:
    """A paged key/value cache: k and v [pages, kv_heads, page_size, head_dim], float16 or bfloat16, the elements of
    a head side by side and the other strides free (a transposed view of [pages, page_size, kv_heads, head_dim] will
    do).  page_size is a multiple of 8.  The handle holds the tensors, not their contents."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for t, name in ((k, "k"), (v, "v")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch.Tensor" % name)
            if t.dtype not in (torch.float16, torch.bfloat16):
                raise TypeError("%s must be float16 or bfloat16, got %s" % (name, t.dtype))
            if t.device.type != "cuda":
                raise ValueError("%s must be on a GPU" % name)
            if t.dim() != 4:
                raise ValueError("%s must be [pages, kv_heads, page_size, head_dim]" % name)
            if t.stride(3) != 1 and t.shape[3] != 1:
                raise ValueError("the elements of a head of %s must be side by side" % name)
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("k and v must have one shape, type and device")
        self.k, self.v = k, v
        self.device, self.dtype, self.gpu = k.device, k.dtype, k.get_device()
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.desc = CacheDesc(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2),
                              v.stride(0), v.stride(1), v.stride(2), self.pages, self.page_size, self.kv_heads,
                              self.head_dim, _TYPES[k.dtype])
        self._ref = ctypes.byref(self.desc)


class KVBatch:
    """The sequences of a call: block_table [B, P] (the pages a sequence holds, in order), query_start [B + 1] (rows
    of its new tokens in the token tensors) and context_lens [B] (its length with them), int32 on the GPU, where the
    kernels read them: they may change between calls and between replays of a captured graph.  max_query_len and
    max_context_len, if known, help to choose a kernel; results do not depend on them."""

    def __init__(self, block_table: torch.Tensor, query_start: torch.Tensor, context_lens: torch.Tensor,
                 max_query_len: int | None = None, max_context_len: int | None = None):
        if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32:
            raise TypeError("block_table must be an int32 tensor")
        if block_table.device.type != "cuda":
            raise ValueError("block_table must be on a GPU")
        if block_table.dim() != 2 or (block_table.stride(1) != 1 and block_table.shape[1] != 1):
            raise ValueError("block_table must be [sequences, pages] with consecutive entries")
        b = block_table.shape[0]
        self.device, self.gpu = block_table.device, block_table.get_device()
        self._keep = (block_table, query_start, context_lens)
        self.seqs = b
        self.slots = None
        self.desc = BatchDesc(block_table.data_ptr(), block_table.stride(0), block_table.shape[1], b,
                              _vector(query_start, torch.int32, "query_start", b + 1, self.gpu),
                              _vector(context_lens, torch.int32, "context_lens", b, self.gpu),
                              *(min(int(n or 0), 2 ** 31 - 1) for n in (max_query_len, max_context_len)))
        self._ref = ctypes.byref(self.desc)


def _same_device(cache: KVCache, batch: KVBatch):
    if batch.gpu != cache.gpu:
        raise ValueError("the batch is on %s, the cache on %s" % (batch.device, cache.device))


def q4_kv_append(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, layout: str = "half", mscale: float = 1.0,
                 positions: torch.Tensor | None = None, q_out: torch.Tensor | None = None, stream=None):
    """Write the new tokens' keys and values (k, v [T, kv_heads, D], any of the three types) into the cache, the keys
    turned on the way as by q4_rope (inv_freq None: not turned) by their positions in the sequence, or by
    `positions` (int32 [T]).  With q [T, q_heads, D] also returns q turned, in the cache's type, in q_out if given.
    No tokens (a step in which no sequence has new ones): nothing to do."""
    on = _on(cache.gpu, stream)
    if on is not None:
        with on:
            return q4_kv_append(cache, batch, k, v, q, inv_freq, layout, mscale, positions, q_out)
    _same_device(cache, batch)
    dev = cache.gpu
    hk, hv = _heads(k, "k", dev), _heads(v, "v", dev)
    t = k.shape[0]
    if k.shape != v.shape or k.shape[1] != cache.kv_heads or k.shape[2] != cache.head_dim:
        raise ValueError("k and v must be [T, %d, %d]" % (cache.kv_heads, cache.head_dim))
    rq = ro = None
    heads = 0
    if q is not None:
        hq = _heads(q, "q", dev)
        heads = q.shape[1]
        if q.shape[0] != t or q.shape[2] != cache.head_dim:
            raise ValueError("q must be [T=%d, heads, %d]" % (t, cache.head_dim))
        if q_out is None:
            q_out = torch.empty((t, heads, cache.head_dim), dtype=cache.dtype, device=cache.device)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        ho = _heads(q_out, "q_out", dev)
        rq, ro = ctypes.byref(hq), ctypes.byref(ho)
    elif q_out is not None:
        raise ValueError("q_out without q")
    r, freq = 0, None
    if inv_freq is not None:
        freq = _vector(inv_freq, torch.float64, "inv_freq", None, dev)
        r = inv_freq.shape[0]
    pos = None if positions is None else _vector(positions, torch.int32, "positions", t, dev)
    kind = _layout(layout)
    if t == 0:
        return q_out
    status = (_lib or load_library()).q4_kv_append(
        cache._ref, batch._ref, ctypes.byref(hk), ctypes.byref(hv), rq, ro, heads, t, pos, freq if r else None, 2 * r,
        kind, mscale, _current_stream(dev))
    if status:
        _check(status)
    return q_out


def attention_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int, tokens: int, window: int = 0) -> int:
    """Bytes of the workspace q4_attention_paged needs for these sizes (0: none); smaller sizes may need more
    (attention_workspace_most)."""
    if tokens == 0:
        return 0
    with torch.cuda.device(cache.device):  # the work is cut for this device
        n = int(load_library().q4_attention_paged_workspace_bytes(cache._ref, batch._ref, q_heads, tokens, window))
    if n == 0 and last_error():
        raise Q4Error(Q4_ERR_INVALID_ARG, last_error())
    return n


def attention_workspace_most(cache: KVCache, q_heads: int, tokens: int) -> int:
    """Bytes of a workspace for every call of q4_attention_paged and q4_attention_tree with up to `tokens` new tokens over
    such a cache, whatever its batch and window."""
    if tokens == 0:
        return 0
    with torch.cuda.device(cache.device):
        n = int(load_library().q4_attention_workspace_most(cache._ref, q_heads, tokens))
    if n == 0:
        raise Q4Error(Q4_ERR_INVALID_ARG, last_error())
    return n


def q4_attention_paged(cache: KVCache, batch: KVBatch, q: torch.Tensor, scale: float | None = None, window: int = 0,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """softmax(scale q K^T) V of the new tokens' queries q [T, q_heads, D] (the cache's type) over the cached keys of
    their sequences up to their own positions, the last `window` of them if window > 0; query head h reads kv head
    h / (q_heads / kv_heads).  scale: 1 / sqrt(D) if None.  Append the new tokens first (q4_kv_append).  out like q;
    lse (float32 [T, q_heads], optional) receives the log of the sum of exponentials; workspace (uint8) at least
    attention_workspace_bytes.  Rows that see nothing are 0.  No tokens: nothing to do."""
    on = _on(cache.gpu, stream)
    if on is not None:
        with on:
            return q4_attention_paged(cache, batch, q, scale, window, out, lse, workspace)
    _same_device(cache, batch)
    dev = cache.gpu
    hq = _heads(q, "q", dev)
    t, h, d = q.shape
    if d != cache.head_dim:
        raise ValueError("q must be [T, heads, %d]" % cache.head_dim)
    if out is None:
        out = q.new_empty((t, h, d))
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ho = _heads(out, "out", dev)
    lp = None
    if lse is not None:
        lp = _ptr(lse, torch.float32, "lse")
        if tuple(lse.shape) != (t, h) or lse.get_device() != dev:
            raise ValueError("lse must be float32 [T, heads] on %s" % cache.device)
    if t == 0:
        return out
    lib = _lib or load_library()
    wp, wb = None, 0
    if workspace is None:
        wb = lib.q4_attention_paged_workspace_bytes(cache._ref, batch._ref, h, t, window)
        if wb:
            workspace = torch.empty(wb, dtype=torch.uint8, device=cache.device)
            wp = workspace.data_ptr()
    else:
        wp, wb = _vector(workspace, torch.uint8, "workspace", None, dev), workspace.shape[0]
    status = lib.q4_attention_paged(cache._ref, batch._ref, ctypes.byref(hq), ctypes.byref(ho), lp, h, t,
                                    scale if scale is not None else d ** -0.5, window, wp, wb, _current_stream(dev))
    if status:
        _check(status)
    return out


class KVStep:
    """The tables of a step, which q4_kv_assign writes: block_table [B, P], held [B], query_start [B + 1],
    context_lens [B], missing [B], free_count [1] and positions [T], int32, slots [T] and, with mask_words > 0, mask
    [T, mask_words], int64; and `batch`, the KVBatch of them.  The last step's tables (block_table, held, free_count)
    are the next one's inputs, so a program keeps two of these and takes them in turn.  table: a tensor [B, P] to
    write the block table to instead of one of its own (say the one it is read from).  Rows of slots, positions and mask
    behind a step's last token (query_start[B]) keep what an earlier step left there; at first they are -1, 0 and 0."""

    def __init__(self, seqs: int, table_pages: int, page_size: int, tokens: int, mask_words: int = 0,
                 max_query_len: int | None = None, max_context_len: int | None = None,
                 table: torch.Tensor | None = None, device="cuda"):
        for n, name in ((seqs, "seqs"), (table_pages, "table_pages"), (tokens, "tokens")):
            if n < 1:
                raise ValueError("%s must be at least 1" % name)
        if mask_words < 0:
            raise ValueError("mask_words must not be negative")

        if table is not None and tuple(table.shape) != (seqs, table_pages):
            raise ValueError("table must be int32 [%d, %d]" % (seqs, table_pages))
        # the small tensors are parts of one, 64 bytes apart
        sizes = [seqs, seqs + 1, seqs, seqs, 1, tokens]
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + -(-n // 16) * 16)
        whole = torch.zeros(starts[-1], dtype=torch.int32, device=device)
        self.held, self.query_start, self.context_lens, self.missing, self.free_count, self.positions = (
            whole[at : at + n] for at, n in zip(starts, sizes))
        self.block_table = table if table is not None else torch.zeros((seqs, table_pages), dtype=torch.int32, device=device)
        longs = torch.zeros((tokens, 1 + mask_words), dtype=torch.int64, device=device).view(-1)
        self.slots = longs[:tokens].fill_(-1)  # no row has a place yet
        self.mask = longs[tokens:].view(tokens, mask_words) if mask_words else None
        self.seqs, self.table_pages, self.page_size, self.tokens, self.mask_words = seqs, table_pages, page_size, tokens, mask_words
        self.batch = KVBatch(self.block_table, self.query_start, self.context_lens, max_query_len, max_context_len)
        self.batch.slots = self.slots  # of this step's tokens: q4_tree_accept counts none without one
        self.device, self.gpu = self.batch.device, self.batch.gpu
        d = StepDesc()
        d.table, d.table_stride = self.block_table.data_ptr(), self.block_table.stride(0)
        d.held, d.query_start, d.context_len = self.held.data_ptr(), self.query_start.data_ptr(), self.context_lens.data_ptr()
        d.missing, d.free_left, d.positions = self.missing.data_ptr(), self.free_count.data_ptr(), self.positions.data_ptr()
        d.slots, d.mask = self.slots.data_ptr(), self.mask.data_ptr() if mask_words else None
        d.mask_words, d.seqs, d.table_pages, d.page_size, d.tokens = mask_words, seqs, table_pages, page_size, tokens
        self._desc = bytes(d)


def q4_kv_assign(step: KVStep, block_table: torch.Tensor, held: torch.Tensor, past_lens: torch.Tensor,
                 new_lens: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
                 parents: torch.Tensor | None = None, stream=None) -> KVStep:
    """Write `step`'s tables from the lengths past_lens and new_lens [B]: a page for each place a sequence needs and
    does not hold (its first held[b] entries of block_table [B, P]), taken from the end of the first free_count[0] of
    free_pages; a sequence whose pages do not fit gets none, and step.missing says how many it lacks.  parents [T]:
    the tree of each sequence's new tokens (a parent's index among them, -1 for none): positions are depths then, and
    the masks the ancestors; without it each token follows the one before.  All int32 on the GPU.  held, past_lens and
    free_count must not be step's own tensors; block_table may be."""
    on = _on(step.gpu, stream)
    if on is not None:
        with on:
            return q4_kv_assign(step, block_table, held, past_lens, new_lens, free_pages, free_count, parents)
    dev = step.gpu
    if not isinstance(block_table, torch.Tensor) or block_table.dtype is not torch.int32:
        raise TypeError("block_table must be an int32 tensor")
    if block_table.get_device() != dev:
        raise ValueError("block_table must be on GPU %d, is on %s" % (dev, block_table.device))
    if tuple(block_table.shape) != (step.seqs, step.table_pages) or (block_table.stride(1) != 1 and step.table_pages != 1):
        raise ValueError("block_table must be [%d, %d] with consecutive entries" % (step.seqs, step.table_pages))
    b, i32 = step.seqs, torch.int32
    d = StepDesc.from_buffer_copy(step._desc)
    d.table_in, d.table_in_stride = block_table.data_ptr(), block_table.stride(0)
    d.held_in, d.past_len = _vector(held, i32, "held", b, dev), _vector(past_lens, i32, "past_lens", b, dev)
    d.new_len, d.free_pages = _vector(new_lens, i32, "new_lens", b, dev), _vector(free_pages, i32, "free_pages", None, dev)
    d.free_capacity, d.free_count = free_pages.shape[0], _vector(free_count, i32, "free_count", 1, dev)
    if parents is not None:
        d.parents = _vector(parents, i32, "parents", step.tokens, dev)
    status = (_lib or load_library()).q4_kv_assign(ctypes.byref(d), _current_stream(dev))
    if status:
        _check(status)
    return step


def _gain(t, name: str, n: int, gpu: int):
    if t is None:
        return None, 0
    kind = _TYPES.get(getattr(t, "dtype", None))
    if kind is None:
        raise TypeError("%s must be a float16, bfloat16 or float32 tensor" % name)
    return _vector(t, t.dtype, name, n, gpu), kind


def q4_norm_rope(x: torch.Tensor, gain: torch.Tensor | None, eps: float = 1e-6, positions: torch.Tensor | None = None,
                 inv_freq: torch.Tensor | None = None, layout: str = "half", mscale: float = 1.0,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q4_rope behind a norm of each head: x [T, H, D] * gain [D] / sqrt(mean(x^2) + eps) (gain None: ones; float16,
    bfloat16 or float32), then turned as by q4_rope; without inv_freq the norm alone.  Statistics and rotation in 32
    bits, rounded once.  out: like x in shape, of any of the types, and may be x itself.  No tokens: nothing to do."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be on a GPU")
    on = _on(dev, stream)
    if on is not None:
        with on:
            return q4_norm_rope(x, gain, eps, positions, inv_freq, layout, mscale, out)
    hx = _heads(x, "x", dev)
    t, h, d = x.shape
    if out is None:
        out = x.new_empty((t, h, d))
    elif out.shape != x.shape:
        raise ValueError("out must have x's shape")
    ho = _heads(out, "out", dev)
    gp, gk = _gain(gain, "gain", d, dev)
    r, freq, pos = 0, None, None
    if inv_freq is not None:
        freq, r = _vector(inv_freq, torch.float64, "inv_freq", None, dev), inv_freq.shape[0]
    if positions is not None:
        pos = _vector(positions, torch.int32, "positions", t, dev)
    elif r:
        raise ValueError("inv_freq without positions")
    kind = _layout(layout)
    if t == 0:
        return out
    status = (_lib or load_library()).q4_norm_rope(
        ctypes.byref(hx), ctypes.byref(ho), gp, gk, eps, pos, freq if r else None, t, h, d, 2 * r, kind, mscale, _current_stream(dev))
    if status:
        _check(status)
    return out


def q4_kv_append_norm(cache: KVCache, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor | None = None,
                      k_gain: torch.Tensor | None = None, q_gain: torch.Tensor | None = None, eps: float = 1e-6,
                      inv_freq: torch.Tensor | None = None, layout: str = "half", mscale: float = 1.0,
                      positions: torch.Tensor | None = None, q_out: torch.Tensor | None = None, stream=None):
    """q4_kv_append with the norm of q4_norm_rope on the heads of k (and of q) before they turn; k_gain and q_gain [D],
    both of one type, None: ones.  positions (int32 [T]) give the angles, as the depths of a tree's tokens do
    (KVStep.positions); the places in the cache are the batch's."""
    on = _on(cache.gpu, stream)
    if on is not None:
        with on:
            return q4_kv_append_norm(cache, batch, k, v, q, k_gain, q_gain, eps, inv_freq, layout, mscale, positions, q_out)
    _same_device(cache, batch)
    dev = cache.gpu
    hk, hv = _heads(k, "k", dev), _heads(v, "v", dev)
    t = k.shape[0]
    if k.shape != v.shape or k.shape[1] != cache.kv_heads or k.shape[2] != cache.head_dim:
        raise ValueError("k and v must be [T, %d, %d]" % (cache.kv_heads, cache.head_dim))
    rq = ro = None
    heads = 0
    if q is not None:
        hq = _heads(q, "q", dev)
        heads = q.shape[1]
        if q.shape[0] != t or q.shape[2] != cache.head_dim:
            raise ValueError("q must be [T=%d, heads, %d]" % (t, cache.head_dim))
        if q_out is None:
            q_out = torch.empty((t, heads, cache.head_dim), dtype=cache.dtype, device=cache.device)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        ho = _heads(q_out, "q_out", dev)
        rq, ro = ctypes.byref(hq), ctypes.byref(ho)
    elif q_out is not None:
        raise ValueError("q_out without q")
    (gq, kind_q), (gk, kind_k) = _gain(q_gain, "q_gain", cache.head_dim, dev), _gain(k_gain, "k_gain", cache.head_dim, dev)
    if q_gain is not None and k_gain is not None and kind_q != kind_k:
        raise TypeError("q_gain and k_gain must have one type")
    r, freq = 0, None
    if inv_freq is not None:
        freq = _vector(inv_freq, torch.float64, "inv_freq", None, dev)
        r = inv_freq.shape[0]
    pos = None if positions is None else _vector(positions, torch.int32, "positions", t, dev)
    kind = _layout(layout)
    if t == 0:
        return q_out
    status = (_lib or load_library()).q4_kv_append_norm(
        cache._ref, batch._ref, ctypes.byref(hk), ctypes.byref(hv), rq, ro, heads, t, gq, gk, kind_q if q_gain is not None else kind_k,
        eps, pos, freq if r else None, 2 * r, kind, mscale, _current_stream(dev))
    if status:
        _check(status)
    return q_out


def _mask(mask: torch.Tensor, rows: int, gpu: int) -> int:
    """Address of masks int64 [rows, words], side by side."""
    if not isinstance(mask, torch.Tensor):
        raise TypeError("mask must be a torch.Tensor")
    if mask.dtype is not torch.int64:
        raise TypeError("mask must be int64, got %s" % mask.dtype)
    if mask.get_device() != gpu:
        raise ValueError("mask must be on GPU %d, is on %s" % (gpu, mask.device))
    if mask.dim() != 2 or mask.shape[0] != rows or mask.shape[1] < 1 or not mask.is_contiguous():
        raise ValueError("mask must be contiguous, [%d, words]" % rows)
    return mask.data_ptr()


def attention_tree_workspace_bytes(cache: KVCache, batch: KVBatch, q_heads: int, tokens: int, window: int = 0) -> int:
    """Bytes of the workspace q4_attention_tree needs for these sizes (0: none); smaller sizes may need more
    (attention_workspace_most)."""
    if tokens == 0:
        return 0
    with torch.cuda.device(cache.device):  # the work is cut for this device
        n = int(load_library().q4_attention_tree_workspace_bytes(cache._ref, batch._ref, q_heads, tokens, window))
    if n == 0 and last_error():
        raise Q4Error(Q4_ERR_INVALID_ARG, last_error())
    return n


def q4_attention_tree(cache: KVCache, batch: KVBatch, q: torch.Tensor, mask: torch.Tensor, scale: float | None = None,
                      window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q4_attention_paged for drafted trees: each new token sees the cached keys before its sequence's new ones (with
    window > 0 those from past + depth - window + 1 on, depth: the new tokens it sees beside itself) and the new tokens
    whose bits its mask has (int64 [T, words], bit j % 64 of word j / 64: the sequence's j-th; KVStep.mask), whatever the
    window: paths longer than it need masks without the tokens outside of it.  Append the new tokens first.  out, lse, workspace as there (attention_tree_workspace_bytes)."""
    on = _on(cache.gpu, stream)
    if on is not None:
        with on:
            return q4_attention_tree(cache, batch, q, mask, scale, window, out, lse, workspace)
    _same_device(cache, batch)
    dev = cache.gpu
    hq = _heads(q, "q", dev)
    t, h, d = q.shape
    if d != cache.head_dim:
        raise ValueError("q must be [T, heads, %d]" % cache.head_dim)
    mp = _mask(mask, t, dev)
    if out is None:
        out = q.new_empty((t, h, d))
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ho = _heads(out, "out", dev)
    lp = None
    if lse is not None:
        lp = _ptr(lse, torch.float32, "lse")
        if tuple(lse.shape) != (t, h) or lse.get_device() != dev:
            raise ValueError("lse must be float32 [T, heads] on %s" % cache.device)
    if t == 0:
        return out
    lib = _lib or load_library()
    wp, wb = None, 0
    if workspace is None:
        wb = lib.q4_attention_tree_workspace_bytes(cache._ref, batch._ref, h, t, window)
        if wb:
            workspace = torch.empty(wb, dtype=torch.uint8, device=cache.device)
            wp = workspace.data_ptr()
    else:
        wp, wb = _vector(workspace, torch.uint8, "workspace", None, dev), workspace.shape[0]
    status = lib.q4_attention_tree(cache._ref, batch._ref, ctypes.byref(hq), ctypes.byref(ho), mp, mask.shape[1], lp, h, t,
                                   scale if scale is not None else d ** -0.5, window, wp, wb, _current_stream(dev))
    if status:
        _check(status)
    return out


class LogitRules:
    """What q4_logits_argmax does to a step's logits; every part may be left out.  Tensors on the GPU, int32 unless
    noted, which the kernel reads when it runs: their contents may change between calls and replays of a graph.

      query_start [B + 1]      rows of each sequence; left out: row t is sequence t of `seqs` (any tensor by sequence
                               says how many)
      history [B, L], history_lens [B], prompt_lens [B]
                               the tokens behind a sequence, the first prompt_lens of them its prompt, the others its answer
      draft [T], mask [T, words] (int64)
                               drafted tokens: each row's answer goes on with those of its sequence that its mask names
                               (KVStep.mask); without mask with those up to its own
      repetition, presence, frequency [B], float32
                               logits of tokens seen are divided (above 0) or multiplied by repetition; those of the
                               answer's tokens lose presence, and frequency for each time
      bias_start [B + 1], bias_tokens [N], bias_values [N] (float32)
                               added to the logits of these tokens; of equal tokens the last counts
      allowed [R, ceil(V / 32)], allowed_rows [T]
                               bit v % 32 of word v / 32: v may be picked, by row of logits or by the row that allowed_rows
                               names (-1: all may)"""

    def __init__(self, query_start=None, history=None, history_lens=None, prompt_lens=None, draft=None, mask=None,
                 repetition=None, presence=None, frequency=None, bias_start=None, bias_tokens=None, bias_values=None,
                 allowed=None, allowed_rows=None, seqs: int | None = None):
        i32, f32 = torch.int32, torch.float32
        named = dict(query_start=query_start, history=history, history_lens=history_lens, prompt_lens=prompt_lens, draft=draft,
                     mask=mask, repetition=repetition, presence=presence, frequency=frequency, bias_start=bias_start,
                     bias_tokens=bias_tokens, bias_values=bias_values, allowed=allowed, allowed_rows=allowed_rows)
        given = [t for t in named.values() if t is not None]
        for name, t in named.items():
            if t is not None and not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch.Tensor" % name)
        if given and given[0].get_device() < 0:
            raise ValueError("the rules must be on a GPU")
        self.gpu = dev = given[0].get_device() if given else None
        self._keep = given
        d = self.desc = RulesDesc()
        sizes = [t.shape[0] - n for t, n in ((query_start, 1), (history, 0), (repetition, 0), (presence, 0), (frequency, 0),
                                             (bias_start, 1)) if t is not None]
        b = seqs if seqs is not None else sizes[0] if sizes else 0
        self.seqs = b
        if b < 1 and (sizes or seqs is not None):
            raise ValueError("no sequences")

        def vector(t, dtype, name, n):
            return None if t is None else _vector(t, dtype, name, n, dev)

        def table(t, name, dtype=i32):
            if t.dtype is not dtype:
                raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
            if t.get_device() != dev:
                raise ValueError("%s must be on GPU %d, is on %s" % (name, dev, t.device))
            if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] != 1):
                raise ValueError("%s must have two dimensions with consecutive entries" % name)
            return t.data_ptr()

        if (history is None) != (history_lens is None) or (prompt_lens is not None and history is None):
            raise ValueError("history goes with history_lens, prompt_lens with both")
        if mask is not None and draft is None:
            raise ValueError("a mask without draft")
        if len({bias_start is None, bias_tokens is None, bias_values is None}) > 1:
            raise ValueError("bias_start, bias_tokens and bias_values go together")
        if allowed_rows is not None and allowed is None:
            raise ValueError("allowed_rows without allowed")
        d.query_start = vector(query_start, i32, "query_start", b + 1)
        if history is not None:
            d.history, d.history_stride, d.history_tokens = table(history, "history"), history.stride(0), history.shape[1]
            if history.shape[0] != b:
                raise ValueError("history must have %d rows" % b)
        d.history_len, d.prompt_len = vector(history_lens, i32, "history_lens", b), vector(prompt_lens, i32, "prompt_lens", b)
        self.rows = None  # of the tensors by row of logits
        if draft is not None:
            d.draft, self.rows = vector(draft, i32, "draft", None), draft.shape[0]
        if mask is not None:
            d.mask, d.mask_words = _mask(mask, self.rows, dev), mask.shape[1]
        d.repetition, d.presence, d.frequency = (vector(t, f32, n, b) for t, n in (
            (repetition, "repetition"), (presence, "presence"), (frequency, "frequency")))
        if bias_start is not None:
            d.bias_start, d.biases = vector(bias_start, i32, "bias_start", b + 1), bias_tokens.shape[0]
            d.bias_tokens, d.bias_values = vector(bias_tokens, i32, "bias_tokens", None), vector(bias_values, f32, "bias_values", d.biases)
        self.words = None
        if allowed is not None:
            d.allowed, d.allowed_stride, d.allowed_rows = table(allowed, "allowed"), allowed.stride(0), allowed.shape[0]
            self.words = allowed.shape[1]
        if allowed_rows is not None:
            if self.rows is None:
                self.rows = allowed_rows.shape[0]
            d.allowed_row = vector(allowed_rows, i32, "allowed_rows", self.rows)
        d.seqs = b
        self._ref = ctypes.byref(d)


def logits_argmax_workspace_bytes(rows: int, vocab: int) -> int:
    """Bytes of workspace for q4_logits_argmax (0: none), enough for every call of up to so many rows and entries."""
    return int(load_library().q4_logits_argmax_workspace_bytes(rows, vocab))


def q4_logits_argmax(logits: torch.Tensor, rules: LogitRules | None = None, out: torch.Tensor | None = None,
                     tokens: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The greedy pick (int32 [T]) of logits [T, V] (float32, float16 or bfloat16, rows may lie apart) under `rules`:
    the lowest index of the largest, -1 for a row in which nothing above -infinity is left.  out (float32 [T, V], may
    be the logits themselves) receives the logits under the rules; workspace (uint8) at least
    logits_argmax_workspace_bytes.  No rows: nothing to do."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    dev = logits.get_device()
    if dev < 0:
        raise ValueError("logits must be on a GPU")
    on = _on(dev, stream)
    if on is not None:
        with on:
            return q4_logits_argmax(logits, rules, out, tokens, workspace)
    kind = _TYPES.get(logits.dtype)
    if kind is None:
        raise TypeError("logits must be float16, bfloat16 or float32, got %s" % logits.dtype)
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] != 1):
        raise ValueError("logits must be [rows, vocabulary] with consecutive entries")
    t, v = logits.shape
    rp = None
    if rules is not None:
        if rules.gpu is not None and rules.gpu != dev:
            raise ValueError("the rules are on GPU %d, the logits on %s" % (rules.gpu, logits.device))
        if rules.rows is not None and rules.rows != t:
            raise ValueError("draft and allowed_rows must have %d rows" % t)
        if rules.words is not None and rules.words != (v + 31) // 32:
            raise ValueError("allowed must have %d words a row" % ((v + 31) // 32))
        if rules.desc.seqs:
            rp = rules._ref
        elif rules.gpu is not None:  # nothing by sequence: as many as there are rows
            d = RulesDesc.from_buffer_copy(rules.desc)
            d.seqs = max(t, 1)
            rp = ctypes.byref(d)
    op, os_ = None, 0
    if out is not None:
        if not isinstance(out, torch.Tensor) or out.dtype is not torch.float32:
            raise TypeError("out must be a float32 tensor")
        if out.shape != logits.shape or out.get_device() != dev or (out.stride(1) != 1 and v != 1):
            raise ValueError("out must be [%d, %d] on GPU %d with consecutive entries" % (t, v, dev))
        op, os_ = out.data_ptr(), out.stride(0)
    if tokens is None:
        tokens = torch.empty(t, dtype=torch.int32, device=logits.device)
    tp = _vector(tokens, torch.int32, "tokens", t, dev)
    if t == 0:
        return tokens
    lib = _lib or load_library()
    wp, wb = None, 0
    if workspace is None:
        wb = lib.q4_logits_argmax_workspace_bytes(t, v)
        if wb:
            workspace = torch.empty(wb, dtype=torch.uint8, device=logits.device)
            wp = workspace.data_ptr()
    else:
        wp, wb = _vector(workspace, torch.uint8, "workspace", None, dev), workspace.shape[0]
    status = lib.q4_logits_argmax(logits.data_ptr(), kind, logits.stride(0), t, v, rp, op, os_, tp, wp, wb, _current_stream(dev))
    if status:
        _check(status)
    return tokens


def q4_tree_accept(batch: KVBatch, choice: torch.Tensor, draft: torch.Tensor, parents: torch.Tensor | None = None,
                   history: torch.Tensor | None = None, out=None, stream=None, slots: torch.Tensor | None = None):
    """(accepted [B], next_tokens [B], path [T], lens [B]), int32, of the trunk's choice behind each drafted token and
    the tokens themselves (int32 [T]): from each sequence's first new token the lowest child (parents as in
    q4_kv_assign; None: a chain) drafted as what was chosen, and so on.  accepted counts the path's tokens, the first
    included; next_tokens is the choice behind its last; path has their indices in the sequence's first rows, then -1;
    lens the context with them alone.  history (int32 [B, L]) receives the path's tokens at the places they have.
    slots (int64 [T]; left out: those of the KVStep whose batch this is): tokens whose slot is below 0, for want of a page
    or behind the table's end, are on no path; a sequence whose first one has none takes nothing (accepted 0), and its
    next_tokens is that token again.
    T is at least 1.  out: the four tensors to write.  Rows of no sequence are left as they are (in a path made here: undefined)."""
    on = _on(batch.gpu, stream)
    if on is not None:
        with on:
            return q4_tree_accept(batch, choice, draft, parents, history, out, None, slots)
    dev, b, i32 = batch.gpu, batch.seqs, torch.int32
    cp = _vector(choice, i32, "choice", None, dev)
    t = choice.shape[0]
    dp = _vector(draft, i32, "draft", t, dev)
    pp = None if parents is None else _vector(parents, i32, "parents", t, dev)
    hp, hs, hn = None, 0, 0
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dtype is not i32:
            raise TypeError("history must be an int32 tensor")
        if history.dim() != 2 or history.shape[0] != b or history.get_device() != dev or (history.stride(1) != 1 and history.shape[1] != 1):
            raise ValueError("history must be [%d, entries] on GPU %d with consecutive entries" % (b, dev))
        hp, hs, hn = history.data_ptr(), history.stride(0), history.shape[1]
    if t == 0:
        raise ValueError("no tokens")
    if out is None:
        made = choice.new_empty((3 * b + t,))
        out = made.split_with_sizes((b, b, t, b))
        ap = made.data_ptr()
        np_, rp, lp = ap + 4 * b, ap + 8 * b, ap + 8 * b + 4 * t
    else:
        accepted, following, path, lens = out
        ap, np_, lp = _vector(accepted, i32, "accepted", b, dev), _vector(following, i32, "next_tokens", b, dev), _vector(lens, i32, "lens", b, dev)
        rp = _vector(path, i32, "path", t, dev)
    sp, rows = None, t
    if slots is not None:
        sp = _vector(slots, torch.int64, "slots", t, dev)
    elif batch.slots is not None:  # (rows behind the step's are of no sequence)
        sp, rows = batch.slots.data_ptr(), min(t, batch.slots.shape[0])
    d = batch.desc
    status = (_lib or load_library()).q4_tree_accept_stored(
        d.query_start, d.context_len, b, cp, dp, pp, sp, rows, ap, np_, rp, lp, hp, hs, hn, _current_stream(dev))
    if status:
        _check(status)
    return out


class KVLayers:
    """The caches of a model's layers, alike in sizes and strides, for q4_kv_move."""

    def __init__(self, caches):
        self.caches = list(caches)
        if not self.caches:
            raise ValueError("no caches")
        self.gpu, self.device = self.caches[0].gpu, self.caches[0].device
        if any(c.gpu != self.gpu for c in self.caches):
            raise ValueError("the caches must be on one GPU")
        self.desc = (CacheDesc * len(self.caches))(*(c.desc for c in self.caches))


def q4_kv_move(layers, batch: KVBatch, path: torch.Tensor, accepted: torch.Tensor, stream=None) -> None:
    """Move the keys and values of each sequence's path (path [T], accepted [B], int32, of q4_tree_accept) to the places
    behind each other that its tokens have, in the caches of all layers (a KVLayers, or one KVCache)."""
    if isinstance(layers, KVCache):
        layers = KVLayers([layers])
    on = _on(layers.gpu, stream)
    if on is not None:
        with on:
            return q4_kv_move(layers, batch, path, accepted)
    _same_device(layers, batch)
    dev = layers.gpu
    pp, ap = _vector(path, torch.int32, "path", None, dev), _vector(accepted, torch.int32, "accepted", batch.seqs, dev)
    if path.shape[0] == 0:
        return
    status = (_lib or load_library()).q4_kv_move(layers.desc, len(layers.caches), batch._ref, pp, ap, path.shape[0], _current_stream(dev))
    if status:
        _check(status)


# Short names.
gemv = q4_0_gemv
gemm_smallm = q4_0_gemm_smallm
gemm_prefill = q4_0_gemm_prefill
rope = q4_rope
kv_append = q4_kv_append
attention_paged = q4_attention_paged
kv_assign = q4_kv_assign
norm_rope = q4_norm_rope
kv_append_norm = q4_kv_append_norm
attention_tree = q4_attention_tree
logits_argmax = q4_logits_argmax
tree_accept = q4_tree_accept
kv_move = q4_kv_move
