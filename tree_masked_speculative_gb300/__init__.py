"""GB300 tree-verify attention: Python binding of the C ABI in include/tree_attn.h.

Every function here only marshals arguments (torch tensors -> pointer, byte
count, dtype code; the current CUDA stream) into the C library; all work runs
in the library's CUDA kernels.  Importing this module loads the in-tree
``_build/libtree_attn.so`` (compiling it first when it is missing or older than
its sources) and raises if that fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch

from . import build as _build_mod

__all__ = [
    "TA_OK", "TreeParams", "QuantParams", "TreeAttentionError", "lib", "library_path",
    "tree_attn_tmp_bytes", "tree_attn_num_splits", "tree_attn_workspace_bytes", "tree_attn_fwd",
    "tree_attn_fwd_causal", "tree_attn_fwd_parents", "tree_attn_fwd_ex", "tree_attn_status_offset",
    "tree_attn_reduce", "tree_attn_fwd_noalloc", "quant_sdpa_num_splits", "quant_sdpa_tmp_bytes",
    "quant_sdpa_fwd", "ta_last_error", "ta_launch_count", "quant_sdpa_uses_tensor_cores",
    "quant_sdpa_kernel_family", "KERNEL_WARP_MMA",
    "ta_test_quant_sdpa_fwd_wait_limit", "quant_sdpa_fwd_tree", "tree_attention", "quant_sdpa", "tree_params", "quant_params",
    "tree_mask_build", "TreeOptions", "KERNEL_AUTO", "KERNEL_CUDA_CORES", "KERNEL_TENSOR_CORES",
    "PlanParams", "AppendParams", "PagedParams", "PromptParams", "PagedStep", "paged_plan", "paged_append",
    "paged_attention", "paged_attention_workspace", "paged_attn_workspace_bytes", "prompt_attention",
    "prompt_attention_workspace", "prompt_attn_workspace_bytes", "ta_test_paged_attn_fwd_wait_limit",
    "ta_test_paged_quant_attn_fwd_wait_limit",
    "RotaryAppendParams", "QuantAppendParams", "PagedQuantParams", "PagedQuantCache", "paged_append_rotary",
    "paged_quant_cache", "paged_quant_append", "paged_quant_read", "paged_quant_attention",
    "paged_quant_attention_workspace", "paged_quant_attn_workspace_bytes", "rotary_table",
]

TA_OK, TA_ERR_CUDA = 0, 5
TA_F32, TA_F16, TA_BF16, TA_U32, TA_I32, TA_I64 = 0, 1, 2, 3, 4, 5
KERNEL_AUTO, KERNEL_CUDA_CORES, KERNEL_TENSOR_CORES, KERNEL_WARP_MMA = 0, 1, 2, 3
MASK_DENSE, MASK_CAUSAL, MASK_PARENTS = 0, 1, 2
STATUS_NAMES = {0: "TA_OK", 1: "TA_ERR_INVALID_ARGUMENT", 2: "TA_ERR_BUFFER_TOO_SMALL",
                3: "TA_ERR_OVERFLOW", 4: "TA_ERR_UNSUPPORTED", 5: "TA_ERR_CUDA"}


class TreeAttentionError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), message))
        self.status = status


class Buf(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("bytes", ctypes.c_uint64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class TreeParams(ctypes.Structure):
    _fields_ = [("n_heads", ctypes.c_uint32), ("n_kv_heads", ctypes.c_uint32),
                ("head_dim", ctypes.c_uint32), ("kv_seq_len", ctypes.c_uint32),
                ("kv_capacity", ctypes.c_uint32), ("scale", ctypes.c_float), ("nwg", ctypes.c_uint32),
                ("q_l", ctypes.c_uint32), ("mask_stride", ctypes.c_uint32)]


class QuantParams(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_uint32), ("n_q_heads", ctypes.c_uint32),
                ("n_kv_heads", ctypes.c_uint32), ("dim", ctypes.c_uint32), ("tokens", ctypes.c_uint32),
                ("bits", ctypes.c_uint32), ("group_size", ctypes.c_uint32),
                ("has_sinks", ctypes.c_uint32), ("window_size", ctypes.c_uint32),
                ("scale", ctypes.c_float), ("nwg", ctypes.c_uint32), ("kernel", ctypes.c_uint32)]


class TreeOptions(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("mask_kind", ctypes.c_int32), ("window_start", ctypes.c_uint32),
                ("reserved", ctypes.c_int32)]


class PlanParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("batch", "page_size", "max_pages", "capacity", "max_tokens",
                                               "reserved")]


class AppendParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in ("tokens", "n_kv_heads", "head_dim", "page_size", "n_pages",
                                                "reserved")] +
                [(n, ctypes.c_uint64) for n in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride",
                                                "page_stride", "head_stride", "token_stride")])


class PagedParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in ("batch", "n_heads", "n_kv_heads", "head_dim", "tokens", "max_q_len",
                                                "window", "page_size", "n_pages", "max_pages", "kernel")] +
                [("scale", ctypes.c_float)] +
                [(n, ctypes.c_uint64) for n in ("q_token_stride", "q_head_stride", "out_token_stride",
                                                "out_head_stride", "page_stride", "head_stride", "token_stride")])


class PromptParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in ("batch", "n_heads", "n_kv_heads", "head_dim", "tokens", "window",
                                                "kernel")] +
                [("scale", ctypes.c_float)] +
                [(n, ctypes.c_uint64) for n in ("q_token_stride", "q_head_stride", "out_token_stride",
                                                "out_head_stride", "k_token_stride", "k_head_stride",
                                                "v_token_stride", "v_head_stride")])


class RotaryAppendParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in ("tokens", "n_heads", "n_kv_heads", "head_dim", "page_size", "n_pages",
                                                "rotary_dim", "interleaved", "max_positions", "reserved")] +
                [(n, ctypes.c_uint64) for n in ("q_token_stride", "q_head_stride", "q_out_token_stride",
                                                "q_out_head_stride", "k_token_stride", "k_head_stride",
                                                "v_token_stride", "v_head_stride", "page_stride", "head_stride",
                                                "token_stride")])


class QuantAppendParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in ("tokens", "n_heads", "n_kv_heads", "head_dim", "page_size", "n_pages",
                                                "group_size", "rotary_dim", "interleaved", "max_positions")] +
                [(n, ctypes.c_uint64) for n in ("q_token_stride", "q_head_stride", "q_out_token_stride",
                                                "q_out_head_stride", "k_token_stride", "k_head_stride",
                                                "v_token_stride", "v_head_stride", "codes_page_stride",
                                                "codes_head_stride", "codes_token_stride", "affine_page_stride",
                                                "affine_head_stride", "affine_token_stride")])


class PagedQuantParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint32) for n in ("batch", "n_heads", "n_kv_heads", "head_dim", "tokens", "max_q_len",
                                                "window", "page_size", "n_pages", "max_pages", "group_size",
                                                "kernel")] +
                [("scale", ctypes.c_float), ("reserved", ctypes.c_uint32)] +
                [(n, ctypes.c_uint64) for n in ("q_token_stride", "q_head_stride", "out_token_stride",
                                                "out_head_stride", "codes_page_stride", "codes_head_stride",
                                                "codes_token_stride", "affine_page_stride", "affine_head_stride",
                                                "affine_token_stride")])


def library_path() -> str:
    return _build_mod.LIB


def _load() -> ctypes.CDLL:
    # (Re)build the in-tree library when it is missing or older than its
    # sources; a failed build raises, so the package never imports without it.
    path = _build_mod.build()
    if not os.path.exists(path):
        raise ImportError("tree_masked_speculative_gb300: %s is missing" % path)
    L = ctypes.CDLL(path)
    P, B = ctypes.c_void_p, ctypes.POINTER(Buf)
    PT, PQ = ctypes.POINTER(TreeParams), ctypes.POINTER(QuantParams)
    u32 = ctypes.c_uint32
    L.tree_attn_tmp_bytes.argtypes = [u32, u32, u32, u32]
    L.tree_attn_tmp_bytes.restype = ctypes.c_size_t
    L.tree_attn_num_splits.argtypes = [PT]
    L.tree_attn_num_splits.restype = u32
    L.tree_attn_workspace_bytes.argtypes = [PT]
    L.tree_attn_workspace_bytes.restype = ctypes.c_size_t
    L.tree_attn_fwd.argtypes = [PT, B, B, B, B, B, B, P]
    L.tree_attn_fwd.restype = ctypes.c_int
    L.tree_attn_fwd_causal.argtypes = [PT, u32, B, B, B, B, B, P]
    L.tree_attn_fwd_causal.restype = ctypes.c_int
    L.tree_attn_fwd_parents.argtypes = [PT, B, B, B, B, B, B, P]
    L.tree_attn_fwd_parents.restype = ctypes.c_int
    L.tree_attn_fwd_ex.argtypes = [PT, ctypes.POINTER(TreeOptions), B, B, B, B, B, B, P]
    L.tree_attn_fwd_ex.restype = ctypes.c_int
    L.tree_attn_status_offset.argtypes = [PT]
    L.tree_attn_status_offset.restype = ctypes.c_size_t
    L.tree_attn_reduce.argtypes = [PT, B, B, P]
    L.tree_attn_reduce.restype = ctypes.c_int
    L.tree_attn_fwd_noalloc.argtypes = [PT, B, B, B, B, B, P]
    L.tree_attn_fwd_noalloc.restype = ctypes.c_int
    L.quant_sdpa_num_splits.argtypes = [PQ]
    L.quant_sdpa_num_splits.restype = u32
    L.quant_sdpa_tmp_bytes.argtypes = [PQ]
    L.quant_sdpa_tmp_bytes.restype = ctypes.c_size_t
    L.quant_sdpa_fwd.argtypes = [PQ] + [B] * 12 + [P]
    L.quant_sdpa_fwd.restype = ctypes.c_int
    L.ta_last_error.argtypes = []
    L.ta_last_error.restype = ctypes.c_char_p
    L.ta_launch_count.argtypes = []
    L.ta_launch_count.restype = ctypes.c_uint64
    L.quant_sdpa_fwd_tree.argtypes = [PQ, u32] + [B] * 12 + [P]
    L.quant_sdpa_fwd_tree.restype = ctypes.c_int
    L.ta_test_quant_sdpa_fwd_wait_limit.argtypes = [u32, PQ] + [B] * 12 + [P]
    L.ta_test_quant_sdpa_fwd_wait_limit.restype = ctypes.c_int
    L.quant_sdpa_uses_tensor_cores.argtypes = [PQ]
    L.quant_sdpa_uses_tensor_cores.restype = ctypes.c_int
    L.quant_sdpa_kernel_family.argtypes = [PQ]
    L.quant_sdpa_kernel_family.restype = ctypes.c_int
    L.tree_mask_build.argtypes = [PT, B, B, P]
    L.tree_mask_build.restype = ctypes.c_int
    L.paged_plan_build.argtypes = [ctypes.POINTER(PlanParams)] + [B] * 13 + [P]
    L.paged_plan_build.restype = ctypes.c_int
    L.paged_kv_append.argtypes = [ctypes.POINTER(AppendParams)] + [B] * 5 + [P]
    L.paged_kv_append.restype = ctypes.c_int
    L.paged_attn_workspace_bytes.argtypes = [ctypes.POINTER(PagedParams)]
    L.paged_attn_workspace_bytes.restype = ctypes.c_size_t
    L.paged_attn_fwd.argtypes = [ctypes.POINTER(PagedParams)] + [B] * 9 + [P]
    L.paged_attn_fwd.restype = ctypes.c_int
    L.ta_test_paged_attn_fwd_wait_limit.argtypes = [u32, ctypes.POINTER(PagedParams)] + [B] * 9 + [P]
    L.ta_test_paged_attn_fwd_wait_limit.restype = ctypes.c_int
    L.ta_test_paged_quant_attn_fwd_wait_limit.argtypes = [u32, ctypes.POINTER(PagedQuantParams)] + [B] * 11 + [P]
    L.ta_test_paged_quant_attn_fwd_wait_limit.restype = ctypes.c_int
    L.prompt_attn_workspace_bytes.argtypes = [ctypes.POINTER(PromptParams)]
    L.prompt_attn_workspace_bytes.restype = ctypes.c_size_t
    L.prompt_attn_fwd.argtypes = [ctypes.POINTER(PromptParams)] + [B] * 6 + [P]
    L.prompt_attn_fwd.restype = ctypes.c_int
    L.paged_rotary_append.argtypes = [ctypes.POINTER(RotaryAppendParams)] + [B] * 9 + [P]
    L.paged_rotary_append.restype = ctypes.c_int
    L.paged_quant_append.argtypes = [ctypes.POINTER(QuantAppendParams)] + [B] * 11 + [P]
    L.paged_quant_append.restype = ctypes.c_int
    L.paged_quant_read.argtypes = [ctypes.POINTER(QuantAppendParams)] + [B] * 7 + [P]
    L.paged_quant_read.restype = ctypes.c_int
    L.paged_quant_attn_workspace_bytes.argtypes = [ctypes.POINTER(PagedQuantParams)]
    L.paged_quant_attn_workspace_bytes.restype = ctypes.c_size_t
    L.paged_quant_attn_fwd.argtypes = [ctypes.POINTER(PagedQuantParams)] + [B] * 11 + [P]
    L.paged_quant_attn_fwd.restype = ctypes.c_int
    return L


lib = _load()

_DTYPE_CODE = {torch.float32: TA_F32, torch.float16: TA_F16, torch.bfloat16: TA_BF16,
               torch.int32: TA_U32}
_U32 = getattr(torch, "uint32", None)
if _U32 is not None:
    _DTYPE_CODE[_U32] = TA_U32


def buf(t: Optional[torch.Tensor], dtype_code: Optional[int] = None):
    """Describe a tensor as a ta_buf passed by reference; None = absent buffer
    (a NULL descriptor).  int32 tensors are passed as U32 (packed words, bool
    masks)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    code = _DTYPE_CODE.get(t.dtype) if dtype_code is None else dtype_code
    if code is None:
        raise ValueError("unsupported dtype %s" % t.dtype)
    return ctypes.byref(Buf(t.data_ptr(), t.numel() * t.element_size(), code, 0))


def raw_buf(ptr: int, nbytes: int, dtype_code: int) -> Buf:
    return Buf(ptr, nbytes, dtype_code, 0)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status: int):
    if status != TA_OK:
        raise TreeAttentionError(status, lib.ta_last_error().decode())


def ta_last_error() -> str:
    return lib.ta_last_error().decode()


def ta_launch_count() -> int:
    return int(lib.ta_launch_count())


def quant_sdpa_uses_tensor_cores(p: QuantParams) -> int:
    return int(lib.quant_sdpa_uses_tensor_cores(ctypes.byref(p)))


def quant_sdpa_kernel_family(p: QuantParams) -> int:
    return int(lib.quant_sdpa_kernel_family(ctypes.byref(p)))


def tree_params(n_heads, n_kv_heads, head_dim, kv_seq_len, kv_capacity, scale, q_l, mask_stride,
                nwg=0) -> TreeParams:
    return TreeParams(n_heads, n_kv_heads, head_dim, kv_seq_len, kv_capacity, scale, nwg, q_l,
                      mask_stride)


def quant_params(batch, n_q_heads, n_kv_heads, dim, tokens, bits, group_size, has_sinks,
                 window_size, scale, nwg=0, kernel=KERNEL_AUTO) -> QuantParams:
    return QuantParams(batch, n_q_heads, n_kv_heads, dim, tokens, bits, group_size, has_sinks,
                       window_size, scale, nwg, kernel)


def tree_attn_tmp_bytes(n_heads: int, head_dim: int, q_l: int, nwg: int) -> int:
    return int(lib.tree_attn_tmp_bytes(n_heads, head_dim, q_l, nwg))


def tree_attn_num_splits(p: TreeParams) -> int:
    return int(lib.tree_attn_num_splits(ctypes.byref(p)))


def tree_attn_workspace_bytes(p: TreeParams) -> int:
    return int(lib.tree_attn_workspace_bytes(ctypes.byref(p)))


def tree_attn_fwd(p: TreeParams, q, k, v, mask, tmp, out, stream=None):
    _check(lib.tree_attn_fwd(ctypes.byref(p), buf(q), buf(k), buf(v), buf(mask), buf(tmp),
                             buf(out), _stream(stream)))


def tree_attn_fwd_parents(p: TreeParams, parents, q, k, v, tmp, out, stream=None):
    _check(lib.tree_attn_fwd_parents(ctypes.byref(p), buf(parents, TA_I32), buf(q), buf(k), buf(v), buf(tmp),
                                     buf(out), _stream(stream)))


def tree_attn_fwd_causal(p: TreeParams, window_start: int, q, k, v, tmp, out, stream=None):
    _check(lib.tree_attn_fwd_causal(ctypes.byref(p), window_start, buf(q), buf(k), buf(v),
                                    buf(tmp), buf(out), _stream(stream)))


def tree_attn_fwd_ex(p: TreeParams, kernel: int, mask_kind: int, window_start: int, q, k, v, mask, tmp, out,
                     stream=None):
    """Main pass with an explicit kernel family (KERNEL_*) and mask form (MASK_*:
    `mask` is the dense mask, unused, or the int32 parent array)."""
    o = TreeOptions(kernel, mask_kind, window_start, 0)
    m = buf(mask, TA_I32) if mask_kind == MASK_PARENTS else (buf(mask) if mask_kind == MASK_DENSE else None)
    _check(lib.tree_attn_fwd_ex(ctypes.byref(p), ctypes.byref(o), buf(q), buf(k), buf(v), m, buf(tmp), buf(out),
                                _stream(stream)))


def tree_attn_status_offset(p: TreeParams) -> int:
    return int(lib.tree_attn_status_offset(ctypes.byref(p)))


def tree_attn_reduce(p: TreeParams, tmp, out, stream=None):
    _check(lib.tree_attn_reduce(ctypes.byref(p), buf(tmp), buf(out), _stream(stream)))


def tree_attn_fwd_noalloc(p: TreeParams, q, k, v, mask, out, stream=None):
    """Main pass + merge with the library's static scratch (no tmp buffer); for
    callers that cannot allocate device memory.  mask=None: implicit causal."""
    _check(lib.tree_attn_fwd_noalloc(ctypes.byref(p), buf(q), buf(k), buf(v), buf(mask), buf(out),
                                     _stream(stream)))


def quant_sdpa_num_splits(p: QuantParams) -> int:
    return int(lib.quant_sdpa_num_splits(ctypes.byref(p)))


def quant_sdpa_tmp_bytes(p: QuantParams) -> int:
    return int(lib.quant_sdpa_tmp_bytes(ctypes.byref(p)))


def _quant_bufs(queries, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, sinks, mask_bool,
                mask_float, tmp, out):
    return (buf(queries), buf(k_packed, TA_U32), buf(k_scales), buf(k_biases), buf(v_packed, TA_U32),
            buf(v_scales), buf(v_biases), buf(sinks), buf(mask_bool, TA_U32) if mask_bool is not None else None,
            buf(mask_float), buf(tmp), buf(out))


def quant_sdpa_fwd(p: QuantParams, queries, k_packed, k_scales, k_biases, v_packed, v_scales,
                   v_biases, sinks, mask_bool, mask_float, tmp, out, stream=None):
    _check(lib.quant_sdpa_fwd(ctypes.byref(p), *_quant_bufs(queries, k_packed, k_scales, k_biases, v_packed,
                                                            v_scales, v_biases, sinks, mask_bool, mask_float,
                                                            tmp, out), _stream(stream)))


def quant_sdpa_fwd_tree(p: QuantParams, q_l: int, parents, queries, k_packed, k_scales, k_biases, v_packed,
                        v_scales, v_biases, sinks, mask_bool, tmp, out, stream=None):
    """Quantized-KV attention of draft-tree rows (row q = node q % q_l) with the
    tree mask as the int32 parent array of the last q_l tokens."""
    b = _quant_bufs(queries, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, sinks, mask_bool, None,
                    tmp, out)
    _check(lib.quant_sdpa_fwd_tree(ctypes.byref(p), q_l, buf(parents, TA_I32), *b[:9], b[10], b[11],
                                   _stream(stream)))


def ta_test_quant_sdpa_fwd_wait_limit(first_wait_polls: int, p: QuantParams, queries, k_packed, k_scales,
                                      k_biases, v_packed, v_scales, v_biases, sinks, mask_bool, mask_float, tmp,
                                      out, stream=None):
    """Test hook: quant_sdpa_fwd (CUDA-core kernel) whose first copy wait per CTA
    gives up after `first_wait_polls` polls (0: at once)."""
    _check(lib.ta_test_quant_sdpa_fwd_wait_limit(first_wait_polls, ctypes.byref(p),
                                                 *_quant_bufs(queries, k_packed, k_scales, k_biases, v_packed,
                                                              v_scales, v_biases, sinks, mask_bool, mask_float,
                                                              tmp, out), _stream(stream)))


# ------------------------------------------------------------- conveniences
def tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, mask: Optional[torch.Tensor],
                   *, n_heads: int, n_kv_heads: int, kv_seq_len: int, scale: float,
                   mask_stride: Optional[int] = None, nwg: int = 0, window_start: int = 0,
                   tmp: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   parents: Optional[torch.Tensor] = None, kernel: int = KERNEL_AUTO,
                   stream=None) -> torch.Tensor:
    """One verify step (main pass + reduce) on device tensors.  mask=None uses the
    implicit causal mask starting at window_start, or, with `parents` (int32
    [q_l] on the device), the tree mask of that parent array.  `kernel` picks
    the main pass's kernel family (KERNEL_*).  Returns out [q_l, n_heads, D]."""
    H, L, D = q.shape
    C = k.shape[1]
    stride = mask_stride if mask_stride is not None else (mask.shape[1] if mask is not None else kv_seq_len)
    p = tree_params(n_heads, n_kv_heads, D, kv_seq_len, C, scale, L, stride, nwg)
    if tmp is None:
        ws = tree_attn_workspace_bytes(p)
        if ws >= 2 ** 63:
            raise TreeAttentionError(1, "invalid tree-attention parameters")
        tmp = torch.empty((ws + 3) // 4, dtype=torch.float32, device=q.device)
    if out is None:
        out = torch.empty((L, n_heads, D), dtype=torch.float32, device=q.device)
    if parents is not None:
        if mask is not None:
            raise ValueError("give either a dense mask or a parent array, not both")
        tree_attn_fwd_ex(p, kernel, MASK_PARENTS, 0, q, k, v, parents, tmp, out, stream)
    elif mask is None:
        tree_attn_fwd_ex(p, kernel, MASK_CAUSAL, window_start, q, k, v, None, tmp, out, stream)
    else:
        tree_attn_fwd_ex(p, kernel, MASK_DENSE, 0, q, k, v, mask, tmp, out, stream)
    tree_attn_reduce(p, tmp, out, stream)
    return out


def quant_sdpa(inputs: dict, *, batch: int, n_q_heads: int, n_kv_heads: int, dim: int, tokens: int,
               bits: int, group_size: int, has_sinks: int, window_size: int, scale: float,
               nwg: int = 0, out_dtype: Optional[torch.dtype] = None, tmp=None, out=None,
               kernel: int = KERNEL_AUTO, tree_parents: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Quantized-KV attention on device tensors (dict as made by workloads.make_quant_inputs).
    With `tree_parents` (int32 [q_l] on the device) the rows are draft-tree nodes
    (row q = node q % q_l) masked by that tree over the last q_l tokens, and the
    dict's float mask is not used."""
    p = quant_params(batch, n_q_heads, n_kv_heads, dim, tokens, bits, group_size, has_sinks,
                     window_size, scale, nwg, kernel)
    dev = inputs["queries"].device
    if tmp is None:
        nb = quant_sdpa_tmp_bytes(p)
        if nb >= 2 ** 63:
            raise TreeAttentionError(1, "invalid quantized-SDPA parameters")
        tmp = torch.zeros(max(1, (nb + 3) // 4), dtype=torch.float32, device=dev)   # error word = 0
    if out is None:
        out = torch.empty((batch * n_q_heads, dim), dtype=out_dtype or inputs["queries"].dtype,
                          device=dev)
    if tree_parents is not None:
        quant_sdpa_fwd_tree(p, int(tree_parents.numel()), tree_parents, inputs["queries"], inputs["k_packed"],
                            inputs["k_scales"], inputs["k_biases"], inputs["v_packed"], inputs["v_scales"],
                            inputs["v_biases"], inputs["sinks"] if has_sinks else None, inputs.get("mask_bool"),
                            tmp, out, stream)
        return out
    quant_sdpa_fwd(p, inputs["queries"], inputs["k_packed"], inputs["k_scales"], inputs["k_biases"],
                   inputs["v_packed"], inputs["v_scales"], inputs["v_biases"],
                   inputs["sinks"] if has_sinks else None, inputs.get("mask_bool"),
                   inputs.get("mask_float"), tmp, out, stream)
    return out


def tree_mask_build(p: TreeParams, parents: torch.Tensor, mask: torch.Tensor, stream=None):
    """Dense tree mask [q_l, mask_stride] f32 from parents [q_l] int32, on the device."""
    _check(lib.tree_mask_build(ctypes.byref(p), buf(parents, TA_I32), buf(mask), _stream(stream)))


# ------------------------------------------------------------------ serving
# Batched requests on a paged K/V cache.  A step plans its pages and slots
# (paged_plan), writes the new K/V rows of each layer (paged_append) and
# attends them (paged_attention); prompt_attention serves whole prompts whose
# K/V are at hand.  Every length is device data: nothing here waits for the GPU.

class PagedStep(NamedTuple):
    """What paged_plan writes: pages held and free after the step, row offsets
    [B + 1], key counts [B], and per new token (-1 behind the last) its cache
    slot (int64) and its position; `status` collects error bits."""
    held: torch.Tensor
    n_free: torch.Tensor
    cu_q: torch.Tensor
    kv_lens: torch.Tensor
    slot_map: torch.Tensor
    positions: torch.Tensor
    status: torch.Tensor


_SERVE_CODE = {torch.float32: TA_F32, torch.float16: TA_F16, torch.bfloat16: TA_BF16, torch.int32: TA_I32,
               torch.int64: TA_I64}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_this_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_BUF = "QQii"
_ABSENT = (0, 0, TA_F32, 0)


class _Entry:
    """A C entry point whose params struct and ta_bufs are packed into one block of
    memory a thread: a serving step makes these calls per layer, and building the
    ctypes objects one by one took longer than the small kernels."""

    def __init__(self, name: str, params: str, n_bufs: int):
        self.layout = struct.Struct("=" + params + _BUF * n_bufs)
        self.offsets = [0] + [struct.calcsize("=" + params) + 24 * i for i in range(n_bufs)]
        self.fn = ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * (n_bufs + 2))((name, lib))
        self.local = threading.local()

    def __call__(self, dev: int, *values):
        local = self.local
        try:
            mem, args = local.mem, local.args
        except AttributeError:
            mem = local.mem = ctypes.create_string_buffer(self.layout.size)
            base = ctypes.addressof(mem)
            args = local.args = tuple(ctypes.c_void_p(base + o) for o in self.offsets)
        try:
            self.layout.pack_into(mem, 0, *values)
        except (struct.error, OverflowError) as e:      # (a float past f32 raises the latter)
            raise ValueError("argument out of range: %s" % e) from None
        status = self.fn(*args, _raw_stream(dev))
        if status != TA_OK:
            raise TreeAttentionError(status, lib.ta_last_error().decode())


_plan_entry = _Entry("paged_plan_build", "6I", 13)
_append_entry = _Entry("paged_kv_append", "6I7Q", 5)
_paged_entry = _Entry("paged_attn_fwd", "11If7Q", 9)
_prompt_entry = _Entry("prompt_attn_fwd", "7If8Q", 6)
_rotary_entry = _Entry("paged_rotary_append", "10I11Q", 9)
_quant_append_entry = _Entry("paged_quant_append", "10I14Q", 11)
_quant_read_entry = _Entry("paged_quant_read", "10I14Q", 7)
_paged_quant_entry = _Entry("paged_quant_attn_fwd", "12IfI10Q", 11)


def _as_stream(stream, dev: int) -> torch.cuda.Stream:
    """`stream` (a torch stream or a handle) on the tensors' device.  The handles 0
    and cudaStreamLegacy (1) are the default stream's: torch would make a new stream
    of a 0."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        return torch.cuda.default_stream(dev) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device=dev)
    if stream.device.index != dev:
        raise ValueError("stream is on %s, the tensors are on cuda:%d" % (stream.device, dev))
    return stream


def _device_of(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0 or not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device, got %s" % t.device)
    return dev


def _flat(t: Optional[torch.Tensor], dev: int):
    """A contiguous tensor on device `dev` as the fields of a ta_buf."""
    if t is None:
        return _ABSENT
    if t.get_device() != dev:
        raise ValueError("all tensors must be on cuda:%d, got %s" % (dev, t.device))
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    code = _SERVE_CODE.get(t.dtype)
    if code is None:
        raise ValueError("unsupported dtype %s" % t.dtype)
    return t.data_ptr(), t.nbytes, code, 0


def _strided(t: torch.Tensor, dev: int, ndim: int, what: str):
    """A tensor with any outer strides as the fields of a ta_buf and its outer
    strides (0 for an axis of one entry, whose stride means nothing, and for a
    contiguous tensor)."""
    if t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got %d" % (what, ndim, t.dim()))
    if t.is_contiguous():
        return _flat(t, dev), (0,) * (ndim - 1)
    if t.get_device() != dev:
        raise ValueError("all tensors must be on cuda:%d, got %s" % (dev, t.device))
    code = _SERVE_CODE.get(t.dtype)
    if code is None:
        raise ValueError("unsupported dtype %s" % t.dtype)
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s: the last dimension must be contiguous" % what)
    extent, outer = shape[-1], []
    for n, s in zip(shape[:-1], stride[:-1]):
        if n > 1 and s == 0:
            raise ValueError("%s: a broadcast dimension is not supported" % what)
        outer.append(s if n > 1 else 0)
        extent += (n - 1) * s
    return (t.data_ptr(), extent * t.element_size() if t.numel() else 0, code, 0), outer


def _contiguous_default(strides, shape):
    """The strides with 0 (an axis of one entry) replaced by the contiguous
    layout's, which C reads 0 as."""
    full, step = [], shape[-1]
    for n in reversed(shape[1:-1]):
        full.append(step)
        step *= n
    full.append(step)
    full.reverse()
    return [s or f for s, f in zip(strides, full)]


def _cache_pair(k_cache, v_cache, dev):
    kb, ks = _strided(k_cache, dev, 4, "k_cache")
    vb, vs = _strided(v_cache, dev, 4, "v_cache")
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape")
    if any(ks) or any(vs):
        ks, vs = _contiguous_default(ks, k_cache.shape), _contiguous_default(vs, v_cache.shape)
        if ks != vs:
            raise ValueError("k_cache and v_cache must have the same strides")
    return kb, vb, ks


def _elsewhere(fn, dev, stream, args, kw):
    """The call made with `stream`, or with the tensors' device, current."""
    with torch.cuda.stream(_as_stream(stream, dev)) if stream is not None else torch.cuda.device(dev):
        return fn(*args, **kw)


def paged_plan(keep_lens: torch.Tensor, new_lens: torch.Tensor, held: torch.Tensor, block_table: torch.Tensor,
               free_pages: torch.Tensor, n_free: torch.Tensor, *, page_size: int, max_tokens: int,
               out=None, stream=None) -> PagedStep:
    """Plan a step: request b keeps keep_lens[b] cached tokens and gets
    new_lens[b] new ones (int32 [B]).  Pages it no longer needs go back to the
    stack free_pages[:n_free], pages it needs are taken from its top; block_table
    [B, max_pages] and free_pages are updated in place.  `out`: the seven tensors
    of a PagedStep to write into (its held and n_free may be the inputs)."""
    dev = _device_of(block_table)
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_plan, dev, stream, (keep_lens, new_lens, held, block_table, free_pages, n_free),
                          dict(page_size=page_size, max_tokens=max_tokens, out=out))
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch, max_pages]")
    batch, width = block_table.shape
    if out is None:
        def new(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=block_table.device)
        out = (new(batch), new(1), new(batch + 1), new(batch), new(max_tokens, torch.int64), new(max_tokens),
               torch.zeros(1, dtype=torch.int32, device=block_table.device))
    step = PagedStep(*out)
    _plan_entry(dev, batch, page_size, width, free_pages.numel(), max_tokens, 0, *_flat(keep_lens, dev),
                *_flat(new_lens, dev), *_flat(held, dev), *_flat(block_table, dev), *_flat(free_pages, dev),
                *_flat(n_free, dev), *_flat(step.held, dev), *_flat(step.n_free, dev), *_flat(step.cu_q, dev),
                *_flat(step.kv_lens, dev), *_flat(step.slot_map, dev), *_flat(step.positions, dev),
                *_flat(step.status, dev))
    return step


def paged_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slot_map: torch.Tensor, stream=None) -> None:
    """Write the rows k_new, v_new [T, Hk, D] to the slots slot_map [T] (int64) of
    the caches [n_pages, Hk, page_size, D]; slots outside the cache (-1) are
    skipped.  No two rows may have the same slot."""
    dev = _device_of(k_cache)
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_append, dev, stream, (k_new, v_new, k_cache, v_cache, slot_map), {})
    kn, ks = _strided(k_new, dev, 3, "k_new")
    vn, vs = _strided(v_new, dev, 3, "v_new")
    kb, vb, cs = _cache_pair(k_cache, v_cache, dev)
    n_pages, hk, ps, d = k_cache.shape
    t, hn, dn = k_new.shape
    if k_new.shape != v_new.shape or hn != hk or dn != d:
        raise ValueError("k_new and v_new must be [T, %d, %d]" % (hk, d))
    if slot_map.dim() != 1 or slot_map.shape[0] < t:
        raise ValueError("slot_map must be [T]")
    _append_entry(dev, t, hk, d, ps, n_pages, 0, *ks, *vs, *cs, *kn, *vn, *kb, *vb, *_flat(slot_map, dev))


def paged_attn_workspace_bytes(p: PagedParams) -> int:
    return int(lib.paged_attn_workspace_bytes(ctypes.byref(p)))


def prompt_attn_workspace_bytes(p: PromptParams) -> int:
    return int(lib.prompt_attn_workspace_bytes(ctypes.byref(p)))


def _workspace(p, device) -> torch.Tensor:
    """The tmp buffer of a call with parameters `p`, its status word zero."""
    query, call, n_bufs = ((paged_attn_workspace_bytes, lib.paged_attn_fwd, 9) if isinstance(p, PagedParams) else
                           (paged_quant_attn_workspace_bytes, lib.paged_quant_attn_fwd, 11)
                           if isinstance(p, PagedQuantParams) else
                           (prompt_attn_workspace_bytes, lib.prompt_attn_fwd, 6))
    nbytes = query(p)
    if nbytes >= 2 ** 63:
        why = ta_last_error()
        # the call itself, without buffers, is refused by the same check and says with which status;
        # parameters that it takes lack a device to size the workspace for
        status = call(ctypes.byref(p), *[None] * n_bufs, None)
        raise TreeAttentionError(status if status != TA_OK and ta_last_error() == why else TA_ERR_CUDA, why)
    ws = torch.empty((nbytes + 3) // 4, dtype=torch.float32, device=device)
    ws[:1].zero_()                                   # the status word
    return ws


def paged_attention_workspace(q: torch.Tensor, k_cache: torch.Tensor, block_table: torch.Tensor, *,
                              max_q_len: int, kernel: int = KERNEL_AUTO, scale: float = 1.0,
                              window: int = 0) -> torch.Tensor:
    """A tmp buffer for paged_attention calls of these shapes (its first 32-bit
    word, zero here, is the status word; calls that overlap must not share it).
    The window changes no size, but a call may be in range only with it."""
    n_pages, hk, ps, d = k_cache.shape
    p = PagedParams(block_table.shape[0], q.shape[1], hk, d, q.shape[0], max_q_len, window, ps, n_pages,
                    block_table.shape[1], kernel, scale)
    with torch.cuda.device(_device_of(q)):
        return _workspace(p, q.device)


def prompt_attention_workspace(q: torch.Tensor, k: torch.Tensor, cu_seqlens: torch.Tensor, *,
                               kernel: int = KERNEL_AUTO, scale: float = 1.0, window: int = 0) -> torch.Tensor:
    """A tmp buffer for prompt_attention calls of these shapes (see
    paged_attention_workspace)."""
    p = PromptParams(cu_seqlens.numel() - 1, q.shape[1], k.shape[1], q.shape[2], q.shape[0], window, kernel, scale)
    with torch.cuda.device(_device_of(q)):
        return _workspace(p, q.device)


def paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    cu_q: torch.Tensor, kv_lens: torch.Tensor, *, scale: float, max_q_len: int, window: int = 0,
                    parents: Optional[torch.Tensor] = None, tmp: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, kernel: int = KERNEL_AUTO, stream=None) -> torch.Tensor:
    """Attention of each request's new tokens over its pages.  q [T, H, D] holds
    the requests' new tokens one behind the other (cu_q [B + 1]); the caches are
    [n_pages, Hk, page_size, D] (any strides) and already hold the new tokens'
    K/V; kv_lens [B] counts all keys.  Token i of q_len sees the keys up to its own
    position kv_len - q_len + i (the last `window` of them), or, with `parents`
    (int32 [T], each request's draft tree by index inside its chunk), the prefix,
    its ancestors and itself; tokens before position 0 (kv_len < q_len) see nothing
    and give zeros.  Returns out [T, H, D] in q's type; rows behind the last request
    are not written.  What only the GPU sees (a page outside the cache, a length out of
    range, a wait that gave up) is ORed into the first 32-bit word of `tmp`, and the rows
    concerned are then not valid: to learn of it, pass a `tmp` from
    paged_attention_workspace.  Without one it goes unreported."""
    dev = _device_of(q)
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_attention, dev, stream, (q, k_cache, v_cache, block_table, cu_q, kv_lens),
                          dict(scale=scale, max_q_len=max_q_len, window=window, parents=parents, tmp=tmp, out=out,
                               kernel=kernel))
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    qb, qs = _strided(q, dev, 3, "q")
    ob, os_ = _strided(out, dev, 3, "out")
    kb, vb, cs = _cache_pair(k_cache, v_cache, dev)
    t, h, d = q.shape
    n_pages, hk, ps, dk = k_cache.shape
    if d != dk:
        raise ValueError("q and the caches must have one head dimension")
    if block_table.dim() != 2 or cu_q.numel() != block_table.shape[0] + 1 or kv_lens.numel() != block_table.shape[0]:
        raise ValueError("block_table must be [batch, max_pages], cu_q [batch + 1] and kv_lens [batch]")
    if parents is not None and parents.numel() < t:         # (an empty one would pass for none)
        raise ValueError("parents must be [%d]" % t)
    batch, width = block_table.shape
    if tmp is None:
        tmp = _workspace(PagedParams(batch, h, hk, d, t, max_q_len, window, ps, n_pages, width, kernel, scale), q.device)
    _paged_entry(dev, batch, h, hk, d, t, max_q_len, window, ps, n_pages, width, kernel, scale, *qs, *os_, *cs, *qb, *kb,
                 *vb, *_flat(block_table, dev), *_flat(cu_q, dev), *_flat(kv_lens, dev), *_flat(parents, dev),
                 *_flat(tmp, dev), *ob)
    return out


def ta_test_paged_attn_fwd_wait_limit(wait_polls: int, p: PagedParams, q, k_cache, v_cache, block_table, cu_q, kv_lens,
                                      parents, tmp, out, stream=None):
    """Test hook: paged_attn_fwd (tensor-core kernel, contiguous tensors) whose waits
    give up after `wait_polls` polls of about 1 us."""
    i32 = TA_I32
    _check(lib.ta_test_paged_attn_fwd_wait_limit(wait_polls, ctypes.byref(p), buf(q), buf(k_cache), buf(v_cache),
                                                 buf(block_table, i32), buf(cu_q, i32), buf(kv_lens, i32),
                                                 buf(parents, i32), buf(tmp), buf(out), _stream(stream)))


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *, scale: float,
                     window: int = 0, tmp: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     kernel: int = KERNEL_AUTO, stream=None) -> torch.Tensor:
    """Causal attention over whole prompts packed one behind the other: q [T, H, D],
    k and v [T, Hk, D] (any token and head strides, as slices of one projection),
    cu_seqlens [B + 1] int32 on the device.  Row i of a prompt sees its rows up to
    i (the last `window` of them).  Returns out [T, H, D] in q's type; rows behind
    the last prompt are not written.  Errors that only the GPU sees are ORed into the
    first 32-bit word of `tmp` (see paged_attention); without a `tmp` from
    prompt_attention_workspace they go unreported."""
    dev = _device_of(q)
    if stream is not None or dev != _this_device():
        return _elsewhere(prompt_attention, dev, stream, (q, k, v, cu_seqlens),
                          dict(scale=scale, window=window, tmp=tmp, out=out, kernel=kernel))
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    qb, qs = _strided(q, dev, 3, "q")
    ob, os_ = _strided(out, dev, 3, "out")
    kb, ks = _strided(k, dev, 3, "k")
    vb, vs = _strided(v, dev, 3, "v")
    t, h, d = q.shape
    if k.shape != v.shape or k.shape[0] != t or k.shape[2] != d:
        raise ValueError("k and v must be [%d, Hk, %d]" % (t, d))
    batch, hk = cu_seqlens.numel() - 1, k.shape[1]
    if tmp is None:
        tmp = _workspace(PromptParams(max(batch, 0), h, hk, d, t, window, kernel, scale), q.device)
    _prompt_entry(dev, batch, h, hk, d, t, window, kernel, scale, *qs, *os_, *ks, *vs, *qb, *kb, *vb,
                  *_flat(cu_seqlens, dev), *_flat(tmp, dev), *ob)
    return out


# ------------------------------------- rotated rows and 4-bit pages (serving)

class PagedQuantCache(NamedTuple):
    """A paged K/V cache in 4 bits: element = scale * code + bias of its group.  Codes
    int32 [n_pages, Hk, page_size, D / 8] (the order of a row's codes: paged_quant_append
    in include/tree_attn.h), affine float16 or bfloat16 [n_pages, Hk, page_size,
    D / group_size, 2], (scale, bias) pairs.  Any page, head and token strides."""
    k_codes: torch.Tensor
    k_affine: torch.Tensor
    v_codes: torch.Tensor
    v_affine: torch.Tensor


def paged_quant_cache(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, *, group_size: int = 64,
                      dtype: torch.dtype = torch.bfloat16, device="cuda") -> PagedQuantCache:
    """An empty (zero) 4-bit cache; `dtype` is the 16-bit type of its scales and of
    the rows that go with it."""
    shape = (n_pages, n_kv_heads, page_size)
    if dtype not in (torch.float16, torch.bfloat16) or group_size not in (32, 64) or head_dim % group_size:
        raise ValueError("dtype must be float16 or bfloat16, group_size 32 or 64, a divisor of head_dim")
    return PagedQuantCache(*[torch.zeros(*shape, *last, dtype=t, device=device) for t, last in
                             ((torch.int32, (head_dim // 8,)), (dtype, (head_dim // group_size, 2))) * 2])


def rotary_table(positions: int, rotary_dim: int, *, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The table [positions, rotary_dim] f32 of paged_append_rotary and paged_quant_append:
    cosines, then sines, of position * base^(-2 i / rotary_dim); angles in 64 bits."""
    if rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and > 0, got %d" % rotary_dim)
    if positions < 0:
        raise ValueError("positions must be >= 0, got %d" % positions)
    if not 0.0 < base < float("inf"):
        raise ValueError("base must be finite and > 0, got %r" % base)
    turn = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def _new_rows(q, k_new, v_new, slot_map, positions, rotary, q_out, hk, d, dev):
    """Checks and fields of the rows that both appends take: sizes, strides, ta_bufs
    (q, k_new, v_new, slot_map, positions, rotary, q_out) and the q_out to return."""
    kn, ks = _strided(k_new, dev, 3, "k_new")
    vn, vs = _strided(v_new, dev, 3, "v_new")
    t = k_new.shape[0]
    if k_new.shape != v_new.shape or tuple(k_new.shape[1:]) != (hk, d):
        raise ValueError("k_new and v_new must be [T, %d, %d]" % (hk, d))
    if slot_map.dim() != 1 or slot_map.shape[0] < t:
        raise ValueError("slot_map must be [T]")
    h, qb, qs, ob, os_ = 0, _ABSENT, (0, 0), _ABSENT, (0, 0)
    if q is not None:
        if q.dim() != 3 or q.shape[0] != t or q.shape[2] != d or q.shape[1] == 0:
            raise ValueError("q must be [%d, H, %d]" % (t, d))
        h = q.shape[1]
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        qb, qs = _strided(q, dev, 3, "q")
        ob, os_ = _strided(q_out, dev, 3, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    pb, tb, r, most = _ABSENT, _ABSENT, 0, 0
    if rotary is not None:
        if positions is None or positions.dim() != 1 or positions.shape[0] < t:
            raise ValueError("positions must be [T]")
        if rotary.dim() != 2 or rotary.shape[1] == 0:
            raise ValueError("rotary must be [positions, rotary_dim]")
        most, r = rotary.shape
        pb, tb = _flat(positions, dev), _flat(rotary, dev)
    elif positions is not None or q is not None:
        raise ValueError("positions and q need a rotary table")
    return t, h, r, most, (*qs, *os_, *ks, *vs), (*qb, *kn, *vn, *_flat(slot_map, dev), *pb, *tb, *ob), q_out


def paged_append_rotary(q: Optional[torch.Tensor], k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, slot_map: torch.Tensor, positions: torch.Tensor,
                        rotary: torch.Tensor, *, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                        stream=None) -> Optional[torch.Tensor]:
    """paged_append with the position rotation on the way: q [T, H, D] and k_new [T, Hk, D]
    turned by positions [T] (int32), the turned keys and v_new written to the slots
    slot_map [T] of the caches.  rotary [positions, R] f32 holds cosines, then sines
    (rotary_table); the first R elements of a head are turned, element i with i + R / 2,
    or, `interleaved`, 2 i with 2 i + 1.  Returns the turned q (in q_out, which may be q;
    None without q).  A token whose position is outside the table stores nothing and its
    q_out row stays as it was."""
    dev = _device_of(k_cache)
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_append_rotary, dev, stream,
                          (q, k_new, v_new, k_cache, v_cache, slot_map, positions, rotary),
                          dict(interleaved=interleaved, q_out=q_out))
    if rotary is None:
        raise ValueError("rotary must be [positions, rotary_dim]")
    kb, vb, cs = _cache_pair(k_cache, v_cache, dev)
    n_pages, hk, ps, d = k_cache.shape
    t, h, r, most, strides, bufs, q_out = _new_rows(q, k_new, v_new, slot_map, positions, rotary, q_out, hk, d, dev)
    _rotary_entry(dev, t, h, hk, d, ps, n_pages, r, bool(interleaved), most, 0, *strides, *cs, *bufs, *kb, *vb)
    return q_out


def _quant_cache(cache, dev):
    """A PagedQuantCache as (n_pages, Hk, page_size, D, group_size, strides, ta_bufs)."""
    kc, ka, vc, va = cache
    cs, fs = kc.shape, ka.shape
    if kc.dtype != torch.int32 or vc.dtype != torch.int32:
        raise ValueError("codes must be int32")
    if cs != vc.shape or fs != va.shape:
        raise ValueError("K and V must have one shape")
    if len(cs) != 4 or len(fs) != 5 or cs[:3] != fs[:3] or fs[4] != 2 or fs[3] == 0:
        raise ValueError("a cache is codes [n_pages, Hk, page_size, D / 8], affine [n_pages, Hk, page_size, D / group, 2]")
    n_pages, hk, ps, words = cs
    groups = fs[3]
    if 8 * words % groups:
        raise ValueError("D / 8 words and D / group pairs a row do not go together")
    if kc.is_contiguous() and vc.is_contiguous() and ka.is_contiguous() and va.is_contiguous():
        if not kc.get_device() == vc.get_device() == ka.get_device() == va.get_device() == dev:
            raise ValueError("all tensors must be on cuda:%d" % dev)
        code = _SERVE_CODE.get(ka.dtype), _SERVE_CODE.get(va.dtype)
        if None in code:
            raise ValueError("unsupported dtype %s" % ka.dtype)
        rows = n_pages * hk * ps
        nc, na = 4 * rows * words, ka.element_size() * rows * groups * 2
        return (n_pages, hk, ps, 8 * words, 8 * words // groups, _NO_STRIDES,
                (kc.data_ptr(), nc, TA_U32, 0, ka.data_ptr(), na, code[0], 0, vc.data_ptr(), nc, TA_U32, 0, va.data_ptr(), na,
                 code[1], 0))
    # a row's pairs stand one behind the other
    if any(x.stride(4) != 1 or (groups > 1 and x.stride(3) != 2) for x in (ka, va)) and ka.numel():
        raise ValueError("a row's (scale, bias) pairs must be contiguous")
    kcb, vcb, c_str = _cache_pair(kc, vc, dev)
    kab, vab, f_str = _cache_pair(*(x.flatten(3) if x.numel() else x.reshape(*fs[:3], -1) for x in (ka, va)), dev)
    return (n_pages, hk, ps, 8 * words, 8 * words // groups, (*c_str, *f_str),
            (kcb[0], kcb[1], TA_U32, 0, *kab, vcb[0], vcb[1], TA_U32, 0, *vab))


_NO_STRIDES = (0,) * 6                           # contiguous


def paged_quant_append(k_new: torch.Tensor, v_new: torch.Tensor, cache: PagedQuantCache, slot_map: torch.Tensor, *,
                       q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                       rotary: Optional[torch.Tensor] = None, interleaved: bool = False,
                       q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Write the rows k_new, v_new [T, Hk, D] to the slots slot_map [T] of a 4-bit cache, each
    group of elements as round((x - min) / scale) with scale = (max - min) / 15.  With
    `rotary` and `positions`, keys and q are turned on the way as in paged_append_rotary
    (the keys unrounded); returns the turned q.  A group with an element that is not
    finite reads as NaN."""
    dev = _device_of(cache[0])
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_quant_append, dev, stream, (k_new, v_new, cache, slot_map),
                          dict(q=q, positions=positions, rotary=rotary, interleaved=interleaved, q_out=q_out))
    n_pages, hk, ps, d, group, cs, cb = _quant_cache(cache, dev)
    t, h, r, most, strides, bufs, q_out = _new_rows(q, k_new, v_new, slot_map, positions, rotary, q_out, hk, d, dev)
    _quant_append_entry(dev, t, h, hk, d, ps, n_pages, group, r, bool(interleaved), most, *strides, *cs, *bufs, *cb)
    return q_out


def paged_quant_read(cache: PagedQuantCache, slot_map: torch.Tensor, *, out=None, stream=None):
    """The rows of slots slot_map [T] (int64) of a 4-bit cache as 16-bit (k, v), each
    [T, Hk, D] in the type of its scales (`out`: the two tensors to write into).  Rows whose
    slot is outside the cache are 0."""
    dev = _device_of(cache[0])
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_quant_read, dev, stream, (cache, slot_map), dict(out=out))
    n_pages, hk, ps, d, group, cs, cb = _quant_cache(cache, dev)
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be [T]")
    t = slot_map.shape[0]
    if out is None:
        out = tuple(torch.empty(t, hk, d, dtype=cache[1].dtype, device=cache[1].device) for _ in range(2))
    k, v = out
    if tuple(k.shape) != (t, hk, d) or k.shape != v.shape:
        raise ValueError("out must be two tensors [%d, %d, %d]" % (t, hk, d))
    kb, ks = _strided(k, dev, 3, "k")
    vb, vs = _strided(v, dev, 3, "v")
    _quant_read_entry(dev, t, 0, hk, d, ps, n_pages, group, 0, 0, 0, 0, 0, 0, 0, *ks, *vs, *cs, *_flat(slot_map, dev), *cb,
                      *kb, *vb)
    return k, v


def paged_quant_attn_workspace_bytes(p: PagedQuantParams) -> int:
    return int(lib.paged_quant_attn_workspace_bytes(ctypes.byref(p)))


def paged_quant_attention_workspace(q: torch.Tensor, cache: PagedQuantCache, block_table: torch.Tensor, *,
                                    max_q_len: int, kernel: int = KERNEL_AUTO, scale: float = 1.0,
                                    window: int = 0) -> torch.Tensor:
    """A tmp buffer for paged_quant_attention calls of these shapes (see
    paged_attention_workspace)."""
    n_pages, hk, ps, words = cache[0].shape
    p = PagedQuantParams(block_table.shape[0], q.shape[1], hk, 8 * words, q.shape[0], max_q_len, window, ps, n_pages,
                         block_table.shape[1], 8 * words // max(1, cache[1].shape[3]), kernel, scale)
    with torch.cuda.device(_device_of(q)):
        return _workspace(p, q.device)


def paged_quant_attention(q: torch.Tensor, cache: PagedQuantCache, block_table: torch.Tensor, cu_q: torch.Tensor,
                          kv_lens: torch.Tensor, *, scale: float, max_q_len: int, window: int = 0,
                          parents: Optional[torch.Tensor] = None, tmp: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, kernel: int = KERNEL_AUTO, stream=None) -> torch.Tensor:
    """paged_attention over a 4-bit cache: the same arguments, masks, `tmp` (from
    paged_quant_attention_workspace) and status bits, with keys and values
    scale * code + bias.  q and out have the type of the cache's scales."""
    dev = _device_of(q)
    if stream is not None or dev != _this_device():
        return _elsewhere(paged_quant_attention, dev, stream, (q, cache, block_table, cu_q, kv_lens),
                          dict(scale=scale, max_q_len=max_q_len, window=window, parents=parents, tmp=tmp, out=out,
                               kernel=kernel))
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape")
    qb, qs = _strided(q, dev, 3, "q")
    ob, os_ = _strided(out, dev, 3, "out")
    n_pages, hk, ps, dk, group, cs, cb = _quant_cache(cache, dev)
    t, h, d = q.shape
    if d != dk:
        raise ValueError("q and the cache must have one head dimension")
    if block_table.dim() != 2 or cu_q.numel() != block_table.shape[0] + 1 or kv_lens.numel() != block_table.shape[0]:
        raise ValueError("block_table must be [batch, max_pages], cu_q [batch + 1] and kv_lens [batch]")
    if parents is not None and parents.numel() < t:         # (an empty one would pass for none)
        raise ValueError("parents must be [%d]" % t)
    batch, width = block_table.shape
    if tmp is None:
        tmp = _workspace(PagedQuantParams(batch, h, hk, d, t, max_q_len, window, ps, n_pages, width, group, kernel,
                                          scale), q.device)
    _paged_quant_entry(dev, batch, h, hk, d, t, max_q_len, window, ps, n_pages, width, group, kernel, scale, 0, *qs, *os_,
                       *cs, *qb, *cb, *_flat(block_table, dev), *_flat(cu_q, dev), *_flat(kv_lens, dev),
                       *_flat(parents, dev), *_flat(tmp, dev), *ob)
    return out


def ta_test_paged_quant_attn_fwd_wait_limit(wait_polls: int, p: PagedQuantParams, q, cache: PagedQuantCache, block_table,
                                            cu_q, kv_lens, parents, tmp, out, stream=None):
    """Test hook: paged_quant_attn_fwd (tensor-core kernel, contiguous tensors) whose waits
    give up after `wait_polls` polls of about 1 us."""
    i32 = TA_I32
    kc, ka, vc, va = cache
    _check(lib.ta_test_paged_quant_attn_fwd_wait_limit(wait_polls, ctypes.byref(p), buf(q), buf(kc, TA_U32), buf(ka),
                                                       buf(vc, TA_U32), buf(va), buf(block_table, i32), buf(cu_q, i32),
                                                       buf(kv_lens, i32), buf(parents, i32), buf(tmp), buf(out),
                                                       _stream(stream)))
