"""ctypes binding of libdflash_attn (argument marshalling only).

Every step of the attention runs in the library's CUDA kernels; this module
only turns torch tensors into the pointers, sizes and strides that
include/dflash_attn.h describes, picks the current CUDA stream, and keeps a
small per-device workspace cache. There is no CPU fallback: if the library is
missing, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libdflash_attn.so")

# dflash_status
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_CHECK, ERR_WORKSPACE = range(6)
# dflash_dtype
BF16, FP32 = 0, 1
# dflash_kernel
KERNELS = {"auto": 0, "simt": 1, "tc": 2, "tc_pair": 3}
# device error bits
DEVERR_PAGE_ID, DEVERR_SEQ_LEN, DEVERR_TIMEOUT, DEVERR_TOKEN_ID, DEVERR_TREE = 1, 2, 4, 8, 16

EXPORTED = (
    "dflash_block_attn",
    "dflash_block_attn_noalloc",
    "dflash_split_combine",
    "dflash_plan_splits",
    "dflash_plan_call",
    "dflash_workspace_bytes",
    "dflash_read_error",
    "dflash_status_string",
    "dflash_last_error_message",
    "dflash_abi_version",
    "dflash_accept_prefix",
    "dflash_accept_workspace_bytes",
    "dflash_project_kv",
    "dflash_project_kv_workspace_bytes",
    "dflash_grouped_conv",
    "dflash_selector_workspace_bytes",
    "dflash_selector_walk",
    "dflash_logprobs_workspace_bytes",
    "dflash_token_logprobs",
    "dflash_tree_attn_workspace_bytes",
    "dflash_tree_attn",
    "dflash_tree_attn_err",
    "dflash_shared_error_word",
    "dflash_tree_accept_workspace_bytes",
    "dflash_tree_accept",
    "dflash_tree_commit",
    "dflash_rope",
    "dflash_append_kv",
    "dflash_cache8_attn_workspace_bytes",
    "dflash_cache8_attn",
)


class Dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("kv_stride_page", ctypes.c_int64),
        ("kv_stride_slot", ctypes.c_int64),
        ("kv_stride_head", ctypes.c_int64),
    ]


class Opts(ctypes.Structure):
    _fields_ = [
        ("num_splits", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
        ("wait_limit_us", ctypes.c_uint32),
    ]


class Plan(ctypes.Structure):
    _fields_ = [
        ("num_splits", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("balanced", ctypes.c_int32),
        ("launches", ctypes.c_int32),
        ("ctas", ctypes.c_int64),
    ]


class RopeFreqs(ctypes.Structure):
    _fields_ = [
        ("turns", ctypes.c_void_p),
        ("rotary_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("gain", ctypes.c_float),
    ]


KERNEL_NAMES = {1: "simt_attn_kernel", 2: "tc_attn_kernel", 3: "tc_pair_attn_kernel"}


class DflashError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"dflash status {status}: {message}")
        self.status = status


_lock = threading.Lock()
_lib = None


def load_library(path: Optional[str] = None):
    """Load libdflash_attn.so (built by build.py) and declare its signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with speculative_decoding_block_dflash_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        dims_p, opts_p = ctypes.POINTER(Dims), ctypes.POINTER(Opts)
        lib.dflash_block_attn.restype = ctypes.c_int
        lib.dflash_block_attn.argtypes = [vp, vp, vp, vp, vp, dims_p, i32, i32, i32, f32, vp, vp, opts_p]
        lib.dflash_block_attn_noalloc.restype = ctypes.c_int
        lib.dflash_block_attn_noalloc.argtypes = [vp, vp, vp, vp, vp, dims_p, i32, i32, i32, f32, vp, vp, i32, i32, vp]
        lib.dflash_split_combine.restype = ctypes.c_int
        lib.dflash_split_combine.argtypes = [vp, vp, i32, i64, i32, i32, vp, vp, vp]
        lib.dflash_plan_splits.restype = i32
        lib.dflash_plan_splits.argtypes = [dims_p, i32, i32, i32, i32]
        lib.dflash_plan_call.restype = ctypes.c_int
        lib.dflash_plan_call.argtypes = [dims_p, i32, i32, i32, i32, ctypes.POINTER(Plan)]
        lib.dflash_workspace_bytes.restype = ctypes.c_size_t
        lib.dflash_workspace_bytes.argtypes = [dims_p, i32, i32]
        lib.dflash_read_error.restype = ctypes.c_int
        lib.dflash_read_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32), i32]
        lib.dflash_status_string.restype = ctypes.c_char_p
        lib.dflash_status_string.argtypes = [ctypes.c_int]
        lib.dflash_last_error_message.restype = ctypes.c_char_p
        lib.dflash_last_error_message.argtypes = []
        lib.dflash_abi_version.restype = i32
        lib.dflash_abi_version.argtypes = []
        lib.dflash_accept_workspace_bytes.restype = ctypes.c_size_t
        lib.dflash_accept_workspace_bytes.argtypes = [i32, i32]
        lib.dflash_accept_prefix.restype = ctypes.c_int
        lib.dflash_accept_prefix.argtypes = [vp, i32, i32, i32, i32, i64, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        lib.dflash_project_kv.restype = ctypes.c_int
        lib.dflash_project_kv.argtypes = [vp, i32, i32, i64, vp, vp, vp, vp, vp, dims_p, vp, vp, ctypes.c_size_t, vp]
        lib.dflash_project_kv_workspace_bytes.restype = ctypes.c_size_t
        lib.dflash_project_kv_workspace_bytes.argtypes = []
        lib.dflash_grouped_conv.restype = ctypes.c_int
        lib.dflash_grouped_conv.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
        lib.dflash_selector_workspace_bytes.restype = ctypes.c_size_t
        lib.dflash_selector_workspace_bytes.argtypes = [i32, i32, i32]
        lib.dflash_selector_walk.restype = ctypes.c_int
        lib.dflash_selector_walk.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp, vp,
                                             vp, vp, ctypes.c_size_t, vp]
        size, u32 = ctypes.c_size_t, ctypes.c_uint32
        lib.dflash_logprobs_workspace_bytes.restype = size
        lib.dflash_logprobs_workspace_bytes.argtypes = [i32, i32, i32]
        lib.dflash_token_logprobs.restype = ctypes.c_int
        lib.dflash_token_logprobs.argtypes = [vp, i32, i32, i32, i64, f32, vp, i32, vp, vp, vp, i32, vp, vp, vp, vp,
                                              size, vp]
        lib.dflash_tree_attn_workspace_bytes.restype = size
        lib.dflash_tree_attn_workspace_bytes.argtypes = [dims_p, i32]
        lib.dflash_tree_attn.restype = ctypes.c_int
        lib.dflash_tree_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, dims_p, i32, i32, f32, vp, vp, i32, vp, size, u32,
                                         vp]
        lib.dflash_tree_attn_err.restype = ctypes.c_int
        lib.dflash_tree_attn_err.argtypes = [vp, vp, vp, vp, vp, vp, vp, dims_p, i32, i32, f32, vp, vp, i32, vp, vp,
                                             size, u32, vp]
        lib.dflash_shared_error_word.restype = ctypes.c_int
        lib.dflash_shared_error_word.argtypes = [ctypes.POINTER(vp)]
        lib.dflash_tree_accept_workspace_bytes.restype = size
        lib.dflash_tree_accept_workspace_bytes.argtypes = []
        lib.dflash_tree_accept.restype = ctypes.c_int
        lib.dflash_tree_accept.argtypes = [vp, i32, i32, i32, i32, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, size, vp]
        lib.dflash_tree_commit.restype = ctypes.c_int
        lib.dflash_tree_commit.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, dims_p, i32, i32, i64, vp, vp]
        freqs_p = ctypes.POINTER(RopeFreqs)
        lib.dflash_rope.restype = ctypes.c_int
        lib.dflash_rope.argtypes = [vp, vp, i32, i32, i32, i32, i64, i64, i64, i64, vp, freqs_p, i32, vp]
        lib.dflash_append_kv.restype = ctypes.c_int
        lib.dflash_append_kv.argtypes = [vp, vp, i32, i64, i64, i64, i64, vp, vp, freqs_p, vp, vp, vp, vp, vp, vp, dims_p,
                                         vp, vp]
        lib.dflash_cache8_attn_workspace_bytes.restype = size
        lib.dflash_cache8_attn_workspace_bytes.argtypes = [dims_p, i32]
        lib.dflash_cache8_attn.restype = ctypes.c_int
        lib.dflash_cache8_attn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, dims_p, i32, i32, i32, f32, vp, vp, i32, vp,
                                           vp, size, u32, vp]
        if path is None:
            _lib = lib
        return lib


def _check(status: int):
    if status != OK:
        lib = load_library()
        msg = lib.dflash_last_error_message().decode() or lib.dflash_status_string(status).decode()
        raise DflashError(status, msg)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def make_dims(q: torch.Tensor, k_cache: torch.Tensor, page_table: torch.Tensor, block_len: int,
              max_seq_len: Optional[int] = None, batch: Optional[int] = None) -> Dims:
    """Dims for q [B*T, Hq, D] and a cache [num_pages, page_size, Hkv, D] (any strides, d contiguous)."""
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q must be [B*T, Hq, D] and k_cache [num_pages, page_size, Hkv, D]")
    B = batch if batch is not None else page_table.shape[0]
    d = Dims()
    d.batch = B
    d.num_q_heads = q.shape[1]
    d.num_kv_heads = k_cache.shape[2]
    d.head_dim = q.shape[2]
    d.page_size = k_cache.shape[1]
    d.num_pages = k_cache.shape[0]
    d.max_pages = page_table.shape[1]
    d.max_seq_len = int(max_seq_len) if max_seq_len else 0
    d.dtype = _dtype_code(q)
    d.kv_stride_page, d.kv_stride_slot, d.kv_stride_head = (int(s) for s in k_cache.stride()[:3])
    return d


def plan_splits(dims: Dims, block_len: int, window: int = 0, requested: int = 0, kernel: str = "auto") -> int:
    n = load_library().dflash_plan_splits(ctypes.byref(dims), int(block_len), int(window), int(requested),
                                          KERNELS[kernel])
    if n < 1:
        _check(-n)
    return n


def plan_info(dims: Dims, block_len: int, window: int = 0, requested: int = 0, kernel: str = "auto") -> dict:
    """What a call with these sizes runs (dflash_plan_call): split count, kernel, whether the
    splits are length-balanced, CTAs of the attention launch and kernel launches per call."""
    plan = Plan()
    _check(load_library().dflash_plan_call(ctypes.byref(dims), int(block_len), int(window), int(requested),
                                           KERNELS[kernel], ctypes.byref(plan)))
    return {"num_splits": plan.num_splits, "kernel": plan.kernel, "kernel_name": KERNEL_NAMES[plan.kernel],
            "balanced": bool(plan.balanced), "launches": plan.launches, "ctas": int(plan.ctas)}


def workspace_bytes(dims: Dims, block_len: int, num_splits: int) -> int:
    n = load_library().dflash_workspace_bytes(ctypes.byref(dims), int(block_len), int(num_splits))
    if n == 0:
        raise DflashError(ERR_INVALID_ARG, "invalid dims for workspace size")
    return n


def _check_attn_inputs(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, block_len: int, out: Optional[torch.Tensor],
                       lse: Optional[torch.Tensor]) -> None:
    """Checks the library cannot make from the pointers and dims alone: the dims carry
    k_cache's geometry only (the kernels and tensor maps read v_cache with it), and the
    index tensors are read as int32. Shared by both attention entry points."""
    if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("v_cache must match k_cache in shape and strides")
    if v_cache.dtype != k_cache.dtype or q.dtype != k_cache.dtype:
        raise TypeError("q, k_cache and v_cache must share one dtype")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if page_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("page_table and seq_lens must be int32")
    if page_table.dim() != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous [B, max_pages] tensor")
    if seq_lens.dim() != 1 or seq_lens.shape[0] != page_table.shape[0] or not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous [B] tensor matching page_table's rows")
    if q.dim() != 3 or q.shape[0] != page_table.shape[0] * int(block_len):
        raise ValueError("q must be [B*block_len, Hq, D] with B = page_table.shape[0]")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    if lse is not None and (tuple(lse.shape) != tuple(q.shape[:2]) or lse.dtype != torch.float32
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [B*block_len, Hq] tensor")
    devs = {t.device for t in (q, k_cache, v_cache, page_table, seq_lens, out, lse) if t is not None}
    if len(devs) != 1 or next(iter(devs)).type != "cuda":
        raise ValueError("every tensor must be on one CUDA device")


_ws_cache = {}


def workspace_for(device: torch.device, nbytes: int) -> torch.Tensor:
    """A zero-initialised, 256-byte aligned device buffer of at least nbytes, cached per device."""
    key = (device.type, device.index)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def _stream_handle(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def block_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
               seq_lens: torch.Tensor, block_len: int, causal: bool = False, window: int = 0,
               scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, num_splits: int = 0, kernel: str = "auto",
               workspace: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
               stream=None, want_lse: bool = True,
               wait_limit_us: int = 0) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """DFlash block attention (include/dflash_attn.h, dflash_block_attn).

    q [B*T, Hq, D]; k_cache, v_cache [num_pages, page_size, Hkv, D] (head_dim
    contiguous); page_table int32 [B, max_pages]; seq_lens int32 [B] on the
    device. Returns (out [B*T, Hq, D] in q's dtype, lse fp32 [B*T, Hq] or None).
    wait_limit_us bounds every device-side wait of the tensor-core kernels (0 = 2 s).
    """
    lib = load_library()
    _check_attn_inputs(q, k_cache, v_cache, page_table, seq_lens, block_len, out, lse)
    dims = make_dims(q, k_cache, page_table, block_len, max_seq_len)
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[2])
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    splits = plan_splits(dims, block_len, window, num_splits, kernel)
    need = workspace_bytes(dims, block_len, splits)
    if workspace is None:
        workspace = workspace_for(q.device, need)
    opts = Opts()
    opts.num_splits = num_splits  # the caller's request: the library re-plans the same count (0 = auto)
    opts.kernel = KERNELS[kernel]
    opts.workspace = workspace.data_ptr()
    opts.workspace_bytes = workspace.numel() * workspace.element_size()
    opts.stream = _stream_handle(stream)
    opts.wait_limit_us = int(wait_limit_us)
    st = lib.dflash_block_attn(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                               seq_lens.data_ptr(), ctypes.byref(dims), int(block_len), int(bool(causal)),
                               int(window), float(scale), out.data_ptr(),
                               lse.data_ptr() if lse is not None else None, ctypes.byref(opts))
    _check(st)
    return out, lse


def block_attn_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                       seq_lens: torch.Tensor, block_len: int, causal: bool = False, window: int = 0,
                       scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, num_splits: int = 0, kernel: str = "auto",
                       max_seq_len: Optional[int] = None, stream=None,
                       want_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """dflash_block_attn_noalloc: the same attention with the library's own fixed
    scratch instead of a workspace, for callers that cannot allocate device memory.
    The library call allocates nothing; for convenience this wrapper allocates out
    (and lse, when want_lse) with torch when they are not given, so a caller that
    must not allocate passes both."""
    lib = load_library()
    _check_attn_inputs(q, k_cache, v_cache, page_table, seq_lens, block_len, out, lse)
    dims = make_dims(q, k_cache, page_table, block_len, max_seq_len)
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[2])
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    st = lib.dflash_block_attn_noalloc(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                                       seq_lens.data_ptr(), ctypes.byref(dims), int(block_len), int(bool(causal)),
                                       int(window), float(scale), out.data_ptr(),
                                       lse.data_ptr() if lse is not None else None, int(num_splits),
                                       KERNELS[kernel], _stream_handle(stream))
    _check(st)
    return out, lse


def split_combine(partial_out: torch.Tensor, partial_lse: torch.Tensor, out_dtype=torch.float32,
                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Log-sum-exp combine (dflash_split_combine): partial_out fp32 [S, rows..., D],
    partial_lse fp32 [S, rows...] -> out [rows..., D] (out_dtype), lse [rows...]."""
    lib = load_library()
    if partial_out.dtype != torch.float32 or partial_lse.dtype != torch.float32:
        raise TypeError("partials must be fp32")
    if not (partial_out.is_contiguous() and partial_lse.is_contiguous()):
        raise ValueError("partials must be contiguous")
    S, D = partial_out.shape[0], partial_out.shape[-1]
    inner = tuple(partial_out.shape[1:-1])
    rows = int(math.prod(inner)) if inner else 1
    if out is None:
        out = torch.empty(inner + (D,), dtype=out_dtype, device=partial_out.device)
    if lse is None:
        lse = torch.empty(inner, dtype=torch.float32, device=partial_out.device)
    st = lib.dflash_split_combine(partial_out.data_ptr(), partial_lse.data_ptr(), S, rows, D,
                                  _dtype_code(out), out.data_ptr(), lse.data_ptr(), _stream_handle(stream))
    _check(st)
    return out, lse


_accept_ws = {}


def accept_workspace_bytes(batch: int, block_len: int) -> int:
    n = load_library().dflash_accept_workspace_bytes(int(batch), int(block_len))
    if n == 0:
        raise DflashError(1, "invalid batch/block_len for the acceptance workspace")
    return n


def accept_prefix(logits: torch.Tensor, draft: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                  accepted: Optional[torch.Tensor] = None, next_token: Optional[torch.Tensor] = None,
                  target_argmax: Optional[torch.Tensor] = None, want_argmax: bool = True,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Longest-prefix acceptance (dflash_accept_prefix): logits [B, T, V] bf16/fp32 (last
    dim contiguous), draft int32 [B, T-1] -> (accepted_len [B], next_token [B], target
    argmax [B, T] or None), int32 on the device. Without a workspace the call uses one cached
    per device: calls that may overlap (different streams) must each pass their own."""
    lib = load_library()
    if logits.dim() != 3 or logits.stride(2) != 1 or logits.stride(0) != logits.shape[1] * logits.stride(1):
        raise ValueError("logits must be [B, T, V] with contiguous rows of a common stride")
    B, T, V = logits.shape
    if draft.dtype != torch.int32 or tuple(draft.shape) != (B, T - 1) or not draft.is_contiguous():
        raise ValueError("draft must be a contiguous int32 [B, T-1] tensor")
    dev = logits.device
    if workspace is None:
        need = accept_workspace_bytes(B, T)
        key = (dev.type, dev.index)
        workspace = _accept_ws.get(key)
        if workspace is None or workspace.numel() < need:
            workspace = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=dev)
            _accept_ws[key] = workspace
    if accepted is None:
        accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=dev)
    if target_argmax is None and want_argmax:
        target_argmax = torch.empty(B, T, dtype=torch.int32, device=dev)
    st = lib.dflash_accept_prefix(logits.data_ptr(), _dtype_code(logits), B, T, V, logits.stride(1),
                                  draft.data_ptr() if draft.numel() else None, accepted.data_ptr(),
                                  next_token.data_ptr(),
                                  target_argmax.data_ptr() if target_argmax is not None else None,
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream))
    _check(st)
    return accepted, next_token, target_argmax


_proj_ws = {}


def project_kv(hidden: torch.Tensor, w_k: torch.Tensor, w_v: torch.Tensor, slot_mapping: torch.Tensor,
               k_cache: torch.Tensor, v_cache: torch.Tensor, device_error: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, split: bool = True, stream=None) -> None:
    """Context K/V projection into the paged cache (dflash_project_kv): hidden [L, H] bf16
    (rows of any stride, last dim contiguous), w_k / w_v [Hkv*D, H] bf16 contiguous,
    slot_mapping int32 [L] (page * page_size + position; < 0 skips the token), caches
    [num_pages, page_size, Hkv, D] bf16 (d contiguous, same strides). device_error: an
    optional int32/uint32 device word that receives DEVERR_* bits. With split (the default)
    the last round's tiles are split in two through a workspace (a zeroed one cached per
    device when none is given: calls that may overlap must each pass their own);
    split=False computes every tile whole."""
    lib = load_library()
    if split and workspace is None and hidden.numel():
        dev = hidden.device
        key = (dev.type, dev.index)
        workspace = _proj_ws.get(key)
        if workspace is None:
            workspace = torch.zeros(lib.dflash_project_kv_workspace_bytes(), dtype=torch.uint8, device=dev)
            _proj_ws[key] = workspace
    if not split:
        workspace = None
    if hidden.dim() != 2 or hidden.stride(1) != 1:
        raise ValueError("hidden must be [L, H] with a contiguous last dimension")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, Hkv, D] of the same shape and strides")
    if k_cache.stride(3) != 1:
        raise ValueError("the caches' head_dim must be contiguous")
    L, H = hidden.shape
    N = k_cache.shape[2] * k_cache.shape[3]
    for name, w in (("w_k", w_k), ("w_v", w_v)):
        if tuple(w.shape) != (N, H) or not w.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{N}, {H}] tensor")
    if slot_mapping.dtype != torch.int32 or tuple(slot_mapping.shape) != (L,) or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be a contiguous int32 [L] tensor")
    for t in (hidden, w_k, w_v, k_cache, v_cache):
        if t.dtype != torch.bfloat16:
            raise TypeError("hidden, weights and caches must be bf16")
    d = Dims()
    d.batch = 1
    d.num_q_heads = k_cache.shape[2]
    d.num_kv_heads = k_cache.shape[2]
    d.head_dim = k_cache.shape[3]
    d.page_size = k_cache.shape[1]
    d.num_pages = k_cache.shape[0]
    d.max_pages = 1
    d.max_seq_len = 0
    d.dtype = BF16
    d.kv_stride_page, d.kv_stride_slot, d.kv_stride_head = (int(s) for s in k_cache.stride()[:3])
    st = lib.dflash_project_kv(hidden.data_ptr() if L else None, L, H, hidden.stride(0) if L else H,
                               w_k.data_ptr(), w_v.data_ptr(), slot_mapping.data_ptr() if L else None,
                               k_cache.data_ptr(), v_cache.data_ptr(), ctypes.byref(d),
                               device_error.data_ptr() if device_error is not None else None,
                               workspace.data_ptr() if workspace is not None else None,
                               workspace.numel() * workspace.element_size() if workspace is not None else 0,
                               _stream_handle(stream))
    _check(st)


def grouped_conv(x: torch.Tensor, base: torch.Tensor, delta: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """DFlash2 grouped dynamic depthwise convolution (dflash_grouped_conv): x [B, T, C] bf16/fp32,
    base float32 [taps, C], delta float32 [B, T, taps, G] -> out [B, T, C] of x's dtype."""
    lib = load_library()
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, T, C] tensor")
    B, T, C = x.shape
    if base.dim() != 2 or base.shape[1] != C or base.dtype != torch.float32 or not base.is_contiguous():
        raise ValueError("base must be a contiguous float32 [taps, C] tensor")
    taps = base.shape[0]
    if (delta.dim() != 4 or tuple(delta.shape[:3]) != (B, T, taps) or delta.dtype != torch.float32
            or not delta.is_contiguous()):
        raise ValueError("delta must be a contiguous float32 [B, T, taps, G] tensor")
    if out is None:
        out = torch.empty_like(x)
    elif out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of x's shape and dtype")
    st = lib.dflash_grouped_conv(x.data_ptr(), out.data_ptr(), _dtype_code(x), B, T, C, taps, delta.shape[3],
                                 base.data_ptr(), delta.data_ptr(), _stream_handle(stream))
    _check(st)
    return out


def selector_workspace_bytes(num_requests: int, num_slots: int, num_candidates: int) -> int:
    n = load_library().dflash_selector_workspace_bytes(int(num_requests), int(num_slots), int(num_candidates))
    if n == 0:
        raise DflashError(ERR_INVALID_ARG, "invalid sizes for the selector workspace")
    return n


_sel_ws = {}


def selector_walk(pred_codebook: torch.Tensor, succ_codebook: torch.Tensor, proj: torch.Tensor,
                  candidates: torch.Tensor, unary: torch.Tensor, anchor: torch.Tensor, temperature: float = 0.0,
                  uniforms: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  tokens: Optional[torch.Tensor] = None, chosen: Optional[torch.Tensor] = None,
                  path_scores: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                  want_scores: bool = True, device_error: Optional[torch.Tensor] = None, stream=None):
    """DFlash2 candidate-selector walk (dflash_selector_walk). Codebooks bf16 [V, E]; proj float32
    [R, S, E]; candidates int32 [R, S, K]; unary float32 [R, S, K]; anchor int32 [R]; uniforms
    float32 [R, S] when temperature > 0. Returns (tokens [R, S], chosen [R, S], path_scores
    [R, S, K] or None, q [R, S, K] or None). Without a workspace the call uses one cached per
    device: calls that may overlap (different streams) must each pass their own."""
    lib = load_library()
    V, E = pred_codebook.shape
    R, S, K = candidates.shape
    for name, t, dt in (("pred_codebook", pred_codebook, torch.bfloat16), ("succ_codebook", succ_codebook, torch.bfloat16),
                        ("proj", proj, torch.float32), ("candidates", candidates, torch.int32),
                        ("unary", unary, torch.float32), ("anchor", anchor, torch.int32)):
        if t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dt} tensor")
    if tuple(succ_codebook.shape) != (V, E) or tuple(proj.shape) != (R, S, E) or tuple(unary.shape) != (R, S, K) \
            or tuple(anchor.shape) != (R,):
        raise ValueError("inconsistent selector shapes")
    dev = candidates.device
    if temperature > 0:
        if uniforms is None or uniforms.dtype != torch.float32 or tuple(uniforms.shape) != (R, S) \
                or not uniforms.is_contiguous():
            raise ValueError("temperature > 0 needs contiguous float32 uniforms [R, S]")
    if workspace is None:
        need = selector_workspace_bytes(R, S, K)
        key = (dev.type, dev.index)
        workspace = _sel_ws.get(key)
        if workspace is None or workspace.numel() < need:
            workspace = torch.zeros(max(need, 1 << 16), dtype=torch.uint8, device=dev)
            _sel_ws[key] = workspace
    if tokens is None:
        tokens = torch.empty((R, S), dtype=torch.int32, device=dev)
    if chosen is None:
        chosen = torch.empty((R, S), dtype=torch.int32, device=dev)
    if path_scores is None and want_scores:
        path_scores = torch.empty((R, S, K), dtype=torch.float32, device=dev)
    if q is None and temperature > 0:
        q = torch.empty((R, S, K), dtype=torch.float32, device=dev)
    st = lib.dflash_selector_walk(pred_codebook.data_ptr(), succ_codebook.data_ptr(), V, E, proj.data_ptr(),
                                  candidates.data_ptr(), unary.data_ptr(), anchor.data_ptr(), R, S, K,
                                  float(temperature), uniforms.data_ptr() if uniforms is not None else None,
                                  tokens.data_ptr(), chosen.data_ptr(),
                                  path_scores.data_ptr() if path_scores is not None else None,
                                  q.data_ptr() if q is not None else None,
                                  device_error.data_ptr() if device_error is not None else None,
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream))
    _check(st)
    return tokens, chosen, path_scores, q


# ---------------------------------------------------------------------------- drafted trees
#
# These calls take a few microseconds on the GPU, so their marshalling is kept short: one attribute read per fact,
# no helper call per tensor, and the raw stream handle where the caller names no stream.


def _stream_on(dev: torch.device, stream) -> torch.cuda.Stream:
    """The stream of a call whose tensors are on `dev`: the given one, or dev's current stream."""
    if stream is None:
        return torch.cuda.current_stream(dev)
    if isinstance(stream, int):
        return torch.cuda.default_stream(dev) if stream == 0 else torch.cuda.ExternalStream(stream, device=dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return stream


def _call_on(dev: torch.device, stream):
    """(context or None, stream handle): a call's allocations and launches happen on its stream and device,
    whatever the current ones are. None: they are the current ones."""
    if stream is None and torch._C._cuda_getDevice() == dev.index:
        return None, torch._C._cuda_getCurrentRawStream(dev.index)
    s = _stream_on(dev, stream)
    return torch.cuda.stream(s), s.cuda_stream


_tree_ws = {}
# tree_attn launches two kernels that share a workspace: another thread's call on the stream must not come between.
_tree_attn_lock = threading.Lock()


def _tree_workspace(op: str, dev: torch.device, stream: int, nbytes: int, zeroed: int) -> torch.Tensor:
    """A workspace for a call without one, its first `zeroed` bytes zero: cached per operator, device and stream, so
    that calls that may overlap never share one. A call that is being captured gets its own, zeroed by the graph."""
    if torch._C._cuda_isCurrentStreamCapturing():
        buf = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if zeroed:
            buf[:zeroed].zero_()
        return buf
    key = (op, dev.index, stream)
    buf = _tree_ws.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        _tree_ws[key] = buf
    return buf


# Words for the device errors of tree_attn calls whose caller gives none. They stand apart from the workspaces, which
# grow and, of captured calls, belong to the graph.
_tree_words = {}  # (device, stream) -> a word of its eager calls, in a block that dflash_read_error may clear
_graph_words = {}  # device -> address of the word of its captured calls, the library's own
_WORD_BLOCK = 256 + 8192


def _tree_word(dev: torch.device, stream: int) -> int:
    if torch._C._cuda_isCurrentStreamCapturing():
        at = _graph_words.get(dev.index)
        if at is None:
            word = ctypes.c_void_p()
            _check(load_library().dflash_shared_error_word(ctypes.byref(word)))
            at = _graph_words[dev.index] = word.value
        return at
    word = _tree_words.get((dev.index, stream))
    if word is None:
        word = torch.zeros(_WORD_BLOCK, dtype=torch.uint8, device=dev)
        word = _tree_words.setdefault((dev.index, stream), word)  # (another thread's, where that was first)
    return word.data_ptr()


def _bad(name: str, shape, dtype):
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)}")


_I32 = torch.int32


def _check_i32(t: torch.Tensor, shape, dev: int, name: str) -> int:
    """The address of a contiguous int32 tensor of `shape` on CUDA device dev."""
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on the CUDA device of the "
                         "other tensors")
    return t.data_ptr()


def _check_ws(ws: torch.Tensor, dev: int) -> int:
    """Bytes of a given workspace."""
    if not ws.is_contiguous() or ws.get_device() != dev:
        raise ValueError("workspace must be contiguous, on the CUDA device of the tensors")
    return ws.numel() * ws.element_size()


def _check_word(t: torch.Tensor, dev: int) -> int:
    if t.element_size() != 4 or t.dtype.is_floating_point or t.numel() < 1 or t.get_device() != dev:
        raise ValueError("device_error must hold a 32-bit integer, on the CUDA device of the tensors")
    return t.data_ptr()


def logprobs_workspace_bytes(num_rows: int, vocab: int, top_k: int) -> int:
    """Workspace bytes of token_logprobs on the current device."""
    n = load_library().dflash_logprobs_workspace_bytes(int(num_rows), int(vocab), int(top_k))
    if n == 0:
        raise DflashError(ERR_INVALID_ARG, "invalid sizes for the log probability workspace")
    return n


def _row_stride(logits: torch.Tensor, rows: int, V: int) -> int:
    """The one stride of the rows of logits [..., V]."""
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("logits must have a contiguous last dimension")
    if rows <= 1 or logits.is_contiguous():
        return V
    # from the innermost dimension of more than one entry outwards
    want = row = None
    for n, st in zip(reversed(logits.shape[:-1]), reversed(logits.stride()[:-1])):
        if n == 1:
            continue
        if row is None:
            row = st
        elif st != want:
            raise ValueError("the rows of logits must have one stride")
        want = st * n
    return row


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top_k: int = 0,
                   temperature: float = 1.0, want_entropy: bool = True, device_error: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Log probabilities, entropy and top tokens of rows of logits (dflash_token_logprobs).

    logits [..., V] bf16/fp32 whose rows have one stride (last dim contiguous); tokens int32 [..., m] (negative
    ids are padding and get -inf). Returns (token_logp [..., m] or None, entropy [...] or None, log_z [...],
    top_tokens int32 [..., top_k] or None, top_logp [..., top_k] or None), float32 unless said. The
    top tokens come largest first, of equal logits the smaller id first: the candidates and unary
    scores of selector_walk. device_error: an optional int32 device word that receives DEVERR_* bits."""
    lib = _lib or load_library()
    shape = logits.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("logits must be [..., V]")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    lead, V = shape[:-1], shape[-1]
    R = math.prod(lead)
    row = _row_stride(logits, R, V)
    code = _dtype_code(logits)
    dev, index = logits.device, logits.get_device()
    m, tok = 0, None
    if tokens is not None:
        m = tokens.shape[-1] if tokens.dim() == len(shape) else -1
        tok = _check_i32(tokens, lead + (m,), index, "tokens") if m else None
        if m <= 0 and tuple(tokens.shape) != tuple(lead) + (0,):
            _bad("tokens", lead + ("m",), "torch.int32")
    word = None if device_error is None else _check_word(device_error, index)
    given_bytes = None if workspace is None else _check_ws(workspace, index)
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        log_z = torch.empty(lead, dtype=torch.float32, device=dev)
        entropy = token_logp = top_tokens = top_logp = None
        if want_entropy:
            entropy = torch.empty(lead, dtype=torch.float32, device=dev)
        if tokens is not None:
            token_logp = torch.empty(lead + (m,), dtype=torch.float32, device=dev)
        if top_k > 0:
            top_tokens = torch.empty(lead + (top_k,), dtype=_I32, device=dev)
            top_logp = torch.empty(lead + (top_k,), dtype=torch.float32, device=dev)
        if workspace is None and R > 0:
            given_bytes = lib.dflash_logprobs_workspace_bytes(R, V, top_k)
            # (0 for sizes that the call itself refuses with the reason)
            workspace = _tree_workspace("token_logprobs", dev, handle, given_bytes, 4 * R) if given_bytes else None
        st = lib.dflash_token_logprobs(
            logits.data_ptr(), code, R, V, row, temperature, tok, m, token_logp.data_ptr() if m else None,
            log_z.data_ptr(), entropy.data_ptr() if want_entropy else None, top_k,
            top_tokens.data_ptr() if top_k > 0 else None, top_logp.data_ptr() if top_k > 0 else None, word,
            None if workspace is None else workspace.data_ptr(), given_bytes or 0, handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)
    return token_logp, entropy, log_z, top_tokens, top_logp


_tree_dims = {}  # (layout of a call) -> (its Dims, their address for ctypes, workspace bytes)


def _tree_cache_dims(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, first: int, hq: int,
                     max_seq_len: Optional[int], T: int):
    """(Dims, byref, tree attention's workspace bytes) of a cache [..., num_pages, page_size, Hkv, D] whose page
    dimension is `first`. Only sizes and strides decide them, so they are made once per layout."""
    shape, strides, dtype, table = k_cache.shape, k_cache.stride(), k_cache.dtype, page_table.shape
    if v_cache.shape != shape or v_cache.stride() != strides or v_cache.dtype is not dtype:
        raise ValueError("v_cache must match k_cache in shape, strides and dtype")
    key = (shape, strides, dtype, table, first, hq, max_seq_len, T, k_cache.get_device())
    hit = _tree_dims.get(key)
    if hit is None:
        if strides[-1] != 1:
            raise ValueError("the caches' head_dim must be contiguous")
        d = Dims()
        d.batch, d.max_pages = table
        d.num_kv_heads, d.head_dim = shape[first + 2], shape[first + 3]
        d.num_q_heads = hq or d.num_kv_heads
        d.page_size, d.num_pages = shape[first + 1], shape[first]
        d.max_seq_len = int(max_seq_len) if max_seq_len else 0
        d.dtype = _dtype_code(k_cache)
        d.kv_stride_page, d.kv_stride_slot, d.kv_stride_head = (int(s) for s in strides[first:first + 3])
        with torch.cuda.device(k_cache.device):
            nbytes = load_library().dflash_tree_attn_workspace_bytes(ctypes.byref(d), T) if hq else 0
        hit = (d, ctypes.byref(d), nbytes)
        if len(_tree_dims) > 256:
            _tree_dims.clear()
        _tree_dims[key] = hit
    return hit


def tree_attn_workspace_bytes(dims: Dims, max_nodes: int) -> int:
    """Workspace bytes of tree_attn with these dims (make_dims) on the current device."""
    lib = load_library()
    n = lib.dflash_tree_attn_workspace_bytes(ctypes.byref(dims), int(max_nodes))
    if n == 0:
        raise DflashError(ERR_INVALID_ARG, lib.dflash_last_error_message().decode())
    return n


def tree_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
              seq_lens: torch.Tensor, parents: torch.Tensor, num_nodes: Optional[torch.Tensor] = None, window: int = 0,
              scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              kernel: str = "auto", workspace: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
              stream=None, want_lse: bool = True, wait_limit_us: int = 0,
              device_error: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of drafted trees over a paged KV cache (dflash_tree_attn).

    q [B*T, Hq, D]; k_cache, v_cache [num_pages, page_size, Hkv, D] (head_dim contiguous), the nodes' own K/V
    among them; page_table int32 [B, max_pages]; seq_lens int32 [B] (context + nodes); parents int32
    [B, T] (-1 for a root, else an earlier node); num_nodes int32 [B] or None (T each). Returns
    (out [B*T, Hq, D] in q's dtype, lse fp32 [B*T, Hq] or None); padding rows of given outputs keep
    what they held, those of new ones are zero. Without a workspace the call uses one of its stream's (or the
    captured graph's). DEVERR_* bits go to device_error, an int32 device word, if given; else to the given workspace's
    error word (read_error); else to a word that tree_attn_error() reads."""
    lib = _lib or load_library()
    qs, ps = q.shape, parents.shape
    if len(qs) != 3 or k_cache.dim() != 4 or len(ps) != 2:
        raise ValueError("q must be [B*T, Hq, D], the caches [num_pages, page_size, Hkv, D] and parents [B, T]")
    if kernel not in ("auto", "simt", "tc"):
        raise ValueError("kernel must be 'auto', 'simt' or 'tc'")
    B, T = ps
    dev, index = q.device, q.get_device()
    if q.dtype is not k_cache.dtype or qs != (B * T, qs[1], k_cache.shape[3]) or not q.is_contiguous():
        _bad("q", (B * T, qs[1], k_cache.shape[3]), k_cache.dtype)
    if index < 0 or k_cache.get_device() != index or v_cache.get_device() != index:
        raise ValueError("q and the caches must be on one CUDA device")
    batch = (B,)
    table_at = _check_i32(page_table, (B, page_table.shape[-1]), index, "page_table")
    lens_at = _check_i32(seq_lens, batch, index, "seq_lens")
    parents_at = _check_i32(parents, ps, index, "parents")
    nodes_at = None if num_nodes is None else _check_i32(num_nodes, batch, index, "num_nodes")
    if out is not None and (out.dtype is not q.dtype or out.shape != qs or not out.is_contiguous()
                            or out.get_device() != index):
        _bad("out", qs, q.dtype)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != qs[:2] or not lse.is_contiguous()
                            or lse.get_device() != index):
        _bad("lse", qs[:2], torch.float32)
    dims, dims_ref, nbytes = _tree_cache_dims(k_cache, v_cache, page_table, 0, qs[1], max_seq_len, T)
    word = None if device_error is None else _check_word(device_error, index)
    if workspace is not None:
        nbytes = _check_ws(workspace, index)
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        fresh = torch.empty if num_nodes is None else torch.zeros
        if workspace is None and nbytes:  # (0: sizes that the call itself refuses with the reason)
            workspace = _tree_workspace("tree_attn", dev, handle, nbytes, 0)
            if word is None:
                word = _tree_word(dev, handle)
        if out is None:
            out = fresh(qs, dtype=q.dtype, device=dev)
        if lse is None and want_lse:
            lse = fresh(qs[:2], dtype=torch.float32, device=dev)
        with _tree_attn_lock:
            st = lib.dflash_tree_attn_err(
                q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), table_at, lens_at, parents_at, nodes_at,
                dims_ref, T, window, 1.0 / math.sqrt(qs[2]) if scale is None else scale, out.data_ptr(),
                None if lse is None else lse.data_ptr(), KERNELS[kernel], word,
                None if workspace is None else workspace.data_ptr(), nbytes, wait_limit_us, handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)
    return out, lse


def tree_attn_error(device=None, stream=None, clear: bool = True) -> int:
    """DEVERR_* bits of the tree_attn and cache8_attn calls without a device_error and a workspace, and of the append_kv
    calls without a device_error: of the stream's, and of the device's captured ones, whatever stream replays them (a replay
    on another stream has to be waited for first); synchronises the stream."""
    dev = torch.device("cuda" if device is None else device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    s = _stream_on(dev, stream)
    with torch.cuda.stream(s):
        word = _tree_words.get((dev.index, s.cuda_stream))
        bits = 0 if word is None else _read_word(word.data_ptr(), clear, s.cuda_stream)
        at = _graph_words.get(dev.index)
        return bits if at is None else bits | _read_word(at, clear, s.cuda_stream)


def tree_accept(logits: torch.Tensor, tokens: torch.Tensor, parents: torch.Tensor,
                num_nodes: Optional[torch.Tensor] = None, want_argmax: bool = True,
                device_error: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Longest accepted path of drafted trees (dflash_tree_accept): logits [B, T, V] bf16/fp32 (rows of one
    stride, last dim contiguous), tokens and parents int32 [B, T], num_nodes int32 [B] or None. Returns
    (accepted_len [B], path [B, T], next_token [B], target argmax [B, T] or None), int32: path holds the
    accepted nodes from the root on, -1 behind them."""
    lib = _lib or load_library()
    shape = logits.shape
    if len(shape) != 3 or shape[2] < 1:
        raise ValueError("logits must be [B, T, V]")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    B, T, V = shape
    row = _row_stride(logits, B * T, V)
    code = _dtype_code(logits)
    dev, index = logits.device, logits.get_device()
    rows, batch = shape[:2], (B,)
    tokens_at = _check_i32(tokens, rows, index, "tokens")
    parents_at = _check_i32(parents, rows, index, "parents")
    nodes_at = None if num_nodes is None else _check_i32(num_nodes, batch, index, "num_nodes")
    word = None if device_error is None else _check_word(device_error, index)
    nbytes = _accept_bytes(lib) if workspace is None else _check_ws(workspace, index)
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        accepted = torch.empty(batch, dtype=_I32, device=dev)
        nxt = torch.empty(batch, dtype=_I32, device=dev)
        path = torch.empty(rows, dtype=_I32, device=dev)
        argmax = torch.empty(rows, dtype=_I32, device=dev) if want_argmax else None
        if workspace is None:
            workspace = _tree_workspace("tree_accept", dev, handle, nbytes, nbytes)
        st = lib.dflash_tree_accept(
            logits.data_ptr(), code, B, T, V, row, tokens_at, parents_at, nodes_at, accepted.data_ptr(),
            path.data_ptr(), nxt.data_ptr(), argmax.data_ptr() if want_argmax else None, word, workspace.data_ptr(), nbytes, handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)
    return accepted, path, nxt, argmax


_accept_ws_bytes = 0


def _accept_bytes(lib) -> int:
    global _accept_ws_bytes
    if not _accept_ws_bytes:
        _accept_ws_bytes = lib.dflash_tree_accept_workspace_bytes()
    return _accept_ws_bytes


def tree_commit(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                path: torch.Tensor, accepted_len: torch.Tensor, num_nodes: Optional[torch.Tensor] = None,
                new_lens: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
                device_error: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the accepted nodes' K/V to consecutive cache positions (dflash_tree_commit): caches
    [num_pages, page_size, Hkv, D], or [layers, num_pages, page_size, Hkv, D] for every layer at once; path
    int32 [B, T] and accepted_len int32 [B] of tree_accept; seq_lens int32 [B] (context + nodes).
    Returns new_lens int32 [B] (context + bonus token + accepted tokens), which may be seq_lens itself."""
    lib = _lib or load_library()
    first = k_cache.dim() - 4
    shape = path.shape
    if first not in (0, 1) or len(shape) != 2:
        raise ValueError("the caches must be [(layers,) num_pages, page_size, Hkv, D] and path [B, T]")
    B, T = shape
    dev, index = k_cache.device, k_cache.get_device()
    if index < 0 or v_cache.get_device() != index:
        raise ValueError("the caches must be on one CUDA device")
    batch = (B,)
    table_at = _check_i32(page_table, (B, page_table.shape[-1]), index, "page_table")
    lens_at = _check_i32(seq_lens, batch, index, "seq_lens")
    path_at = _check_i32(path, shape, index, "path")
    accepted_at = _check_i32(accepted_len, batch, index, "accepted_len")
    nodes_at = None if num_nodes is None else _check_i32(num_nodes, batch, index, "num_nodes")
    if new_lens is not None:
        _check_i32(new_lens, batch, index, "new_lens")
    dims, dims_ref, _ = _tree_cache_dims(k_cache, v_cache, page_table, first, 0, max_seq_len, T)
    word = None if device_error is None else _check_word(device_error, index)
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        if new_lens is None:
            new_lens = torch.empty(batch, dtype=_I32, device=dev)
        st = lib.dflash_tree_commit(
            k_cache.data_ptr(), v_cache.data_ptr(), table_at, lens_at, path_at, accepted_at, nodes_at,
            new_lens.data_ptr(), dims_ref, T, k_cache.shape[0] if first else 1, k_cache.stride(0) if first else 0,
            word, handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)
    return new_lens


# ---------------------------------------------------------------------------- rotary positions and the 8-bit cache

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
_PI_TIMES_10_60 = 3141592653589793238462643383279502884197169399375105820974944


class Rope:
    """The frequencies of a rotation (make_rope), on a device: what rope and append_kv take."""

    def __init__(self, turns: torch.Tensor, layout: str, gain: float):
        if turns.dtype is not torch.int64 or turns.dim() != 1 or not turns.is_contiguous() or turns.numel() < 1:
            raise ValueError("turns must be a contiguous int64 [rotary_dim / 2] tensor")
        if layout not in ROPE_LAYOUTS:
            raise ValueError("layout must be 'half' or 'interleaved'")
        if not (math.isfinite(gain) and gain > 0):
            raise ValueError("gain must be finite and > 0")
        self.turns, self.layout, self.gain = turns, layout, float(gain)
        self.rotary_dim = 2 * turns.numel()
        self._freqs = RopeFreqs(turns.data_ptr(), self.rotary_dim, ROPE_LAYOUTS[layout], self.gain)
        self._ref = ctypes.byref(self._freqs)
        self._index = turns.get_device()


def make_rope(rotary_dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "none", factor: float = 1.0,
              original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, gain: Optional[float] = None,
              inv_freq=None, device="cuda") -> Rope:
    """The rotation of heads whose first rotary_dim dims turn: pair i by p f_i at position p, f_i = base^(-2i / rotary_dim).

    layout "half" pairs dims i and i + rotary_dim / 2, "interleaved" 2i and 2i + 1. Scalings for contexts `factor` times
    as long: "linear" divides every f_i by it (position interpolation); "ntk" takes the base base * factor^(r / (r - 2)),
    r = rotary_dim, which leaves the fastest pair as it is and divides the slowest by factor. "yarn" and "yarn_index" (Peng et
    al., YaRN, 2023) divide the pairs that turn less than beta_slow times in original_len positions, keep those that turn more
    than beta_fast times, blend linearly between, and scale cosine and sine by a gain of 0.1 ln(factor) + 1. They differ in what
    the blend is linear in: in "yarn" the number of turns, as the paper's text defines it; in "yarn_index" the pair's index,
    from the last pair of more than beta_fast turns to the first of less than beta_slow. Models published with such a scaling
    are as a rule trained and served with the latter: take "yarn_index" for a checkpoint unless it says otherwise. (For base
    10^4, 128 dims, factor 4 and 32768 positions 24 of the 64 frequencies differ, by up to 42 %.) inv_freq (numbers or a tensor
    of rotary_dim / 2) gives the f_i instead, gain another factor of cosine and sine. The table is made on the host, exactly
    from 64-bit floats."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and >= 2")
    if inv_freq is not None:
        if scaling != "none":
            raise ValueError("give inv_freq or a scaling")
        f = [float(x) for x in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq)]
        if len(f) != rotary_dim // 2:
            raise ValueError("inv_freq must hold rotary_dim / 2 numbers")
    else:
        if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor > 0):
            raise ValueError("base and factor must be finite and > 0")
        if scaling == "ntk":
            if rotary_dim == 2:
                raise ValueError("'ntk' needs rotary_dim > 2")
            base = base * factor ** (rotary_dim / (rotary_dim - 2))
        f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling in ("yarn", "yarn_index"):
            if original_len < 1 or not beta_fast > beta_slow:
                raise ValueError("'yarn' needs original_len >= 1 and beta_fast > beta_slow")
            if scaling == "yarn_index":
                if not (base > 1 and beta_slow > 0):
                    raise ValueError("'yarn_index' needs base > 1 and beta_slow > 0")
                # the index at which a pair makes so many turns, the blend's ends rounded outwards and kept within the head
                first, last = (rotary_dim * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))
                               for turns in (beta_fast, beta_slow))
                first, last = max(math.floor(first), 0), min(math.ceil(last), rotary_dim - 1)
            for i, x in enumerate(f):
                if scaling == "yarn":
                    keep = (original_len * x / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)
                else:
                    keep = (last - i) / (last - first) if last > first else float(i <= first)
                keep = min(1.0, max(0.0, keep))
                f[i] = x / factor * (1 - keep) + x * keep
            if gain is None:
                gain = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        elif scaling not in ("none", "ntk"):
            raise ValueError("scaling must be 'none', 'linear', 'ntk', 'yarn' or 'yarn_index'")
    if not all(math.isfinite(x) for x in f):
        raise ValueError("frequencies must be finite")
    turns = []
    for x in f:
        num, den = x.as_integer_ratio()  # of x / 2 pi turns, the nearest multiple of 2^-64, modulo a turn
        num, den = num * 10 ** 60 * 2 ** 64, den * 2 * _PI_TIMES_10_60
        t = (2 * num + den) // (2 * den) % 2 ** 64
        turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return Rope(torch.tensor(turns, dtype=torch.int64).to(device), layout, 1.0 if gain is None else gain)


def _check_rope(rope: Rope, index: int):
    if rope._index != index:
        raise ValueError("the rope must be on the CUDA device of the other tensors")
    return rope._ref


def rope(x: torch.Tensor, positions: torch.Tensor, rope: Rope, inverse: bool = False, out: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """Rotary positions (dflash_rope): x [N, H, D] bf16/fp32 (last dim contiguous, any other strides), positions int32 [N].
    Returns out of x's shape and dtype (a new contiguous tensor, out, or x itself when out is x). inverse turns back,
    which takes the gradient of the result to the gradient of x; autograd records a call without an out, and one of an x
    that requires a gradient is refused with it."""
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("x requires a gradient: a call with an out is not recorded by autograd")
        return _Turn.apply(x, positions, rope, bool(inverse), stream)
    lib = _lib or load_library()
    shape = x.shape
    if len(shape) != 3 or not x.is_cuda:
        raise ValueError("x must be a CUDA tensor [N, H, D]")
    N, H, D = shape
    code = _dtype_code(x)
    dev, index = x.device, x.get_device()
    pos_at = _check_i32(positions, (N,), index, "positions")
    ref = _check_rope(rope, index)
    xs = x.stride()
    if D > 1 and xs[2] != 1:
        raise ValueError("x must have a contiguous last dimension")
    if out is not None:
        os = out.stride()
        if out.shape != shape or out.dtype is not x.dtype or (D > 1 and os[2] != 1) or out.get_device() != index:
            raise ValueError("out must have x's shape, dtype and device and a contiguous last dimension")
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
            os = out.stride()
        st = lib.dflash_rope(x.data_ptr(), out.data_ptr(), code, N, H, D, xs[0], xs[1], os[0], os[1], pos_at, ref,
                             int(inverse), handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)
    return out


class _Turn(torch.autograd.Function):
    """rope as autograd records it: the map is linear, and its transpose is the turn back."""

    @staticmethod
    def forward(ctx, x, positions, turns, inverse, stream):
        ctx.save_for_backward(positions)
        ctx.turns, ctx.inverse = turns, inverse
        return rope(x, positions, turns, inverse=inverse, stream=stream)

    @staticmethod
    def backward(ctx, grad):
        (positions,) = ctx.saved_tensors
        if grad.dim() == 3 and grad.shape[2] > 1 and grad.stride(2) != 1:  # (that of a sum is one number, repeated)
            grad = grad.contiguous()
        return rope(grad, positions, ctx.turns, inverse=not ctx.inverse), None, None, None, None


_E4M3 = torch.float8_e4m3fn
_cache_dims = {}  # (layout of a call) -> (its Dims, their address for ctypes, cache8_attn's workspace bytes)


def _cache8_dims(k_cache: torch.Tensor, v_cache: torch.Tensor, table, hq: int, code: int, max_seq_len: Optional[int], T: int):
    """(Dims, byref, workspace bytes of cache8_attn or 0) of a cache [num_pages, page_size, Hkv, D], made once per layout."""
    shape, strides, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape or v_cache.stride() != strides or v_cache.dtype is not dtype:
        raise ValueError("the caches must be [num_pages, page_size, Hkv, D] of the same shape, strides and dtype")
    key = (shape, strides, dtype, table, hq, code, max_seq_len, T, k_cache.get_device())
    hit = _cache_dims.get(key)
    if hit is None:
        if strides[3] != 1:
            raise ValueError("the caches' head_dim must be contiguous")
        d = Dims()
        d.batch, d.max_pages = table
        d.num_kv_heads, d.head_dim = shape[2], shape[3]
        d.num_q_heads = hq or d.num_kv_heads
        d.page_size, d.num_pages = shape[1], shape[0]
        d.max_seq_len = int(max_seq_len) if max_seq_len else 0
        d.dtype = code
        d.kv_stride_page, d.kv_stride_slot, d.kv_stride_head = (int(x) for x in strides[:3])
        with torch.cuda.device(k_cache.device):
            nbytes = load_library().dflash_cache8_attn_workspace_bytes(ctypes.byref(d), T) if T else 0
        hit = (d, ctypes.byref(d), nbytes)
        if len(_cache_dims) > 256:
            _cache_dims.clear()
        _cache_dims[key] = hit
    return hit


def _check_scale(t: torch.Tensor, shape, dev: int, name: str) -> int:
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 [num_pages, Hkv] tensor on the CUDA device of the caches")
    return t.data_ptr()


def append_kv(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
              seq_lens: torch.Tensor, starts: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
              positions: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None, max_seq_len: Optional[int] = None,
              device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """Appends new keys, rotated by `rope`, and values to the paged cache (dflash_append_kv).

    k, v [N, Hkv, D] bf16/fp32 (last dim contiguous); caches [num_pages, page_size, Hkv, D] of the same dtype, or
    float8_e4m3fn with k_scale and v_scale float32 [num_pages, Hkv]; page_table int32 [B, max_pages]; seq_lens int32 [B],
    the new tokens counted. Request b's rows are starts[b] .. starts[b + 1] - 1 (int32 [B + 1]; None: N / B each), and go to
    the last positions of its seq_lens[b]. positions int32 [N]: what the keys are rotated to, if not to their place in the
    cache. Caches and scales are written in place. device_error: an int32 device word that receives DEVERR_* bits (tokens of
    a bad length, table of starts or page id are left out); without one tree_attn_error() reads them."""
    lib = _lib or load_library()
    shape = k.shape
    if len(shape) != 3 or not k.is_cuda or v.shape != shape or v.dtype is not k.dtype:
        raise ValueError("k and v must be CUDA tensors [N, Hkv, D] of one dtype")
    N = shape[0]
    dev, index = k.device, k.get_device()
    code = _dtype_code(k)
    if v.get_device() != index or k_cache.get_device() != index or v_cache.get_device() != index:
        raise ValueError("k, v and the caches must be on one CUDA device")
    ks, vs = k.stride(), v.stride()
    if shape[2] > 1 and (ks[2] != 1 or vs[2] != 1):
        raise ValueError("k and v must have a contiguous last dimension")
    e4m3 = k_scale is not None
    if k_cache.dtype is not (_E4M3 if e4m3 else k.dtype) or e4m3 != (v_scale is not None):
        raise ValueError("the caches must be of k's dtype, or float8_e4m3fn with k_scale and v_scale")
    if k_cache.dim() != 4 or k_cache.shape[2:] != shape[1:]:
        raise ValueError("the caches must be [num_pages, page_size, Hkv, D] with the heads and dims of k")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B = page_table.shape[0]
    table_at = _check_i32(page_table, (B, page_table.shape[1]), index, "page_table")
    lens_at = _check_i32(seq_lens, (B,), index, "seq_lens")
    starts_at = None if starts is None else _check_i32(starts, (B + 1,), index, "starts")
    pos_at = None if positions is None else _check_i32(positions, (N,), index, "positions")
    scales = (k_cache.shape[0], shape[1])
    k_scale_at = _check_scale(k_scale, scales, index, "k_scale") if e4m3 else None
    v_scale_at = _check_scale(v_scale, scales, index, "v_scale") if e4m3 else None
    ref = None if rope is None else _check_rope(rope, index)
    word = None if device_error is None else _check_word(device_error, index)
    _, dims_ref, _ = _cache8_dims(k_cache, v_cache, page_table.shape, 0, code, max_seq_len, 0)
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        if word is None:
            word = _tree_word(dev, handle)
        st = lib.dflash_append_kv(k.data_ptr(), v.data_ptr(), N, ks[0], ks[1], vs[0], vs[1], starts_at, pos_at, ref,
                                  k_cache.data_ptr(), v_cache.data_ptr(), k_scale_at, v_scale_at, table_at, lens_at,
                                  dims_ref, word, handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)


def cache8_attn_workspace_bytes(dims: Dims, max_queries: int) -> int:
    """Workspace bytes of cache8_attn with these dims (make_dims) on the current device."""
    lib = load_library()
    n = lib.dflash_cache8_attn_workspace_bytes(ctypes.byref(dims), int(max_queries))
    if n == 0:
        raise DflashError(ERR_INVALID_ARG, lib.dflash_last_error_message().decode())
    return n


def cache8_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                v_scale: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor, block_len: int,
                num_queries: Optional[torch.Tensor] = None, parents: Optional[torch.Tensor] = None, causal: bool = False,
                window: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, kernel: str = "auto", workspace: Optional[torch.Tensor] = None,
                max_seq_len: Optional[int] = None, stream=None, want_lse: bool = True, wait_limit_us: int = 0,
                device_error: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention over an e4m3 paged cache with a scale per page and head (dflash_cache8_attn).

    q [B*T, Hq, D] bf16/fp32, T = block_len in [1, 256]; k_cache, v_cache float8_e4m3fn [num_pages, page_size, Hkv, D]
    (head_dim contiguous), k_scale, v_scale float32 [num_pages, Hkv]: append_kv's; page_table int32 [B, max_pages];
    seq_lens int32 [B], the queries' own keys counted; num_queries int32 [B] or None (T each). The mask is block_attn's
    (causal or not, window) or, with parents int32 [B, T], tree_attn's. Returns (out [B*T, Hq, D] in q's dtype, lse fp32
    [B*T, Hq] or None); padding rows of given outputs keep what they held, those of new ones are zero. Workspaces and
    errors are as tree_attn's: without a device_error and a workspace tree_attn_error() reads the bits."""
    lib = _lib or load_library()
    qs = q.shape
    if len(qs) != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q must be [B*T, Hq, D], the caches [num_pages, page_size, Hkv, D] and page_table [B, max_pages]")
    if kernel not in ("auto", "simt", "tc"):
        raise ValueError("kernel must be 'auto', 'simt' or 'tc'")
    B, T = page_table.shape[0], int(block_len)
    dev, index = q.device, q.get_device()
    code = _dtype_code(q)
    if qs != (B * T, qs[1], k_cache.shape[3]) or not q.is_contiguous():
        _bad("q", (B * T, qs[1], k_cache.shape[3]), q.dtype)
    if k_cache.dtype is not _E4M3:
        raise TypeError("the caches must be float8_e4m3fn")
    if index < 0 or k_cache.get_device() != index or v_cache.get_device() != index:
        raise ValueError("q and the caches must be on one CUDA device")
    batch = (B,)
    table_at = _check_i32(page_table, (B, page_table.shape[1]), index, "page_table")
    lens_at = _check_i32(seq_lens, batch, index, "seq_lens")
    nodes_at = None if num_queries is None else _check_i32(num_queries, batch, index, "num_queries")
    parents_at = None if parents is None else _check_i32(parents, (B, T), index, "parents")
    scales = (k_cache.shape[0], k_cache.shape[2])
    k_scale_at = _check_scale(k_scale, scales, index, "k_scale")
    v_scale_at = _check_scale(v_scale, scales, index, "v_scale")
    if out is not None and (out.dtype is not q.dtype or out.shape != qs or not out.is_contiguous()
                            or out.get_device() != index):
        _bad("out", qs, q.dtype)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != qs[:2] or not lse.is_contiguous()
                            or lse.get_device() != index):
        _bad("lse", qs[:2], torch.float32)
    _, dims_ref, nbytes = _cache8_dims(k_cache, v_cache, page_table.shape, qs[1], code, max_seq_len, T)
    word = None if device_error is None else _check_word(device_error, index)
    if workspace is not None:
        nbytes = _check_ws(workspace, index)
    ctx, handle = _call_on(dev, stream)
    if ctx is not None:
        ctx.__enter__()
    try:
        fresh = torch.empty if num_queries is None else torch.zeros
        if workspace is None and nbytes:  # (0: sizes that the call itself refuses with the reason)
            workspace = _tree_workspace("cache8_attn", dev, handle, nbytes, 0)
            if word is None:
                word = _tree_word(dev, handle)
        if out is None:
            out = fresh(qs, dtype=q.dtype, device=dev)
        if lse is None and want_lse:
            lse = fresh(qs[:2], dtype=torch.float32, device=dev)
        with _tree_attn_lock:
            st = lib.dflash_cache8_attn(
                q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale_at, v_scale_at, table_at, lens_at, nodes_at,
                parents_at, dims_ref, T, int(causal), window, 1.0 / math.sqrt(qs[2]) if scale is None else scale,
                out.data_ptr(), None if lse is None else lse.data_ptr(), KERNELS[kernel], word,
                None if workspace is None else workspace.data_ptr(), nbytes, wait_limit_us, handle)
    finally:
        if ctx is not None:
            ctx.__exit__(None, None, None)
    if st:
        _check(st)
    return out, lse


def read_error(workspace: Optional[torch.Tensor] = None, clear: bool = True, stream=None) -> int:
    """The workspace's device error word (DEVERR_* bits); synchronises the stream."""
    lib = load_library()
    if workspace is None:
        if not torch.cuda.is_available():
            return 0
        workspace = _ws_cache.get(("cuda", torch.cuda.current_device()))
        if workspace is None:
            return 0
    return _read_word(workspace.data_ptr(), clear, _stream_handle(stream))


def _read_word(at: int, clear: bool, stream: int) -> int:
    word = ctypes.c_uint32(0)
    st = load_library().dflash_read_error(at, stream, ctypes.byref(word), int(bool(clear)))
    if st not in (OK, ERR_DEVICE_CHECK):
        _check(st)
    return int(word.value)


def abi_version() -> int:
    return int(load_library().dflash_abi_version())
