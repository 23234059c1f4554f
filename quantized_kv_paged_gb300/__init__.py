"""Python binding of libqkvp: paged MLA decode over a quantized (FP8 E4M3 / NVFP4) latent KV cache.

Argument marshalling only: every function below forwards to the C entry point of the same name
(``include/qkvp.h``) with raw device pointers and the current torch CUDA stream. All computation runs
in the library's CUDA kernels. There is no fallback: if the library is missing, ``load()`` raises.
PyTorch is used for device memory and streams.
"""
from __future__ import annotations

import ctypes
import itertools
import operator
import os
import threading
from array import array

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libqkvp.so")

QKVP_OK, QKVP_E_INVALID, QKVP_E_UNSUPPORTED, QKVP_E_WORKSPACE, QKVP_E_CUDA = 0, -1, -2, -3, -4
KV_FP8_E4M3, KV_NVFP4, KV_BF16, KV_FP8_PER_TOKEN = 1, 2, 3, 4
PAGE_BYTES_FP8_PER_TOKEN = 64 * (576 + 4)   # 64 rows of E4M3 codes, then 64 FP32 token scales
SRC_FP8_E4M3, SRC_BF16 = 1, 2
ALGO_AUTO, ALGO_MMA_SYNC, ALGO_TCGEN05, ALGO_MMA_FP8, ALGO_TCGEN05_TOKENS = 0, 1, 2, 3, 4
CACHE_E4M3, CACHE_INT8 = 1, 2
ROPE_HALVES, ROPE_PAIRS = 0, 1
LATENT_DIM, V_DIM, PAGE_SIZE = 576, 512, 64

EXPORTS = ["kv_append_quant", "mla_decode_plan", "mla_decode_run", "mla_decode_attend",
           "mla_decode_combine", "mla_decode_noalloc", "kv_pool_cast_bf16", "kv_gather_fp8",
           "kv_gather_pages_bf16", "mla_append_rope", "gqa_append_rope", "gqa_decode_plan", "gqa_decode_run",
           "gqa_tree_plan", "gqa_tree_run", "gqa_tree_commit", "kv_pages_workspace", "kv_pages_copy", "kv_pages_fork",
           "kv_pages_grow", "kv_pages_free", "kv_pages_compact", "qkvp_encode_f32", "qkvp_status_string", "qkvp_version"]


class qkvp_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_heads", "page_size", "kv_dtype", "algo", "num_workers", "ctas_per_worker",
        "num_segments", "num_split_requests", "num_empty_requests", "max_worker_pages",
        "min_worker_pages", "num_partials", "max_request_segments",
        "num_wide_requests")] + [
        ("total_pages", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_uint64), ("table_bytes", ctypes.c_uint64),
        ("partial_o_offset", ctypes.c_uint64), ("partial_lse_offset", ctypes.c_uint64),
        ("status_offset", ctypes.c_uint64), ("magic", ctypes.c_uint64)]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class gqa_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_heads", "num_kv_heads", "head_dim", "page_size", "cache_dtype", "window", "sinks",
        "num_workers", "warps_per_worker", "num_segments", "num_split_groups", "max_group_segments", "num_partials",
        "max_worker_pages", "min_worker_pages", "table_entries", "reserved")] + [
        ("total_pages", ctypes.c_int64), ("total_tokens", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_uint64), ("table_bytes", ctypes.c_uint64),
        ("partial_o_offset", ctypes.c_uint64), ("partial_lse_offset", ctypes.c_uint64),
        ("status_offset", ctypes.c_uint64), ("magic", ctypes.c_uint64)]

    as_dict = qkvp_plan.as_dict


class qkvp_tree_plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_heads", "num_kv_heads", "head_dim", "page_size", "cache_dtype", "window", "sinks", "num_tokens",
        "max_drafted", "num_workers", "num_segments", "num_joins", "max_join_segments", "num_partials",
        "max_worker_pages", "min_worker_pages", "table_entries", "row_copies", "reserved")] + [
        ("total_pages", ctypes.c_int64)] + [(n, ctypes.c_uint64) for n in (
            "workspace_bytes", "table_bytes", "partial_o_offset", "partial_lse_offset", "status_offset", "magic")]

    as_dict = qkvp_plan.as_dict


class qkvp_page_state(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("table", "held", "lens", "refs", "free_list", "free_count")] + [
        ("rows", ctypes.c_int32), ("row_pages", ctypes.c_int32), ("num_pages", ctypes.c_int64)]


class QkvpError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


_lib = None
_lock = threading.Lock()


def load(path: str | None = None):
    """Load libqkvp.so (built by ``quantized_kv_paged_gb300.build``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libqkvp.so not found at {p}: run quantized_kv_paged_gb300.build.build()")
        L = ctypes.CDLL(p)
        c = ctypes
        vp, i32, i64, u64, f32 = c.c_void_p, c.c_int32, c.c_int64, c.c_uint64, c.c_float
        L.kv_append_quant.argtypes = [vp, i32, i64, vp, vp, vp, i32, f32, i32, i64, vp]
        L.mla_decode_plan.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, u64, vp,
                                      c.POINTER(qkvp_plan)]
        L.mla_decode_run.argtypes = [c.POINTER(qkvp_plan), vp, vp, vp, i64, vp, f32, f32, vp, vp,
                                     vp, u64, vp]
        L.mla_decode_attend.argtypes = L.mla_decode_run.argtypes
        L.mla_decode_combine.argtypes = [c.POINTER(qkvp_plan), f32, vp, vp, vp, u64, vp]
        L.mla_decode_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, i64, vp, f32,
                                         f32, vp, vp, vp]
        L.kv_pool_cast_bf16.argtypes = [vp, i64, vp, vp]
        L.kv_gather_fp8.argtypes = [vp, vp, i32, f32, i32, i64, vp, vp, i64, vp, i32, i64, vp, vp]
        L.kv_gather_pages_bf16.argtypes = [vp, i32, i64, vp, i64, vp, vp]
        L.mla_append_rope.argtypes = [vp, i64, vp, i64, i64, vp, vp, vp, i64, i32, vp, i64, i64, i32, vp,
                                      vp, vp, i32, f32, i32, i64, vp]
        L.gqa_append_rope.argtypes = [vp, i64, vp, i64, i64, vp, vp, i32, vp, vp, i64, vp, vp, i64, i32,
                                      i32, i32, i32, vp, vp, i32, i32, i64, vp, i64, i32, vp, vp]
        L.gqa_decode_plan.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, vp, u64,
                                      vp, c.POINTER(gqa_plan)]
        L.gqa_decode_run.argtypes = [c.POINTER(gqa_plan), vp, vp, vp, i64, vp, f32, vp, vp, vp, u64, vp]
        L.gqa_tree_plan.argtypes = [vp, vp, vp] + [i32] * 10 + [vp, u64, vp, c.POINTER(qkvp_tree_plan)]
        L.gqa_tree_run.argtypes = [c.POINTER(qkvp_tree_plan), vp, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, u64, vp]
        L.gqa_tree_commit.argtypes = [vp, vp, i32, vp, i32, vp, vp, i64, vp, vp, i32, i32, i32, i32, i32, i64, vp]
        L.kv_pages_workspace.argtypes = [i64, i32, i32, c.POINTER(u64)]
        pool, state = vp, c.POINTER(qkvp_page_state)      # pool: qkvp_pool array
        L.kv_pages_copy.argtypes = [pool, i32, vp, vp, i64, i64, vp]
        L.kv_pages_fork.argtypes = [pool, i32, state, vp, vp, i32, vp, vp, u64, vp]
        L.kv_pages_grow.argtypes = [state, vp, vp, i32, vp, vp, u64, vp]
        L.kv_pages_free.argtypes = [state, vp, i32, vp, u64, vp]
        L.kv_pages_compact.argtypes = [pool, i32, state, vp, u64, vp]
        L.qkvp_encode_f32.argtypes = [vp, i64, i32, vp, vp]
        L.qkvp_status_string.restype = c.c_char_p
        L.qkvp_status_string.argtypes = [c.c_int]
        for fn in EXPORTS:
            if fn != "qkvp_status_string":
                getattr(L, fn).restype = c.c_int
        _lib = L
        return L


def status_string(status: int) -> str:
    return load().qkvp_status_string(status).decode()


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _table(kv_indptr, kv_len):
    """The host page table as contiguous int32 arrays; kv_indptr must have len(kv_len) + 1 entries
    (the library reads kv_indptr[r + 1] for every request r)."""
    indptr = np.ascontiguousarray(kv_indptr, dtype=np.int32)
    lens = np.ascontiguousarray(kv_len, dtype=np.int32)
    if indptr.ndim != 1 or lens.ndim != 1 or indptr.shape[0] != lens.shape[0] + 1:
        raise ValueError(f"kv_indptr needs len(kv_len) + 1 = {lens.shape[0] + 1} entries, got {indptr.shape}")
    return indptr, lens


def _check(fn, status, raise_on_error):
    if status != QKVP_OK and raise_on_error:
        raise QkvpError(fn, status)
    return status


def kv_append_quant(src, src_dtype: int, slot_mapping, kv_data, kv_scale, kv_dtype: int,
                    global_scale: float = 1.0, num_pages: int | None = None,
                    page_size: int = PAGE_SIZE, stream=None, raise_on_error: bool = True) -> int:
    """Quantize-on-append of src [n, 576] into the paged pool at slot_mapping (see qkvp.h)."""
    n = int(src.shape[0]) if src is not None else 0
    if num_pages is None:
        num_pages = int(kv_data.shape[0])
    st = load().kv_append_quant(_ptr(src), src_dtype, n, _ptr(slot_mapping), _ptr(kv_data),
                                _ptr(kv_scale), kv_dtype, float(global_scale), page_size,
                                int(num_pages), _stream(stream))
    return _check("kv_append_quant", st, raise_on_error)


def mla_decode_plan(kv_indptr, kv_len, num_heads: int, kv_dtype: int, num_sms: int = 0,
                    min_splits: int = 0, algo: int = ALGO_AUTO, workspace=None,
                    page_size: int = PAGE_SIZE, stream=None, raise_on_error: bool = True):
    """Plan the split; with workspace=None only sizes are computed. Returns a qkvp_plan."""
    indptr, lens = _table(kv_indptr, kv_len)
    plan = qkvp_plan()
    ws = _ptr(workspace)
    nbytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
    st = load().mla_decode_plan(indptr.ctypes.data, lens.ctypes.data, int(lens.shape[0]),
                                num_heads, page_size, kv_dtype, num_sms, min_splits, algo, ws,
                                nbytes, _stream(stream) if ws else None, ctypes.byref(plan))
    _check("mla_decode_plan", st, raise_on_error)
    plan.status = st
    return plan


def mla_decode_run(plan: qkvp_plan, q, kv_data, kv_scale, num_pages: int, kv_indices,
                   sm_scale: float, global_scale: float, out, lse, workspace, stream=None,
                   raise_on_error: bool = True) -> int:
    """Decode one layer: out [B, H, 512] bf16 and lse [B, H] float32 (lse may be None)."""
    nbytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
    st = load().mla_decode_run(ctypes.byref(plan), _ptr(q), _ptr(kv_data), _ptr(kv_scale),
                               int(num_pages), _ptr(kv_indices), float(sm_scale),
                               float(global_scale), _ptr(out), _ptr(lse), _ptr(workspace), nbytes,
                               _stream(stream))
    return _check("mla_decode_run", st, raise_on_error)


def mla_decode_attend(plan: qkvp_plan, q, kv_data, kv_scale, num_pages: int, kv_indices,
                      sm_scale: float, global_scale: float, out, lse, workspace, stream=None,
                      raise_on_error: bool = True) -> int:
    """The split-KV decode kernel alone (first half of mla_decode_run)."""
    nbytes = int(workspace.numel() * workspace.element_size())
    st = load().mla_decode_attend(ctypes.byref(plan), _ptr(q), _ptr(kv_data), _ptr(kv_scale),
                                  int(num_pages), _ptr(kv_indices), float(sm_scale),
                                  float(global_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                  nbytes, _stream(stream))
    return _check("mla_decode_attend", st, raise_on_error)


def mla_decode_combine(plan: qkvp_plan, global_scale: float, out, lse, workspace, stream=None,
                       raise_on_error: bool = True) -> int:
    """The log-sum-exp merge of split partials (second half of mla_decode_run)."""
    nbytes = int(workspace.numel() * workspace.element_size())
    st = load().mla_decode_combine(ctypes.byref(plan), float(global_scale), _ptr(out), _ptr(lse),
                                   _ptr(workspace), nbytes, _stream(stream))
    return _check("mla_decode_combine", st, raise_on_error)


def mla_decode_noalloc(kv_indptr, kv_len, num_heads: int, kv_dtype: int, q, kv_data, kv_scale,
                       num_pages: int, kv_indices, sm_scale: float, global_scale: float, out, lse,
                       num_sms: int = 0, min_splits: int = 0, stream=None,
                       raise_on_error: bool = True) -> int:
    """Plan + decode with the library's fixed scratch array, for callers that cannot allocate
    device memory (see qkvp.h for the size limit and the sharing rules)."""
    indptr, lens = _table(kv_indptr, kv_len)
    st = load().mla_decode_noalloc(indptr.ctypes.data, lens.ctypes.data, int(lens.shape[0]), num_heads,
                                   kv_dtype, num_sms, min_splits, _ptr(q), _ptr(kv_data),
                                   _ptr(kv_scale), int(num_pages), _ptr(kv_indices), float(sm_scale),
                                   float(global_scale), _ptr(out), _ptr(lse), _stream(stream))
    return _check("mla_decode_noalloc", st, raise_on_error)


def kv_pool_cast_bf16(src, out, stream=None, raise_on_error: bool = True) -> int:
    """The cast-then-attend baseline's pool-wide FP8 -> BF16 cast."""
    st = load().kv_pool_cast_bf16(_ptr(src), int(src.numel()), _ptr(out), _stream(stream))
    return _check("kv_pool_cast_bf16", st, raise_on_error)


def kv_gather_fp8(kv_data, kv_scale, kv_dtype: int, global_scale: float, kv_indptr, kv_indices, tok_indptr,
                  out, num_pages: int | None = None, page_size: int = PAGE_SIZE, stream=None,
                  raise_on_error: bool = True) -> int:
    """Extend-path gather of each request's tokens into the FP8 workspace out [T, 576] (see qkvp.h).
    kv_indptr / kv_indices int32 and tok_indptr int64 are device tensors."""
    if num_pages is None:
        num_pages = int(kv_data.shape[0])
    batch = int(tok_indptr.shape[0]) - 1
    st = load().kv_gather_fp8(_ptr(kv_data), _ptr(kv_scale), kv_dtype, float(global_scale), page_size,
                              int(num_pages), _ptr(kv_indptr), _ptr(kv_indices), int(kv_indices.numel()),
                              _ptr(tok_indptr), batch, int(out.shape[0]), _ptr(out), _stream(stream))
    return _check("kv_gather_fp8", st, raise_on_error)


def kv_gather_pages_bf16(kv_data, page_ids, out, num_pages: int | None = None, page_size: int = PAGE_SIZE,
                         stream=None, raise_on_error: bool = True) -> int:
    """Gather-then-cast baseline: pool pages page_ids (device int32) cast into out [n, 64, 576] BF16."""
    if num_pages is None:
        num_pages = int(kv_data.shape[0])
    st = load().kv_gather_pages_bf16(_ptr(kv_data), page_size, int(num_pages), _ptr(page_ids),
                                     int(page_ids.numel()), _ptr(out), _stream(stream))
    return _check("kv_gather_pages_bf16", st, raise_on_error)


class _Torch:
    """What the checked entry points take from torch, which is imported on the first of their calls. Their
    checks run on every call of a decode step, so they are written for few attribute reads: one look at
    each tensor's type, shape, layout and device, all against the first tensor's device."""
    ready = False

    @classmethod
    def get(cls):
        if not cls.ready:
            import torch
            cls.torch = torch
            cls.bf16, cls.f32, cls.i32, cls.i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
            cls.u32 = torch.uint32
            # for looks over lists of tensors
            cls.ptr, cls.size, cls.same_size, cls.device = torch.Tensor.data_ptr, torch.Tensor.size, torch.Tensor.is_same_size, torch.Tensor.get_device
            cls.contiguous, cls.dtype, cls.nbytes = torch.Tensor.is_contiguous, operator.attrgetter("dtype"), operator.attrgetter("nbytes")
            cls.codes = (torch.uint8, torch.int8, torch.float8_e4m3fn)
            # the current stream's handle without a Stream object around it, where this torch has the call
            cls.handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda device: torch.cuda.current_stream(device).cuda_stream)
            cls.ready = True
        return cls


def _alike(name: str, tensors, dtypes, T, here: int):
    """Refuses tensors that do not lie in memory as the first one does, of another type or on another device. A call takes two
    for each layer, so each look goes over the whole list."""
    first = tensors[0]
    if (not all(map(T.same_size, tensors, itertools.repeat(first))) or not all(map(T.contiguous, tensors)) or
            not set(map(T.dtype, tensors)) <= dtypes or set(map(T.device, tensors)) != {here}):
        for i, t in enumerate(tensors):
            if t.shape != first.shape or not t.is_contiguous() or t.dtype not in dtypes or t.get_device() != here:
                _refuse(f"{name}[{i}]", t, first.shape, dtypes, "a contiguous layout", here)


def _refuse(name: str, t, shape, dtype, layout: str, here: int):
    if t.get_device() != here:
        raise ValueError(f"tensors need to be on one device, the current CUDA device: {name} is on {t.device}")
    raise ValueError(f"{name} needs the shape {tuple(shape)}, the type {dtype} and {layout}; got {tuple(t.shape)}, {t.dtype}, "
                     f"strides {t.stride()}")


def _dense(name: str, t, shape, dtype, here: int):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != here:
        _refuse(name, t, shape, dtype, "a contiguous layout", here)


def _rows(name: str, t, n: int, heads: int, dim: int, dtype, here: int):
    """Row stride of a [n, heads, dim] tensor (heads 0: [n, dim]) whose rows are dense. The stride of an extent
    of one says nothing: such a tensor counts as dense."""
    stride = t.stride()
    if heads == 0:
        if t.shape != (n, dim) or t.dtype is not dtype or stride[1] != 1 or t.get_device() != here:
            _refuse(name, t, (n, dim), dtype, "dense rows", here)
        return stride[0] if n > 1 else dim
    if t.shape != (n, heads, dim) or t.dtype is not dtype or stride[2] != 1 or (stride[1] != dim and heads > 1) or t.get_device() != here:
        _refuse(name, t, (n, heads, dim), dtype, "dense rows", here)
    return stride[0] if n > 1 else heads * dim


# bytes of a latent pool's page and of its scales, by kv_dtype
_LATENT_PAGE = {KV_FP8_E4M3: (PAGE_SIZE * LATENT_DIM, 0), KV_NVFP4: (PAGE_SIZE * LATENT_DIM // 2, PAGE_SIZE * LATENT_DIM // 16),
                KV_FP8_PER_TOKEN: (PAGE_BYTES_FP8_PER_TOKEN, 0)}


def _latent_pool(kv_data, kv_scale, kv_dtype: int, num_pages: int, here: int):
    page, scales = _LATENT_PAGE.get(kv_dtype, (0, 0))
    for name, t, need in (("kv_data", kv_data, page), ("kv_scale", kv_scale, scales)):
        if t is None:
            continue
        if t.get_device() != here:
            raise ValueError("tensors need to be on one device, the current CUDA device: the pool is on another")
        if not t.is_contiguous() or t.nbytes < num_pages * need:
            raise ValueError(f"{name} needs a contiguous layout and the bytes of {num_pages} pages, {need} each; got {tuple(t.shape)}, "
                             f"{t.dtype}, strides {t.stride()}")


def _launch_on(stream, here: int):
    """The stream to launch on. The launch goes to the current device, so the tensors have to be there."""
    if here < 0 or here != _Torch.torch.cuda.current_device():
        raise ValueError(f"tensors need to be on the current CUDA device, got device index {here}")
    if stream is None:
        return _Torch.handle(here)
    return stream if isinstance(stream, int) else stream.cuda_stream


def mla_append_rope(c_kv, k_pe, slot_mapping, positions, cos_sin, rope_style: int, kv_data, kv_scale,
                    kv_dtype: int, q_pe=None, q=None, global_scale: float = 1.0,
                    num_pages: int | None = None, page_size: int = PAGE_SIZE, stream=None,
                    raise_on_error: bool = True) -> int:
    """Append latent rows [c_kv | rotated k_pe] at slot_mapping, quantized, and rotate q_pe [n, H, 64] into
    the last 64 dims of q [n, H, 576] (see qkvp.h). c_kv [n, 512], k_pe [n, 64] and q_pe may be slices with
    their own row strides; cos_sin float32 [max_positions, 64]."""
    T = _Torch.get()
    n, here = c_kv.shape[0], c_kv.get_device()
    c_stride = _rows("c_kv", c_kv, n, 0, V_DIM, T.bf16, here)
    pe_stride = _rows("k_pe", k_pe, n, 0, 64, T.bf16, here)
    _dense("slot_mapping", slot_mapping, (n,), T.i64, here)
    _dense("positions", positions, (n,), T.i64, here)
    max_positions = cos_sin.shape[0]
    _dense("cos_sin", cos_sin, (max_positions, 64), T.f32, here)
    if num_pages is None:
        num_pages = kv_data.shape[0]
    _latent_pool(kv_data, kv_scale, kv_dtype, num_pages, here)
    heads = tok_stride = head_stride = 0
    q_at = pe_at = None
    if q is not None or q_pe is not None:
        if q is None or q_pe is None or q.dim() != 3:
            raise ValueError("q_pe [n, H, 64] and q [n, H, 576] go together")
        heads = q.shape[1]
        _dense("q", q, (n, heads, LATENT_DIM), T.bf16, here)
        stride = q_pe.stride()
        if q_pe.shape != (n, heads, 64) or q_pe.dtype is not T.bf16 or stride[2] != 1 or q_pe.get_device() != here:
            _refuse("q_pe", q_pe, (n, heads, 64), T.bf16, "a dense last dimension", here)
        if heads:
            head_stride = stride[1] if heads > 1 else 64
            tok_stride = stride[0] if n > 1 else 64
            q_at, pe_at = q.data_ptr(), q_pe.data_ptr()
    on = _launch_on(stream, here)
    st = (_lib or load()).mla_append_rope(
        c_kv.data_ptr(), c_stride, k_pe.data_ptr(), pe_stride, n, slot_mapping.data_ptr(), positions.data_ptr(),
        cos_sin.data_ptr(), max_positions, rope_style, pe_at, tok_stride, head_stride, heads, q_at,
        kv_data.data_ptr(), kv_scale if kv_scale is None else kv_scale.data_ptr(), kv_dtype, global_scale, page_size,
        num_pages, on)
    return st if st == QKVP_OK else _check("mla_append_rope", st, raise_on_error)


def _head_pool(kv_data, kv_scale, T, here: int):
    """(pages, KV heads, head dim) of a head pool."""
    shape = kv_data.shape
    if len(shape) != 5 or shape[1] != 2 or shape[3] != PAGE_SIZE or kv_data.dtype not in T.codes or not kv_data.is_contiguous() or kv_data.get_device() != here:
        _refuse("kv_data", kv_data, ("pages", 2, "heads", PAGE_SIZE, "dim"), T.codes, "a contiguous layout", here)
    pages, _, heads, _, dim = shape
    _dense("kv_scale", kv_scale, (pages, 2, heads), T.f32, here)
    return pages, heads, dim


def gqa_append_rope(k, v, tok_indptr, kv_len, kv_indptr, kv_indices, cos_sin, rope_style: int, kv_data,
                    kv_scale, cache_dtype: int, q=None, q_out=None, positions=None, stream=None,
                    raise_on_error: bool = True) -> int:
    """Append K (rotated) and V heads [n, Hkv, D] to the head pool kv_data uint8 [pages, 2, Hkv, 64, D] with
    kv_scale float32 [pages, 2, Hkv], and rotate q [n, H, D] into q_out (see qkvp.h). k, v and q may be
    slices of one projection; request r's tokens are tok_indptr[r] .. tok_indptr[r + 1] - 1 and go behind
    its kv_len[r] cached ones. cos_sin float32 [max_positions, rot_dim], or None: no rotation."""
    T = _Torch.get()
    n, here = k.shape[0], k.get_device()
    pages, heads_kv, dim = _head_pool(kv_data, kv_scale, T, here)
    batch, nnz = kv_len.shape[0], kv_indices.shape[0]
    bf16, i32 = T.bf16, T.i32
    k_stride, v_stride = _rows("k", k, n, heads_kv, dim, bf16, here), _rows("v", v, n, heads_kv, dim, bf16, here)
    _dense("tok_indptr", tok_indptr, (batch + 1,), i32, here)
    _dense("kv_len", kv_len, (batch,), i32, here)
    _dense("kv_indptr", kv_indptr, (batch + 1,), i32, here)
    _dense("kv_indices", kv_indices, (nnz,), i32, here)
    max_positions = rot = heads = q_stride = 0
    cs_at = pos_at = q_at = out_at = None
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            _refuse("cos_sin", cos_sin, ("positions", "rot_dim"), T.f32, "a contiguous layout", here)
        max_positions, rot = shape = cos_sin.shape
        _dense("cos_sin", cos_sin, shape, T.f32, here)
        cs_at = cos_sin.data_ptr()
    if positions is not None:
        _dense("positions", positions, (n,), T.i64, here)
        pos_at = positions.data_ptr()
    if q is not None or q_out is not None:
        if q is None or q_out is None or q_out.dim() != 3:
            raise ValueError("q and q_out [n, H, D] go together")
        heads = q_out.shape[1]
        _dense("q_out", q_out, (n, heads, dim), bf16, here)
        if heads:
            q_stride = _rows("q", q, n, heads, dim, bf16, here)
            q_at, out_at = q.data_ptr(), q_out.data_ptr()
    on = _launch_on(stream, here)
    st = (_lib or load()).gqa_append_rope(
        k.data_ptr(), k_stride, v.data_ptr(), v_stride, n, tok_indptr.data_ptr(), kv_len.data_ptr(), batch,
        kv_indptr.data_ptr(), kv_indices.data_ptr(), nnz, pos_at, cs_at, max_positions, rot, rope_style, heads_kv, dim,
        kv_data.data_ptr(), kv_scale.data_ptr(), cache_dtype, PAGE_SIZE, pages, q_at, q_stride, heads, out_at, on)
    return st if st == QKVP_OK else _check("gqa_append_rope", st, raise_on_error)


def _workspace(t, here: int):
    if t.get_device() != here:
        raise ValueError("tensors need to be on one device, the current CUDA device: the workspace is on another")
    if not t.is_contiguous():
        raise ValueError(f"workspace needs a contiguous layout, got strides {t.stride()}")


def gqa_decode_plan(kv_indptr, kv_len, num_heads: int, num_kv_heads: int, head_dim: int, cache_dtype: int,
                    window: int = 0, sinks: int = 0, num_sms: int = 0, min_splits: int = 0, workspace=None,
                    page_size: int = PAGE_SIZE, stream=None, raise_on_error: bool = True):
    """Plan a head-pool decode on the host; with workspace=None only sizes are computed. Returns a gqa_plan."""
    indptr, lens = _table(kv_indptr, kv_len)
    plan = gqa_plan()
    ws, nbytes, on = None, 0, None
    if workspace is not None:
        _Torch.get()
        here = workspace.get_device()
        _workspace(workspace, here)
        on = _launch_on(stream, here)
        ws, nbytes = workspace.data_ptr(), workspace.nbytes
    st = load().gqa_decode_plan(indptr.ctypes.data, lens.ctypes.data, int(lens.shape[0]), num_heads,
                                num_kv_heads, head_dim, page_size, cache_dtype, window, sinks, num_sms,
                                min_splits, ws, nbytes, on, ctypes.byref(plan))
    _check("gqa_decode_plan", st, raise_on_error)
    plan.status = st
    return plan


def gqa_decode_run(plan: gqa_plan, q, kv_data, kv_scale, kv_indices, sm_scale: float, out, lse, workspace,
                   stream=None, raise_on_error: bool = True) -> int:
    """Decode one layer over a head pool: q, out bf16 [B, H, D], lse float32 [B, H] or None; kv_data and
    kv_scale as for gqa_append_rope."""
    T = _Torch.get()
    batch, heads, dim = plan.batch, plan.num_heads, plan.head_dim
    here = q.get_device()
    _dense("q", q, (batch, heads, dim), T.bf16, here)
    _dense("out", out, (batch, heads, dim), T.bf16, here)
    pages, heads_kv, kv_dim = _head_pool(kv_data, kv_scale, T, here)
    if heads_kv != plan.num_kv_heads or kv_dim != dim:
        raise ValueError(f"kv_data has {heads_kv} heads of {kv_dim}, the plan {plan.num_kv_heads} of {dim}")
    entries = kv_indices.shape[0]
    _dense("kv_indices", kv_indices, (entries,), T.i32, here)
    if entries < plan.table_entries:
        raise ValueError(f"kv_indices has {entries} entries, the plan's page table {plan.table_entries}")
    lse_at = None
    if lse is not None:
        _dense("lse", lse, (batch, heads), T.f32, here)
        lse_at = lse.data_ptr()
    _workspace(workspace, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).gqa_decode_run(ctypes.byref(plan), q.data_ptr(), kv_data.data_ptr(), kv_scale.data_ptr(), pages,
                                         kv_indices.data_ptr(), sm_scale, out.data_ptr(), lse_at, workspace.data_ptr(),
                                         workspace.nbytes, on)
    return st if st == QKVP_OK else _check("gqa_decode_run", st, raise_on_error)


def gqa_tree_plan(kv_indptr, kv_len, tok_indptr, num_heads: int, num_kv_heads: int, head_dim: int, cache_dtype: int,
                  window: int = 0, sinks: int = 0, num_sms: int = 0, min_splits: int = 0, workspace=None,
                  page_size: int = PAGE_SIZE, stream=None, raise_on_error: bool = True):
    """Plan the attention of drafted tokens on the host: request r's last tok_indptr[r + 1] - tok_indptr[r] of kv_len[r]
    tokens are drafted. With workspace=None only sizes are computed. Returns a qkvp_tree_plan."""
    indptr, lens = _table(kv_indptr, kv_len)
    tok, _ = _table(tok_indptr, lens)
    plan = qkvp_tree_plan()
    ws, nbytes, on = None, 0, None
    if workspace is not None:
        _Torch.get()
        here = workspace.get_device()
        _workspace(workspace, here)
        on = _launch_on(stream, here)
        ws, nbytes = workspace.data_ptr(), workspace.nbytes
    st = load().gqa_tree_plan(indptr.ctypes.data, lens.ctypes.data, tok.ctypes.data, int(lens.shape[0]), num_heads,
                              num_kv_heads, head_dim, page_size, cache_dtype, window, sinks, num_sms, min_splits, ws,
                              nbytes, on, ctypes.byref(plan))
    _check("gqa_tree_plan", st, raise_on_error)
    plan.status = st
    return plan


def gqa_tree_run(plan: qkvp_tree_plan, q, kv_data, kv_scale, kv_indices, tree_mask, sm_scale: float, out, lse,
                 workspace, stream=None, raise_on_error: bool = True) -> int:
    """Attention of one layer's drafted tokens over a head pool: q, out bf16 [n, H, D], lse float32 [n, H] or None;
    tree_mask int32 [n, words], bit k of a row set for the k-th drafted token that it sees, or None for chains."""
    T = _Torch.get()
    n, heads, dim = plan.num_tokens, plan.num_heads, plan.head_dim
    here = q.get_device()
    _dense("q", q, (n, heads, dim), T.bf16, here)
    _dense("out", out, (n, heads, dim), T.bf16, here)
    pages, heads_kv, kv_dim = _head_pool(kv_data, kv_scale, T, here)
    if heads_kv != plan.num_kv_heads or kv_dim != dim:
        raise ValueError(f"kv_data has {heads_kv} heads of {kv_dim}, the plan {plan.num_kv_heads} of {dim}")
    entries = kv_indices.shape[0]
    _dense("kv_indices", kv_indices, (entries,), T.i32, here)
    if entries < plan.table_entries:
        raise ValueError(f"kv_indices has {entries} entries, the plan's page table {plan.table_entries}")
    mask_at, words = None, 0
    if tree_mask is not None:
        words = tree_mask.shape[-1]
        if tree_mask.dtype is not T.i32 and tree_mask.dtype is not T.u32 or tree_mask.shape != (n, words) or not tree_mask.is_contiguous() or tree_mask.get_device() != here:
            _refuse("tree_mask", tree_mask, (n, "words"), T.i32, "a contiguous layout", here)
        mask_at = tree_mask.data_ptr()
        if words * 32 < plan.max_drafted:
            raise ValueError(f"tree_mask has {words} words a token, the plan's trees have up to {plan.max_drafted} tokens")
        if n == 0:
            mask_at, words = None, 0
    lse_at = None
    if lse is not None:
        _dense("lse", lse, (n, heads), T.f32, here)
        lse_at = lse.data_ptr()
    _workspace(workspace, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).gqa_tree_run(ctypes.byref(plan), q.data_ptr(), kv_data.data_ptr(), kv_scale.data_ptr(), pages,
                                       kv_indices.data_ptr(), mask_at, words, sm_scale, out.data_ptr(), lse_at,
                                       workspace.data_ptr(), workspace.nbytes, on)
    return st if st == QKVP_OK else _check("gqa_tree_run", st, raise_on_error)


def gqa_tree_commit(kv_data, kv_scale, cache_dtype: int, kv_len, kv_indptr, kv_indices, path, path_len, stream=None,
                    raise_on_error: bool = True) -> int:
    """Move the accepted drafted tokens right behind the cached ones in every layer: kv_data and kv_scale are lists of the
    layers' head pools, path int32 [batch, max_path] ascending indices of drafted tokens, path_len int32 [batch],
    kv_len int32 [batch] the tokens before the drafted ones (see qkvp.h)."""
    T = _Torch.get()
    layers = len(kv_data)
    if layers != len(kv_scale):
        raise ValueError(f"{layers} layers of kv_data and {len(kv_scale)} of kv_scale")
    here = kv_len.get_device()
    pages, heads, dim = 0, 1, 64
    if layers:
        pages, heads, dim = _head_pool(kv_data[0], kv_scale[0], T, here)
        _alike("kv_data", kv_data, set(T.codes), T, here)
        _alike("kv_scale", kv_scale, {T.f32}, T, here)
    batch, nnz, i32 = kv_len.shape[0], kv_indices.shape[0], T.i32
    max_path = path.shape[-1]
    _dense("kv_len", kv_len, (batch,), i32, here)
    _dense("kv_indptr", kv_indptr, (batch + 1,), i32, here)
    _dense("kv_indices", kv_indices, (nnz,), i32, here)
    _dense("path", path, (batch, max_path), i32, here)
    _dense("path_len", path_len, (batch,), i32, here)
    on = _launch_on(stream, here)
    data, scales = array("Q", map(T.ptr, kv_data)), array("Q", map(T.ptr, kv_scale))
    st = (_lib or load()).gqa_tree_commit(data.buffer_info()[0], scales.buffer_info()[0], layers, kv_len.data_ptr(), batch, kv_indptr.data_ptr(),
                                          kv_indices.data_ptr(), nnz, path.data_ptr(), path_len.data_ptr(), max_path,
                                          heads, dim, cache_dtype, PAGE_SIZE, pages, on)
    return st if st == QKVP_OK else _check("gqa_tree_commit", st, raise_on_error)


def kv_pages_workspace(num_pages: int, rows: int, n: int) -> int:
    """Bytes of the workspace of the kv_pages_* calls, for lists of up to n entries. It has to be zero before its first use."""
    size = ctypes.c_uint64()
    _check("kv_pages_workspace", load().kv_pages_workspace(num_pages, rows, n, ctypes.byref(size)), True)
    return size.value


def _pools(pools, num_pages: int, T, here: int):
    """The pools as the C array (data, page_bytes); every one a contiguous tensor with a page for each first index. A call
    takes one or two for each layer, so each look goes over the whole list."""
    try:
        rows = set(map(T.size, pools, itertools.repeat(0)))
    except IndexError:                         # a tensor without dimensions
        rows = set()
    sizes = list(map(T.nbytes, pools))
    if pools and (rows != {num_pages} or set(map(T.device, pools)) != {here} or not all(map(T.contiguous, pools)) or 0 in sizes):
        for i, t in enumerate(pools):
            if t.get_device() != here:
                raise ValueError(f"tensors need to be on one device, the current CUDA device: pool {i} is on {t.device}")
            if t.dim() < 1 or t.shape[0] != num_pages or not t.is_contiguous() or t.nbytes == 0:
                raise ValueError(f"pool {i} needs a contiguous layout and {num_pages} pages; got {tuple(t.shape)}, strides {t.stride()}")
    arr = array("q", bytes(16 * len(pools)))
    arr[::2] = array("q", map(T.ptr, pools))
    arr[1::2] = array("q", [n // num_pages for n in sizes])
    return arr


def _page_state(table, held, lens, refs, free_list, free_count, T, here: int):
    i32 = T.i32
    if table.dim() != 2:
        _refuse("table", table, ("rows", "pages"), i32, "a contiguous layout", here)
    rows, row_pages = shape = table.shape
    pages = refs.shape[0]
    for name, t, want in (("table", table, shape), ("held", held, (rows,)), ("lens", lens, (rows,)), ("refs", refs, (pages,)),
                          ("free_list", free_list, (pages,)), ("free_count", free_count, (1,))):
        _dense(name, t, want, i32, here)
    return qkvp_page_state(table.data_ptr(), held.data_ptr(), lens.data_ptr(), refs.data_ptr(), free_list.data_ptr(),
                           free_count.data_ptr(), rows, row_pages, pages)


def kv_pages_copy(pools, src, dst, stream=None, raise_on_error: bool = True) -> int:
    """Copy page src[i] to page dst[i] (int32 device tensors) in every tensor of the list pools, each [num_pages, ...]."""
    T = _Torch.get()
    here, n = src.get_device(), src.shape[0]
    _dense("src", src, (n,), T.i32, here)
    _dense("dst", dst, (n,), T.i32, here)
    pages = pools[0].shape[0] if len(pools) and pools[0].dim() else 0
    arr = _pools(pools, pages, T, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).kv_pages_copy(arr.buffer_info()[0], len(pools), src.data_ptr(), dst.data_ptr(), n, pages, on)
    return st if st == QKVP_OK else _check("kv_pages_copy", st, raise_on_error)


def kv_pages_fork(pools, table, held, lens, refs, free_list, free_count, parents, children, status, workspace, stream=None,
                  raise_on_error: bool = True) -> int:
    """Rows children[i] become copies of rows parents[i]: full pages are shared, a started one is copied in every tensor of
    pools. status[i] is 1 where that was done (see qkvp.h)."""
    T = _Torch.get()
    here, n = table.get_device(), parents.shape[0]
    state = _page_state(table, held, lens, refs, free_list, free_count, T, here)
    for name, t in (("parents", parents), ("children", children), ("status", status)):
        _dense(name, t, (n,), T.i32, here)
    arr = _pools(pools, refs.shape[0], T, here)
    _workspace(workspace, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).kv_pages_fork(arr.buffer_info()[0], len(pools), ctypes.byref(state), parents.data_ptr(), children.data_ptr(), n,
                                        status.data_ptr(), workspace.data_ptr(), workspace.nbytes, on)
    return st if st == QKVP_OK else _check("kv_pages_fork", st, raise_on_error)


def kv_pages_grow(table, held, lens, refs, free_list, free_count, rows, tokens, status, workspace, stream=None,
                  raise_on_error: bool = True) -> int:
    """Rows rows[i] get the pages that tokens[i] tokens need. status[i] is 1 where that was done (see qkvp.h)."""
    T = _Torch.get()
    here, n = table.get_device(), rows.shape[0]
    state = _page_state(table, held, lens, refs, free_list, free_count, T, here)
    for name, t in (("rows", rows), ("tokens", tokens), ("status", status)):
        _dense(name, t, (n,), T.i32, here)
    _workspace(workspace, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).kv_pages_grow(ctypes.byref(state), rows.data_ptr(), tokens.data_ptr(), n, status.data_ptr(),
                                        workspace.data_ptr(), workspace.nbytes, on)
    return st if st == QKVP_OK else _check("kv_pages_grow", st, raise_on_error)


def kv_pages_free(table, held, lens, refs, free_list, free_count, rows, workspace, stream=None,
                  raise_on_error: bool = True) -> int:
    """Rows rows[i] give their pages back; what nobody holds any more joins the free list (see qkvp.h)."""
    T = _Torch.get()
    here, n = table.get_device(), rows.shape[0]
    state = _page_state(table, held, lens, refs, free_list, free_count, T, here)
    _dense("rows", rows, (n,), T.i32, here)
    _workspace(workspace, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).kv_pages_free(ctypes.byref(state), rows.data_ptr(), n, workspace.data_ptr(), workspace.nbytes, on)
    return st if st == QKVP_OK else _check("kv_pages_free", st, raise_on_error)


def kv_pages_compact(pools, table, held, lens, refs, free_list, free_count, workspace, stream=None,
                     raise_on_error: bool = True) -> int:
    """Move the pages with references to the lowest ids, in every tensor of pools, tables and counts with them (see qkvp.h)."""
    T = _Torch.get()
    here = table.get_device()
    state = _page_state(table, held, lens, refs, free_list, free_count, T, here)
    arr = _pools(pools, refs.shape[0], T, here)
    _workspace(workspace, here)
    on = _launch_on(stream, here)
    st = (_lib or load()).kv_pages_compact(arr.buffer_info()[0], len(pools), ctypes.byref(state), workspace.data_ptr(), workspace.nbytes, on)
    return st if st == QKVP_OK else _check("kv_pages_compact", st, raise_on_error)


def qkvp_encode_f32(x, fmt: int, codes, stream=None, raise_on_error: bool = True) -> int:
    """Device E4M3 (fmt 1) / E2M1 (fmt 2) rounding of FP32 values, one code byte each."""
    st = load().qkvp_encode_f32(_ptr(x), int(x.numel()), fmt, _ptr(codes), _stream(stream))
    return _check("qkvp_encode_f32", st, raise_on_error)


def qkvp_version() -> int:
    return load().qkvp_version()
