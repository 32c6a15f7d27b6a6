"""Python binding of libsfi, the GB300 decode-attention hot path of Slow-Fast
Inference (SFI) with Vegas-style aggregated selection.

This module only marshals arguments: every step of the path runs in the CUDA
kernels of ``_lib/libsfi.so`` (built in-tree from ``csrc/`` by
``__graft_entry__.build()``).  Importing it without the built library raises
ImportError; there is no CPU fallback.  Functions carry the C names declared
in ``include/sfi.h`` and take torch tensors (device memory) or None for the
nullable pointers; ``stream`` is a torch.cuda.Stream, a raw cudaStream_t
handle, or None for torch's current stream.
"""
from __future__ import annotations

import array
import ctypes
import os
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libsfi.so")

SFI_OK, SFI_ERR_INVALID_ARG, SFI_ERR_UNSUPPORTED, SFI_ERR_CAPACITY, SFI_ERR_WORKSPACE, SFI_ERR_CUDA = range(6)
SFI_F32, SFI_BF16 = 0, 1
SFI_SELECT_FUSED, SFI_SELECT_LOGIT_SUM_SEQ, SFI_SELECT_LOGIT_SUM_HEAD = 0, 1, 2
SFI_DEV_LEN_OVER_CAP, SFI_DEV_BAD_INDEX, SFI_DEV_WAIT_TIMEOUT, SFI_DEV_ITEMS_OVERFLOW = 1, 2, 4, 8
SFI_DEV_REFINE, SFI_DEV_NO_PAGES = 16, 32


class sfi_layout(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32),
                ("head_dim", c_int32), ("dtype", c_int32), ("max_len", c_int32),
                ("kv_offset", c_void_p), ("kv_cap", c_void_p), ("len", c_void_p)]


class sfi_params(ctypes.Structure):
    _fields_ = [("n_sink", c_int32), ("window", c_int32), ("k", c_int32),
                ("lam", c_float), ("mode", c_int32)]


class sfi_refine(ctypes.Structure):
    _fields_ = [("nms_radius", c_int32), ("nms_sigma", c_float), ("excl_beta", c_float)]


class sfi_ctx_desc(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32),
                ("head_dim", c_int32), ("dtype", c_int32), ("max_len", c_int32),
                ("n_layers", c_int32), ("params", sfi_params), ("budget", c_int32),
                ("async_select", c_int32), ("refine", sfi_refine)]


class sfi_packed_layout(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32),
                ("head_dim", c_int32), ("dtype", c_int32), ("total_q", c_int32),
                ("total_k", c_int32), ("q_stride", c_int64), ("k_stride", c_int64),
                ("v_stride", c_int64), ("out_stride", c_int64), ("cu_q", c_void_p),
                ("cu_k", c_void_p)]


class sfi_paged_layout(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("n_q_heads", c_int32), ("n_kv_heads", c_int32),
                ("head_dim", c_int32), ("dtype", c_int32), ("page_size", c_int32),
                ("n_pages", c_int32), ("max_pages", c_int32), ("page_stride", c_int64),
                ("page_table", c_void_p), ("len", c_void_p)]


class sfi_page_store(ctypes.Structure):
    _fields_ = [("ref", c_void_p), ("k", c_void_p), ("v", c_void_p), ("n_layers", c_int32),
                ("layer_stride", c_int64)]


_L = POINTER(sfi_layout)
_P = POINTER(sfi_params)
_PL, _PS = POINTER(sfi_paged_layout), POINTER(sfi_page_store)
# name -> (restype, argtypes); every function declared in include/sfi.h
EXPORTS = {
    "sfi_last_error": (c_char_p, []),
    "sfi_read_status": (c_int32, [c_void_p, POINTER(c_uint32), c_void_p]),
    "sfi_device_sm_count": (c_int32, []),
    "sfi_set_wait_limit": (c_int32, [ctypes.c_int64]),
    "sfi_slow_attn_workspace_size": (c_size_t, [_L]),
    "sfi_slow_attn": (c_int32, [_L, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_size_t, c_void_p]),
    "sfi_select_workspace_size": (c_size_t, [_L, _P]),
    "sfi_select": (c_int32, [_L, _P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_size_t, c_void_p]),
    "sfi_select_refined_workspace_size": (c_size_t, [_L, _P, POINTER(sfi_refine)]),
    "sfi_select_refined": (c_int32, [_L, _P, POINTER(sfi_refine), c_void_p, c_void_p, c_void_p,
                                     c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_fast_attn_workspace_size": (c_size_t, [_L, _P]),
    "sfi_fast_attn": (c_int32, [_L, _P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_verify_attn_workspace_size": (c_size_t, [_L, c_int32]),
    "sfi_verify_attn": (c_int32, [_L, c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_fast_attn_noalloc": (c_int32, [_L, _P, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                        c_void_p, c_void_p]),
    "sfi_prefill_attn_workspace_size": (c_size_t, [POINTER(sfi_packed_layout)]),
    "sfi_prefill_attn": (c_int32, [POINTER(sfi_packed_layout), c_void_p, c_void_p, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_paged_workspace_size": (c_size_t, [_PL]),
    "sfi_paged_attn": (c_int32, [_PL, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_size_t, c_void_p]),
    "sfi_paged_append": (c_int32, [_PL, c_int32, c_void_p, c_void_p, c_int64, c_int64, c_void_p,
                                   c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_pages_extend": (c_int32, [_PL, _PS, c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_pages_fork": (c_int32, [_PL, _PS, c_void_p, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
    "sfi_pages_free": (c_int32, [_PL, _PS, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
    "sfi_pages_compact": (c_int32, [_PL, _PS, c_void_p, c_void_p, c_size_t, c_void_p]),
    "sfi_pages_copy": (c_int32, [_PL, _PS, c_void_p, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]),
    "sfi_ctx_create": (c_int32, [POINTER(sfi_ctx_desc), POINTER(c_void_p)]),
    "sfi_ctx_destroy": (c_int32, [c_void_p]),
    "sfi_decode_step": (c_int32, [c_void_p, c_int32, c_void_p, _L, c_void_p, c_void_p, c_void_p,
                                  c_void_p, c_void_p]),
    "sfi_schedule": (c_int32, [c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p]),
    "sfi_ctx_reset": (c_int32, [c_void_p]),
    "sfi_ctx_read_status": (c_int32, [c_void_p, POINTER(c_uint32), c_void_p]),
    "sfi_ctx_profile": (c_int32, [c_void_p, c_int32]),
    "sfi_ctx_profile_read": (c_int32, [c_void_p, POINTER(ctypes.c_double), POINTER(ctypes.c_int64),
                                       POINTER(ctypes.c_double), POINTER(ctypes.c_int64)]),
    "sfi_ctx_slow_mask": (c_int32, [c_void_p, c_void_p]),
    "sfi_ctx_selection": (c_int32, [c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libsfi is not built ({LIB_PATH} missing): run `python -c \"import __graft_entry__ as g; "
            f"g.build()\"` first.  There is no CPU fallback.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class SfiError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib.sfi_last_error().decode(errors="replace")
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != SFI_OK:
        raise SfiError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libsfi takes device tensors")
    return t.data_ptr()


# (torch.cuda.current_stream() builds a Stream object: 2.9 us a call against 0.1)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return SFI_F32
    if dt == torch.bfloat16:
        return SFI_BF16
    raise ValueError(f"unsupported dtype {dt}")


class Layout:
    """Batch/cache geometry of one layer: owns the device arrays the C layout points to.

    ``kv_offset[b]`` (elements), ``kv_cap[b]`` and ``len[b]`` describe where
    sequence b's [H_kv][cap][d] block lives and how long it is."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 kv_offset: Sequence[int], kv_cap: Sequence[int], lens: Sequence[int],
                 max_len: int, device="cuda"):
        self.B = len(kv_cap)
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.dtype = dtype
        self.max_len = int(max_len)
        self.kv_offset = torch.tensor(list(kv_offset), dtype=torch.int64, device=device)
        self.kv_cap = torch.tensor(list(kv_cap), dtype=torch.int32, device=device)
        self.len = torch.tensor(list(lens), dtype=torch.int32, device=device)
        self._c = None

    def set_lens(self, lens: Sequence[int]) -> None:
        self.len.copy_(torch.tensor(list(lens), dtype=torch.int32))

    @property
    def c(self) -> sfi_layout:
        return sfi_layout(self.B, self.n_q_heads, self.n_kv_heads, self.head_dim,
                          dtype_code(self.dtype), self.max_len, self.kv_offset.data_ptr(),
                          self.kv_cap.data_ptr(), self.len.data_ptr())


def params(n_sink: int, window: int, k: int, lam: float, mode: int = SFI_SELECT_FUSED) -> sfi_params:
    return sfi_params(int(n_sink), int(window), int(k), float(lam), int(mode))


def workspace_size(layout: Layout) -> int:
    c = layout.c
    return int(lib.sfi_slow_attn_workspace_size(ctypes.byref(c)))


def alloc_workspace(layout: Layout) -> torch.Tensor:
    """A zero-filled device workspace for every call of this geometry."""
    n = workspace_size(layout)
    if n == 0:
        raise SfiError("sfi_slow_attn_workspace_size", SFI_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def sfi_slow_attn(layout: Layout, q, k, v, out, f_out=None, knorm_out=None, ws=None, stream=None):
    c = layout.c
    _check("sfi_slow_attn", lib.sfi_slow_attn(
        ctypes.byref(c), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(f_out), _ptr(knorm_out),
        _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def sfi_select(layout: Layout, prm: sfi_params, evidence, knorm, idx_out, count_out, s_out=None,
               ws=None, stream=None):
    c = layout.c
    _check("sfi_select", lib.sfi_select(
        ctypes.byref(c), ctypes.byref(prm), _ptr(evidence), _ptr(knorm), _ptr(idx_out),
        _ptr(count_out), _ptr(s_out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def sfi_select_refined(layout: Layout, prm: sfi_params, ref: sfi_refine, f, knorm, idx_out,
                       count_out, s_out=None, ws=None, stream=None):
    c = layout.c
    _check("sfi_select_refined", lib.sfi_select_refined(
        ctypes.byref(c), ctypes.byref(prm), ctypes.byref(ref), _ptr(f), _ptr(knorm), _ptr(idx_out),
        _ptr(count_out), _ptr(s_out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def select_refined_workspace_size(layout: Layout, prm: sfi_params, ref: sfi_refine) -> int:
    return int(lib.sfi_select_refined_workspace_size(ctypes.byref(layout.c), ctypes.byref(prm),
                                                     ctypes.byref(ref)))


def sfi_fast_attn(layout: Layout, prm: sfi_params, q, k, v, idx, count, out, ws=None, stream=None):
    c = layout.c
    _check("sfi_fast_attn", lib.sfi_fast_attn(
        ctypes.byref(c), ctypes.byref(prm), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(count),
        _ptr(out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def sfi_schedule(is_boundary, have_sel, since, budget: int):
    """Host-only schedule step on numpy arrays (uint8, uint8, int32; updated in place).
    Returns the slow mask (uint8 [B])."""
    import numpy as np
    B = len(is_boundary)
    ib = np.ascontiguousarray(is_boundary, np.uint8)
    out = np.zeros(B, np.uint8)
    assert have_sel.dtype == np.uint8 and since.dtype == np.int32
    _check("sfi_schedule", lib.sfi_schedule(B, int(budget), ib.ctypes.data, have_sel.ctypes.data,
                                            since.ctypes.data, out.ctypes.data))
    return out


def verify_workspace(layout: Layout, n_rows: int) -> torch.Tensor:
    """A zero-filled workspace for sfi_verify_attn with n_rows chain rows."""
    c = layout.c
    n = int(lib.sfi_verify_attn_workspace_size(ctypes.byref(c), int(n_rows)))
    if n == 0:
        raise SfiError("sfi_verify_attn_workspace_size", SFI_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def sfi_verify_attn(layout: Layout, n_rows: int, collect_rows, q, k, v, out, logitsum_out=None,
                    ws=None, stream=None):
    rows = list(collect_rows or [])
    arr = (c_int32 * max(1, len(rows)))(*rows)
    c = layout.c
    _check("sfi_verify_attn", lib.sfi_verify_attn(
        ctypes.byref(c), int(n_rows), arr, len(rows), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
        _ptr(logitsum_out), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))


def sfi_fast_attn_noalloc(layout: Layout, prm: sfi_params, q, k, v, idx, count, out, stream=None):
    """The fast step without a workspace (scratch in a fixed array inside the
    library), for callers that may not allocate on the path that runs it."""
    c = layout.c
    _check("sfi_fast_attn_noalloc", lib.sfi_fast_attn_noalloc(
        ctypes.byref(c), ctypes.byref(prm), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(count),
        _ptr(out), _stream(stream)))


def _want(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, device: torch.device,
          inner: bool = False) -> torch.Tensor:
    """Refuse a tensor of another shape, type or device, or one that is not dense (with
    ``inner``: not dense behind its first dimension)."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} lies on {t.device}, the layout on {device}")
    if not t.is_contiguous() and not (inner and t[0].is_contiguous()):
        raise ValueError(f"{name} must be dense{' behind its first dimension' if inner else ''}")
    if inner and shape[0] > 1 and t.stride(0) < shape[1] * shape[2]:
        # (an expanded row has stride 0, which the C calls read as rows without gaps)
        raise ValueError(f"{name}: rows {t.stride(0)} elements apart overlap")
    return t


def _device_of(name: str, t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name}: libsfi takes device tensors")
    return t.device


def _here(device: torch.device, stream) -> None:
    """The kernels run on the current device, so the tensors and the stream must be its own."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors lie on {device}, but cuda:{torch.cuda.current_device()} is current")
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")


class PackedLayout:
    """Prompts packed one after another: sequence b's query rows are
    cu_q[b]..cu_q[b + 1] of [total_q, H_q, d], its key rows cu_k[b]..cu_k[b + 1]
    of [total_k, H_kv, d] (cu_*: int32 device tensors of batch + 1 entries)."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 cu_q: torch.Tensor, cu_k: torch.Tensor, total_q: int, total_k: int):
        self.device = _device_of("cu_q", cu_q)
        self.B = cu_q.numel() - 1
        _want("cu_q", cu_q, (self.B + 1,), torch.int32, self.device)
        _want("cu_k", cu_k, (self.B + 1,), torch.int32, self.device)
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.dtype = n_q_heads, n_kv_heads, head_dim, dtype
        self.cu_q, self.cu_k = cu_q, cu_k
        self.total_q, self.total_k = int(total_q), int(total_k)
        self._c = sfi_packed_layout(self.B, n_q_heads, n_kv_heads, head_dim, dtype_code(dtype),
                                    self.total_q, self.total_k, 0, 0, 0, 0, cu_q.data_ptr(),
                                    cu_k.data_ptr())


def prefill_workspace(layout: PackedLayout) -> torch.Tensor:
    """A zero-filled workspace for sfi_prefill_attn."""
    n = int(lib.sfi_prefill_attn_workspace_size(ctypes.byref(layout._c)))
    if n == 0:
        raise SfiError("sfi_prefill_attn_workspace_size", SFI_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=layout.device)


def sfi_prefill_attn(layout: PackedLayout, q, k, v, out, lse_out=None, ws=None, stream=None):
    """q, out [total_q, H_q, d], k, v [total_k, H_kv, d], bf16, heads dense, any row stride (slices
    of a joint projection); lse_out [total_q, H_q] fp32."""
    L, c = layout, sfi_packed_layout.from_buffer_copy(layout._c)
    _here(L.device, stream)
    rq, rk = (L.total_q, L.n_q_heads, L.head_dim), (L.total_k, L.n_kv_heads, L.head_dim)
    _want("q", q, rq, L.dtype, L.device, True)
    _want("k", k, rk, L.dtype, L.device, True)
    _want("v", v, rk, L.dtype, L.device, True)
    _want("out", out, rq, L.dtype, L.device, True)
    if lse_out is not None:
        _want("lse_out", lse_out, rq[:2], torch.float32, L.device)
    # (a row stride only means something where there is a second row)
    c.q_stride, c.out_stride = (t.stride(0) if L.total_q > 1 else 0 for t in (q, out))
    c.k_stride, c.v_stride = (t.stride(0) if L.total_k > 1 else 0 for t in (k, v))
    _check("sfi_prefill_attn", lib.sfi_prefill_attn(
        ctypes.byref(c), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse_out), *_ws(ws, L.device),
        _stream(stream)))


class PagedLayout:
    """A KV cache in pages: sequence b's position i lies in row i % page_size of
    page page_table[b, i // page_size] (page_table [B, max_pages], len [B], int32
    device tensors, shared with the caller).  One layer's pool is
    [n_pages, H_kv, page_size, d]; ``page_stride`` is the distance of its pages in
    elements where they are not one after another (0: they are)."""

    def __init__(self, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 page_size: int, n_pages: int, page_table: torch.Tensor, len: torch.Tensor,
                 page_stride: int = 0):
        self.device = _device_of("page_table", page_table)
        if page_table.dim() != 2:
            raise ValueError("page_table: expected [batch, max_pages]")
        self.B, self.max_pages = page_table.shape
        _want("page_table", page_table, (self.B, self.max_pages), torch.int32, self.device)
        _want("len", len, (self.B,), torch.int32, self.device)
        self.n_q_heads, self.n_kv_heads, self.head_dim, self.dtype = n_q_heads, n_kv_heads, head_dim, dtype
        self.page_size, self.n_pages, self.page_stride = page_size, n_pages, page_stride
        self.page_table, self.len = page_table, len
        self._pool_shape = (n_pages, n_kv_heads, page_size, head_dim)
        self._page_strides = (page_size * head_dim, head_dim, 1)
        self.c = sfi_paged_layout(self.B, n_q_heads, n_kv_heads, head_dim, dtype_code(dtype), page_size,
                                  n_pages, self.max_pages, page_stride, page_table.data_ptr(),
                                  len.data_ptr())

    def _pool(self, name: str, t: torch.Tensor, layers: int = 0) -> torch.Tensor:
        """Refuse a tensor that is not a pool ([layers,] n_pages, H_kv, page_size, d) of this layout."""
        want = (layers,) + self._pool_shape if layers else self._pool_shape
        if t.dtype is not self.dtype or t.shape != want or t.device != self.device:
            raise ValueError(f"{name}: expected {self.dtype} {want} on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device}")
        apart = self.page_stride or self.n_kv_heads * self.page_size * self.head_dim
        strides = t.stride()[-4:]
        if strides[1:] != self._page_strides and not t[(0,) * (t.dim() - 3)].is_contiguous():
            raise ValueError(f"{name}: a page must be dense")
        if self.n_pages > 1 and strides[0] != apart:
            raise ValueError(f"{name}: pages lie {strides[0]} elements apart, the layout says {apart}")
        return t


class PageStore:
    """The page counts ref [n_pages] (int32) and the pools k, v of the layers that the
    bookkeeping moves: [n_pages, H_kv, page_size, d] or [layers, n_pages, H_kv, page_size, d]."""

    def __init__(self, ref: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
        self.ref, self.k, self.v = ref, k, v
        if k.shape != v.shape or k.stride() != v.stride() or k.dim() not in (4, 5):
            raise ValueError("k and v must be pools of the same shape and strides")
        self.layers = k.shape[0] if k.dim() == 5 else 0
        self.c = sfi_page_store(_ptr(ref), _ptr(k), _ptr(v), max(1, self.layers),
                                k.stride(0) if self.layers > 1 else 0)

    def _check(self, layout: PagedLayout) -> "PageStore":
        _want("ref", self.ref, (layout.n_pages,), torch.int32, layout.device)
        layout._pool("k", self.k, self.layers)
        layout._pool("v", self.v, self.layers)
        return self


def paged_workspace(layout: PagedLayout) -> torch.Tensor:
    """A zero-filled workspace for every paged call of this geometry."""
    n = int(lib.sfi_paged_workspace_size(ctypes.byref(layout.c)))
    if n == 0:
        raise SfiError("sfi_paged_workspace_size", SFI_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=layout.device)


def _ws(ws, device: torch.device):
    if ws is None:
        return None, 0
    if ws.device != device:
        raise ValueError(f"the workspace lies on {ws.device}, the layout on {device}")
    return _ptr(ws), ws.numel() * ws.element_size()


def sfi_paged_attn(layout: PagedLayout, q, k, v, out, lse_out=None, ws=None, stream=None):
    """q [B, H_q, d], k, v one layer's pools; out [B, H_q, d] and lse_out [B, H_q] fp32."""
    L = layout
    _here(L.device, stream)
    rq = (L.B, L.n_q_heads, L.head_dim)
    _want("q", q, rq, L.dtype, L.device)
    L._pool("k", k)
    L._pool("v", v)
    _want("out", out, rq, torch.float32, L.device)
    if lse_out is not None:
        _want("lse_out", lse_out, rq[:2], torch.float32, L.device)
    _check("sfi_paged_attn", lib.sfi_paged_attn(
        ctypes.byref(L.c), _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse_out), *_ws(ws, L.device),
        _stream(stream)))


def sfi_paged_append(layout: PagedLayout, k_new, v_new, k, v, cu_new=None, ws=None, stream=None):
    """k_new, v_new [rows, H_kv, d] (heads dense, any row stride) into the pools k, v; cu_new
    [B + 1] int32, or None: one row per sequence.  Sequences that sfi_pages_extend refused on the
    same workspace are left out."""
    L = layout
    _here(L.device, stream)
    new = (k_new.shape[0], L.n_kv_heads, L.head_dim)
    _want("k_new", k_new, new, L.dtype, L.device, True)
    _want("v_new", v_new, new, L.dtype, L.device, True)
    L._pool("k", k)
    L._pool("v", v)
    if cu_new is not None:
        _want("cu_new", cu_new, (L.B + 1,), torch.int32, L.device)
    ks, vs = (t.stride(0) if new[0] > 1 else 0 for t in (k_new, v_new))
    _check("sfi_paged_append", lib.sfi_paged_append(
        ctypes.byref(L.c), new[0], _ptr(k_new), _ptr(v_new), ks, vs, _ptr(cu_new), _ptr(k), _ptr(v),
        *_ws(ws, L.device), _stream(stream)))


def _ids(v):
    """A host list of sequences as C ints: (their array, its address, how many)."""
    ids = array.array("i", v)
    return ids, ids.buffer_info()[0], len(ids)


def sfi_pages_extend(layout: PagedLayout, store: PageStore, n_new=None, ws=None, stream=None):
    """Every sequence grows by n_new[b] positions (int32 [B] on the device; None: by one, if it
    holds any), with new pages where it needs them."""
    _here(layout.device, stream)
    if n_new is not None:
        _want("n_new", n_new, (layout.B,), torch.int32, layout.device)
    _check("sfi_pages_extend", lib.sfi_pages_extend(
        ctypes.byref(layout.c), ctypes.byref(store._check(layout).c), _ptr(n_new),
        *_ws(ws, layout.device), _stream(stream)))


def sfi_pages_fork(layout: PagedLayout, store: PageStore, src, dst, ws=None, stream=None):
    """The empty sequences dst[i] become copies of src[i] (host lists)."""
    _here(layout.device, stream)
    (_s, s, n), (_d, d, m) = _ids(src), _ids(dst)
    if n != m:
        raise ValueError(f"{n} sources, but {m} destinations")
    _check("sfi_pages_fork", lib.sfi_pages_fork(
        ctypes.byref(layout.c), ctypes.byref(store._check(layout).c), s, d, n, *_ws(ws, layout.device),
        _stream(stream)))


def sfi_pages_free(layout: PagedLayout, store: PageStore, seqs, ws=None, stream=None):
    """The listed sequences (host list) give up their pages."""
    _here(layout.device, stream)
    _s, s, n = _ids(seqs)
    _check("sfi_pages_free", lib.sfi_pages_free(
        ctypes.byref(layout.c), ctypes.byref(store._check(layout).c), s, n, *_ws(ws, layout.device),
        _stream(stream)))


def sfi_pages_compact(layout: PagedLayout, store: PageStore, new_id=None, ws=None, stream=None):
    """Used pages move to the lowest places; new_id (int32 [n_pages]) gets where each went."""
    _here(layout.device, stream)
    if new_id is not None:
        _want("new_id", new_id, (layout.n_pages,), torch.int32, layout.device)
    _check("sfi_pages_compact", lib.sfi_pages_compact(
        ctypes.byref(layout.c), ctypes.byref(store._check(layout).c), _ptr(new_id),
        *_ws(ws, layout.device), _stream(stream)))


def sfi_pages_copy(layout: PagedLayout, store: PageStore, src, dst, ws=None, stream=None):
    """Whole pages src[i] -> dst[i] in every layer (int32 device tensors)."""
    _here(layout.device, stream)
    n = src.numel()
    _want("src", src, (n,), torch.int32, layout.device)
    _want("dst", dst, (n,), torch.int32, layout.device)
    _check("sfi_pages_copy", lib.sfi_pages_copy(
        ctypes.byref(layout.c), ctypes.byref(store._check(layout).c), _ptr(src), _ptr(dst), n,
        *_ws(ws, layout.device), _stream(stream)))


def sfi_read_status(ws: torch.Tensor, stream=None) -> int:
    st = c_uint32(0)
    _check("sfi_read_status", lib.sfi_read_status(_ptr(ws), ctypes.byref(st), _stream(stream)))
    return int(st.value)


class DecodeContext:
    """sfi_ctx wrapper: per-layer selections plus the slow/fast schedule.

    ``refine`` (an ``sfi_refine``) applies Soft-NMS / cross-head exclusivity
    at every refresh; None keeps the plain Top-K."""

    def __init__(self, batch: int, n_q_heads: int, n_kv_heads: int, head_dim: int, dtype: torch.dtype,
                 max_len: int, n_layers: int, prm: sfi_params, budget: int,
                 async_select: bool = True, refine: Optional[sfi_refine] = None):
        desc = sfi_ctx_desc(batch, n_q_heads, n_kv_heads, head_dim, dtype_code(dtype), max_len,
                            n_layers, prm, budget, int(bool(async_select)),
                            refine if refine is not None else sfi_refine(0, 0.0, 0.0))
        h = c_void_p()
        _check("sfi_ctx_create", lib.sfi_ctx_create(ctypes.byref(desc), ctypes.byref(h)))
        self.h = h
        self.batch, self.n_kv_heads, self.k = batch, n_kv_heads, prm.k

    def close(self) -> None:
        if self.h:
            lib.sfi_ctx_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def step(self, layer: int, is_boundary, layout: Layout, q, k, v, out, stream=None) -> None:
        """sfi_decode_step; is_boundary is a host uint8 sequence (read at layer 0)."""
        buf = None
        if is_boundary is not None:
            buf = (ctypes.c_uint8 * self.batch)(*[int(x) for x in is_boundary])
        c = layout.c
        _check("sfi_decode_step", lib.sfi_decode_step(
            self.h, int(layer), buf, ctypes.byref(c), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
            _stream(stream)))

    def reset(self) -> None:
        _check("sfi_ctx_reset", lib.sfi_ctx_reset(self.h))

    def profile(self, enable: bool) -> None:
        _check("sfi_ctx_profile", lib.sfi_ctx_profile(self.h, int(bool(enable))))

    def profile_read(self):
        """(attention ms, attention launches, evidence+selector ms, their launches)."""
        am, sm = ctypes.c_double(), ctypes.c_double()
        al, sl = ctypes.c_int64(), ctypes.c_int64()
        _check("sfi_ctx_profile_read", lib.sfi_ctx_profile_read(
            self.h, ctypes.byref(am), ctypes.byref(al), ctypes.byref(sm), ctypes.byref(sl)))
        return am.value, al.value, sm.value, sl.value

    def read_status(self, stream=None) -> int:
        """OR of the context's device status words (cleared); waits for the stream."""
        v = c_uint32(0)
        _check("sfi_ctx_read_status", lib.sfi_ctx_read_status(self.h, ctypes.byref(v),
                                                              _stream(stream)))
        return int(v.value)

    def slow_mask(self):
        buf = (ctypes.c_uint8 * self.batch)()
        _check("sfi_ctx_slow_mask", lib.sfi_ctx_slow_mask(self.h, buf))
        return [int(x) for x in buf]

    def selection(self, layer: int, stream=None):
        """Copies of the layer's selection: (idx [B, H_kv, k], count [B, H_kv]) int32."""
        idx = torch.empty(self.batch, self.n_kv_heads, self.k, dtype=torch.int32, device="cuda")
        cnt = torch.empty(self.batch, self.n_kv_heads, dtype=torch.int32, device="cuda")
        _check("sfi_ctx_selection", lib.sfi_ctx_selection(self.h, int(layer), _ptr(idx), _ptr(cnt),
                                                          _stream(stream)))
        return idx, cnt
