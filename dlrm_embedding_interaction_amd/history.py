"""Event histories: windowed attention over ragged histories and the 8-bit paged history cache.

Thin marshalling over the ``dlrm_history_*`` calls of ``include/dlrm_mi355x.h``, re-exported by the
package: ``history_attention`` and ``HistoryCache``.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import DLRM_OK, _check, _dev, _vp, load

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ALL_EVENTS = 1 << 30    # a window that no history reaches


class _Attention(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("window", ctypes.c_int64), ("sinks", ctypes.c_int64),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class _Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_pages", "page_events", "n_kv_heads", "head_dim", "n_slots",
                                              "max_pages")] + \
               [(n, _vp) for n in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs", "free_pages", "counters")]


def declare(L: ctypes.CDLL) -> None:
    i32, i64, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    att, cache = ctypes.POINTER(_Attention), ctypes.POINTER(_Cache)
    L.dlrm_history_attention.argtypes = [att, i64, i64, _vp, i32, _vp, i64, _vp, i64, _vp, i64, _vp, _vp, i64, _vp]
    L.dlrm_history_workspace_bytes.argtypes = [cache, i64, i32, i32]
    L.dlrm_history_workspace_bytes.restype = size
    L.dlrm_history_init.argtypes = [cache, _vp]
    L.dlrm_history_append.argtypes = [cache, i64, _vp, i32, i64, _vp, i32, _vp, i64, _vp, i64, _vp, size, _vp]
    L.dlrm_history_lookup.argtypes = [cache, att, i64, _vp, i32, _vp, i64, _vp, i64, _vp, size, _vp]
    L.dlrm_history_fork.argtypes = [cache, i64, _vp, _vp, _vp, size, _vp]
    L.dlrm_history_truncate.argtypes = [cache, i64, _vp, _vp, _vp, size, _vp]
    L.dlrm_history_trim.argtypes = [cache, i64, _vp, i64, i64, _vp, size, _vp]
    L.dlrm_history_compact.argtypes = [cache, _vp, size, _vp]
    for f in ("attention", "init", "append", "lookup", "fork", "truncate", "trim", "compact"):
        getattr(L, f"dlrm_history_{f}").restype = ctypes.c_int


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, dims: int, device: torch.device) -> int:
    """Row stride of (..., heads, head_dim) rows whose heads lie side by side."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    shape = t.shape
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    heads, dim = shape[-2], shape[-1]
    if t.is_contiguous():
        return max(heads * dim, 1)
    stride = t.stride()
    if (dim > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != dim):
        raise ValueError(f"the heads of one row of {name} must lie side by side")
    if dims == 4 and shape[0] > 1 and shape[1] > 1 and stride[0] != shape[1] * stride[1]:
        raise ValueError(f"{name} must have evenly spaced rows")
    n = t.numel() // max(1, heads * dim)
    return (stride[0] if dims == 3 or shape[1] == 1 else stride[1]) if n > 1 else max(heads * dim, 1)


def _offsets(t: torch.Tensor, device: torch.device) -> int:
    """Width of the offsets in bytes."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("offsets must be a CUDA (HIP) tensor")
    if t.dtype is not torch.int64 and t.dtype is not torch.int32:
        raise TypeError("offsets must be int32 or int64")
    if t.dim() != 1 or t.device != device or not t.is_contiguous():
        raise ValueError(f"offsets must be 1-D and contiguous on {device}")
    return 8 if t.dtype is torch.int64 else 4


_ATTENTION = {}     # descriptors by their values


def _attention(dtype, heads, kv, dim, window, sinks, scale):
    key = (dtype, heads, kv, dim, window, sinks, scale)
    ref = _ATTENTION.get(key)
    if ref is None:
        if len(_ATTENTION) > 1024:
            _ATTENTION.clear()
        a = _Attention(DTYPES[dtype], heads, kv, dim, int(window), int(sinks),
                       dim ** -0.5 if scale is None else float(scale), 0)
        ref = _ATTENTION[key] = ctypes.byref(a)
    return ref


def _i32(t: torch.Tensor, name: str, device: torch.device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_cuda or not t.is_contiguous():
        _dev(t, torch.int32, name)
    if t.dim() != 1 or t.device != device:
        raise ValueError(f"{name} must be 1-D on {device}")
    return t


def _stream(device: torch.device) -> int:
    """The current stream's handle, without the stream object that a call this short would notice."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def history_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor,
                      window: int = ALL_EVENTS, sinks: int = 0, scale: Optional[float] = None,
                      padding: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Every event of ragged histories attends to its own history -> (N, n_heads, head_dim).

    ``q`` (N, n_heads, head_dim), ``k`` and ``v`` (N, n_kv_heads, head_dim), all fp32, bf16 or fp16; rows may be
    columns of a wider tensor.  History b is rows [offsets[b], offsets[b + 1]); rows before offsets[0], usually 0, are
    no one's and are not written.  An event sees the last ``window`` events of its history, itself included, and the
    first ``sinks``, but none whose ``padding`` byte is set."""
    if not isinstance(q, torch.Tensor) or q.dtype not in DTYPES:
        raise TypeError("q must be an fp32, bf16 or fp16 tensor")
    dev, dtype = q.device, q.dtype
    ld_q, ld_k, ld_v = _rows(q, "q", dtype, 3, dev), _rows(k, "k", dtype, 3, dev), _rows(v, "v", dtype, 3, dev)
    n, heads, dim = q.shape
    kshape = k.shape
    if kshape != v.shape or kshape[0] != n or kshape[2] != dim:
        raise ValueError("k and v must be (N, n_kv_heads, head_dim) beside q's (N, n_heads, head_dim)")
    ib = _offsets(offsets, dev)
    if padding is not None:
        if padding.dtype == torch.bool:
            padding = padding.view(torch.uint8)
        _dev(padding, torch.uint8, "padding")
        if tuple(padding.shape) != (n,) or padding.device != dev:
            raise ValueError("padding must hold one byte for each event")
    if out is None:
        out = torch.empty((n, heads, dim), dtype=dtype, device=dev)
        ld_out = max(heads * dim, 1)
    else:
        ld_out = _rows(out, "out", dtype, 3, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    rc = load().dlrm_history_attention(_attention(dtype, heads, kshape[1], dim, window, sinks, scale),
                                       offsets.shape[0], n, offsets.data_ptr(), ib, q.data_ptr(), ld_q, k.data_ptr(),
                                       ld_k, v.data_ptr(), ld_v, None if padding is None else padding.data_ptr(),
                                       out.data_ptr(), ld_out, _stream(dev))
    if rc != DLRM_OK:
        _check(rc, "dlrm_history_attention")
    return out


class HistoryCache:
    """Keys and values of many histories in 8 bits, on pages of a common pool.

    ``n_slots`` histories of up to ``max_pages`` pages of ``page_events`` events.  Slots are int32 CUDA tensors.
    Calls run on the current stream and never wait for the GPU; ``n_free`` and ``n_refused`` read it back.  Lookups
    change nothing but the count of refused slots and may run on several streams, and in several graphs, at once."""

    def __init__(self, n_pages: int, n_slots: int, max_pages: int, n_kv_heads: int, head_dim: int,
                 page_events: int = 64, device="cuda"):
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        codes = dict(dtype=torch.uint8, device=dev)
        scales = dict(dtype=torch.float32, device=dev)
        self._bind(torch.empty((n_pages, n_kv_heads, page_events, head_dim), **codes),
                   torch.empty((n_pages, n_kv_heads, head_dim, page_events), **codes),
                   torch.empty((n_pages, n_kv_heads), **scales), torch.empty((n_pages, n_kv_heads), **scales),
                   torch.empty((n_slots, max_pages), **i32), torch.empty(n_slots, **i32), torch.empty(n_pages, **i32),
                   torch.empty(n_pages, **i32), torch.empty(4, **i32))
        _check(load().dlrm_history_init(self._ref, _stream(self.device)), "dlrm_history_init")

    @classmethod
    def wrap(cls, k, v, k_scale, v_scale, table, lens, refs, free_pages, counters) -> "HistoryCache":
        """A cache over buffers that are filled already."""
        self = cls.__new__(cls)
        self._bind(k, v, k_scale, v_scale, table, lens, refs, free_pages, counters)
        return self

    def _bind(self, k, v, k_scale, v_scale, table, lens, refs, free_pages, counters):
        load()
        for t, d, n in ((k, torch.uint8, "k"), (v, torch.uint8, "v"), (k_scale, torch.float32, "k_scale"),
                        (v_scale, torch.float32, "v_scale"), (table, torch.int32, "table"),
                        (lens, torch.int32, "lens"), (refs, torch.int32, "refs"),
                        (free_pages, torch.int32, "free_pages"), (counters, torch.int32, "counters")):
            _dev(t, d, n)
            if t.device != k.device:
                raise ValueError(f"{n} must be on {k.device}")
        if k.dim() != 4 or table.dim() != 2:
            raise ValueError("k must be (n_pages, n_kv_heads, page_events, head_dim), table (n_slots, max_pages)")
        pages, kv, pe, dim = k.shape
        if (tuple(v.shape) != (pages, kv, dim, pe) or tuple(k_scale.shape) != (pages, kv) or
                tuple(v_scale.shape) != (pages, kv) or tuple(lens.shape) != (table.shape[0],) or
                tuple(refs.shape) != (pages,) or tuple(free_pages.shape) != (pages,) or tuple(counters.shape) != (4,)):
            raise ValueError("shape mismatch")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.table, self.lens, self.refs, self.free_pages, self.counters = table, lens, refs, free_pages, counters
        self.device = k.device
        self.n_kv_heads, self.head_dim, self.page_events = kv, dim, pe
        self.n_slots = table.shape[0]
        self._desc = _Cache(pages, pe, kv, dim, table.shape[0], table.shape[1], k.data_ptr(), v.data_ptr(),
                            k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(), lens.data_ptr(),
                            refs.data_ptr(), free_pages.data_ptr(), counters.data_ptr())
        self._ref = ctypes.byref(self._desc)
        self._ws = {}           # stream -> workspace: calls on two streams may overlap
        self._need = {}

    def _workspace(self, stream: int, batch: int, queries: int = 0, heads: int = 0):
        """(address, bytes, the tensor that holds them) for one call on the stream."""
        key = (batch, queries, heads)
        need = self._need.get(key)
        if need is None:
            need = max(256, int(load().dlrm_history_workspace_bytes(self._ref, batch, queries, heads)))
            if len(self._need) > 256:
                self._need.clear()
            self._need[key] = need
        if torch.cuda.is_current_stream_capturing():
            # The graph's own, from its pool: replays may run on any stream, beside calls and other graphs.  The pool
            # keeps the memory for the graph once the tensor is gone.
            return self._new_workspace(need)
        ws = self._ws.get(stream)
        if ws is None or ws[1] < need:
            ws = self._ws[stream] = self._new_workspace(need)
        return ws

    def _new_workspace(self, size: int):
        t = torch.empty(size, dtype=torch.uint8, device=self.device)
        return t.data_ptr(), size, t

    def _slots(self, slots: Optional[torch.Tensor], batch: int):
        if slots is None:
            if batch > self.n_slots:
                raise ValueError("more histories than slots")
            return None
        _i32(slots, "slots", self.device)
        if slots.shape[0] != batch:
            raise ValueError("one slot for each history")
        return slots.data_ptr()

    def append(self, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor,
               slots: Optional[torch.Tensor] = None) -> None:
        """Events behind histories: rows [offsets[b], offsets[b + 1]) of ``k`` and ``v`` (N, n_kv_heads, head_dim)
        go behind history slots[b] (b without slots).  Histories without room are refused whole (``n_refused``); pages
        are promised in batch order, so that one refused for want of them leaves none for those behind it."""
        if not isinstance(k, torch.Tensor) or k.dtype not in DTYPES:
            raise TypeError("k must be an fp32, bf16 or fp16 tensor")
        ld_k, ld_v = (_rows(t, n, k.dtype, 3, self.device) for t, n in ((k, "k"), (v, "v")))
        if k.shape != v.shape or tuple(k.shape[1:]) != (self.n_kv_heads, self.head_dim):
            raise ValueError("k and v must be (N, n_kv_heads, head_dim)")
        ib = _offsets(offsets, self.device)
        batch = offsets.shape[0]
        s = _stream(self.device)
        ws = self._workspace(s, batch)
        rc = load().dlrm_history_append(self._ref, batch, self._slots(slots, batch), DTYPES[k.dtype], k.shape[0],
                                        offsets.data_ptr(), ib, k.data_ptr(), ld_k, v.data_ptr(), ld_v,
                                        ws[0], ws[1], s)
        _check(rc, "dlrm_history_append")

    def lookup(self, q: torch.Tensor, window: int = ALL_EVENTS, sinks: int = 0, scale: Optional[float] = None,
               slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Queries (batch, n_heads, head_dim) or (batch, queries, n_heads, head_dim) over the histories slots[b]
        (b without slots): the last ``window`` events and the first ``sinks`` of each -> out of q's shape."""
        if not isinstance(q, torch.Tensor) or q.dtype not in DTYPES:
            raise TypeError("q must be an fp32, bf16 or fp16 tensor")
        if q.dim() not in (3, 4):
            raise ValueError("q must be (batch, n_heads, head_dim) or (batch, queries, n_heads, head_dim)")
        ld_q = _rows(q, "q", q.dtype, q.dim(), self.device)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
            ld_out = max(q.shape[-2] * q.shape[-1], 1)
        else:
            ld_out = _rows(out, "out", q.dtype, q.dim(), self.device)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        batch, heads, dim = q.shape[0], q.shape[-2], q.shape[-1]
        queries = q.shape[1] if q.dim() == 4 else 1
        a = _attention(q.dtype, heads, self.n_kv_heads, dim, window, sinks, scale)
        s = _stream(self.device)
        ws = self._workspace(s, batch, queries, heads)
        rc = load().dlrm_history_lookup(self._ref, a, batch, self._slots(slots, batch), queries,
                                        q.data_ptr(), ld_q, out.data_ptr(), ld_out, ws[0], ws[1], s)
        _check(rc, "dlrm_history_lookup")
        return out

    def fork(self, src: torch.Tensor, dst: torch.Tensor) -> None:
        """History dst[i] becomes a copy of src[i] on shared pages; an append copies what it has to."""
        _i32(src, "src", self.device)
        _i32(dst, "dst", self.device)
        if src.shape != dst.shape:
            raise ValueError("one destination for each source")
        s = _stream(self.device)
        ws = self._workspace(s, 1)
        _check(load().dlrm_history_fork(self._ref, src.shape[0], src.data_ptr(), dst.data_ptr(), ws[0], ws[1],
                                        s), "dlrm_history_fork")

    def truncate(self, slots: torch.Tensor, new_lens: Optional[torch.Tensor] = None) -> None:
        """Cut histories to their first new_lens[i] events (none: free them)."""
        _i32(slots, "slots", self.device)
        if new_lens is not None:
            _i32(new_lens, "new_lens", self.device)
            if new_lens.shape != slots.shape:
                raise ValueError("one length for each slot")
        s = _stream(self.device)
        ws = self._workspace(s, 1)
        _check(load().dlrm_history_truncate(self._ref, slots.shape[0], slots.data_ptr(),
                                            new_lens.data_ptr() if new_lens is not None else None, ws[0],
                                            ws[1], s), "dlrm_history_truncate")

    def free(self, slots: torch.Tensor) -> None:
        """Empty histories; their pages go back to the pool."""
        self.truncate(slots)

    def trim(self, slots: torch.Tensor, window: int, sinks: int = 0) -> None:
        """Give back the pages that no later lookup with this window and these sinks reads."""
        _i32(slots, "slots", self.device)
        s = _stream(self.device)
        ws = self._workspace(s, 1)
        _check(load().dlrm_history_trim(self._ref, slots.shape[0], slots.data_ptr(), int(window), int(sinks),
                                        ws[0], ws[1], s), "dlrm_history_trim")

    def compact(self) -> None:
        """Move the used pages to the front of the pool."""
        s = _stream(self.device)
        ws = self._workspace(s, 1)
        _check(load().dlrm_history_compact(self._ref, ws[0], ws[1], s), "dlrm_history_compact")

    @property
    def n_free(self) -> int:
        """Pages that appends can take (waits for the GPU)."""
        return int(self.counters[0].item())

    @property
    def n_refused(self) -> int:
        """Histories refused so far, for want of pages or for a bad slot or length (waits for the GPU)."""
        return int(self.counters[1].item())
