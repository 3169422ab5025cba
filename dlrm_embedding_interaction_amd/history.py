"""Event histories: windowed attention over ragged histories, the 8-bit paged history cache and its continuation
with beams.

Thin marshalling over the ``dlrm_history_*`` calls of ``include/dlrm_mi355x.h``, re-exported by the
package: ``history_attention``, ``history_select`` and ``HistoryCache``.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

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


class _Select(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("beams", ctypes.c_int32), ("keep", ctypes.c_int32),
                ("end_item", ctypes.c_int32), ("n_items", ctypes.c_int64)]


def declare(L: ctypes.CDLL) -> None:
    i32, i64, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    att, cache, select = ctypes.POINTER(_Attention), ctypes.POINTER(_Cache), ctypes.POINTER(_Select)
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
    L.dlrm_history_reorder.argtypes = [cache, i64, i32, _vp, _vp, _vp, size, _vp]
    L.dlrm_history_shared_workspace_bytes.argtypes = [cache, i64, i64, i32, i32]
    L.dlrm_history_shared_workspace_bytes.restype = size
    L.dlrm_history_lookup_shared.argtypes = [cache, att, i64, _vp, i64, _vp, i32, i32, _vp, i64, _vp, i64, _vp, size,
                                             _vp]
    L.dlrm_history_select_workspace_bytes.argtypes = [select, i64]
    L.dlrm_history_select_workspace_bytes.restype = size
    L.dlrm_history_select.argtypes = [select, i64, _vp, i64, _vp, _vp, i64, _vp, _vp, _vp, _vp, _vp, size, _vp]
    for f in ("attention", "init", "append", "lookup", "fork", "truncate", "trim", "compact", "reorder",
              "lookup_shared", "select"):
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


_SELECT = {}        # descriptors and workspace sizes by their values


def _bytes(t: torch.Tensor, name: str, device: torch.device) -> torch.Tensor:
    """A tensor of bytes or truth values as bytes."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor of bool or uint8")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t.view(torch.uint8) if t.dtype is torch.bool else t


def _item_rows(t: torch.Tensor, name: str) -> int:
    """Row stride of (groups, beams, items) rows."""
    groups, beams, items = t.shape
    stride = t.stride()
    if items > 1 and stride[2] != 1:
        raise ValueError(f"the items of one row of {name} must lie side by side")
    if groups > 1 and beams > 1 and stride[0] != beams * stride[1]:
        raise ValueError(f"{name} must have evenly spaced rows")
    return stride[1] if beams > 1 else (stride[0] if groups > 1 else max(items, 1))


def history_select(logits: torch.Tensor, scores: Optional[torch.Tensor] = None, keep: Optional[int] = None,
                   allowed: Optional[torch.Tensor] = None, ended: Optional[torch.Tensor] = None,
                   end_item: int = -1) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The best continuations of groups of beams -> (scores, parents, items), each (groups, keep).

    ``logits`` (groups, beams, items), fp32, bf16 or fp16: of each beam's next item; rows may be columns of a wider
    tensor.  ``scores`` (groups, beams) fp32: the sums of log-probabilities so far (none: 0).  A continuation's score
    is its beam's plus the log-probability of its item; the ``keep`` (none: as many as there are beams) best of each
    group come in descending order, equal ones by beam, then by logit and item; what is missing is -inf, -1 and -1.
    ``allowed`` (items,) or (groups, beams, items), truth values: items that may be taken.  ``ended`` (groups, beams),
    truth values: beams that are carried over as they are, with ``end_item`` as their item.  A beam whose score is not
    finite, or with NaN or +inf among its allowed logits, gives no continuations.  Scores of different beams that lie
    within 4e-9 may come in either order.  Items are masked by -inf or ``allowed``: in a row of nothing but the lowest
    value of fp32 or bf16 every item has the log-probability 0, since the logarithm of its sum is one 64-bit number."""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in DTYPES or not logits.is_cuda:
        raise TypeError("logits must be a CUDA (HIP) tensor of fp32, bf16 or fp16")
    if logits.dim() != 3:
        raise ValueError("logits must be (groups, beams, items)")
    dev = logits.device
    groups, beams, items = logits.shape
    keep, end_item = beams if keep is None else int(keep), int(end_item)
    if not 0 <= keep < 2 ** 31 or not -2 ** 31 <= end_item < 2 ** 31:
        raise ValueError("keep and end_item must fit 32 bits, and keep not be negative")
    ld = _item_rows(logits, "logits")
    if scores is not None:
        _dev(scores, torch.float32, "scores")
        if tuple(scores.shape) != (groups, beams) or scores.device != dev:
            raise ValueError(f"scores must be (groups, beams) on {dev}")
    ld_allowed = 0
    if allowed is not None:
        allowed = _bytes(allowed, "allowed", dev)
        if tuple(allowed.shape) == (items,):
            if items > 1 and allowed.stride(0) != 1:
                raise ValueError("the items of one row of allowed must lie side by side")
        elif tuple(allowed.shape) == (groups, beams, items):
            ld_allowed = _item_rows(allowed, "allowed")
        else:
            raise ValueError("allowed must be (items,) or (groups, beams, items)")
    if ended is not None:
        ended = _bytes(ended, "ended", dev)
        if tuple(ended.shape) != (groups, beams) or not ended.is_contiguous():
            raise ValueError("ended must be contiguous (groups, beams)")
    if dev.index != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return history_select(logits, scores, keep, allowed, ended, end_item)
    key = (logits.dtype, beams, keep, end_item, items, groups)
    entry = _SELECT.get(key)
    if entry is None:
        d = _Select(DTYPES[logits.dtype], beams, keep, end_item, items)
        if len(_SELECT) > 1024:
            _SELECT.clear()
        entry = _SELECT[key] = (ctypes.byref(d), int(load().dlrm_history_select_workspace_bytes(ctypes.byref(d),
                                                                                                groups)))
    if not entry[1]:                    # refused below, and nothing written
        groups_out, keep_out = 1, 1
    else:
        groups_out, keep_out = groups, keep
    ws = torch.empty(max(entry[1], 256), dtype=torch.uint8, device=dev)
    out_scores = torch.empty((groups_out, keep_out), dtype=torch.float32, device=dev)
    out = torch.empty((2, groups_out, keep_out), dtype=torch.int32, device=dev)
    rc = load().dlrm_history_select(entry[0], groups, logits.data_ptr(), ld,
                                    None if scores is None else scores.data_ptr(),
                                    None if allowed is None else allowed.data_ptr(), ld_allowed,
                                    None if ended is None else ended.data_ptr(), out_scores.data_ptr(),
                                    out[0].data_ptr(), out[1].data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev))
    if rc != DLRM_OK:
        _check(rc, "dlrm_history_select")
    return out_scores, out[0], out[1]


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

    def _workspace(self, stream: int, batch: int, queries: int = 0, heads: int = 0, groups: int = 0):
        """(address, bytes, the tensor that holds them) for one call on the stream."""
        key = (batch, queries, heads, groups)
        need = self._need.get(key)
        if need is None:
            L = load()
            need = max(256, int(L.dlrm_history_shared_workspace_bytes(self._ref, batch, groups, queries, heads)
                                if groups else L.dlrm_history_workspace_bytes(self._ref, batch, queries, heads)))
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

    def _queries(self, q, window, sinks, scale, out):
        """The checked arguments of a lookup."""
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
        return a, batch, queries, heads, ld_q, out, ld_out

    def lookup(self, q: torch.Tensor, window: int = ALL_EVENTS, sinks: int = 0, scale: Optional[float] = None,
               slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Queries (batch, n_heads, head_dim) or (batch, queries, n_heads, head_dim) over the histories slots[b]
        (b without slots): the last ``window`` events and the first ``sinks`` of each -> out of q's shape."""
        a, batch, queries, heads, ld_q, out, ld_out = self._queries(q, window, sinks, scale, out)
        s = _stream(self.device)
        ws = self._workspace(s, batch, queries, heads)
        rc = load().dlrm_history_lookup(self._ref, a, batch, self._slots(slots, batch), queries,
                                        q.data_ptr(), ld_q, out.data_ptr(), ld_out, ws[0], ws[1], s)
        if rc != DLRM_OK:
            _check(rc, "dlrm_history_lookup")
        return out

    def lookup_shared(self, q: torch.Tensor, groups: Union[int, torch.Tensor], window: int = ALL_EVENTS, sinks: int = 0,
                      scale: Optional[float] = None, slots: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """``lookup`` of histories in groups that share what came first, as forks of one history do: the events that
        lie on the same pages in all of a group are read once for the group.

        ``groups``: how many histories of the batch, one behind the other, each group has; or ascending offsets
        (n_groups,), group g being the histories [groups[g], groups[g + 1]).  What is shared is found in the page
        lists, so that the result is ``lookup``'s whatever the groups are, up to the order of its sums.  Where little
        can be seen (by the table's width, the window and the batch) histories are looked up one by one."""
        a, batch, queries, heads, ld_q, out, ld_out = self._queries(q, window, sinks, scale, out)
        if isinstance(groups, torch.Tensor):
            ib, n_groups, at = _offsets(groups, self.device), groups.shape[0], groups.data_ptr()
        else:
            groups = int(groups)
            if groups < 1 or batch % groups != 0:
                raise ValueError("the batch must hold whole groups")
            ib, n_groups, at = 8, batch // groups, None
        if self.device.index != torch._C._cuda_getDevice():
            with torch.cuda.device(self.device):
                return self.lookup_shared(q, groups, window, sinks, scale, slots, out)
        s = _stream(self.device)
        ws = self._workspace(s, batch, queries, heads, max(n_groups, 1))
        rc = load().dlrm_history_lookup_shared(self._ref, a, batch, self._slots(slots, batch), n_groups, at, ib, queries,
                                               q.data_ptr(), ld_q, out.data_ptr(), ld_out, ws[0], ws[1], s)
        if rc != DLRM_OK:
            _check(rc, "dlrm_history_lookup_shared")
        return out

    def reorder(self, parents: torch.Tensor, slots: Optional[torch.Tensor] = None) -> None:
        """The histories of groups change places, all at once: in each group g history slots[g, i] becomes what
        slots[g, parents[g, i]] was, on shared pages; a parent of -1 frees it.

        ``parents`` (groups, beams) int32, as ``history_select`` gives them; ``slots`` the same shape (none: 0, 1,
        2 ...).  A parent may come any number of times; slots may come once in the call."""
        _dev(parents, torch.int32, "parents")
        if parents.dim() != 2 or parents.device != self.device:
            raise ValueError(f"parents must be (groups, beams) on {self.device}")
        if slots is not None:
            _dev(slots, torch.int32, "slots")
            if slots.shape != parents.shape or slots.device != self.device:
                raise ValueError("one slot for each parent")
        if self.device.index != torch._C._cuda_getDevice():
            with torch.cuda.device(self.device):
                return self.reorder(parents, slots)
        s = _stream(self.device)
        ws = self._workspace(s, 1)
        _check(load().dlrm_history_reorder(self._ref, parents.shape[0], parents.shape[1],
                                           None if slots is None else slots.data_ptr(), parents.data_ptr(), ws[0],
                                           ws[1], s), "dlrm_history_reorder")

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
