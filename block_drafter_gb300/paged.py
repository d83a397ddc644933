"""Paged K/V cache of the target model: append, attention, accumulated weights, eviction.

``PagedCache`` wraps one layer's pools and calls the library's ``bd_paged_*`` entry points
(``include/blockdrafter.h`` states their semantics); all computation happens in its kernels.

    cache = PagedCache(k_pool, v_pool, n_q_heads=32)         # [pages, KV heads, page size, D]
    batch = cache.batch(page_table, seq_len, row_start, n_rows=rows, max_rows=16, max_len=32768)
    cache.append(batch, k, v)                                # the rows' keys and values
    cache.attention(batch, q, out, lse=lse, window=4096, n_sink=4)
    cache.weights(batch, q, lse, score, score_in=score, rows_used=accepted)
    cache.evict(batch, score, 8192, kept, new_len, n_sink=4, n_recent=512, score_out=score)

A batch holds the addresses of its device arrays: a program that updates lengths, row starts
and page tables in place keeps one batch (and its captured graphs) for many steps.  Calls run
on the given stream, or on the current stream of the pools' device.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import binding as B


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle without building a torch.cuda.Stream (2.8 us a call), where torch has it.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)

_TYPES = {torch.bfloat16: B.BF16, torch.float16: B.F16, torch.float32: B.F32}


def _stream_of(handle: int, device: torch.device) -> torch.cuda.Stream:
    # 0 and 1 are the default stream's handles; an ExternalStream of 0 would be a new stream
    return torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device=device)


def _capturing(stream: torch.cuda.Stream) -> bool:
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _need(ok: bool, msg: str):
    if not ok:
        raise ValueError(msg)


class PagedBatch:
    """One batch of requests; made by ``PagedCache.batch``."""

    def __init__(self, cache: "PagedCache", page_table: torch.Tensor, seq_len: torch.Tensor,
                 row_start: Optional[torch.Tensor], n_rows: int, max_rows: int, max_len: int,
                 workspace: Optional[torch.Tensor]):
        n = page_table.shape[0] if page_table.dim() == 2 else -1
        for name, t, shape in (("page_table", page_table, page_table.shape if n >= 0 else None),
                               ("seq_len", seq_len, (n,)), ("row_start", row_start, (n + 1,))):
            if t is None and name == "row_start" and n_rows == 0:
                continue
            _need(t is not None and t.dtype == torch.int32 and shape is not None
                  and tuple(t.shape) == tuple(shape) and t.is_contiguous(),
                  f"{name}: a contiguous int32 tensor is wanted (page_table [requests, pages], "
                  "seq_len [requests], row_start [requests + 1])")
            cache._on_device(name, t)
        self.n_requests, self.n_rows, self.max_len = n, int(n_rows), int(max_len)
        self.q_shape = (self.n_rows, cache.n_q_heads, cache.head_dim)
        self.kv_shape = (self.n_rows, cache.n_kv_heads, cache.head_dim)
        self.lse_shape = (self.n_rows, cache.n_q_heads)
        self.tensors = (page_table, seq_len, row_start)
        self.struct = B.PagedBatch(n, page_table.shape[1], int(n_rows), int(max_rows), int(max_len),
                                   page_table.data_ptr(), seq_len.data_ptr(),
                                   None if row_start is None else row_start.data_ptr())
        nbytes = B.paged_workspace_bytes(cache.struct, n, int(max_rows))
        # Streams that the batch's own workspace is known to; None: the caller's workspace.
        self.streams = None
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=cache.device)
            self.home = _current_stream(cache.index)
            self.streams = {self.home}
        cache._on_device("workspace", workspace)
        _need(workspace.is_contiguous(), "workspace: a contiguous tensor is wanted")
        self.workspace = workspace
        self.ws_ptr = workspace.data_ptr()
        self.ws_bytes = workspace.numel() * workspace.element_size()

    def _use_on(self, handle: int):
        """First use of the batch's own workspace on a stream other than the one it was allocated on: what that one
        has queued comes first (its memory may have been something else's), and the memory goes to no other use
        before the stream's calls are done.  In a capture there is nothing to wait for that it could hold."""
        device = self.workspace.device
        home, other = (_stream_of(h, device) for h in (self.home, handle))
        if not (_capturing(other) or _capturing(home)):
            other.wait_stream(home)
        self.workspace.record_stream(other)
        self.streams.add(handle)


class PagedCache:
    """k, v: pools [pages, KV heads, page size, D] of bf16 or fp16 (any strides that are equal
    for both, with D contiguous -- a [pages, page size, KV heads, D] pool is passed permuted)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, n_q_heads: int):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.stride() == v.stride(),
              "k and v: two pools [pages, KV heads, page size, D] of one shape, type and layout are wanted")
        _need(k.dtype in _TYPES, f"pools of {k.dtype} are not supported")
        _need(k.stride(3) == 1, "the D values of a slot must be contiguous")
        self.k, self.v, self.dtype, self.device, self.index = k, v, k.dtype, k.device, k.get_device()
        self.n_q_heads, self.n_kv_heads, self.head_dim = int(n_q_heads), k.shape[1], k.shape[3]
        self.scale = 1.0 / math.sqrt(self.head_dim)
        self.struct = B.PagedKv(self.n_q_heads, self.n_kv_heads, self.head_dim, _TYPES[k.dtype],
                                k.shape[2], k.shape[0], k.stride(0), k.stride(1), k.stride(2),
                                k.data_ptr(), v.data_ptr())
        B.paged_workspace_bytes(self.struct, 1, 1)  # the library's checks of the pools
        self._on_device("v", v)

    # The checks of a call are written for their cost: a decoding step makes one call per layer.
    def _on_device(self, name: str, t: torch.Tensor):
        if t.get_device() != self.index or self.index < 0:
            raise ValueError(f"{name} is on {t.device}, the pools on {self.device} (a CUDA device is wanted)")

    def _rows(self, name: str, t: torch.Tensor, shape: tuple) -> int:
        """Row stride of a row tensor [n_rows, heads, D]."""
        if t.shape != shape or t.dtype is not self.dtype:
            raise ValueError(f"{name}: {list(shape)} of {self.dtype} is wanted, got {list(t.shape)} of {t.dtype}")
        row, head, one = t.stride()
        if one != 1 or (head != shape[2] and shape[1] != 1):
            raise ValueError(f"{name}: a row's heads must be contiguous")
        if t.get_device() != self.index:
            self._on_device(name, t)
        return row

    def _floats(self, name: str, t: torch.Tensor, rows: int, width: int) -> int:
        """Row stride of an fp32 matrix with at least ``width`` columns."""
        s, n = t.stride(), t.shape
        if len(n) != 2 or t.dtype is not torch.float32 or n[0] != rows or n[1] < width or (s[1] != 1 and n[1] > 1) or s[0] < n[1]:
            raise ValueError(f"{name}: float32 [{rows}, >= {width}] with contiguous rows is wanted, got {list(n)} of {t.dtype}")
        if t.get_device() != self.index:
            self._on_device(name, t)
        return s[0]

    def _ints(self, name: str, t: torch.Tensor, shape):
        if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous int32 {list(shape)} is wanted, got {list(t.shape)} of {t.dtype}")
        if t.get_device() != self.index:
            self._on_device(name, t)

    def _lse(self, lse: torch.Tensor, batch: PagedBatch):
        if lse.dtype is not torch.float32 or lse.shape != batch.lse_shape or not lse.is_contiguous():
            raise ValueError(f"lse: contiguous float32 {list(batch.lse_shape)} is wanted")
        if lse.get_device() != self.index:
            self._on_device("lse", lse)

    def _handle(self, stream) -> int:
        """The given stream's handle, or that of the pools' device's current one."""
        return _current_stream(self.index) if stream is None else getattr(stream, "cuda_stream", stream)

    def _call(self, fn, *args, stream: int):
        """The library's call on the pools' device."""
        if torch.cuda.current_device() == self.index:
            fn(self.struct, *args, stream)
        else:
            with torch.cuda.device(self.index):
                fn(self.struct, *args, stream)

    def batch(self, page_table: torch.Tensor, seq_len: torch.Tensor, row_start: Optional[torch.Tensor],
              n_rows: int, max_rows: int, max_len: int, workspace: Optional[torch.Tensor] = None) -> PagedBatch:
        """page_table int32 [requests, pages], seq_len int32 [requests] (this step's rows counted),
        row_start int32 [requests + 1]; max_rows (at most n_rows) and max_len bound every request's rows and
        length.  The schedules go by these bounds: close ones are faster than loose ones.
        workspace: a uint8 tensor to share between batches used in order on one stream.  Without one the batch
        allocates its own, which it keeps from other uses until its calls are done, on whatever streams they ran;
        a stream given by its handle must outlive the batch.  Captured calls hold the addresses of the batch's
        arrays and of its workspace: keep the batch as long as their graphs are replayed."""
        return PagedBatch(self, page_table, seq_len, row_start, n_rows, max_rows, max_len, workspace)

    def append(self, batch: PagedBatch, k_new: torch.Tensor, v_new: torch.Tensor, stream=None):
        """Stores the rows' keys and values ([n_rows, KV heads, D]) in their slots."""
        ks = self._rows("k_new", k_new, batch.kv_shape)
        vs = self._rows("v_new", v_new, batch.kv_shape)
        self._call(B.paged_append, batch.struct, k_new.data_ptr(), ks, v_new.data_ptr(), vs, stream=self._handle(stream))

    def attention(self, batch: PagedBatch, q: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                  window: int = 0, n_sink: int = 0, scale: Optional[float] = None, stream=None):
        """Attention of the rows q [n_rows, query heads, D] into out, causal, optionally through a
        sliding window beside n_sink first slots; lse float32 [n_rows, query heads] or None.
        scale: 1/sqrt(D) if None."""
        qs = self._rows("q", q, batch.q_shape)
        os = self._rows("out", out, batch.q_shape)
        if lse is not None:
            self._lse(lse, batch)
        stream = self._handle(stream)
        if batch.streams is not None and stream not in batch.streams:
            batch._use_on(stream)
        self._call(B.paged_attention, batch.struct, q.data_ptr(), qs, out.data_ptr(), os,
                   None if lse is None else lse.data_ptr(), window, n_sink,
                   self.scale if scale is None else scale, batch.ws_ptr, batch.ws_bytes, stream=stream)

    def weights(self, batch: PagedBatch, q: torch.Tensor, lse: torch.Tensor, score_out: torch.Tensor,
                score_in: Optional[torch.Tensor] = None, decay: float = 1.0,
                rows_used: Optional[torch.Tensor] = None, window: int = 0, n_sink: int = 0,
                scale: Optional[float] = None, stream=None):
        """score_out[b, j] = decay * score_in[b, j] + the attention weight slot j got from the first
        rows_used[b] rows (all if None), over all heads; score_in may be score_out, or None for zero."""
        qs = self._rows("q", q, batch.q_shape)
        self._lse(lse, batch)
        stride = self._floats("score_out", score_out, batch.n_requests, batch.max_len)
        if score_in is not None:
            _need(self._floats("score_in", score_in, batch.n_requests, batch.max_len) == stride,
                  "score_in and score_out: the same row stride is wanted")
        if rows_used is not None:
            self._ints("rows_used", rows_used, (batch.n_requests,))
        self._call(B.paged_weights, batch.struct, q.data_ptr(), qs, lse.data_ptr(),
                   None if rows_used is None else rows_used.data_ptr(), window, n_sink,
                   self.scale if scale is None else scale, decay,
                   None if score_in is None else score_in.data_ptr(), score_out.data_ptr(), stride, stream=self._handle(stream))

    def evict(self, batch: PagedBatch, score: torch.Tensor, budget: int, kept: torch.Tensor, len_out: torch.Tensor,
              n_sink: int = 0, n_recent: int = 0, dst_table: Optional[torch.Tensor] = None,
              score_out: Optional[torch.Tensor] = None, stream=None):
        """Requests longer than budget keep their first n_sink, last n_recent and best-scored slots;
        kept int32 [requests, budget] and len_out int32 [requests] say which and how many.  The kept
        slots move, in order, to the pages of dst_table (int32 [requests, pages]) or, if None, up in
        their own.  score_out (may be score) takes the kept slots' scores; len_out may be the
        batch's seq_len."""
        stride = self._floats("score", score, batch.n_requests, batch.max_len)
        _need(isinstance(budget, int) and budget >= 1, "budget must be >= 1")
        self._ints("kept", kept, (batch.n_requests, budget))
        self._ints("len_out", len_out, (batch.n_requests,))
        width = 0
        if dst_table is not None:
            width = dst_table.shape[-1] if dst_table.dim() else 0
            self._ints("dst_table", dst_table, (batch.n_requests, width))
        ostride = 0
        if score_out is not None:
            ostride = self._floats("score_out", score_out, batch.n_requests, min(budget, batch.max_len))
        self._call(B.paged_evict, batch.struct, score.data_ptr(), stride, budget, n_sink, n_recent,
                   None if dst_table is None else dst_table.data_ptr(), width, kept.data_ptr(),
                   len_out.data_ptr(), None if score_out is None else score_out.data_ptr(), ostride, stream=self._handle(stream))
