"""PyTorch-side helper around the 4-bit memory cache: device buffers and streams only.

``MemoryCache`` owns (or is given) the page buffer and the page accounts, and calls the
``clef_cache_*`` entry points on torch's current stream.  All arithmetic happens in
libclef_head.so.  A serving step is

    slots, cu = cache.plan(want, n_slots)        # pages and slots of the new tokens
    cache.append(k, v, slots)                    # their keys and values, into 4 bits
    out, lse = cache.attend(q, cu, max_q)        # their attention over the whole memory

and ``plan`` with smaller lengths gives pages back.  Nothing here waits for the GPU;
``device_status`` does, and reports what the kernels met (a bad slot, pages that ran out).
The cache holds numbers, not gradients: tensors that require one are refused while grad
mode is on.
"""
from typing import Optional, Tuple

import torch

from . import binding as B

_DTYPES = {torch.bfloat16: B.BF16, torch.float16: B.FP16, torch.float32: B.FP32}
_ROW_DTYPES = {torch.bfloat16: B.BF16, torch.float16: B.FP16}
_INT32 = torch.int32


def stream_handle(stream: Optional[torch.cuda.Stream] = None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


# A decoding step calls this layer a few times for every layer of a model, so the host's share of
# a call matters: no device guard and no Stream object where the current device is the cache's.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else None
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _refuse(why):
    raise B.ClefError(1, why)


def _overlap(a, b):
    """Whether the memory of two tensors, from the first value to the last, has bytes in common."""
    if not a.numel() or not b.numel():
        return False
    (a0, a1), (b0, b1) = ((t.data_ptr(), t.data_ptr() + t.element_size() *
                           (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))) for t in (a, b))
    return a0 < b1 and b0 < a1


class MemoryCache:
    """Pages of 4-bit keys and values, and who holds them.

    ``n_pages`` pages of ``page`` tokens (16 .. 256, a power of two) of ``heads`` heads of
    ``head_dim`` 64 or 128; page accounts for ``requests`` requests of at most ``max_len``
    tokens.  ``data`` (uint8, of ``size_bytes``) and ``state`` (int32, of ``state_size``: the free
    count, the lengths, the free pages and the block table, one after the other) may be
    buffers of the caller, taken as they are; otherwise they are made here, empty.
    """

    def __init__(self, n_pages: int, page: int = 64, heads: int = 16, head_dim: int = 64, requests: int = 1,
                 max_len: int = 16384, device="cuda", data: Optional[torch.Tensor] = None,
                 state: Optional[torch.Tensor] = None):
        self.n_pages, self.page, self.heads, self.head_dim = int(n_pages), int(page), int(heads), int(head_dim)
        self.requests, self.max_len = int(requests), int(max_len)
        self.struct = B.ClefCache(0, self.n_pages, self.page, self.heads, self.head_dim)
        self.size_bytes = B.clef_cache_size(self.struct)
        if not 1 <= self.requests <= B.CACHE_MAX_REQUESTS or self.max_len < 1:
            _refuse("MemoryCache: requests or max_len out of range")
        self.width = -(-self.max_len // self.page)
        n, p = self.requests, self.n_pages
        self.state_size = 1 + n + p + n * self.width
        # index 0 where no number is given, so that the current device may differ from the cache's
        self.device = torch.empty(0, device=device).device
        if data is None:
            data = torch.zeros(self.size_bytes, dtype=torch.uint8, device=self.device)
        elif data.dtype != torch.uint8 or data.numel() != self.size_bytes or not data.is_contiguous() or \
                data.device != self.device:
            _refuse("MemoryCache: data is not a contiguous uint8 tensor of size_bytes on the device")
        if state is None:
            state = torch.full((self.state_size,), -1, dtype=torch.int32, device=self.device)
            state[0] = p
            state[1:1 + n] = 0
            state[1 + n:1 + n + p] = torch.arange(p - 1, -1, -1, dtype=torch.int32, device=self.device)
        elif state.dtype != torch.int32 or state.numel() != self.state_size or not state.is_contiguous() or \
                state.device != self.device:
            _refuse("MemoryCache: state is not a contiguous int32 tensor of state_size on the device")
        self.data, self.state = data, state
        self.struct.data = data.data_ptr()
        self.free_count, self.lengths = state[:1], state[1:1 + n]
        self.free_pages, self.block_table = state[1 + n:1 + n + p], state[1 + n + p:].view(n, self.width)
        self.flags = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._index = self.device.index if self.device.type == "cuda" else None
        self._flags = self.flags.data_ptr()
        self._accounts = [x.data_ptr() for x in (self.lengths, self.block_table, self.free_pages, self.free_count)]
        self._lib = B.load()
        self._space = {}  # workspace bytes of the sizes that attend has met

    # ------------------------------------------------------------- checks

    def checked_slots(self, slots: torch.Tensor) -> torch.Tensor:
        if slots.dtype is not _INT32 or slots.dim() != 1 or not slots.is_contiguous() or slots.device != self.device:
            _refuse(f"slots and offsets: a contiguous int32 vector on {self.device}")
        return slots

    def checked_table(self, table: Optional[torch.Tensor], n: int) -> torch.Tensor:
        if table is None:
            table = self.block_table
        if table.dtype is not _INT32 or table.dim() != 2 or table.shape[0] < n or not table.is_contiguous() or \
                table.device != self.device:
            _refuse(f"block_table: contiguous int32 [requests, pages] on {self.device}")
        return table

    def _elsewhere(self):
        """Whether another device than the cache's is current (the call is then made inside a guard)."""
        if self._index is None:
            _refuse("the cache is not on a GPU")
        return _current_device() != self._index

    def _rows(self, t, what):
        """The type, shape and strides of rows [tokens, heads, head_dim]."""
        dtype, shape, strides = _ROW_DTYPES.get(t.dtype), t.shape, t.stride()
        if dtype is None or len(shape) != 3 or shape[2] != self.head_dim or strides[2] != 1 or t.device != self.device:
            _refuse(f"{what}: bf16 or fp16 [tokens, heads, {self.head_dim}], values contiguous, on {self.device}")
        if t.requires_grad and torch.is_grad_enabled():
            _refuse(f"{what} requires a gradient, which a 4-bit cache does not pass on")
        return dtype, shape, strides

    # ---------------------------------------------------------- operators

    def plan(self, want: torch.Tensor, n_slots: int, slots: Optional[torch.Tensor] = None,
             cu: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Take the requests' lengths to ``want`` (int32 [requests]): the slots of the tokens
        gained, request by request, -1 behind them (int32 [n_slots]), and their running sum
        (int32 [requests + 1])."""
        if want.dtype is not _INT32 or want.dim() != 1 or want.numel() != self.requests or \
                not want.is_contiguous() or want.device != self.device:
            _refuse(f"want: contiguous int32 [requests] on {self.device}")
        if slots is not None and self.checked_slots(slots).numel() != n_slots:
            _refuse("slots: int32 [n_slots]")
        if cu is not None and self.checked_slots(cu).numel() != self.requests + 1:
            _refuse("cu: int32 [requests + 1]")
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self.plan(want, n_slots, slots, cu)
        if slots is None:
            slots = torch.empty(n_slots, dtype=_INT32, device=self.device)
        if cu is None:
            cu = torch.empty(self.requests + 1, dtype=_INT32, device=self.device)
        lengths, table, free_pages, free_count = self._accounts
        status = self._lib.clef_cache_plan(self.struct, self.requests, lengths, want.data_ptr(), table, self.width,
                                           free_pages, free_count, cu.data_ptr(), slots.data_ptr(), n_slots,
                                           self._flags, _raw_stream(self._index))
        if status:
            raise B.ClefError(status, "clef_cache_plan")
        return slots, cu

    def append(self, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, head0: int = 0):
        """Store key and value rows [tokens, heads, head_dim] (bf16 or fp16, any row and head
        strides) in ``slots``, as cache heads ``head0`` on.  Negative slots skip their row."""
        dtype, (n, heads, _), ks = self._rows(k, "k")
        v_dtype, v_shape, vs = self._rows(v, "v")
        if v_dtype != dtype or v_shape[0] != n or v_shape[1] != heads:
            _refuse("k and v: one shape and type")
        if self.checked_slots(slots).numel() != n:
            _refuse("slots: one a row")
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self.append(k, v, slots, head0)
        status = self._lib.clef_cache_append(self.struct, n, head0, heads, dtype, k.data_ptr(), ks[0], ks[1],
                                             v.data_ptr(), vs[0], vs[1], slots.data_ptr(), self._flags,
                                             _raw_stream(self._index))
        if status:
            raise B.ClefError(status, "clef_cache_append")

    def read(self, slots: torch.Tensor, dtype=torch.bfloat16, head0: int = 0,
             heads: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """What the rows of ``slots`` stand for: k, v [tokens, heads, head_dim] in ``dtype``
        (bf16, fp16 or fp32); zeros for negative slots."""
        if dtype not in _DTYPES:
            _refuse("read: bf16, fp16 or fp32")
        heads = self.heads - head0 if heads is None else heads
        n = self.checked_slots(slots).numel()
        if heads < 1:
            _refuse("read: no heads")
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self.read(slots, dtype, head0, heads)
        k = torch.empty((n, heads, self.head_dim), dtype=dtype, device=self.device)
        v = torch.empty_like(k)
        status = self._lib.clef_cache_read(self.struct, n, head0, heads, _DTYPES[dtype], slots.data_ptr(),
                                           k.data_ptr(), v.data_ptr(), self._flags, _raw_stream(self._index))
        if status:
            raise B.ClefError(status, "clef_cache_read")
        return k, v

    def attend(self, q: torch.Tensor, cu_q: torch.Tensor, max_q: int, scale: Optional[float] = None,
               causal: bool = True, head0: int = 0, kv_heads: Optional[int] = None,
               block_table: Optional[torch.Tensor] = None, lengths: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Attention of query rows [total, q_heads, head_dim] over their requests' memory: the
        output in q's type and the scores' log-sum (fp32 [total, q_heads]).

        ``cu_q`` (int32 [B + 1]) holds each request's first row, ``max_q`` bounds the rows of
        one request.  With ``causal`` the queries are the request's last tokens, otherwise
        each sees the whole memory.  Query heads share the ``kv_heads`` cache heads from
        ``head0`` on evenly (all of the cache's by default).  ``block_table`` and ``lengths``
        default to the cache's own.  A row that sees nothing gives 0 and -inf; rows behind
        the last request are not written (not set at all without ``out``, which must lie apart
        from ``q``)."""
        dtype, (total, q_heads, _), strides = self._rows(q, "q")
        n = self.checked_slots(cu_q).numel() - 1
        lengths = self.lengths if lengths is None else self.checked_slots(lengths)
        table = self.checked_table(block_table, n)
        pages = table.shape[1]
        if n < 1 or lengths.numel() < n:
            _refuse("cu_q, lengths: one entry a request")
        if kv_heads is None:
            kv_heads = self.heads - head0
        if scale is None:
            scale = self.head_dim ** -0.5
        if out is not None and (out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or
                                out.device != self.device or _overlap(out, q)):
            _refuse("out: contiguous, of q's shape and type, apart from q")
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self.attend(q, cu_q, max_q, scale, causal, head0, kv_heads, table, lengths, out)
        if out is None:
            out = torch.empty((total, q_heads, self.head_dim), dtype=q.dtype, device=self.device)
        lse = torch.empty((total, q_heads), dtype=torch.float32, device=self.device)
        # a buffer of the call's own: overlapping calls and captured graphs never share one
        n_bytes = self._space.get((n, total, q_heads, pages))
        if n_bytes is None:
            if len(self._space) >= 4096:
                self._space.clear()
            n_bytes = B.clef_cache_attend_workspace(self.struct, n, total, max(q_heads, 1), pages * self.page)
            self._space[n, total, q_heads, pages] = n_bytes
        space = torch.empty(n_bytes, dtype=torch.uint8, device=self.device) if n_bytes else None
        status = self._lib.clef_cache_attend(self.struct, n, total, max_q, q_heads, head0, kv_heads, dtype, q.data_ptr(),
                                             strides[0], strides[1], cu_q.data_ptr(), table.data_ptr(), pages,
                                             lengths.data_ptr(), scale, 1 if causal else 0, out.data_ptr(),
                                             lse.data_ptr(), self._flags, space.data_ptr() if n_bytes else None, n_bytes,
                                             _raw_stream(self._index))
        if status:
            raise B.ClefError(status, "clef_cache_attend")
        return out, lse

    def device_status(self) -> int:
        """Waits for the current stream, reads and clears what the kernels reported."""
        if self._elsewhere():
            with torch.cuda.device(self._index):
                return self.device_status()
        return B.clef_cache_status(self._flags, _raw_stream(self._index))
