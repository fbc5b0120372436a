"""Paged key/value cache for streams of frames, through the C ABI (bsa_kv_* in include/bsa.h).

KVCache keeps the keys and values of the tokens seen so far; each new chunk of tokens (a frame,
its camera and register tokens, one token) is appended and attends over the cache:

    cache = KVCache(seqs=1, heads=16, kv_heads=16, pages=2048, page_tokens=64, max_pages=2048, fmt="e4m3")
    chunk = cache.extend([782])                        # 782 new tokens of sequence 0: pages and lengths
    cache.append(k, v, chunk.cu_new)                   # k, v: [782, 16, 64] bf16
    o = cache.attend(q, chunk.cu_new, chunk.max_new, unit=782)     # frame-wise causal
    K, V = cache.read_all(0)                           # [tokens, 16, 64] bf16, e.g. for a global layer

A program that keeps its own pools and page tables wraps them with KVCache.over(...) and calls
append / attend / read with its own offsets. Device tables are read when the kernels run, so
captured calls replay with what the tables then hold.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import _lib

_POOL_DTYPE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@dataclass
class Chunk:
    """New tokens of every sequence: packed rows cu_new[s] .. cu_new[s + 1] - 1."""
    cu_new: torch.Tensor
    max_new: int
    rows: int


class KVCache:
    """One layer's cache. Calls on one KVCache share its workspace and status word: calls that may
    overlap on the GPU (other streams) need a KVCache each, over the same pools if need be.

    A call runs on the current stream or on the one whose handle it is given. The cache's own tensors are
    kept until such work is done; the tensors passed to a call are the caller's to keep, and a stream that
    was given must live as long as the cache."""

    def __init__(self, seqs: int, heads: int, kv_heads: int, pages: int, page_tokens: int, max_pages: int,
                 fmt: str = "bf16", head_dim: int = 64, device: str | torch.device = "cuda"):
        if fmt not in _lib.KV_FORMATS:
            raise ValueError(f"fmt must be one of {tuple(_lib.KV_FORMATS)}")
        _int32(seqs=seqs, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_tokens=page_tokens, pages=pages,
               max_pages=max_pages)
        sizes = _lib.bsa_kv_cache(seqs, heads, kv_heads, head_dim, page_tokens, pages, max_pages,
                                  _lib.KV_FORMATS[fmt])
        _lib.bsa_kv_workspace_size(sizes)              # refuses what the kernels do not take
        dev = _device(device)
        shape = (pages, kv_heads, page_tokens, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8 if fmt == "e4m3" else torch.bfloat16, device=dev)
                for _ in range(2))
        ks = vs = None
        if fmt == "e4m3":
            k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            ks, vs = (torch.zeros(shape[:3], dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
                      for _ in range(2))
        self._bind(k, v, ks, vs, torch.full((seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(seqs, dtype=torch.int32, device=dev), heads)
        self._table = torch.full((seqs, max_pages), -1, dtype=torch.int32)
        self._free = list(range(pages - 1, -1, -1))
        self.lengths = [0] * seqs

    @classmethod
    def over(cls, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor, heads: int,
             k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None) -> "KVCache":
        """A cache over the caller's pools [pages, kv_heads, page_tokens, 64] (bf16, or e4m3 with scales
        [pages, kv_heads, page_tokens]) and tables (page_table [seqs, max_pages], kv_len [seqs], int32). The
        caller keeps the tables; extend, release, forget and read_all are not available."""
        self = cls.__new__(cls)
        self._bind(k, v, k_scale, v_scale, page_table, kv_len, heads)
        self._table = None
        return self

    def _bind(self, k, v, k_scale, v_scale, page_table, kv_len, heads) -> None:
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in _POOL_DTYPE.values():
            raise ValueError("k and v must be bf16 or float8_e4m3fn pools [pages, kv_heads, page_tokens, head_dim]")
        self.fmt = "bf16" if k.dtype == torch.bfloat16 else "e4m3"
        pages, kv_heads, page_tokens, head_dim = k.shape
        if page_table.dim() != 2 or kv_len.shape != page_table.shape[:1]:
            raise ValueError("page_table must be [seqs, max_pages] and kv_len [seqs]")
        tensors = [k, v, page_table, kv_len]
        if self.fmt == "e4m3":
            for t in (k_scale, v_scale):
                if t is None or t.shape != k.shape[:3] or t.dtype not in (torch.float8_e8m0fnu, torch.uint8):
                    raise ValueError("an e4m3 cache needs k_scale and v_scale, float8_e8m0fnu or uint8 "
                                     "[pages, kv_heads, page_tokens]")
                tensors.append(t)
        if page_table.dtype != torch.int32 or kv_len.dtype != torch.int32:
            raise ValueError("page_table and kv_len must be int32")
        _int32(seqs=page_table.shape[0], max_pages=page_table.shape[1], heads=heads)
        if any(t.device != k.device or not t.is_contiguous() for t in tensors):
            raise ValueError("the cache's tensors must be contiguous and on one device")
        self.device, self.heads, self.kv_heads, self.head_dim = k.device, heads, kv_heads, head_dim
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.page_table, self.kv_len, self.page_tokens = page_table, kv_len, page_tokens
        ptr = (lambda t: None if t is None else t.data_ptr())
        self.c = _lib.bsa_kv_cache(page_table.shape[0], heads, kv_heads, head_dim, page_tokens, pages,
                                   page_table.shape[1], _lib.KV_FORMATS[self.fmt], ptr(k), ptr(v), ptr(k_scale),
                                   ptr(v_scale), ptr(page_table), ptr(kv_len))
        self.seqs = page_table.shape[0]
        self._index = self.device.index
        with torch.cuda.device(self.device) if self.device.type == "cuda" else contextlib.nullcontext():
            self.ws_bytes = _lib.bsa_kv_workspace_size(self.c)
        self._lib = _lib.load()
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._tensors = tensors + [self.workspace, self.status]
        self._streams = set()                           # that waited for them, and that they are kept for
        self._made = None                               # on the stream that made them, the first of these
        if self.device.type == "cuda":
            self._streams.add(_raw_stream(self._index))
            if not self._capturing(None):
                self._made = torch.cuda.Event()
                self._made.record(torch.cuda.current_stream(self.device))
        self._ref = ctypes.byref(self.c)
        self._ws_ptr, self._status_ptr = self.workspace.data_ptr(), self.status.data_ptr()

    @property
    def own_tables(self) -> bool:
        """Whether the cache keeps pages and lengths itself (not KVCache.over)."""
        return self._table is not None

    # steps --------------------------------------------------------------------------
    # A short call is over on the GPU in a few microseconds, so what happens here per call is kept
    # to the checks themselves.
    def append(self, k: torch.Tensor, v: torch.Tensor, cu_new: torch.Tensor, stream: int | None = None) -> None:
        """Writes the new tokens' keys and values ([rows, kv_heads, 64] bf16, one row stride) to the ends
        of their sequences, whose kv_len and pages count them already."""
        rows, stride = self._rows("k", k, self.kv_heads)
        if self._rows("v", v, self.kv_heads) != (rows, stride):
            raise ValueError("k and v must have the same rows and row stride")
        self._offsets("cu_new", cu_new, self.seqs + 1)
        self._call("bsa_kv_append", self._lib.bsa_kv_append, stream, rows, cu_new.data_ptr(), k.data_ptr(), v.data_ptr(),
                   stride, self._status_ptr)

    def attend(self, q: torch.Tensor, cu_new: torch.Tensor, max_new: int, unit: int = 0, window: int = 0,
               sink: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               stream: int | None = None) -> torch.Tensor:
        """Attention of the new tokens' queries ([rows, heads, 64] bf16) over their sequences, which hold
        the tokens already. unit: tokens per causal unit (tokens per frame: frame-wise; 1: token-wise; 0: all
        see all). window, sink: only the last `window` units and the first `sink` tokens. max_new: the most
        new tokens of a sequence, or a bound; it chooses the kernel. lse: optional float32 [heads, rows] for
        ln sum exp."""
        if (max_new | unit | window | sink) >> 31:
            _int32(max_new=max_new, unit=unit, window=window, sink=sink)
        rows, stride = self._rows("q", q, self.heads)
        if out is None:
            out = self._result(rows, self.heads, stream)
        out_rows, out_stride = self._rows("out", out, self.heads)
        if out_rows != rows:
            raise ValueError("out must have q's rows")
        lse_ptr = None
        if lse is not None:
            if (lse.shape != (self.heads, rows) or lse.dtype is not torch.float32 or lse.device != self.device
                    or not lse.is_contiguous()):
                raise ValueError(f"lse must be a contiguous float32 tensor {(self.heads, rows)} on {self.device}")
            lse_ptr = lse.data_ptr()
        self._offsets("cu_new", cu_new, self.seqs + 1)
        self._call("bsa_kv_attention", self._lib.bsa_kv_attention, stream, rows, max_new, unit, window, sink,
                   cu_new.data_ptr(), q.data_ptr(), stride, out.data_ptr(), out_stride, lse_ptr, self._ws_ptr,
                   self.ws_bytes, self._status_ptr)
        return out

    def read(self, cu_rows: torch.Tensor, first: torch.Tensor, rows: int | None = None, out=None,
             stream: int | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """Positions first[s], first[s] + 1, ... of each sequence as packed bf16 rows (k, v)
        [rows, kv_heads, 64]; tokens without a page read as zeros. `rows` or `out` = (k, v) sets the size."""
        if out is None:
            if rows is None:
                raise ValueError("read needs rows or out")
            out = tuple(self._result(rows, self.kv_heads, stream) for _ in range(2))
        k, v = out
        n, stride = self._rows("k", k, self.kv_heads)
        if self._rows("v", v, self.kv_heads) != (n, stride):
            raise ValueError("k and v must have the same rows and row stride")
        self._offsets("cu_rows", cu_rows, self.seqs + 1)
        self._offsets("first", first, self.seqs)
        self._call("bsa_kv_read", self._lib.bsa_kv_read, stream, n, cu_rows.data_ptr(), first.data_ptr(), k.data_ptr(),
                   v.data_ptr(), stride, self._status_ptr)
        return k, v

    def check_status(self, stream: int | None = None) -> int:
        """Waits for the stream; the first device-side error since the last check (0: none)."""
        with torch.cuda.device(self.device):
            return _lib.bsa_check_status(self._status_ptr, _raw_stream(self._index) if stream is None else stream)

    # pages and lengths kept by the cache itself ------------------------------------------
    def extend(self, counts, stream: int | None = None) -> Chunk:
        """Makes room for counts[s] new tokens of each sequence: takes pages, updates the device tables (in
        stream order) and returns the chunk's offsets. Raises before any change if the pages do not suffice.
        The tables are copied from host memory, which waits for the stream's earlier work and cannot be
        captured: capture append and attend, and extend between the replays."""
        self._own(stream)
        counts = [int(n) for n in counts]
        if len(counts) != self.seqs or min(counts) < 0:
            raise ValueError(f"extend needs {self.seqs} counts >= 0")
        P, width = self.page_tokens, self._table.shape[1]
        spans = [(-(-m // P), -(-(m + n) // P)) for m, n in zip(self.lengths, counts)]
        if any(b > width for _, b in spans):
            raise RuntimeError(f"a sequence would exceed max_pages = {width}")
        if sum(b - a for a, b in spans) > len(self._free):
            raise RuntimeError(f"{sum(b - a for a, b in spans)} pages needed, {len(self._free)} free")
        cu = [0]
        for s, (a, b) in enumerate(spans):
            for t in range(a, b):
                self._table[s, t] = self._free.pop()
            self.lengths[s] += counts[s]
            cu.append(cu[-1] + counts[s])
        return Chunk(self._upload(stream, cu), max(counts), cu[-1])

    def forget(self, seq: int, start: int, stop: int, stream: int | None = None) -> None:
        """Gives back the pages that lie wholly inside positions [start, stop) of a sequence: their tokens no
        longer exist for later calls. The sequence's last page, if not full, stays."""
        self._own(stream)
        seq = self._seq(seq)
        P = self.page_tokens
        for t in range(-(-max(start, 0) // P), min(stop, self.lengths[seq]) // P):
            if self._table[seq, t] >= 0:
                self._free.append(int(self._table[seq, t]))
                self._table[seq, t] = -1
        self._upload(stream)

    def release(self, seq: int, stream: int | None = None) -> None:
        """Empties a sequence."""
        self._own(stream)
        seq = self._seq(seq)
        self._free += [int(p) for p in self._table[seq] if p >= 0]
        self._table[seq] = -1
        self.lengths[seq] = 0
        self._upload(stream)

    def read_all(self, seq: int, stream: int | None = None) -> tuple[torch.Tensor, torch.Tensor]:
        """Every position of a sequence, (k, v) [tokens, kv_heads, 64] bf16."""
        self._own(stream)
        seq = self._seq(seq)
        n = self.lengths[seq]
        with self._torch_stream(stream):
            cu = torch.tensor([0] * (seq + 1) + [n] * (self.seqs - seq), dtype=torch.int32).to(self.device)
            first = torch.zeros(self.seqs, dtype=torch.int32, device=self.device)
        return self.read(cu, first, rows=n, stream=stream)

    # helpers ------------------------------------------------------------------------------
    def _own(self, stream) -> None:
        """Refuses, before any change, what needs tables of the cache's own that can be copied from the host now."""
        if not self.own_tables:
            raise RuntimeError("the caller keeps this cache's tables")
        if self.device.type == "cuda" and self._capturing(stream):
            raise RuntimeError("tables copied from the host cannot be part of a capture: call this outside of it")

    def _seq(self, seq: int) -> int:
        """Negative ones count from the end, as in a list."""
        if not -self.seqs <= seq < self.seqs:
            raise IndexError(f"sequence {seq} of {self.seqs}")
        return seq % self.seqs

    def _upload(self, stream, cu=()) -> torch.Tensor:
        """The tables to the device; offsets too, as a tensor of their own."""
        if self.device.type == "cuda":
            handle = _raw_stream(self._index) if stream is None else stream
            if handle not in self._streams:
                self._join(handle)
        with self._torch_stream(stream):
            self.page_table.copy_(self._table)
            self.kv_len.copy_(torch.tensor(self.lengths, dtype=torch.int32))
            return torch.tensor(cu, dtype=torch.int32).to(self.device)

    def _rows(self, name: str, x: torch.Tensor, heads: int) -> tuple[int, int]:
        shape, stride = x.shape, x.stride()
        if (len(shape) != 3 or shape[1] != heads or shape[2] != self.head_dim or x.dtype is not torch.bfloat16
                or x.device != self.device or stride[2] != 1 or stride[1] != self.head_dim):
            raise ValueError(f"{name} must be a bf16 tensor [rows, {heads}, {self.head_dim}] on {self.device} whose "
                             "rows are contiguous")
        return shape[0], stride[0] if shape[0] > 1 else heads * self.head_dim

    def _result(self, rows: int, heads: int, stream) -> torch.Tensor:
        """Memory for a result: that of the stream that writes it (a block of the current stream's memory may
        still be in use by work queued there), kept for the current stream too, which will read it."""
        with self._torch_stream(stream):
            x = torch.empty((rows, heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
        if stream is not None:
            x.record_stream(torch.cuda.current_stream(self.device))
        return x

    def _offsets(self, name: str, x: torch.Tensor, n: int) -> None:
        if x.dtype is not torch.int32 or x.dim() != 1 or len(x) != n or x.device != self.device or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor [{n}] on {self.device}")

    def _call(self, name: str, fn, stream, *args) -> None:
        """fn(cache, *args, stream) on the cache's device, on its current stream unless one is given."""
        if stream is None:
            stream = _raw_stream(self._index)
        if stream not in self._streams:
            self._join(stream)
        if _current_device() == self._index:
            code = fn(self._ref, *args, stream)
        else:
            with torch.cuda.device(self.device):
                code = fn(self._ref, *args, stream)
        if code:
            _lib._check(name, code)

    def _join(self, stream: int) -> None:
        """Once for each stream: it waits until the cache's tensors are made (a capture needs no wait: it begins
        with all work done), and they are kept for it, so that their memory waits for its work when they are
        dropped."""
        other = torch.cuda.ExternalStream(stream, device=self.device)
        if self._made is not None and not self._capturing(stream):
            other.wait_event(self._made)
        for t in self._tensors:
            t.record_stream(other)
        self._streams.add(stream)

    def _capturing(self, stream) -> bool:
        if stream is None or stream == _raw_stream(self._index):
            if _current_device() == self._index:
                return torch.cuda.is_current_stream_capturing()
            with torch.cuda.device(self.device):
                return torch.cuda.is_current_stream_capturing()
        with self._torch_stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def _torch_stream(self, stream):
        if stream is None:
            return contextlib.nullcontext()
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device))


_MOST = 2 ** 31 - 1


def _int32(**sizes) -> None:
    """The ABI's integers have 32 bits; what lies outside would be cut to others without a word."""
    for name, n in sizes.items():
        if not -_MOST <= n <= _MOST:
            raise ValueError(f"{name} = {n} does not fit 32 bits")


def _device(device) -> torch.device:
    dev = torch.device(device)
    return torch.device("cuda", torch.cuda.current_device()) if dev.type == "cuda" and dev.index is None else dev


# current_stream().cuda_stream and current_device() without the objects in between (several
# microseconds a call)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
