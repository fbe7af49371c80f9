"""Paged KV cache for several sequences, and the operators that work on its pages.

`PagedCache` describes device memory (its own, or tensors given to it) to libmk.so's paged
entry points: sequences grow, end, fork and move by pages, new keys and values are normed,
rotated and appended, and new tokens attend over the pages. `qk_norm_rope` is the norm and
rotation without a cache. Argument checks and marshalling only; every step runs in the library's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import math
import struct
from typing import Optional, Tuple

import torch

from . import _abi
from ._abi import MkPagedCache, MkQkRope, check

_DTYPES = {torch.float32: _abi.MK_DT_F32, torch.bfloat16: _abi.MK_DT_BF16}
_BF16 = torch.bfloat16
_load_library = _abi.load_library
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device
# mk_qk_rope in one piece (filling a ctypes structure field by field costs more than the call)
_ROPE = struct.Struct("@6idf4xPqPqPqPPPqPqPPiiPP")
assert _ROPE.size == C.sizeof(MkQkRope)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class _Here:
    """The tensors' device and its current stream are current already: the raw stream, and nothing to undo."""
    __slots__ = ("raw",)

    def __init__(self, raw: int):
        self.raw = raw

    def __enter__(self) -> int:
        return self.raw

    def __exit__(self, *exc) -> None:
        return None


@contextlib.contextmanager
def _there(device: torch.device, stream: Optional[torch.cuda.Stream]):
    if stream is None:
        with torch.cuda.device(device):
            yield _raw_stream(device.index)
    else:
        _need(stream.device == device, f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _on(device: torch.device, stream: Optional[torch.cuda.Stream]):
    """A context with the tensors' device current, on `stream` or the device's current stream, so that what is
    allocated in it belongs to that stream; gives the raw stream. The usual case costs next to nothing."""
    if stream is None and _current_device() == device.index:
        return _Here(_raw_stream(device.index))
    return _there(device, stream)


def _used_on(stream: Optional[torch.cuda.Stream], *tensors: Optional[torch.Tensor]) -> None:
    """Arguments of a call on a stream that was given: their memory is not reused before it has run there."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


# Tensors are compared by device index here: every caller has made sure that the index means CUDA.
def _ints(t: torch.Tensor, what: str, index: int) -> int:
    if t.dtype is not torch.int32 or t.dim() != 1 or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-D int32 tensor on cuda:{index}")
    return t.data_ptr()


def _heads(t: torch.Tensor, what: str, index: int, dtype, rows: int, d: int) -> Tuple[int, int, int]:
    """Address, pitch and heads of t [rows][heads][d], heads next to each other; rows may be strided."""
    shape, st = t.shape, t.stride()
    if (len(shape) != 3 or t.dtype is not dtype or t.get_device() != index or shape[0] != rows or shape[2] != d or st[2] != 1
            or (shape[1] > 1 and st[1] != d)):
        raise ValueError(f"{what} must be {dtype} [{rows}][heads][{d}] on cuda:{index} with its heads contiguous")
    # a single row has no pitch of its own; any that holds the row will do
    return t.data_ptr(), st[0] if rows > 1 else shape[1] * d, shape[1]


def _gain(t: torch.Tensor, index: int, d: int) -> int:
    if t.dtype is not _BF16 or t.shape != (d,) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"a gain must be a contiguous bfloat16 tensor of {d} on cuda:{index}")
    return t.data_ptr()


class PagedCache:
    """A KV cache cut into pages (see mk_paged_cache in include/mk.h).

    k, v: bfloat16 [layers][pages][kv heads][page size][head dim], any strides whose entries
    are contiguous (the same for both). table: int32 [sequences][max pages], -1 where a
    sequence has no page. len: int32 [sequences]. ref: int32 [pages], table entries per page.
    All stay the caller's tensors and are updated in place, on the device, in stream order.
    A captured call uses the cache's own arrays too: keep the cache as long as its graphs.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, len: torch.Tensor, ref: torch.Tensor,
                 fixed: bool = False):
        self.fixed = fixed      # pages that belong to something else (a model): resize, fork and compact are refused
        self.lib = _abi.load_library()
        _need(k.is_cuda and k.dim() == 5 and k.dtype == torch.bfloat16 and v.dtype == torch.bfloat16, "k and v must be 5-D bfloat16 CUDA tensors")
        _need(v.shape == k.shape and v.stride() == k.stride() and v.device == k.device and k.stride(4) == 1,
              "k and v must agree in shape, strides and device, entries contiguous")
        for t, n, what in ((table, 2, "table"), (len, 1, "len"), (ref, 1, "ref")):
            _need(t.dtype == torch.int32 and t.dim() == n and t.device == k.device and t.is_contiguous(),
                  f"{what} must be a contiguous {n}-D int32 tensor on {k.device}")
        _need(len.shape[0] == table.shape[0], "table and len disagree in the number of sequences")
        _need(ref.shape[0] == k.shape[1], "ref must have one entry per page")
        self.k, self.v, self.table, self.len, self.ref = k, v, table, len, ref
        self.device, self._index = k.device, k.get_device()
        c = self._c = MkPagedCache()
        c.k, c.v = k.data_ptr(), v.data_ptr()
        c.n_layers, c.n_pages, c.kv_heads, c.page_size, c.head_dim = k.shape
        # a dimension of one entry is never stepped over: give it a stride that holds what lies within
        st, inner = [0] * 4, c.head_dim
        for i in (3, 2, 1, 0):
            st[i] = k.stride(i) if k.shape[i] > 1 else inner
            inner = max(inner, st[i] * k.shape[i])
        c.layer_stride, c.page_stride, c.head_stride, c.slot_stride = st
        c.n_seqs, c.max_pages = table.shape
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        self.work = torch.zeros(int(self.lib.mk_pages_work_ints(C.byref(c))), dtype=torch.int32, device=k.device)
        c.table, c.len, c.ref = table.data_ptr(), len.data_ptr(), ref.data_ptr()
        c.work, c.err = self.work.data_ptr(), self.err.data_ptr()
        self._p, self._address = C.byref(c), C.addressof(c)
        self._d, self._kv_heads, self._n_seqs = c.head_dim, c.kv_heads, c.n_seqs
        self._scale = 1.0 / math.sqrt(c.head_dim)
        self._scratch = (0, 0, 0)                # rows, query heads and the bytes for calls of this shape, replaced in one piece
        self._attention = self.lib.mk_paged_attention
        self._bytes = torch.empty(0, dtype=torch.uint8, device=k.device)
        # err and work are made on the stream that is current now; the others wait for that (see _first_use)
        self._streams = set()
        with torch.cuda.device(k.device):
            self._made = None if torch.cuda.is_current_stream_capturing() else torch.cuda.current_stream().record_event()

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, kv_heads: int, page_size: int, head_dim: int, n_seqs: int, max_pages: int,
              device="cuda") -> "PagedCache":
        """A cache of its own memory, every page free."""
        dev = torch.device(device)
        k, v = (torch.zeros((n_layers, n_pages, kv_heads, page_size, head_dim), dtype=torch.bfloat16, device=dev) for _ in "kv")
        return cls(k, v, torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(n_seqs, dtype=torch.int32, device=dev), torch.zeros(n_pages, dtype=torch.int32, device=dev))

    # ---- streams ----
    def _first_use(self, stream: Optional[torch.cuda.Stream]) -> None:
        """Where the stream of a call has not worked on this cache yet: it waits until the cache's own arrays are made,
        and none of its memory is given to anything else before that stream has run, should the cache be dropped after a call."""
        if (_raw_stream(self._index) if stream is None else stream.cuda_stream) in self._streams:
            return
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        _need(stream.device == self.device, f"the stream is on {stream.device}, the tensors on {self.device}")
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
        if not capturing:                        # (a capture cannot wait for what it does not hold)
            self._streams.add(stream.cuda_stream)
            if self._made is not None:
                stream.wait_event(self._made)
        for t in (self.k, self.v, self.table, self.len, self.ref, self.work, self.err):
            t.record_stream(stream)

    def _on(self, stream: Optional[torch.cuda.Stream]):
        self._first_use(stream)
        return _on(self.device, stream)

    # ---- pages ----
    def _movable(self) -> None:
        _need(not self.fixed, "the pages of this cache belong to a model and keep their places")

    def resize(self, seqs: torch.Tensor, lens: torch.Tensor, stream=None) -> None:
        """Set the lengths of different sequences, taking and giving back pages (mk_pages_resize)."""
        self._movable()
        s, l = _ints(seqs, "seqs", self._index), _ints(lens, "lens", self._index)   # noqa: E741
        _need(seqs.numel() == lens.numel(), "seqs and lens differ in length")
        with self._on(stream) as st:
            check(self.lib.mk_pages_resize(self._p, s, l, seqs.numel(), st))
        _used_on(stream, seqs, lens)

    def free(self, seqs: torch.Tensor, stream=None) -> None:
        """Give back every page of these sequences."""
        self._movable()
        s = _ints(seqs, "seqs", self._index)
        with self._on(stream) as st:
            check(self.lib.mk_pages_resize(self._p, s, None, seqs.numel(), st))
        _used_on(stream, seqs)

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Make sequence dst[i] a continuation of src[i], sharing its full pages (mk_pages_fork)."""
        self._movable()
        a, b = _ints(src, "src", self._index), _ints(dst, "dst", self._index)
        _need(src.numel() == dst.numel(), "src and dst differ in length")
        with self._on(stream) as st:
            check(self.lib.mk_pages_fork(self._p, a, b, src.numel(), st))
        _used_on(stream, src, dst)

    def compact(self, stream=None) -> None:
        """Move the used pages to the lowest ids (mk_pages_compact)."""
        self._movable()
        with self._on(stream) as st:
            check(self.lib.mk_pages_compact(self._p, st))

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, source: Optional["PagedCache"] = None, stream=None) -> None:
        """Copy page src[i] of `source` (or of this cache) to page dst[i] of this cache (mk_pages_copy)."""
        f = self if source is None else source
        _need(f.device == self.device, "the caches are on different devices")
        a, b = _ints(src, "src", self._index), _ints(dst, "dst", self._index)
        _need(src.numel() == dst.numel(), "src and dst differ in length")
        f._first_use(stream)
        with self._on(stream) as st:
            check(self.lib.mk_pages_copy(f._p, self._p, a, b, src.numel(), st))
        _used_on(stream, src, dst)

    # ---- new tokens ----
    def append(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_start: torch.Tensor,
               seqs: Optional[torch.Tensor] = None, *, q_gain: Optional[torch.Tensor] = None,
               k_gain: Optional[torch.Tensor] = None, eps: float = 1e-6, theta: float = 1e7, rot_dim: Optional[int] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Norm (where a gain is given) and rotate the queries and keys of new rows and store keys and values in
        their pages (mk_qk_norm_rope). Rows seq_start[i] .. seq_start[i+1]-1 are the last positions of sequence
        seqs[i] (or i), whose length already counts them. Returns the bfloat16 queries (rows of no sequence are not written)."""
        return _rope(self.device, q, k, v, None, q_gain, k_gain, eps, theta, rot_dim, out, None, self, layer, seq_start, seqs,
                     self._d, stream)[0]

    def attention(self, layer: int, q: torch.Tensor, seq_start: torch.Tensor, seqs: Optional[torch.Tensor] = None, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Causal attention of new rows over their sequences' pages (mk_paged_attention); q bfloat16
        [rows][query heads][head dim], scale 1/sqrt(head dim) unless given. Returns bfloat16 like q (rows of no sequence are not written)."""
        index, rows, d = self._index, q.shape[0], self._d
        qp, ldq, hq = _heads(q, "q", index, _BF16, rows, d)
        start, ids, n = _new_rows(seq_start, seqs, self._n_seqs, index)
        if out is not None:
            op, ldo, ho = _heads(out, "out", index, _BF16, rows, d)
            _need(ho == hq, "out must have q's shape")
        else:
            op, ldo = 0, hq * d
        with self._on(stream) as st:
            for_rows, for_heads, size = self._scratch
            if for_rows != rows or for_heads != hq:  # asked with the tensors' device current: it goes by that GPU
                size = max(32, self.lib.mk_paged_attention_scratch(self._p, rows, hq))
                self._scratch = rows, hq, size
            if out is None:
                out = torch.empty_like(q)
                op = out.data_ptr()
            scratch = self._bytes.new_empty(size)
            rc = self._attention(self._p, layer, qp, ldq, rows, hq, start, ids, n, self._scale if scale is None else scale, op, ldo,
                                 scratch.data_ptr(), size, st)
        if rc:
            check(rc)
        _used_on(stream, q, seq_start, seqs, out)
        return out

    def sync(self, stream=None) -> None:
        """Wait for the stream and raise if a call found bad ids, lengths or too few pages (the word is then cleared)."""
        with self._on(stream):                    # read and cleared there: in order with the calls on that stream
            bits = int(self.err.item())
            if bits:
                self.err.zero_()
        if bits:
            names = [n for b, n in ((_abi.MK_DEVERR_BAD_PAGE, "a sequence, page, length or position out of range, or an id given twice"),
                                    (_abi.MK_DEVERR_NO_PAGES, "not enough free pages"),
                                    (_abi.MK_DEVERR_PIPE_TIMEOUT, "a pipeline wait gave up")) if bits & b]
            raise _abi.MkError(_abi.MK_ERR_DEVICE, f"paged cache: {', '.join(names)} (device word 0x{bits:x})")


def _new_rows(seq_start, seqs, n_seqs, index) -> Tuple[int, Optional[int], int]:
    start = _ints(seq_start, "seq_start", index)
    n = seq_start.shape[0] - 1
    _need(n >= 0, "seq_start must have one entry more than there are sequences")
    if seqs is None:
        _need(n <= n_seqs, "more sequences than the cache has")
        return start, None, n
    _need(seqs.shape[0] == n, "seqs must have one entry less than seq_start")
    return start, _ints(seqs, "seqs", index), n


def _rope(dev, q, k, v, positions, q_gain, k_gain, eps, theta, rot_dim, q_out, k_out, cache, layer, seq_start, seqs, d, stream):
    dtype, rows, index = q.dtype, q.shape[0], dev.index
    dt = _DTYPES.get(dtype)
    _need(dt is not None, "q must be float32 or bfloat16")
    qp, ldq, hq = _heads(q, "q", index, dtype, rows, d)
    kp, ldk, hkv = _heads(k, "k", index, dtype, rows, d)
    vp = ldv = pos = start = ids = cp = n = qop = kop = ldko = 0
    if cache is not None:
        vp, ldv, hv = _heads(v, "v", index, dtype, rows, d)
        _need(hkv == cache._kv_heads and hv == hkv, "k and v must have the cache's heads")
        start, ids, n = _new_rows(seq_start, seqs, cache._n_seqs, index)
        cp = cache._address
    else:
        pos = _ints(positions, "positions", index)
        _need(positions.shape[0] == rows, "one position per row")
        ldko = hkv * d
        if k_out is not None:
            kop, ldko, h = _heads(k_out, "the key output", index, _BF16, rows, d)
            _need(h == hkv, "the key output must have k's shape")
    ldqo = hq * d
    if q_out is not None:
        qop, ldqo, h = _heads(q_out, "the query output", index, _BF16, rows, d)
        _need(h == hq, "the query output must have q's shape")
    gq = 0 if q_gain is None else _gain(q_gain, index, d)
    gk = 0 if k_gain is None else _gain(k_gain, index, d)

    with (_on(dev, stream) if cache is None else cache._on(stream)) as st:
        # a fresh output is contiguous: the heads of a row are, and rows that are further apart are packed
        if q_out is None:
            q_out = torch.empty_like(q, dtype=_BF16)
            qop = q_out.data_ptr()
        if cache is None and k_out is None:
            k_out = torch.empty_like(k, dtype=_BF16)
            kop = k_out.data_ptr()
        rc = _load_library().mk_qk_norm_rope(
            _ROPE.pack(dt, rows, hq, hkv, d, d if rot_dim is None else rot_dim, theta, eps, qp, ldq, kp, ldk, vp, ldv, gq, gk, qop, ldqo,
                       kop, ldko, pos, cp, layer, n, start, ids or 0), st)
    if rc:
        check(rc)
    _used_on(stream, q, k, v, positions, q_gain, k_gain, q_out, k_out, seq_start, seqs)
    return q_out, k_out


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, *, q_gain: Optional[torch.Tensor] = None,
                 k_gain: Optional[torch.Tensor] = None, eps: float = 1e-6, theta: float = 1e7, rot_dim: Optional[int] = None,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-head norm (where a gain is given) and rotation of q, k [rows][heads][head dim] (float32 or bfloat16) at the
    given int32 positions; returns bfloat16 tensors (mk_qk_norm_rope without a cache)."""
    _need(q.is_cuda and q.dim() == 3, "q must be a CUDA tensor [rows][heads][head dim]")
    return _rope(q.device, q, k, None, positions, q_gain, k_gain, eps, theta, rot_dim, q_out, k_out, None, 0, None, None,
                 q.shape[2], stream)
