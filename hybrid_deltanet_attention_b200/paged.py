"""Paged KV cache for several sequences, and the operators that work on its pages.

`PagedCache` describes device memory (its own, or tensors given to it) to libmk.so's paged
entry points: sequences grow, end, fork and move by pages, new keys and values are normed,
rotated and appended, and new tokens attend over the pages. `qk_norm_rope` is the norm and
rotation without a cache. Argument checks and marshalling only; every step runs in the library's kernels.
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional, Tuple

import torch

from . import _abi
from ._abi import MkPagedCache, MkQkRope, check

_DTYPES = {torch.float32: _abi.MK_DT_F32, torch.bfloat16: _abi.MK_DT_BF16}


def _stream_of(device: torch.device, stream: Optional[torch.cuda.Stream]) -> torch.cuda.Stream:
    if stream is None:
        return torch.cuda.current_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return stream


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _ints(t: torch.Tensor, what: str, device: torch.device) -> int:
    if t.dtype != torch.int32 or t.dim() != 1 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-D int32 tensor on {device}")
    return t.data_ptr()


def _heads(t: torch.Tensor, what: str, device: torch.device, dtype, rows: int, d: int) -> None:
    """t is [rows][heads][d], heads next to each other; rows may be strided."""
    if (t.dim() != 3 or t.dtype != dtype or t.device != device or t.shape[0] != rows or t.shape[2] != d
            or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != d)):
        raise ValueError(f"{what} must be {dtype} [{rows}][heads][{d}] on {device} with its heads contiguous")


def _pitch(t: torch.Tensor) -> int:
    # a single row has no pitch of its own; any that holds the row will do
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _gain(t: Optional[torch.Tensor], device: torch.device, d: int):
    if t is None:
        return None
    if t.dtype != torch.bfloat16 or t.shape != (d,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"a gain must be a contiguous bfloat16 tensor of {d} on {device}")
    return t.data_ptr()


class PagedCache:
    """A KV cache cut into pages (see mk_paged_cache in include/mk.h).

    k, v: bfloat16 [layers][pages][kv heads][page size][head dim], any strides whose entries
    are contiguous (the same for both). table: int32 [sequences][max pages], -1 where a
    sequence has no page. len: int32 [sequences]. ref: int32 [pages], table entries per page.
    All stay the caller's tensors and are updated in place, on the device, in stream order.
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
        self.device = k.device
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
        self._p = C.byref(c)
        self._scale = 1.0 / math.sqrt(c.head_dim)

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, kv_heads: int, page_size: int, head_dim: int, n_seqs: int, max_pages: int,
              device="cuda") -> "PagedCache":
        """A cache of its own memory, every page free."""
        dev = torch.device(device)
        k, v = (torch.zeros((n_layers, n_pages, kv_heads, page_size, head_dim), dtype=torch.bfloat16, device=dev) for _ in "kv")
        return cls(k, v, torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(n_seqs, dtype=torch.int32, device=dev), torch.zeros(n_pages, dtype=torch.int32, device=dev))

    # ---- pages ----
    def _movable(self) -> None:
        _need(not self.fixed, "the pages of this cache belong to a model and keep their places")

    def resize(self, seqs: torch.Tensor, lens: torch.Tensor, stream=None) -> None:
        """Set the lengths of different sequences, taking and giving back pages (mk_pages_resize)."""
        self._movable()
        s, l = _ints(seqs, "seqs", self.device), _ints(lens, "lens", self.device)   # noqa: E741
        _need(seqs.numel() == lens.numel(), "seqs and lens differ in length")
        with torch.cuda.device(self.device):
            check(self.lib.mk_pages_resize(self._p, s, l, seqs.numel(), _stream_of(self.device, stream).cuda_stream))

    def free(self, seqs: torch.Tensor, stream=None) -> None:
        """Give back every page of these sequences."""
        self._movable()
        s = _ints(seqs, "seqs", self.device)
        with torch.cuda.device(self.device):
            check(self.lib.mk_pages_resize(self._p, s, None, seqs.numel(), _stream_of(self.device, stream).cuda_stream))

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Make sequence dst[i] a continuation of src[i], sharing its full pages (mk_pages_fork)."""
        self._movable()
        a, b = _ints(src, "src", self.device), _ints(dst, "dst", self.device)
        _need(src.numel() == dst.numel(), "src and dst differ in length")
        with torch.cuda.device(self.device):
            check(self.lib.mk_pages_fork(self._p, a, b, src.numel(), _stream_of(self.device, stream).cuda_stream))

    def compact(self, stream=None) -> None:
        """Move the used pages to the lowest ids (mk_pages_compact)."""
        self._movable()
        with torch.cuda.device(self.device):
            check(self.lib.mk_pages_compact(self._p, _stream_of(self.device, stream).cuda_stream))

    def copy_pages(self, src: torch.Tensor, dst: torch.Tensor, source: Optional["PagedCache"] = None, stream=None) -> None:
        """Copy page src[i] of `source` (or of this cache) to page dst[i] of this cache (mk_pages_copy)."""
        f = self if source is None else source
        _need(f.device == self.device, "the caches are on different devices")
        a, b = _ints(src, "src", self.device), _ints(dst, "dst", self.device)
        _need(src.numel() == dst.numel(), "src and dst differ in length")
        with torch.cuda.device(self.device):
            check(self.lib.mk_pages_copy(f._p, self._p, a, b, src.numel(), _stream_of(self.device, stream).cuda_stream))

    # ---- new tokens ----
    def append(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, seq_start: torch.Tensor,
               seqs: Optional[torch.Tensor] = None, *, q_gain: Optional[torch.Tensor] = None,
               k_gain: Optional[torch.Tensor] = None, eps: float = 1e-6, theta: float = 1e7, rot_dim: Optional[int] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Norm (where a gain is given) and rotate the queries and keys of new rows and store keys and values in
        their pages (mk_qk_norm_rope). Rows seq_start[i] .. seq_start[i+1]-1 are the last positions of sequence
        seqs[i] (or i), whose length already counts them. Returns the bfloat16 queries."""
        c = self._c
        return _rope(self.device, q, k, v, None, q_gain, k_gain, eps, theta, rot_dim, out, None, self, layer, seq_start, seqs,
                     c.head_dim, stream)[0]

    def attention(self, layer: int, q: torch.Tensor, seq_start: torch.Tensor, seqs: Optional[torch.Tensor] = None, *,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Causal attention of new rows over their sequences' pages (mk_paged_attention); q bfloat16
        [rows][query heads][head dim], scale 1/sqrt(head dim) unless given. Returns bfloat16 like q."""
        c, dev = self._c, self.device
        rows = q.shape[0]
        _heads(q, "q", dev, torch.bfloat16, rows, c.head_dim)
        start, ids, n = _new_rows(seq_start, seqs, c, dev)
        st = _stream_of(dev, stream)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            if out is None:
                out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
            else:
                _heads(out, "out", dev, torch.bfloat16, rows, c.head_dim)
                _need(out.shape == q.shape, "out must have q's shape")
            need = self.lib.mk_paged_attention_scratch(self._p, rows, q.shape[1])
            scratch = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
            check(self.lib.mk_paged_attention(self._p, layer, q.data_ptr(), _pitch(q), rows, q.shape[1], start, ids, n,
                                              self._scale if scale is None else scale, out.data_ptr(), _pitch(out),
                                              scratch.data_ptr(), scratch.numel(), st.cuda_stream))
        return out

    def sync(self, stream=None) -> None:
        """Wait for the stream and raise if a call found bad ids, lengths or too few pages (the word is then cleared)."""
        _stream_of(self.device, stream).synchronize()
        bits = int(self.err.item())
        if bits:
            self.err.zero_()
            names = [n for b, n in ((_abi.MK_DEVERR_BAD_PAGE, "a sequence, page, length or position out of range, or an id given twice"),
                                    (_abi.MK_DEVERR_NO_PAGES, "not enough free pages"),
                                    (_abi.MK_DEVERR_PIPE_TIMEOUT, "a pipeline wait gave up")) if bits & b]
            raise _abi.MkError(_abi.MK_ERR_DEVICE, f"paged cache: {', '.join(names)} (device word 0x{bits:x})")


def _new_rows(seq_start, seqs, c, dev) -> Tuple[int, Optional[int], int]:
    start = _ints(seq_start, "seq_start", dev)
    n = seq_start.shape[0] - 1
    _need(n >= 0, "seq_start must have one entry more than there are sequences")
    if seqs is None:
        _need(n <= c.n_seqs, "more sequences than the cache has")
        return start, None, n
    _need(seqs.shape[0] == n, "seqs must have one entry less than seq_start")
    return start, _ints(seqs, "seqs", dev), n


def _rope(dev, q, k, v, positions, q_gain, k_gain, eps, theta, rot_dim, q_out, k_out, cache, layer, seq_start, seqs, d, stream):
    dt = _DTYPES.get(q.dtype)
    _need(dt is not None, "q must be float32 or bfloat16")
    _need(q.dim() == 3 and k.dim() == 3, "q and k must be [rows][heads][head dim]")
    rows = q.shape[0]
    _heads(q, "q", dev, q.dtype, rows, d)
    _heads(k, "k", dev, q.dtype, rows, d)
    a = MkQkRope()
    a.dtype, a.rows, a.q_heads, a.kv_heads, a.head_dim = dt, rows, q.shape[1], k.shape[1], d
    a.rot_dim = d if rot_dim is None else rot_dim
    a.eps, a.theta = eps, theta
    a.q, a.ldq, a.k, a.ldk = q.data_ptr(), _pitch(q), k.data_ptr(), _pitch(k)
    a.q_gain, a.k_gain = _gain(q_gain, dev, d), _gain(k_gain, dev, d)
    if cache is not None:
        _heads(v, "v", dev, q.dtype, rows, d)
        _need(k.shape[1] == cache._c.kv_heads and v.shape[1] == cache._c.kv_heads, "k and v must have the cache's heads")
        a.v, a.ldv = v.data_ptr(), _pitch(v)
        a.seq_start, a.seqs, a.n = _new_rows(seq_start, seqs, cache._c, dev)
        a.cache, a.layer = C.addressof(cache._c), layer
    else:
        a.positions = _ints(positions, "positions", dev)
        _need(positions.shape[0] == rows, "one position per row")
    st = _stream_of(dev, stream)
    with torch.cuda.device(dev), torch.cuda.stream(st):
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        else:
            _heads(q_out, "the query output", dev, torch.bfloat16, rows, d)
            _need(q_out.shape == q.shape, "the query output must have q's shape")
        a.q_out, a.ldq_out = q_out.data_ptr(), _pitch(q_out)
        if cache is None:
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
            else:
                _heads(k_out, "the key output", dev, torch.bfloat16, rows, d)
                _need(k_out.shape == k.shape, "the key output must have k's shape")
            a.k_out, a.ldk_out = k_out.data_ptr(), _pitch(k_out)
        check(_abi.load_library().mk_qk_norm_rope(C.byref(a), st.cuda_stream))
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
