"""Paged key-value cache: torch layer over alspec_paged_*.

``PagedCache`` holds (or wraps) the page pools and writes and reads them;
``PagedDecoder`` runs attention of one new token per sequence over a cache.
Both check the tensors they are given, launch on the current stream of the
cache's device (or the stream passed in) and raise ``AlspecError`` on a
non-OK status.
"""
from __future__ import annotations

import torch

from . import alspec as _c
from .alspec import AlspecError

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_CODES = {torch.float32: _c.ALSPEC_F32, torch.bfloat16: _c.ALSPEC_BF16,
          torch.float8_e4m3fn: _c.ALSPEC_E4M3}


_FLOATS = (torch.float32, torch.bfloat16)

# The raw handle of the current stream; torch.cuda.current_stream builds an
# object around it, which took longer (2.2 us) than the checks and the launch
# of a small call.  (A build of torch without CUDA has neither name, nor
# tensors that would get as far.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _device(device):
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"a CUDA device is needed, not {device}")
    return torch.device("cuda", torch.cuda.current_device()) if device.index is None else device


def _stream(stream, index):
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _on(index, fn, *args):
    """fn(*args) with device `index` current."""
    if _current_device() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _empty(shape, dtype, device, stream):
    """An output made for a call on `stream`: from that stream's memory, so
    that nothing earlier on the current one still uses it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _settle(device):
    """What a constructor has zeroed is there for calls on any stream."""
    if not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(device).synchronize()


def _want(ok, what):
    if not ok:
        raise ValueError(what)


def _index(t, name, n, device):
    """Address of an int32 [n] tensor that the kernels index with."""
    if not (t.dtype is torch.int32 and t.shape == (n,) and t.device == device
            and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous int32 tensor of {n} on {device} is needed, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t, device):
    """(batch, max_pages) of a page table."""
    shape = t.shape
    if not (t.dtype is torch.int32 and len(shape) == 2 and t.device == device
            and t.is_contiguous() and shape[0] > 0 and shape[1] > 0):
        raise ValueError("page_table: a contiguous int32 tensor [batch, max_pages] on the "
                         f"cache's device {device} is needed, got {t.dtype} {tuple(shape)} on "
                         f"{t.device}")
    return shape


def _take_error(err, code, stream, device):
    """(status, word) of an error word, read and cleared; synchronizes."""
    s = torch.cuda.current_stream(device) if stream is None else stream
    with torch.cuda.device(device), torch.cuda.stream(s):
        word = int(err.item())
        err.zero_()
    return (code if word else _c.ALSPEC_OK), word


class PagedCache:
    """Page pools of one layer.

    ``k_pages`` and ``v_pages`` are [n_pages, n_kv_heads, page_size, head_dim]
    views of the pools ("f32", "bf16" or "e4m3"; with ``token_major`` a page's
    memory is [page_size, n_kv_heads, head_dim]); ``k_scales`` and
    ``v_scales`` (e4m3 only) hold one fp32 factor per row,
    [n_pages, n_kv_heads, page_size].  Token t of a sequence lives in slot
    t % page_size of page ``page_table[b, t // page_size]``.
    """

    def __init__(self, n_pages, page_size, n_kv_heads, head_dim, dtype="bf16", device=None,
                 token_major=False):
        dt = _DTYPES.get(dtype, dtype)
        _want(dt in _CODES, f"dtype {dtype!r}: one of {sorted(_DTYPES)} is needed")
        _want(min(n_pages, page_size, n_kv_heads, head_dim) >= 1, "sizes must be positive")
        device = _device(device)
        shape = ((n_pages, page_size, n_kv_heads, head_dim) if token_major
                 else (n_pages, n_kv_heads, page_size, head_dim))
        k, v = (torch.zeros(shape, dtype=dt, device=device) for _ in range(2))
        if token_major:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        ks = vs = None
        if dt is torch.float8_e4m3fn:
            ks, vs = (torch.zeros((n_pages, n_kv_heads, page_size), device=device)
                      for _ in range(2))
        self._wrap(k, v, ks, vs)

    @classmethod
    def from_tensors(cls, k_pages, v_pages, k_scales=None, v_scales=None):
        """A cache over existing pools: [n_pages, n_kv_heads, page_size,
        head_dim] tensors of equal strides with consecutive elements in a
        row, and for e4m3 their contiguous fp32 scales."""
        self = cls.__new__(cls)
        self._wrap(k_pages, v_pages, k_scales, v_scales)
        return self

    def _wrap(self, k, v, ks, vs):
        _want(k.dim() == 4 and k.shape == v.shape and k.dtype is v.dtype and k.dtype in _CODES
              and k.device == v.device and k.is_cuda,
              "k_pages and v_pages: two CUDA tensors [n_pages, n_kv_heads, page_size, head_dim] "
              "of one shape and type (fp32, bf16 or float8_e4m3fn) are needed")
        n, h, s, d = k.shape
        # The stride of a dimension of one index says nothing: take the one
        # that the contiguous layout would have.
        flat = (h * s * d, s * d, d, 1)
        strides = [tuple(c if m == 1 else x for m, x, c in zip(k.shape, t.stride(), flat))
                   for t in (k, v)]
        _want(strides[0] == strides[1] and strides[0][3] == 1 and min(strides[0]) > 0,
              "k_pages and v_pages need equal strides, none of them 0, and consecutive elements "
              "in a row")
        quantised = k.dtype is torch.float8_e4m3fn
        for name, t in (("k_scales", ks), ("v_scales", vs)):
            if quantised:
                _want(t is not None and t.dtype is torch.float32 and tuple(t.shape) == (n, h, s)
                      and t.is_contiguous() and t.device == k.device,
                      f"{name}: e4m3 pages need contiguous fp32 scales [n_pages, n_kv_heads, "
                      "page_size] on their device")
            else:
                _want(t is None, f"{name}: only e4m3 pages have scales")
        self.k_pages, self.v_pages, self.k_scales, self.v_scales = k, v, ks, vs
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n, h, s, d
        self.dtype, self.device = k.dtype, k.device
        self.err = torch.zeros(1, dtype=torch.int32, device=self.device)
        page, head, token = strides[0][:3]
        self.desc = _c.alspec_paged_cache(
            k.data_ptr(), v.data_ptr(), ks.data_ptr() if quantised else None,
            vs.data_ptr() if quantised else None, page, head, token, n, s, h, d,
            _CODES[k.dtype], 0)
        self._index = self.device.index
        # Sizes and strides that no entry point takes are refused here.
        if _c.alspec_paged_workspace_size(self.desc, 1, h) == 0:
            raise AlspecError(_c.ALSPEC_ERR_UNSUPPORTED, "alspec_paged_workspace_size")
        _settle(self.device)

    def append(self, k, v, positions, page_table, seq_ids=None, stream=None):
        """Write new tokens' rows: k, v [n, n_kv_heads, head_dim] (fp32 or
        bf16, token rows may be slices of wider ones), positions int32 [n]
        (negative: padding, skipped), page_table int32 [batch, max_pages],
        seq_ids int32 [n] or None (token i is sequence i's).  Bad sequences,
        positions and pages are skipped and set ALSPEC_DEVERR_PAGE, read with
        device_error().  A token named twice gets a mixture of its values."""
        n = k.shape[0]
        row = (n, self.n_kv_heads, self.head_dim)
        dev, one_head = self.device, self.n_kv_heads == 1
        kt, vt = k.stride(), v.stride()
        if not (k.shape == row and v.shape == row and k.dtype in _FLOATS and v.dtype is k.dtype
                and k.device == dev and v.device == dev and kt[2] == 1 and vt[2] == 1
                and (n <= 1 or (kt[0] > 0 and vt[0] > 0))
                and (one_head or (kt[1] == self.head_dim and vt[1] == self.head_dim))):
            raise ValueError("k and v: [n, n_kv_heads, head_dim] tensors in fp32 or bf16 (both "
                             f"alike) on {dev}, heads side by side, rows not broadcast, "
                             f"are needed, got {k.dtype} {tuple(k.shape)} and {v.dtype} "
                             f"{tuple(v.shape)}")
        batch, max_pages = _table(page_table, dev)
        pos = _index(positions, "positions", n, dev)
        seq = 0 if seq_ids is None else _index(seq_ids, "seq_ids", n, dev)
        if n == 0:
            return
        st = _on(self._index, _c._lib.alspec_paged_append, self.desc, k.data_ptr(), v.data_ptr(),
                 _CODES[k.dtype], 0 if n == 1 else kt[0], 0 if n == 1 else vt[0], pos, seq, n,
                 page_table.data_ptr(), batch, max_pages, self.err.data_ptr(),
                 _stream(stream, self._index))
        if st:
            raise AlspecError(st, "alspec_paged_append")

    def gather(self, page_table, seq_lens, k_out, v_out, stream=None):
        """Read pages back: rows [0, seq_lens[b]) of k_out and v_out [batch,
        n_kv_heads, max_seq_len, head_dim] (fp32 or bf16, contiguous) get the
        values of sequence b; the rows behind keep theirs.  Returns them."""
        dev = self.device
        batch, max_pages = _table(page_table, dev)
        shape = k_out.shape
        if not (len(shape) == 4 and shape[0] == batch and shape[1] == self.n_kv_heads
                and shape[2] > 0 and shape[3] == self.head_dim and v_out.shape == shape
                and k_out.dtype in _FLOATS and v_out.dtype is k_out.dtype
                and k_out.device == dev and v_out.device == dev
                and k_out.is_contiguous() and v_out.is_contiguous()):
            raise ValueError("k_out and v_out: contiguous tensors [batch, n_kv_heads, "
                             f"max_seq_len, head_dim] in fp32 or bf16 (both alike) on {dev} are "
                             f"needed, got {k_out.dtype} {tuple(shape)} and {v_out.dtype} "
                             f"{tuple(v_out.shape)}")
        lens = _index(seq_lens, "seq_lens", batch, dev)
        st = _on(self._index, _c._lib.alspec_paged_gather, self.desc, page_table.data_ptr(),
                 max_pages, lens, batch, shape[2], _CODES[k_out.dtype], k_out.data_ptr(),
                 v_out.data_ptr(), self.err.data_ptr(), _stream(stream, self._index))
        if st:
            raise AlspecError(st, "alspec_paged_gather")
        return k_out, v_out

    def device_error(self, stream=None):
        """(status, error word) that append and gather left, read and
        cleared; synchronizes the stream."""
        return _take_error(self.err, _c.ALSPEC_ERR_DEVICE_DATA, stream, self.device)


class PagedDecoder:
    """Attention of one new token per sequence over a PagedCache, for batches
    of one size; owns the workspace, so one call at a time (calls on one
    stream are)."""

    def __init__(self, cache, batch, n_q_heads, n_sink=0, window=0, scale=0.0, timeout_ms=0):
        self.cache, self.batch, self.n_q_heads = cache, int(batch), int(n_q_heads)
        self.n_sink, self.window, self.scale = int(n_sink), int(window), float(scale)
        self.timeout_ms = int(timeout_ms)
        self._index = cache.device.index
        nbytes = _on(self._index, _c.alspec_paged_workspace_size, cache.desc, self.batch,
                     self.n_q_heads)
        if nbytes == 0:
            raise AlspecError(_c.ALSPEC_ERR_INVALID_ARG, "alspec_paged_workspace_size")
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=cache.device)
        self.workspace_bytes = nbytes
        self.q_dtype = torch.float32 if cache.dtype is torch.float32 else torch.bfloat16
        self._shape = (self.batch, self.n_q_heads, cache.head_dim)
        _settle(cache.device)

    def decode(self, q, page_table, seq_lens, out=None, lse=None, stream=None):
        """q [batch, n_q_heads, head_dim] (fp32 for fp32 pages, else bf16;
        rows may be slices of wider ones) over sequence b's first
        seq_lens[b] tokens (0: zeros), or with n_sink + window > 0 over its
        sink set.  Fills out (fp32 or bf16; new: q's type) and, if given, lse
        (fp32 [batch, n_q_heads], natural logarithm), which overlap no input;
        returns out.  A new out belongs to the stream of the call.  Pages
        without a token attended to need no table entry."""
        c = self.cache
        dev, shape = c.device, self._shape
        qt = q.stride()
        if not (q.shape == shape and q.dtype is self.q_dtype and q.device == dev and qt[2] == 1
                and (shape[0] == 1 or qt[0] > 0) and (shape[1] == 1 or qt[1] == shape[2])):
            raise ValueError(f"q: {self.q_dtype} {shape} on {dev}, heads side by side, rows not "
                             f"broadcast, is needed, got {q.dtype} {tuple(q.shape)} on {q.device}")
        if out is None:
            out = _empty(shape, q.dtype, dev, stream)
        elif not (out.shape == shape and out.dtype in _FLOATS and out.device == dev
                  and out.is_contiguous()):
            raise ValueError(f"out: a contiguous fp32 or bf16 tensor {shape} on {dev} is needed, "
                             f"got {out.dtype} {tuple(out.shape)} on {out.device}")
        if lse is not None and not (lse.shape == shape[:2] and lse.dtype is torch.float32
                                    and lse.device == dev and lse.is_contiguous()):
            raise ValueError(f"lse: a contiguous fp32 tensor {shape[:2]} on {dev} is needed")
        batch, max_pages = _table(page_table, dev)
        if batch != self.batch:
            raise ValueError(f"page_table: {self.batch} rows are needed, got {batch}")
        lens = _index(seq_lens, "seq_lens", batch, dev)
        st = _on(self._index, _c._lib.alspec_paged_decode, c.desc, q.data_ptr(),
                 0 if batch == 1 else qt[0], shape[1], page_table.data_ptr(), max_pages, lens,
                 batch, self.n_sink, self.window, self.scale, _CODES[out.dtype], out.data_ptr(),
                 0 if lse is None else lse.data_ptr(), self.timeout_ms,
                 self.workspace.data_ptr(), self.workspace_bytes, _stream(stream, self._index))
        if st:
            raise AlspecError(st, "alspec_paged_decode")
        return out

    def device_error(self, stream=None):
        """(status, error word) of the workspace; see alspec_get_device_error."""
        return _on(self._index, _c.alspec_get_device_error, self.workspace.data_ptr(),
                   self.workspace_bytes, _stream(stream, self._index))
