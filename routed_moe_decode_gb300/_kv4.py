"""Kv4Cache: a paged K/V cache in 4 bits, the attention over it and the calls on its pages."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._routing import _raw_stream

KV4_NO_PAGE = 0x1
KV4_BAD_PAGE = 0x2
KV4_NONFINITE = 0x4
KV4_BAD_SEQ = 0x8
KV4_TIMEOUT = 0x10

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


class Kv4Cache:
    """Keys and values of `layers` layers in `pages` pages of page_size tokens each (include/moe_kv4.h
    has the page format, the rounding and the steps' rows).

    Tensors (made here where they are not given, empty; the caller may read them, and write them
    between steps):
        pool  [layers, pages, page bytes] uint8
        table [seqs, max_pages] int32   page numbers of each sequence's tokens, -1 past them
        lens  [seqs] int32              tokens of each sequence
        refs  [pages] int32             table entries that point at each page (0: free)
    k_scale, v_scale: FP32 tensor scales of the values.  One cache's calls are ordered on one stream,
    and its device is the current one when they are made.

    A step: reserve(new_tokens); for every layer append(...) and attend(...); compact(keep, ...).
    Rows of a step are those of sequence 0, then of sequence 1, ...; cu_rows [seqs + 1] int32 on the
    device holds where each sequence's begin.
    """

    def __init__(self, layers, pages, kv_heads, head_dim, page_size, seqs, max_pages, pool=None, table=None, lens=None,
                 refs=None, k_scale=1.0, v_scale=1.0, device="cuda"):
        self._lib = _lib.lib()
        a = self._args = _lib.Kv4Args()
        a.layers, a.pages, a.kv_heads, a.head_dim = int(layers), int(pages), int(kv_heads), int(head_dim)
        a.page_size, a.seqs, a.max_pages = int(page_size), int(seqs), int(max_pages)
        a.k_scale, a.v_scale = float(k_scale), float(v_scale)
        self._ref = ctypes.byref(a)
        _lib._check("moe_kv4_check", self._lib.moe_kv4_check(self._ref))
        self.page_bytes = int(self._lib.moe_kv4_page_bytes(self._ref))
        if pool is not None:
            device = pool.device
        self.pool = self._tensor("pool", pool, (a.layers, a.pages, self.page_bytes), torch.uint8, 0, device)
        self.device = self.pool.device
        self._index = self.device.index
        self.table = self._tensor("table", table, (a.seqs, a.max_pages), torch.int32, -1, self.device)
        self.lens = self._tensor("lens", lens, (a.seqs,), torch.int32, 0, self.device)
        self.refs = self._tensor("refs", refs, (a.pages,), torch.int32, 0, self.device)
        n = int(self._lib.moe_kv4_workspace_bytes(self._ref))
        self._ws = torch.empty(n + 256, dtype=torch.uint8, device=self.device)
        a.pool, a.table, a.lens, a.refs = (t.data_ptr() for t in (self.pool, self.table, self.lens, self.refs))
        a.workspace = self._ws.data_ptr() + (-self._ws.data_ptr()) % 256
        a.workspace_bytes = n
        self._call("moe_kv4_workspace_init", None)
        self.kv_heads, self.head_dim, self.seqs = a.kv_heads, a.head_dim, a.seqs
        self._default_scale = 1.0 / math.sqrt(a.head_dim)
        self._attend, self._append, self._read = (self._lib.moe_kv4_attend, self._lib.moe_kv4_append,
                                                  self._lib.moe_kv4_read)

    @staticmethod
    def _tensor(name, t, shape, dtype, fill, device):
        if t is None:
            return torch.full(shape, fill, dtype=dtype, device=device)
        if tuple(t.shape) != shape or t.dtype is not dtype or not t.is_contiguous() or not t.is_cuda or \
                t.device != torch.device(device):
            raise ValueError(f"{name}: contiguous {list(shape)} of {dtype} on {device}")
        return t

    def _call(self, fn, stream, *args):
        rc = getattr(self._lib, fn)(self._ref, *args, _raw_stream(self._index, stream))
        if rc != 0:
            raise _lib.MoeError(fn, rc)

    def _new(self, make, shape, dtype, stream):
        """A result that the call makes: of the stream that it runs on, as whose its memory is filled and given back."""
        if stream is None:
            return make(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return make(shape, dtype=dtype, device=self.device)

    def _ints(self, name, t, n):
        if t.dtype is not torch.int32 or t.get_device() != self._index or not t.is_contiguous() or t.dim() != 1 or \
                (n is not None and t.shape[0] != n):
            raise ValueError(f"{name}: contiguous int32{'' if n is None else f' [{n}]'} on {self.device}")
        return t.data_ptr()

    def _rows(self, name, t, heads):
        """Type code, strides and rows of a [rows, heads, head_dim] tensor whose channels are consecutive."""
        dtype = _DTYPES.get(t.dtype)
        shape, stride = t.shape, t.stride()
        if dtype is None or len(shape) != 3 or shape[2] != self.head_dim or (heads and shape[1] != heads) or \
                stride[2] != 1 or t.get_device() != self._index:
            raise ValueError(f"{name}: [rows, {heads or 'heads'}, {self.head_dim}] of bfloat16 or float16 on "
                             f"{self.device} with consecutive channels")
        return dtype, stride[0], stride[1], shape[0]

    def append(self, layer, k, v, cu_rows, stream=None):
        """Quantise the step's K and V rows, [rows, kv_heads, head_dim] of bfloat16 or float16, into
        the pages (row and head strides multiples of 8)."""
        dtype, k_row, k_head, rows = self._rows("k", k, self.kv_heads)
        v_dtype, v_row, v_head, v_rows = self._rows("v", v, self.kv_heads)
        if v_dtype != dtype or v_rows != rows:
            raise ValueError("k and v: of one type and as many rows")
        rc = self._append(self._ref, layer, k.data_ptr(), k_row, k_head, v.data_ptr(), v_row, v_head, dtype,
                          self._ints("cu_rows", cu_rows, self.seqs + 1), rows, _raw_stream(self._index, stream))
        if rc != 0:
            raise _lib.MoeError("moe_kv4_append", rc)

    def read(self, layer, cu_rows, rows=None, dtype=torch.bfloat16, out=None, stream=None):
        """The values held for the step's rows: (k, v), [rows, kv_heads, head_dim] each, in `out` if
        given (a pair of contiguous tensors), else new ones of `rows` rows and `dtype`."""
        if out is None:
            if rows is None:
                raise ValueError("rows or out is needed")
            out = tuple(self._new(torch.zeros, (rows, self.kv_heads, self.head_dim), dtype, stream) for _ in range(2))
        k, v = out
        code, _, _, n = self._rows("out[0]", k, self.kv_heads)
        v_code, _, _, v_n = self._rows("out[1]", v, self.kv_heads)
        if v_code != code or v_n != n or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("out: two contiguous tensors of one type and as many rows")
        rc = self._read(self._ref, layer, k.data_ptr(), v.data_ptr(), code, self._ints("cu_rows", cu_rows, self.seqs + 1),
                        n, _raw_stream(self._index, stream))
        if rc != 0:
            raise _lib.MoeError("moe_kv4_read", rc)
        return out

    def attend(self, layer, q, cu_rows, max_rows, scale=None, window=0, tree=None, out=None, lse=None, stream=None):
        """Attention of the step's query rows, q [rows, q_heads, head_dim], over their sequences'
        tokens.  max_rows: the largest number of rows of a sequence, as far as the host knows; scale
        (default head_dim ** -0.5); window > 0: a row sees that many tokens back, itself included;
        tree [rows] int64: bit j set where the row sees the step's token j.  Returns out (like q,
        contiguous), or (out, lse) if lse [rows, q_heads] float32 is given."""
        dtype, q_row, q_head, rows = self._rows("q", q, None)
        heads = q.shape[1]
        if out is None:
            out = self._new(torch.empty, (rows, heads, self.head_dim), q.dtype, stream)
        elif out.shape != q.shape or out.dtype is not q.dtype or out.get_device() != self._index or not out.is_contiguous():
            raise ValueError("out: contiguous, of q's shape and type")
        if lse is not None and (lse.shape != (rows, heads) or lse.dtype is not torch.float32 or
                                lse.get_device() != self._index or not lse.is_contiguous()):
            raise ValueError("lse: contiguous [rows, q_heads] of float32")
        if tree is not None and (tree.dtype is not torch.int64 or tree.shape != (rows,) or
                                 tree.get_device() != self._index or not tree.is_contiguous()):
            raise ValueError("tree: contiguous [rows] of int64")
        rc = self._attend(self._ref, layer, q.data_ptr(), q_row, q_head, heads, dtype,
                          self._ints("cu_rows", cu_rows, self.seqs + 1), rows, max_rows,
                          self._default_scale if scale is None else scale, window,
                          None if tree is None else tree.data_ptr(), out.data_ptr(),
                          None if lse is None else lse.data_ptr(), _raw_stream(self._index, stream))
        if rc != 0:
            raise _lib.MoeError("moe_kv4_attend", rc)
        return out if lse is None else (out, lse)

    def reserve(self, new_tokens, stream=None):
        """Room for new_tokens[s] more tokens of every sequence ([seqs] int32 on the device): lens grows,
        pages are added, and a shared page that the step will write is replaced by a copy.  A sequence that
        gets no room (KV4_NO_PAGE) keeps its lens, and the step's calls leave its rows out."""
        self._call("moe_kv4_reserve", stream, self._ints("new_tokens", new_tokens, self.seqs))

    def fork(self, src, dst, stream=None):
        """Sequence dst[i] becomes a copy of sequence src[i], sharing its pages (int32, on the device)."""
        n = src.shape[0]
        self._call("moe_kv4_fork", stream, self._ints("src", src, None), self._ints("dst", dst, n), n)

    def trim(self, to_tokens, stream=None):
        """Cut every sequence to at most to_tokens[s] tokens (0 frees it)."""
        self._call("moe_kv4_trim", stream, self._ints("to_tokens", to_tokens, self.seqs))

    def compact(self, keep, cu_rows, max_rows, stream=None):
        """Keep the step's rows with keep[r] != 0 ([rows] uint8): they move together on every layer and
        every sequence is cut to them.  At most 64 rows a sequence."""
        if keep.dtype is not torch.uint8 or keep.dim() != 1 or keep.device != self.device or not keep.is_contiguous():
            raise ValueError(f"keep: contiguous [rows] of uint8 on {self.device}")
        self._call("moe_kv4_compact", stream, keep.data_ptr(), self._ints("cu_rows", cu_rows, self.seqs + 1),
                   keep.shape[0], max_rows)

    def status(self, clear=True, stream=None):
        """The cache's status bits (KV4_*), waiting for the stream."""
        bits = ctypes.c_uint32(0)
        rc = self._lib.moe_kv4_read_status(self._ref, 1 if clear else 0, ctypes.byref(bits), _raw_stream(self._index, stream))
        if rc not in (_lib.MOE_OK, _lib.MOE_ERR_DEVICE):
            raise _lib.MoeError("moe_kv4_read_status", rc)
        return int(bits.value)


def selftest_kv4_attend(cache, layer, q, cu_rows, max_rows, out, stuck, wait_limit_cycles, stream=None):
    """cache.attend(layer, q, cu_rows, max_rows, out=out) with every wait of the kernels limited to
    `wait_limit_cycles`, and with `stuck` the waits for copies never met (include/moe_selftest.h)."""
    dtype, q_row, q_head, rows = cache._rows("q", q, None)
    _lib._check("moe_selftest_kv4_attend", cache._lib.moe_selftest_kv4_attend(
        cache._ref, layer, q.data_ptr(), q_row, q_head, q.shape[1], dtype, cache._ints("cu_rows", cu_rows, cache.seqs + 1),
        rows, max_rows, cache._default_scale, out.data_ptr(), int(stuck), int(wait_limit_cycles), _raw_stream(cache._index, stream)))
    return out
