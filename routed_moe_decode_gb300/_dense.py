"""The dense path in 8 bits: RmsNorm, quantize_rows, Fp8Linear and token_logprobs (include/moe_dense.h)."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._routing import _DTYPES, _raw_stream

_quantize_rows = _token_logprobs = None  # the library's functions, looked up at the first call

DENSE_BAD_OFFSETS = 0x1
DENSE_TIMEOUT = 0x2

_E4M3 = torch.float8_e4m3fn


def _empty(shape, dtype, device, stream):
    """A result that a call makes: of the stream that it runs on, as whose its memory is given back."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class Fp8Rows:
    """Rows in 8 bits: codes [rows, k] float8_e4m3fn (consecutive channels) and scales [rows, ceil(k / 128)] float32
    with any strides; value = code * scale of its row and block of 128 channels."""

    __slots__ = ("codes", "scales", "device", "_index")

    def __init__(self, codes, scales):
        if codes.dtype is not _E4M3 or codes.dim() != 2 or (codes.shape[1] > 1 and codes.stride(1) != 1) or not codes.is_cuda:
            raise ValueError("codes: [rows, k] of float8_e4m3fn on a CUDA device with consecutive channels")
        if scales.dtype is not torch.float32 or scales.shape != (codes.shape[0], -(-codes.shape[1] // 128)) or \
                scales.device != codes.device:
            raise ValueError(f"scales: [{codes.shape[0]}, {-(-codes.shape[1] // 128)}] of float32 on {codes.device}")
        self.codes, self.scales, self.device, self._index = codes, scales, codes.device, codes.get_device()

    @classmethod
    def empty(cls, rows, k, device="cuda", stream=None):
        """Rows to be written: code rows a multiple of 16 bytes apart, a block's scales together (as the products
        read them best)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return cls.empty(rows, k, device)
        self = object.__new__(cls)
        if k % 16:
            codes = torch.empty((rows, -(-k // 16) * 16), dtype=_E4M3, device=device)
            self.codes = codes[:, :k]
        else:
            self.codes = codes = torch.empty((rows, k), dtype=_E4M3, device=device)
        self.scales = torch.empty_strided((rows, -(-k // 128)), (1, rows), dtype=torch.float32, device=device)
        self.device, self._index = codes.device, codes.get_device()
        return self


def _rows_to_write(out, rows, k, index):
    if out.codes.shape != (rows, k) or out._index != index:
        raise ValueError(f"8-bit rows: [{rows}, {k}] on cuda:{index}")
    return out


def _same_place(out, out_strides, of, of_strides):
    """An output in an input's place has its strides (those of a dimension of one element say nothing)."""
    if of is not None and out_strides != of_strides and out.data_ptr() == of.data_ptr() and out.numel() and \
            any(n > 1 and a != b for n, a, b in zip(out.shape, out_strides, of_strides)):
        raise ValueError("an output in an input's place has its strides")


class RmsNorm:
    """Root-mean-square norm, with the residual's addition before it and rows in 8 bits after it (moe_rms_norm).

    weight [d] float32, bfloat16 or float16; one_plus: multiplies by 1 + weight.
    """

    def __init__(self, weight, eps=1e-6, one_plus=False):
        if weight.dim() != 1 or weight.dtype not in _DTYPES or not weight.is_contiguous() or not weight.is_cuda:
            raise ValueError("weight: contiguous [d] of float32, bfloat16 or float16 on a CUDA device")
        self.weight, self.eps, self.one_plus = weight, float(eps), bool(one_plus)
        self.d, self._index = weight.shape[0], weight.get_device()
        self._weight_dtype = _DTYPES[weight.dtype]
        self._norm = _lib.lib().moe_rms_norm

    def __call__(self, x, residual=None, normed=True, residual_out=None, quantize=False, stream=None):
        """x [rows, d] or [outer, inner, d] (consecutive channels, any other strides) of float32, bfloat16 or float16.
        Returns (normed, residual_out, rows in 8 bits), each None where it is not made:
          normed: True for a new tensor, a tensor of x's shape and type to write (x or the residual itself, if
            need be), False for none;
          residual [rows, d] of x's type: h = x + residual is what is normed, and residual_out (a new tensor, or the one
            given, which may be x or the residual) receives it; residual_out=False: it is not written;
          quantize: True for new Fp8Rows of [rows, d] (outer * inner rows), Fp8Rows to write, False for none.
        """
        d, index, shape, strides = self.d, self._index, x.shape, x.stride()
        dtype, dims = _DTYPES.get(x.dtype), len(shape)
        if dtype is None or not 2 <= dims <= 3 or shape[-1] != d or (strides[-1] != 1 and d > 1) or x.get_device() != index:
            raise ValueError(f"x: [rows, {d}] or [outer, inner, {d}] of float32, bfloat16 or float16 on cuda:{index} with "
                             "consecutive channels")
        outer, inner = shape[0], shape[1] if dims == 3 else 1
        x_inner = strides[1] if dims == 3 else 0
        residual_ptr = sum_ptr = normed_ptr = codes_ptr = scales_ptr = None
        r_stride = ro_stride = n_outer = n_inner = code_stride = scale_row = scale_block = 0
        if residual is not None:
            if residual.dtype is not x.dtype or residual.shape != shape or dims != 2 or \
                    (residual.stride(1) != 1 and d > 1) or residual.get_device() != index:
                raise ValueError(f"residual: of x's type and shape, which is [rows, {d}], with consecutive channels")
            residual_ptr, r_stride = residual.data_ptr(), residual.stride(0)
            if residual_out is None:
                residual_out, ro_stride = torch.empty(shape, dtype=x.dtype, device=x.device) if stream is None else \
                    _empty(shape, x.dtype, x.device, stream), d
                sum_ptr = residual_out.data_ptr()
            elif residual_out is False:
                residual_out = None
            else:
                if residual_out.dtype is not x.dtype or residual_out.shape != shape or \
                        (residual_out.stride(1) != 1 and d > 1) or residual_out.get_device() != index:
                    raise ValueError(f"residual_out: of x's type and shape with consecutive channels on cuda:{index}")
                _same_place(residual_out, residual_out.stride(), x, strides)
                _same_place(residual_out, residual_out.stride(), residual, residual.stride())
                sum_ptr, ro_stride = residual_out.data_ptr(), residual_out.stride(0)
        elif residual_out is not None and residual_out is not False:
            raise ValueError("residual_out needs a residual")
        else:
            residual_out = None
        if normed is True:
            normed, n_outer, n_inner = torch.empty(shape, dtype=x.dtype, device=x.device) if stream is None else \
                _empty(shape, x.dtype, x.device, stream), inner * d, d
            normed_ptr = normed.data_ptr()
        elif normed is False or normed is None:
            normed = None
        else:
            to = normed.stride()
            if normed.dtype is not x.dtype or normed.shape != shape or (to[-1] != 1 and d > 1) or normed.get_device() != index:
                raise ValueError(f"normed: of x's type and shape with consecutive channels on cuda:{index}")
            _same_place(normed, to, x, strides)
            if residual is not None:
                _same_place(normed, to, residual, residual.stride())
            normed_ptr, n_outer, n_inner = normed.data_ptr(), to[0], to[1] if dims == 3 else 0
        fp8 = None
        if quantize is not False and quantize is not None:
            rows = outer * inner
            fp8 = Fp8Rows.empty(rows, d, x.device, stream) if quantize is True else _rows_to_write(quantize, rows, d, index)
            codes_ptr, scales_ptr, code_stride = fp8.codes.data_ptr(), fp8.scales.data_ptr(), fp8.codes.stride(0)
            scale_row, scale_block = fp8.scales.stride()
        rc = self._norm(outer, inner, d, dtype, x.data_ptr(), strides[0], x_inner, residual_ptr, r_stride,
                        self.weight.data_ptr(), self._weight_dtype, self.one_plus, self.eps, sum_ptr, ro_stride, normed_ptr, n_outer, n_inner,
                        codes_ptr, code_stride, scales_ptr, scale_row, scale_block, _raw_stream(index, stream))
        if rc != 0:
            raise _lib.MoeError("moe_rms_norm", rc)
        return normed, residual_out, fp8


def quantize_rows(x, gated=False, out=None, stream=None):
    """x [rows, d] of float32, bfloat16 or float16 (consecutive channels) as Fp8Rows (in `out`, if given); gated: x is
    [rows, 2 d], gate then up, and silu(gate) * up is quantised."""
    dtype, index, (row, channel) = _DTYPES.get(x.dtype), x.get_device(), x.stride() if x.dim() == 2 else (0, 0)
    rows, d = x.shape if x.dim() == 2 else (0, 0)
    if dtype is None or x.dim() != 2 or (channel != 1 and d > 1) or index < 0 or (gated and d % 2):
        raise ValueError("x: [rows, d] (gated: [rows, 2 d]) of float32, bfloat16 or float16 on a CUDA device with "
                         "consecutive channels")
    if gated:
        d //= 2
    global _quantize_rows
    if _quantize_rows is None:
        _quantize_rows = _lib.lib().moe_quantize_rows
    out = Fp8Rows.empty(rows, d, x.device, stream) if out is None else _rows_to_write(out, rows, d, index)
    scale_row, scale_block = out.scales.stride()
    rc = _quantize_rows(rows, d, 1 if gated else 0, dtype, x.data_ptr(), row, out.codes.data_ptr(),
                        out.codes.stride(0), out.scales.data_ptr(), scale_row, scale_block, _raw_stream(index, stream))
    if rc != 0:
        raise _lib.MoeError("moe_quantize_rows", rc)
    return out


class Fp8Linear:
    """Products with a block-scaled 8-bit weight (moe_fp8_matmul): codes [n, k] float8_e4m3fn and scales
    [ceil(n / 128), ceil(k / 128)] float32, or one weight for each group of rows, codes [groups, n, k] and
    scales [groups, ceil(n / 128), ceil(k / 128)]; both contiguous, k a multiple of 16.
    """

    def __init__(self, codes, scales):
        if codes.dtype is not _E4M3 or codes.dim() not in (2, 3) or not codes.is_contiguous() or not codes.is_cuda:
            raise ValueError("codes: contiguous [n, k] or [groups, n, k] of float8_e4m3fn on a CUDA device")
        self.n, self.k = codes.shape[-2:]
        self.groups = codes.shape[0] if codes.dim() == 3 else 0
        shape = codes.shape[:-2] + (-(-self.n // 128), -(-self.k // 128))
        if scales.dtype is not torch.float32 or scales.shape != shape or not scales.is_contiguous() or \
                scales.device != codes.device:
            raise ValueError(f"scales: contiguous {list(shape)} of float32 on {codes.device}")
        if codes.dim() == 3 and self.groups == 0:
            raise ValueError("no groups")
        self.codes, self.scales, self.device, self._index = codes, scales, codes.device, codes.get_device()
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        if not torch.cuda.is_current_stream_capturing():  # products of other streams may set it from now on
            torch.cuda.current_stream(self.device).synchronize()
        self._matmul = _lib.lib().moe_fp8_matmul
        # an empty product: what the library thinks of the sizes
        _lib._check("moe_fp8_matmul", self._matmul(0, self.n, self.k, self.groups, None, 0, None, 0, 0, None, None, None,
                                                   None, 0, 0, None, None))

    def __call__(self, x, offsets=None, out=None, dtype=torch.bfloat16, stream=None):
        """x: Fp8Rows [rows, k]; the product [rows, n] in `out` (consecutive channels) if given, else a new tensor of
        `dtype`.  With groups, offsets [groups + 1] int32 on the device: rows offsets[g] .. offsets[g + 1] - 1 meet weight
        g; rows of no group are left as they were."""
        index, n = self._index, self.n
        rows, k = x.codes.shape
        if k != self.k or x._index != index:
            raise ValueError(f"x: [rows, {self.k}] on cuda:{index}")
        if out is None:
            out, out_stride = torch.empty((rows, n), dtype=dtype, device=self.device) if stream is None else \
                _empty((rows, n), dtype, self.device, stream), n
        else:
            out_stride, channel = out.stride() if out.dim() == 2 else (0, 0)
            if out.shape != (rows, n) or (channel != 1 and n > 1) or out.get_device() != index:
                raise ValueError(f"out: [{rows}, {n}] with consecutive channels on cuda:{index}")
        out_dtype = _DTYPES.get(out.dtype)
        if out_dtype is None:
            raise ValueError("out is of float32, bfloat16 or float16")
        if self.groups:
            if offsets is None or offsets.dtype is not torch.int32 or offsets.shape != (self.groups + 1,) or \
                    not offsets.is_contiguous() or offsets.get_device() != index:
                raise ValueError(f"offsets: contiguous int32 [{self.groups + 1}] on cuda:{index}")
            offsets = offsets.data_ptr()
        elif offsets is not None:
            raise ValueError("offsets need a weight with groups")
        scale_row, scale_block = x.scales.stride()
        rc = self._matmul(rows, n, k, self.groups, x.codes.data_ptr(), x.codes.stride(0), x.scales.data_ptr(), scale_row,
                          scale_block, self.codes.data_ptr(), self.scales.data_ptr(), offsets, out.data_ptr(), out_stride,
                          out_dtype, self._status.data_ptr(), _raw_stream(index, stream))
        if rc != 0:
            raise _lib.MoeError("moe_fp8_matmul", rc)
        return out

    def status(self, clear=True, stream=None):
        """The status bits (DENSE_*) of the products that are ordered before this call on the stream, and of others that ran by then;
        waits for the stream.  A bit that a product of another stream sets meanwhile is in this result or in the next."""
        bits = ctypes.c_uint32(0)
        rc = _lib.lib().moe_dense_read_status(self._status.data_ptr(), 1 if clear else 0, ctypes.byref(bits),
                                              _raw_stream(self._index, stream))
        if rc not in (_lib.MOE_OK, _lib.MOE_ERR_DEVICE):
            raise _lib.MoeError("moe_dense_read_status", rc)
        return int(bits.value)


class TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor  # [rows, n] (or [rows]) float32
    lse: torch.Tensor       # [rows] float32
    entropy: torch.Tensor   # [rows] float32
    top_ids: Optional[torch.Tensor]       # [rows, top] int32
    top_logprobs: Optional[torch.Tensor]  # [rows, top] float32


def token_logprobs(logits, tokens, top=0, scale=1.0, stream=None):
    """Log probabilities of tokens [rows, n] or [rows] int32 under the softmax of scale * logits [rows, vocab] (float32,
    bfloat16 or float16; consecutive columns), with every row's log-sum-exp, entropy and its `top` best tokens (equal
    logits: the lower id first).  A token outside the vocabulary has log probability -infinity (moe_token_logprobs)."""
    dtype, index = _DTYPES.get(logits.dtype), logits.get_device()
    if dtype is None or logits.dim() != 2 or index < 0 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits: [rows, vocab] of float32, bfloat16 or float16 on a CUDA device with consecutive columns")
    rows, vocab = logits.shape
    shape, strides = tokens.shape, tokens.stride()
    n = shape[1] if len(shape) == 2 else 1
    if tokens.dtype is not torch.int32 or not 1 <= len(shape) <= 2 or shape[0] != rows or tokens.get_device() != index or \
            (len(shape) == 2 and strides[1] != 1 and n > 1):
        raise ValueError(f"tokens: [{rows}, n] or [{rows}] of int32 on cuda:{index} with consecutive columns")
    global _token_logprobs
    if _token_logprobs is None:
        _token_logprobs = _lib.lib().moe_token_logprobs
    device, f32 = logits.device, torch.float32
    ids = best = ids_ptr = best_ptr = None
    if stream is None:
        empty = torch.empty
        logprobs, lse, entropy = empty(shape, dtype=f32, device=device), empty(rows, dtype=f32, device=device), \
            empty(rows, dtype=f32, device=device)
        if top > 0:
            ids, best = empty((rows, top), dtype=torch.int32, device=device), empty((rows, top), dtype=f32, device=device)
    else:
        logprobs, lse, entropy = _empty(shape, f32, device, stream), _empty(rows, f32, device, stream), _empty(rows, f32, device, stream)
        if top > 0:
            ids, best = _empty((rows, top), torch.int32, device, stream), _empty((rows, top), f32, device, stream)
    if top > 0:
        ids_ptr, best_ptr = ids.data_ptr(), best.data_ptr()
    rc = _token_logprobs(rows, vocab, dtype, logits.data_ptr(), logits.stride(0), scale, tokens.data_ptr(), n, strides[0], top,
                         logprobs.data_ptr(), lse.data_ptr(), entropy.data_ptr(), ids_ptr, best_ptr, _raw_stream(index, stream))
    if rc != 0:
        raise _lib.MoeError("moe_token_logprobs", rc)
    return TokenLogprobs(logprobs, lse, entropy, ids, best)


def selftest_fp8_matmul(linear, x, out, stuck, wait_limit_cycles, offsets=None, stream=None):
    """Fp8Linear's product with its waits limited, one of them stuck if asked for (include/moe_selftest.h)."""
    scale_row, scale_block = x.scales.stride()
    _lib._check("moe_selftest_fp8_matmul", _lib.lib().moe_selftest_fp8_matmul(
        x.codes.shape[0], linear.n, linear.k, linear.groups, x.codes.data_ptr(), x.codes.stride(0), x.scales.data_ptr(),
        scale_row, scale_block, linear.codes.data_ptr(), linear.scales.data_ptr(),
        None if offsets is None else offsets.data_ptr(), out.data_ptr(), out.stride(0), _DTYPES[out.dtype],
        linear._status.data_ptr(), int(stuck), int(wait_limit_cycles), _raw_stream(linear._index, stream)))
