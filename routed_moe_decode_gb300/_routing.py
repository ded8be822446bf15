"""Routing: the grouped router (sigmoid or softmax scores, selection bias, expert groups)."""
from __future__ import annotations

import ctypes

import torch

from . import _lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


_devices = 0  # CUDA devices that there are, counted at the first call


def _raw_stream(index, stream=None):
    """The handle of `stream`, or of the current stream, for a call on tensors of CUDA device `index`.  A launch goes to
    the current device (handle 0 is that device's default stream), so another device than the tensors' is refused;
    where there is one device it is not asked for, which takes 0.2 us."""
    global _devices
    if _devices != 1:
        _devices = _devices or torch.cuda.device_count()
        current = torch.cuda.current_device()
        if current != index:
            raise ValueError(f"the tensors lie on cuda:{index} and the current device is cuda:{current}: call it under "
                             f"torch.cuda.device({index})")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device.index != index:
        raise ValueError(f"the tensors lie on cuda:{index} and the stream is one of {stream.device}")
    return stream.cuda_stream


class Routing:
    """How a layer selects and weights its experts (moe_route_grouped in include/moe.h).

    E experts, k of them per token; score "sigmoid" or "softmax"; `groups` consecutive groups of
    E / groups experts, of which the `keep_groups` best (group_score "max": their largest key,
    "top2": the sum of their two largest) stay in the selection; renormalise: the weights are
    divided by their sum; scale multiplies them.
    """

    def __init__(self, E, k, score="softmax", groups=1, keep_groups=None, group_score="max", renormalise=True,
                 scale=1.0):
        if score not in ("softmax", "sigmoid"):
            raise ValueError(f"score is 'softmax' or 'sigmoid', not {score!r}")
        if group_score not in ("max", "top2"):
            raise ValueError(f"group_score is 'max' or 'top2', not {group_score!r}")
        self.E, self.k = int(E), int(k)
        self._args = _lib.RoutingArgs(self.E, self.k, int(score == "softmax"), int(groups),
                                      int(groups if keep_groups is None else keep_groups), int(group_score == "top2"),
                                      int(bool(renormalise)), float(scale))
        self._ref = ctypes.byref(self._args)
        self._route = _lib.lib().moe_route_grouped
        _lib._check("moe_route_grouped", self._route(self._ref, 0, None, self.E, 0, None, None, None, None))

    def route(self, logits, bias, ids, weights, stream=None):
        """logits [T, E] (float32, bfloat16 or float16, rows may be strided) and bias [E] float32 or
        None to ids [T, k] int32 and weights [T, k] float32, both contiguous."""
        T, E = logits.shape
        dtype = _DTYPES.get(logits.dtype)
        if dtype is None or E != self.E or (E > 1 and logits.stride(1) != 1):
            raise ValueError(f"logits: [T, {self.E}] of float32, bfloat16 or float16 with consecutive columns")
        if ids.dtype is not torch.int32 or weights.dtype is not torch.float32 or \
                ids.shape != (T, self.k) or weights.shape != (T, self.k) or \
                not ids.is_contiguous() or not weights.is_contiguous():
            raise ValueError(f"ids, weights: contiguous [{T}, {self.k}] of int32 and float32")
        if bias is not None and (bias.dtype is not torch.float32 or bias.shape != (E,) or not bias.is_contiguous()):
            raise ValueError(f"bias: contiguous [{E}] of float32")
        index = logits.get_device()
        if index < 0 or ids.get_device() != index or weights.get_device() != index or \
                (bias is not None and bias.get_device() != index):
            raise ValueError("logits, bias, ids and weights lie on one CUDA device")
        rc = self._route(self._ref, T, logits.data_ptr(), logits.stride(0) if T > 1 else E, dtype,
                         None if bias is None else bias.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                         _raw_stream(index, stream))
        if rc != 0:
            raise _lib.MoeError("moe_route_grouped", rc)
        return ids, weights
