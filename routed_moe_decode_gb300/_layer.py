"""MoeLayer: owns the workspace and the per-call ids/weights buffers of one layer shape."""
from __future__ import annotations

import torch

from . import _lib


class MoeLayer:
    """Routed MoE layer of a fixed shape on one CUDA device.

    __call__ runs the whole layer and returns the BF16 output [T, d]: with the automatic
    kernel choice one moe_layer call (fused router + plan front for moderate T * k), else
    router, plan and experts as three C-ABI calls on the current stream.  Weights are a dict of device tensors:
    w13_codes [E, 2*ffn, d/2] uint8, w13_scales [E, 2*ffn, d/16] uint8 (E4M3),
    w2_codes [E, d, ffn/2] uint8, w2_scales [E, d, ffn/16] uint8, and the FP32 tensor
    scales w13_ts / w2_ts (Python floats).  With `routing` (a Routing of the same E and k) the
    experts are selected and weighted by it, with the call's router_bias, instead of by softmax
    top-k; the call is then router, plan and experts as three C-ABI calls.
    """

    def __init__(self, T, d, ffn, E, k, device="cuda", algo=_lib.ALGO_AUTO, routing=None):
        if routing is not None and (routing.E, routing.k) != (E, k):
            raise ValueError(f"routing selects {routing.k} of {routing.E} experts, the layer {k} of {E}")
        self.routing = routing
        self.shape = _lib.shape_of(T, d, ffn, E, k)
        rc = _lib.check_shape(self.shape)
        if rc != _lib.MOE_OK:
            raise _lib.MoeError("moe_check_shape", rc)
        self.device = torch.device(device)
        self.algo = algo
        self.ws = _lib.Workspace(self.shape, device=self.device)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=self.device)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=self.device)

    def route(self, logits, router_bias=None):
        if self.routing is not None:
            return self.routing.route(logits, router_bias, self.ids, self.weights)
        if router_bias is not None:
            raise ValueError("router_bias needs a routing")
        _lib.route_topk(self.shape, logits, self.ids, self.weights)
        return self.ids, self.weights

    def plan(self):
        _lib.plan(self.shape, self.ids, self.weights, self.ws)

    def experts(self, hidden, w, residual=None, out=None):
        if out is None:
            out = torch.empty((self.shape.T, self.shape.d), dtype=torch.bfloat16, device=self.device)
        _lib.forward(self.shape, hidden, w, residual, out, self.ws, self.algo)
        return out

    def __call__(self, logits, hidden, w, residual=None, out=None, router_bias=None):
        if self.algo == _lib.ALGO_AUTO and self.routing is None and router_bias is None:
            if out is None:
                out = torch.empty((self.shape.T, self.shape.d), dtype=torch.bfloat16, device=self.device)
            _lib.layer(self.shape, logits, hidden, w, residual, out, self.ids, self.weights, self.ws)
            return out
        self.route(logits, router_bias)
        self.plan()
        return self.experts(hidden, w, residual, out)

    def status(self, clear=True):
        return _lib.read_status(self.ws, clear)
