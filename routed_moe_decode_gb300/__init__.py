"""Routed mixture-of-experts layer (softmax top-k router, NVFP4 experts, fused un-route)
for GB300 (sm_103a): the C-ABI library libroutedmoe.so plus a thin ctypes binding.

High-level use (torch tensors on a CUDA device):

    import routed_moe_decode_gb300 as moe
    layer = moe.MoeLayer(T, d, ffn, E, k)
    out = layer(logits, hidden, weights, residual)     # weights: dict of NVFP4 tensors

    cache = moe.Kv4Cache(layers, pages, kv_heads, head_dim, page_size, seqs, max_pages)
    routing = moe.Routing(E, k, score="sigmoid", groups=8, keep_groups=4, group_score="top2")
    # a step: cache.reserve, per layer cache.append / cache.attend / MoeLayer(..., routing=routing),
    # then cache.compact (examples/verify_step.py)

    norm, linear = moe.RmsNorm(weight), moe.Fp8Linear(codes, scales)     # the dense path in 8 bits
    _, residual, rows = norm(x, residual, normed=False, quantize=True)   # also quantize_rows(x, gated=...)
    out = linear(rows)                                                   # weights of groups: linear(rows, offsets)
    scores = moe.token_logprobs(logits, tokens, top=8)

The package contains no compute of its own: every step runs in the library's kernels.
"""
from ._lib import (ALGO_AUTO, ALGO_MMA, ALGO_SIMT, ALGO_TCGEN05, ALGO_WIDE, MOE_DEV_BAD_EXPERT_ID, MOE_DEV_H_SATURATED, MOE_DEV_Y_SATURATED,
                   MOE_DEV_HIDDEN_RANGE, MOE_DEV_TIMEOUT, MoeError, Shape, Workspace, auto_algo, check_shape, forward,
                   forward_expert_kernels, forward_experts, forward_prepare, forward_unroute, front,
                   forward_experts_expert_range, layer, layer_expert_range, layer_launches, forward_unroute_gated, layer_expert_scales, layer_from_hidden, layer_gated, lib, plan, plan_expert_range, plan_summary, router_logits, selftest_expert_part, selftest_expert_timeout, plan_views, read_status, route_topk, shape_of, unroute_fused,
                   workspace_bytes)
from ._dense import (DENSE_BAD_OFFSETS, DENSE_TIMEOUT, Fp8Linear, Fp8Rows, RmsNorm, TokenLogprobs, quantize_rows,
                     selftest_fp8_matmul, token_logprobs)
from ._kv4 import KV4_BAD_PAGE, KV4_BAD_SEQ, KV4_NO_PAGE, KV4_NONFINITE, KV4_TIMEOUT, Kv4Cache, selftest_kv4_attend
from ._layer import MoeLayer
from ._routing import Routing

__all__ = ["DENSE_BAD_OFFSETS", "DENSE_TIMEOUT", "Fp8Linear", "Fp8Rows", "RmsNorm", "TokenLogprobs", "quantize_rows", "selftest_fp8_matmul", "token_logprobs", "KV4_BAD_PAGE", "KV4_BAD_SEQ", "KV4_NONFINITE", "KV4_NO_PAGE", "KV4_TIMEOUT", "Kv4Cache", "Routing", "ALGO_AUTO", "ALGO_MMA", "ALGO_SIMT", "ALGO_TCGEN05", "ALGO_WIDE", "MOE_DEV_BAD_EXPERT_ID", "MOE_DEV_H_SATURATED", "MOE_DEV_Y_SATURATED",
           "MOE_DEV_HIDDEN_RANGE", "MOE_DEV_TIMEOUT", "MoeError", "MoeLayer", "Shape", "Workspace",
           "auto_algo", "check_shape", "forward", "forward_expert_kernels", "forward_experts", "forward_prepare", "forward_unroute", "front", "forward_experts_expert_range", "layer", "layer_expert_range", "layer_launches", "forward_unroute_gated", "layer_expert_scales", "layer_from_hidden", "layer_gated", "lib", "plan", "plan_expert_range", "plan_summary", "router_logits", "selftest_expert_part", "selftest_expert_timeout", "plan_views", "read_status",
           "route_topk", "selftest_kv4_attend", "shape_of", "unroute_fused", "workspace_bytes"]
