"""The grouped router on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_moe_decode_gb300 as m
    return m


def plain(l, bias, k, score, groups, keep, group_score, renormalise, scale):
    """ids and weights in 64 bits, and the smallest gap between keys (and group scores) that the selection
    depends on: where it is far above FP32 rounding the selection has to agree exactly."""
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    T, E = l.shape
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            m = l.max(1, keepdims=True)
            p = np.where(l == -np.inf, 0.0, np.exp(l - np.where(np.isfinite(m), m, 0.0)))
            t = p.sum(1, keepdims=True)
            s = np.divide(p, t, out=np.zeros_like(p), where=t > 0)
        key = l if score == "softmax" and bias is None else s + (0.0 if bias is None else bias)
    key = np.where(np.isnan(key), -np.inf, key)
    ids, w, gaps = np.zeros((T, k), dtype=np.int64), np.zeros((T, k)), np.full(T, np.inf)
    size = E // groups
    for t in range(T):
        kk = key[t].copy()
        if keep < groups:
            g = kk.reshape(groups, size)
            top = -np.sort(-g, axis=1)
            gs = top[:, 0] + top[:, 1] if group_score == "top2" and size > 1 else top[:, 0]
            gs = np.where(np.isnan(gs), -np.inf, gs)
            order = sorted(range(groups), key=lambda i: (-gs[i], i))
            a, b = gs[order[keep - 1]], gs[order[keep]]
            if np.isfinite(a) and np.isfinite(b) and a != b:
                gaps[t] = min(gaps[t], (a - b) / max(abs(a), abs(b)))
            allowed = [e for i in sorted(order[:keep]) for e in range(i * size, (i + 1) * size)]
        else:
            allowed = list(range(E))
        order = sorted(allowed, key=lambda e: (-kk[e], e))
        ids[t] = order[:k]
        v = kk[order[:k + 1]]
        v = v[np.isfinite(v)]
        d = v[:-1] - v[1:]
        d = d[d != 0] / np.maximum(np.abs(v[:-1]), np.abs(v[1:]))[d != 0]
        if len(d):
            gaps[t] = min(gaps[t], d.min())
        w[t] = s[t, ids[t]]
        if renormalise:
            w[t] = scale * w[t] / w[t].sum() if w[t].sum() > 0 else 0.0
        else:
            w[t] *= scale
    return ids, w, gaps


def check(moe, logits, bias, k, score, groups=1, keep=None, group_score="max", renormalise=True, scale=1.0):
    keep = keep or groups
    T, E = logits.shape
    r = moe.Routing(E, k, score=score, groups=groups, keep_groups=keep, group_score=group_score, renormalise=renormalise,
                    scale=scale)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, dtype=torch.float32, device="cuda")
    r.route(logits, bias, ids, w)
    want_ids, want_w, gaps = plain(logits.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy(), k,
                                   score, groups, keep, group_score, renormalise, scale)
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    sure = gaps > 1e-5
    assert sure.mean() > 0.9
    assert np.array_equal(ids[sure], want_ids[sure])
    # score: exp to 2 ulp, one addition, one division (softmax: a sum of E terms, exp of a difference of
    # logits up to 2^8 with 2^-24 relative error); weight: a sum of k and a division
    tol = 2.0 ** -24 * (12 + 2 * k + (E / 32 + 20 if score == "softmax" else 0))
    assert (np.abs(w - want_w)[sure] <= tol * np.abs(want_w)[sure] + 1e-37).all()
    return ids, w


@pytest.mark.parametrize("E,groups,keep", [(512, 8, 4), (256, 8, 4), (160, 8, 3), (64, 1, 1), (96, 3, 2), (512, 16, 5), (1024, 32, 8),
                                           (17, 1, 1), (34, 17, 9), (40, 5, 2), (30, 30, 11), (320, 4, 4)])
@pytest.mark.parametrize("score,group_score", [("sigmoid", "top2"), ("softmax", "max"), ("sigmoid", "max")])
def test_shapes(moe, E, groups, keep, score, group_score):
    g = torch.Generator().manual_seed(E + groups)
    T, k = 37, min(8, keep * E // groups)
    logits = torch.randn((T, E), generator=g).cuda()
    bias = (0.1 * torch.randn(E, generator=g)).cuda() if score == "sigmoid" else None
    check(moe, logits, bias, k, score, groups, keep, group_score, scale=2.5)


@pytest.mark.parametrize("E,groups,keep", [(512, 8, 4), (64, 16, 3), (40, 5, 2), (96, 3, 1), (1024, 32, 8), (24, 24, 9)])
def test_softmax_groups_ranked_by_two_scores(moe, E, groups, keep):
    # the sum is of scores, whether there is a bias of zeros or none: a sum of logits would rank groups by the product
    g = torch.Generator().manual_seed(E)
    logits = (2 * torch.randn((64, E), generator=g)).cuda()
    k = min(6, keep * E // groups)
    with_zeros = check(moe, logits, torch.zeros(E, device="cuda"), k, "softmax", groups, keep, "top2")
    r = moe.Routing(E, k, score="softmax", groups=groups, keep_groups=keep, group_score="top2")
    ids, w = torch.empty((64, k), dtype=torch.int32, device="cuda"), torch.empty((64, k), device="cuda")
    r.route(logits, None, ids, w)
    assert np.array_equal(ids.cpu().numpy(), with_zeros[0]) and np.array_equal(w.double().cpu().numpy(), with_zeros[1])
    # by hand: scores e^5 + e^-5 against e + e
    two = torch.tensor([[1.0, 1.0, 5.0, -5.0]], device="cuda")
    ids, w = torch.empty((1, 2), dtype=torch.int32, device="cuda"), torch.empty((1, 2), device="cuda")
    moe.Routing(4, 2, score="softmax", groups=2, keep_groups=1, group_score="top2").route(two, None, ids, w)
    assert ids.tolist() == [[2, 3]]


@pytest.mark.parametrize("E,offset", [(512, 1), (512, 4), (100, 3), (500, 4)])
def test_bias_alignment(moe, E, offset):
    g = torch.Generator().manual_seed(E + offset)
    logits = torch.randn((37, E), generator=g).cuda()
    bias = (0.1 * torch.randn(E + offset, generator=g)).cuda()[offset:]
    check(moe, logits, bias, 8, "sigmoid", 4, 2, "top2")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("stride", [0, 1, 8])
def test_types_and_strides(moe, dtype, stride):
    g = torch.Generator().manual_seed(stride)
    wide = (2 * torch.randn((21, 128 + stride), generator=g)).to(dtype).cuda()
    logits = wide[:, stride:] if stride == 1 else wide[:, :128]
    check(moe, logits, None, 6, "softmax", renormalise=False, scale=0.5)
    check(moe, logits, (0.2 * torch.randn(128, generator=g)).cuda(), 6, "sigmoid", 4, 2, "top2")


@pytest.mark.parametrize("T", [1, 3, 5, 4097])
def test_token_counts_and_all_experts(moe, T):
    g = torch.Generator().manual_seed(T)
    logits = torch.randn((T, 64), generator=g).cuda()
    check(moe, logits[:300], None, 32, "softmax")
    r = moe.Routing(64, 4, score="sigmoid")
    ids, w = torch.empty((T, 4), dtype=torch.int32, device="cuda"), torch.empty((T, 4), device="cuda")
    r.route(logits, None, ids, w)
    assert np.array_equal(ids.cpu().numpy(), torch.sort(logits.cpu(), dim=1, descending=True, stable=True).indices[:, :4].numpy())
    check(moe, torch.randn((9, 8), generator=g).cuda(), None, 8, "sigmoid", 2, 2, "top2")


def test_ties_go_to_the_lower_index(moe):
    logits = torch.zeros((5, 256), device="cuda")
    logits[1, 100:140] = 1.0
    logits[2] = 300.0   # sigmoid saturates at 1
    logits[3, ::2] = -0.0
    logits[4] = torch.arange(256, device="cuda").float() // 64
    for score, gs in (("sigmoid", "top2"), ("softmax", "max")):
        ids, _ = check(moe, logits, None, 10, score, 8, 3, gs)
        assert list(ids[0]) == list(range(10)) and list(ids[2]) == list(range(10)) and list(ids[3]) == list(range(10))
        assert list(ids[1]) == list(range(100, 110)) and list(ids[4]) == list(range(192, 202))


def test_extreme_logits_and_biases(moe):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    g = torch.Generator().manual_seed(1)
    logits = torch.randn((8, 128), generator=g).cuda()
    logits[0, :] = -inf
    logits[1, 5:] = -inf
    logits[2, ::3] = nan
    logits[3, 7] = inf
    logits[4, :] = low
    logits[5, 3:] = low
    logits[6, :] = nan
    bias = torch.zeros(128, device="cuda")
    for score in ("sigmoid", "softmax"):
        _, w = check(moe, logits, None, 8, score)
        assert np.isfinite(w).all()
        bias[:64], bias[100] = -inf, nan
        _, w = check(moe, logits, bias, 8, score, 4, 3, "top2")
        assert np.isfinite(w).all()
        bias.zero_()


def test_fp32_selection_is_reproducible_by_the_same_operations(moe):
    # the scores as written, each operation rounded once in FP32, give the same selection on every row
    g = torch.Generator().manual_seed(3)
    T, E, k, groups, keep = 4096, 512, 10, 8, 4
    logits, bias = torch.randn((T, E), generator=g).cuda(), (0.1 * torch.randn(E, generator=g)).cuda()
    r = moe.Routing(E, k, score="sigmoid", groups=groups, keep_groups=keep, group_score="top2")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    r.route(logits, bias, ids, w)
    key = 1.0 / (1.0 + torch.exp(-logits)) + bias
    top = key.reshape(T, groups, -1).sort(dim=-1, descending=True, stable=True).values
    kept = (top[..., 0] + top[..., 1]).sort(dim=-1, descending=True, stable=True).indices[:, :keep]
    allowed = torch.zeros((T, groups), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
    key = key.masked_fill(~allowed.repeat_interleave(E // groups, 1), -float("inf"))
    assert torch.equal(ids.long(), key.sort(dim=-1, descending=True, stable=True).indices[:, :k])


def test_feeds_the_plan_and_the_experts(moe):
    # grouped routing, then plan and experts, equals the layer's own path when the selection is the same
    import moe_inputs as mi
    from gpu_helpers import bf16_tensor, device_weights
    cfg = mi.CONFIGS["tiny"]
    inp = mi.gen_layer(cfg, seed=0)
    w = device_weights(inp, "cuda")
    logits, hidden = torch.from_numpy(inp["logits"]).cuda(), bf16_tensor(inp["hidden"], "cuda")
    layer = moe.MoeLayer(cfg.T, cfg.d, cfg.ffn, cfg.E, cfg.k)
    want = layer(logits, hidden, w)
    ids, wts = layer.ids.clone(), layer.weights.clone()
    moe.Routing(cfg.E, cfg.k, score="softmax").route(logits, None, layer.ids, layer.weights)
    assert torch.equal(ids, layer.ids) and torch.allclose(wts, layer.weights, rtol=1e-6)
    layer.plan()
    assert torch.allclose(layer.experts(hidden, w).float(), want.float(), rtol=2.0 ** -7, atol=1e-3)


def test_refusals(moe):
    for kw in (dict(E=12, k=2, groups=5), dict(E=16, k=6, groups=4, keep_groups=1), dict(E=16, k=0), dict(E=16, k=17),
               dict(E=16, k=2, groups=4, keep_groups=5)):
        with pytest.raises(moe.MoeError):
            moe.Routing(**kw)
    with pytest.raises(moe.MoeError):
        moe.Routing(2048, 8)
    with pytest.raises(ValueError):
        moe.Routing(16, 2, score="tanh")
    r = moe.Routing(16, 2)
    l = torch.zeros((3, 16), device="cuda")
    ids, w = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    for bad in (l.double(), l[:, :8], l.t().contiguous().t()):
        with pytest.raises(ValueError):
            r.route(bad, None, ids, w)
    with pytest.raises(ValueError):
        r.route(l, torch.zeros(15, device="cuda"), ids, w)
    with pytest.raises(ValueError):
        r.route(l, None, ids.long(), w)
    with pytest.raises(ValueError):
        r.route(l, None, ids[:2], w)
    r.route(l[:0], None, ids[:0], w[:0])
