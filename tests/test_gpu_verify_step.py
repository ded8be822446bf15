"""The operators around the routed layer as a step runs them: the example, and the layer with a routing."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv4_plain as P
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs_and_accounts_for_its_tokens(example):
    m, kept = example.main(prompts=(37, 64, 5), steps=3)
    c = m.cache
    assert c.status() == 0
    assert c.lens.tolist() == [n + k for n, k in zip((37, 64, 5, 37), kept.tolist())]
    table, refs = c.table.cpu().numpy(), c.refs.cpu().numpy()
    used = [-(-int(n) // 32) for n in c.lens.tolist()]
    for s, n in enumerate(used):
        assert (table[s, :n] >= 0).all() and (table[s, n:] == -1).all()
    assert np.array_equal(np.bincount(table[table >= 0], minlength=len(refs)), refs)
    assert table[0, 0] == table[3, 0] and table[0, 1] != table[3, 1]  # the full page is shared, the written one is not
    c.trim(torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (c.refs == 0).all()


def test_step_attends_to_what_the_cache_holds(example):
    # a step's attention equals plain attention over the values that the cache gives back
    m = example.Decoder(seqs=2, seed=3)
    c = m.cache
    gen = torch.Generator(device="cuda").manual_seed(5)
    rows = [40, 23]
    cu = torch.tensor([0, 40, 63], dtype=torch.int32, device="cuda")
    m.forward(torch.randn(63, m.d, generator=gen, device="cuda").to(torch.bfloat16), cu, torch.tensor(rows, dtype=torch.int32, device="cuda"))
    q = torch.randn(63, 8, 64, generator=gen, device="cuda").to(torch.bfloat16)
    for layer in range(m.layers):
        out = c.attend(layer, q, cu, max_rows=40).double().cpu().numpy()
        k, v = (t.double().cpu().numpy() for t in c.read(layer, cu, rows=63))
        qn = q.double().cpu().numpy()
        for s, first in enumerate((0, 40)):
            for r in (0, 7, rows[s] - 1):
                for h in range(8):
                    at = slice(first, first + r + 1)
                    ref = P.attend_row(qn[first + r, h], k[at, h // 4], v[at, h // 4], np.ones(r + 1, bool), 0.125)[0]
                    # p rounded to FP16 and the output to BF16 (tests/test_gpu_kv4.py has the terms); values up to 4
                    assert np.abs(out[first + r, h] - ref).max() <= 2.0 ** -8 * np.abs(ref).max() + 4 * 2.0 ** -10


def test_step_in_a_graph_gives_the_same(example):
    m = example.Decoder(seqs=3, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    prompt, cu0 = torch.randn(90, m.d, generator=gen, device="cuda").to(torch.bfloat16), ints([0, 30, 61, 90])
    m.forward(prompt, cu0, ints([30, 31, 29]))
    start = m.cache.lens.clone()
    x, cu, new = torch.randn(12, m.d, generator=gen, device="cuda").to(torch.bfloat16), ints([0, 4, 8, 12]), ints([4, 4, 4])
    keep = torch.tensor([1, 0, 1, 0] * 3, dtype=torch.uint8, device="cuda")

    def step():
        out = m.forward(x, cu, new)
        m.cache.compact(keep, cu, max_rows=4)
        return out

    want = step().clone()
    lens = m.cache.lens.clone()
    m.cache.trim(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # lengths and pages return to the start before the capture and the replay
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(m.cache.lens, lens) and m.cache.status() == 0


def test_layer_with_a_routing(example):
    import routed_moe_decode_gb300 as moe
    import moe_inputs as mi
    from gpu_helpers import bf16_tensor, device_weights
    cfg = mi.CONFIGS["tiny"]
    inp = mi.gen_layer(cfg, seed=0)
    w = device_weights(inp, "cuda")
    logits, hidden, res = torch.from_numpy(inp["logits"]).cuda(), bf16_tensor(inp["hidden"], "cuda"), bf16_tensor(inp["residual"], "cuda")
    bias = torch.linspace(-0.3, 0.3, cfg.E, device="cuda")
    r = moe.Routing(cfg.E, cfg.k, score="sigmoid", groups=4, keep_groups=2, group_score="top2", scale=1.5)
    layer = moe.MoeLayer(cfg.T, cfg.d, cfg.ffn, cfg.E, cfg.k, routing=r)
    out = layer(logits, hidden, w, res, router_bias=bias)
    s = 1.0 / (1.0 + torch.exp(-logits.double())) + bias.double()
    top = s.view(cfg.T, 4, -1).topk(2, -1).values.sum(-1).topk(2, -1).indices
    mask = torch.zeros(cfg.T, 4, dtype=torch.bool, device="cuda").scatter_(1, top, True).repeat_interleave(cfg.E // 4, 1)
    ids = s.masked_fill(~mask, -1e9).topk(cfg.k, -1).indices
    assert torch.equal(layer.ids.long(), ids)
    assert layer.status() == 0
    # the same experts and weights through the plain calls
    ids32, wts = layer.ids.clone(), layer.weights.clone()
    other = moe.MoeLayer(cfg.T, cfg.d, cfg.ffn, cfg.E, cfg.k)
    moe.plan(other.shape, ids32, wts, other.ws)
    assert torch.equal(other.experts(hidden, w, res), out)
    with pytest.raises(ValueError):
        moe.MoeLayer(cfg.T, cfg.d, cfg.ffn, cfg.E, cfg.k, routing=moe.Routing(2 * cfg.E, cfg.k))
    with pytest.raises(ValueError):
        other(logits, hidden, w, res, router_bias=bias)
