"""The dense path's operators together, as a step runs them: against the plain implementations, captured in graphs, on other
streams, at sizes past 32 bits, and in the example."""
import importlib.util
import os

import pytest
import torch

import dense_plain as P
from conftest import ROOT
from test_gpu_dense import BF16, FP16, FP32, NORM_REL, U, check_product, check_quantized, gen, half_step, make_weight, moe, rand  # noqa: F401

pytestmark = pytest.mark.gpu


class Block:
    """norm -> gate and up -> silu(gate) * up -> down -> residual and norm -> vocabulary -> log probabilities."""

    def __init__(self, moe, g, d, ffn, vocab, dtype=BF16):
        self.moe = moe
        self.codes = [make_weight(g, 2 * ffn, d), make_weight(g, d, ffn), make_weight(g, vocab, d)]
        self.up, self.down, self.head = (moe.Fp8Linear(c, s / (d ** 0.5 * 50)) for c, s in self.codes)
        self.norms = [moe.RmsNorm((1 + 0.1 * rand(g, d)).to(dtype)) for _ in range(2)]

    def __call__(self, x, tokens, stream=None):
        kw = dict(stream=stream)
        s = {}
        _, _, s["rows"] = self.norms[0](x, normed=False, quantize=True, **kw)
        s["wide"] = self.up(s["rows"], **kw)
        s["act"] = self.moe.quantize_rows(s["wide"], gated=True, **kw)
        s["delta"] = self.down(s["act"], **kw)
        s["normed"], s["sum"], s["last"] = self.norms[1](s["delta"], residual=x, quantize=True, **kw)
        s["logits"] = self.head(s["last"], dtype=FP32, **kw)
        s["scores"] = self.moe.token_logprobs(s["logits"], tokens, top=4, **kw)
        return s


def tensors(s):
    for v in s.values():
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, tuple):
            yield from (t for t in v if t is not None)
        else:
            yield v.codes.view(torch.uint8)
            yield v.scales


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(tensors(a), tensors(b)))


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
def test_block_stage_by_stage(moe, rows):  # noqa: F811
    g = gen(rows)
    d, ffn, vocab = 512, 768, 3001
    b = Block(moe, g, d, ffn, vocab)
    x = rand(g, rows, d, dtype=BF16)
    tokens = torch.randint(0, vocab, (rows, 2), generator=g, device="cuda").to(torch.int32)
    s = b(x, tokens)
    check_quantized(s["rows"], P.rms_norm(x, b.norms[0].weight, 1e-6, False), NORM_REL)
    check_product(s["wide"], s["rows"], b.up.codes, b.up.scales)
    a, u = s["wide"][:, :ffn].double(), s["wide"][:, ffn:].double()
    check_quantized(s["act"], a / (1 + torch.exp(-a)) * u, 8 * U)
    check_product(s["delta"], s["act"], b.down.codes, b.down.scales)
    assert torch.equal(s["sum"], (x.float() + s["delta"].float()).to(BF16))
    want = P.rms_norm(s["sum"], b.norms[1].weight, 1e-6, False)
    assert ((s["normed"].double() - want).abs() <= half_step(want, BF16) * (1 + 2.0 ** -8) + want.abs() * NORM_REL).all()
    check_quantized(s["last"], want, NORM_REL)
    check_product(s["logits"], s["last"], b.head.codes, b.head.scales)
    x64 = s["logits"].double()
    lse = torch.logsumexp(x64, -1)
    # tests/test_gpu_dense.py has the terms
    assert ((s["scores"].lse.double() - lse).abs() <= 1e-5 + 4 * U * lse.abs()).all()
    given = x64.gather(1, tokens.long()) - lse[:, None]
    assert ((s["scores"].logprobs.double() - given).abs() <= 1e-5 + 4 * U * (given.abs() + lse.abs()[:, None])).all()
    assert torch.equal(s["scores"].top_ids.long(), torch.sort(s["logits"], dim=-1, descending=True, stable=True).indices[:, :4])
    for linear in (b.up, b.down, b.head):
        assert linear.status() == 0


@pytest.mark.parametrize("rows", [3, 300])
def test_graphs_on_two_streams_give_the_same(moe, rows):  # noqa: F811
    """Two captured runs share weights and nothing else, so they may run at the same time; new inputs are read at replay."""
    g = gen(7)
    d, ffn, vocab = 256, 384, 20000
    b = Block(moe, g, d, ffn, vocab)
    inputs = [rand(g, rows, d, dtype=BF16) for _ in range(4)]
    tokens = torch.randint(0, vocab, (rows, 1), generator=g, device="cuda").to(torch.int32)
    want = [b(x, tokens) for x in inputs]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        x, stream, graph = inputs[i].clone(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            b(x, tokens)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                s = b(x, tokens)
        graphs.append((x, stream, graph, s))
    torch.cuda.synchronize()
    for at in (0, 2):
        for i, (x, stream, graph, s) in enumerate(graphs):
            with torch.cuda.stream(stream):
                x.copy_(inputs[at + i])
                for _ in range(5):
                    graph.replay()
        torch.cuda.synchronize()
        for i, (x, stream, graph, s) in enumerate(graphs):
            assert same(s, want[at + i])
    assert b.up.status() == b.down.status() == b.head.status() == 0


def test_a_stream_of_its_own(moe):  # noqa: F811
    """The stream argument: inputs made on it, outputs of it, while another stream is busy."""
    g = gen(8)
    b = Block(moe, g, 256, 256, 5000)
    x = rand(g, 64, 256, dtype=BF16)
    tokens = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    want = b(x, tokens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        busy = busy @ busy * 1e-3
    with torch.cuda.stream(side):
        y = x * 1
    got = b(y, tokens, stream=side)
    side.synchronize()
    assert same(got, want)


def test_eager_calls_between_two_streams(moe):  # noqa: F811
    g = gen(9)
    b = Block(moe, g, 256, 256, 5000)
    x = [rand(g, 40, 256, dtype=BF16) for _ in range(2)]
    tokens = torch.zeros(40, 1, dtype=torch.int32, device="cuda")
    want = [b(v, tokens) for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = b(x[i], tokens)
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_a_status_bit_is_read_once_whatever_the_streams(moe):  # noqa: F811
    """A product of one stream sets its bit at any moment of a read on another: one of two reads has it."""
    g = gen(10)
    x = moe.quantize_rows(rand(g, 20, 128))
    linear = moe.Fp8Linear(*make_weight(g, 4, 128, 128))
    bad = torch.tensor([0, 5, 5, 25, 30], dtype=torch.int32, device="cuda")
    out = torch.zeros(20, 128, device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    both = 0
    for i in range(4000):
        with torch.cuda.stream(side):
            torch.cuda._sleep(1 + 100 * (i % 500))  # moments up to 25 us apart
        linear(x, offsets=bad, out=out, stream=side)
        first = linear.status(stream=main)
        side.synchronize()
        second = linear.status(stream=main)
        assert first | second == moe.DENSE_BAD_OFFSETS, i
        both += first == second
    assert both == 0 and linear.status(stream=main) == 0
    # a read that does not clear leaves the bit
    linear(x, offsets=bad, out=out, stream=main)
    assert linear.status(clear=False, stream=main) == linear.status(stream=main) == moe.DENSE_BAD_OFFSETS
    assert linear.status(clear=False, stream=main) == 0


def test_a_new_weight_on_a_busy_stream(moe):  # noqa: F811
    """The status word is clear before a product of another stream can set it."""
    g = gen(11)
    x = moe.quantize_rows(rand(g, 20, 128))
    codes, scales = make_weight(g, 4, 128, 128)
    bad = torch.tensor([0, 5, 5, 25, 30], dtype=torch.int32, device="cuda")
    out = torch.zeros(20, 128, device="cuda")
    side, busy = torch.cuda.Stream(), torch.cuda.Stream()
    moe.Fp8Linear(codes, scales)(x, offsets=bad, out=out)
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(100_000_000)  # ~50 ms
        linear = moe.Fp8Linear(codes, scales)
    linear(x, offsets=bad, out=out, stream=side)
    side.synchronize()
    busy.synchronize()
    assert linear.status(stream=side) == moe.DENSE_BAD_OFFSETS


# ---- past 32 bits: the last rows of arrays of more than 2^31 elements equal the same rows alone ----

def test_many_logits(moe):  # noqa: F811
    vocab, rows = 131072, 16500
    logits = torch.empty(rows, vocab, dtype=BF16, device="cuda")
    logits[-3:] = rand(gen(1), 3, vocab, dtype=BF16)
    logits[:-3] = 0
    tokens = torch.full((rows, 1), 131071, dtype=torch.int32, device="cuda")
    got, few = moe.token_logprobs(logits, tokens, top=3), moe.token_logprobs(logits[-3:].clone(), tokens[-3:], top=3)
    assert torch.equal(got.top_ids[-3:], few.top_ids)
    # one CTA a row and a cluster's parts add up in other orders
    assert ((got.lse[-3:] - few.lse).abs() <= 1e-5).all() and (got.top_ids[0].tolist() == [0, 1, 2])


def test_many_normed_rows(moe):  # noqa: F811
    d, rows = 16384, 132000
    x = torch.zeros(rows, d, dtype=BF16, device="cuda")
    x[-2:] = rand(gen(2), 2, d, dtype=BF16)
    norm = moe.RmsNorm(torch.ones(d, device="cuda"))
    n, _, q = norm(x, quantize=True)
    a, _, b = norm(x[-2:].clone(), quantize=True)
    assert torch.equal(n[-2:], a) and torch.equal(q.scales[-2:], b.scales)
    assert torch.equal(q.codes[-2:].view(torch.uint8), b.codes.view(torch.uint8)) and (n[:2] == 0).all()
    del n
    p = moe.quantize_rows(x)
    assert torch.equal(p.codes[-2:].view(torch.uint8), moe.quantize_rows(x[-2:].clone()).codes.view(torch.uint8))


@pytest.mark.parametrize("groups", [0, 3])
def test_many_outputs(moe, groups):  # noqa: F811
    rows, n, k = 70000, 32768, 16
    g = gen(3)
    codes, scales = make_weight(g, *((groups,) if groups else ()), n, k)
    linear = moe.Fp8Linear(codes, scales)
    x = moe.quantize_rows(rand(g, rows, k))
    offsets = torch.tensor([0, 100, 69000, rows], dtype=torch.int32, device="cuda") if groups else None
    out = linear(x, offsets=offsets)
    assert linear.status() == 0
    tail = moe.Fp8Rows(x.codes[-200:], x.scales[-200:])
    check_product(out[-200:], tail, codes[-1] if groups else codes, scales[-1] if groups else scales)
    del out


def test_as_many_grouped_rows_as_there_can_be(moe):  # noqa: F811
    """Rows and groups whose sum passes 2^31 (81 GB; only the last rows hold anything)."""
    rows, n, k, groups = 0x7fffff00, 8, 16, 1024
    g = gen(4)
    codes, scales = make_weight(g, groups, n, k)
    linear = moe.Fp8Linear(codes, scales)
    few = moe.quantize_rows(rand(g, 300, k))
    x = moe.Fp8Rows.empty(rows, k)
    x.codes[-300:], x.scales[-300:] = few.codes, few.scales
    edges = torch.linspace(0, rows, groups + 1, dtype=torch.float64).to(torch.int32)
    edges[-1], edges[-2] = rows, rows - 300
    out = torch.empty(rows, n + 1, dtype=BF16, device="cuda")
    out[-300:] = 7
    linear(x, offsets=edges.cuda(), out=out[:, :n])
    assert linear.status() == 0
    check_product(out[-300:, :n], few, codes[-1], scales[-1])
    assert (out[-300:, n:] == 7).all()
    del x, out
    torch.cuda.empty_cache()


def test_example_with_the_dense_path_in_8_bits():
    spec = importlib.util.spec_from_file_location("verify_step", os.path.join(ROOT, "examples", "verify_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    decoder, kept = m.main(prompts=(37, 64, 5), steps=3, fp8=True)
    c = decoder.cache
    assert c.status() == 0 and decoder.head.status() == 0
    assert c.lens.tolist() == [n + k for n, k in zip((37, 64, 5, 37), kept.tolist())]
    assert all(w["qkv"].status() == 0 and w["out"].status() == 0 for w in decoder.weights)
