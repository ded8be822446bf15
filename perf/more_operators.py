"""Timed cases of the dense path around the routed-MoE layer, in 8-bit floating point.

  norm      the residual's addition and a root-mean-square norm of its rounded sum, as rows of the input's type
            and as E4M3 codes with one FP32 scale for each row and 128 channels;
  quantize  rows, or silu(gate) * up of a fused projection, as such codes and scales;
  matmul    rows of codes times a weight of codes (one FP32 scale for 128 x 128 of it);
  grouped   the same with a weight of its own for every group of consecutive rows (ragged, empty ones among them);
  logprobs  log probabilities of given tokens, log-sum-exp, entropy and the best alternatives of every row.

A block of 128 values v is stored with the scale s = max|v| / 448 (FP32) and the codes E4M3(v / s), to nearest even;
code 0 where s is 0.  out[t, n] = sum over blocks b of xs[t, b] ws[n / 128, b] (sum of x[t, k] w[n, k] over the block).
Alternatives are ordered by the logit itself, equal ones by the lower id.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = dict(bfloat16=torch.bfloat16, float16=torch.float16, float32=torch.float32)


def listed():
    return [
        # a verify step of one request: latency is all
        dict(name="norm verify step", op="norm", rows=4, d=2048, residual=True, normed=True, fp8=True, dtype="bfloat16"),
        # a prefill chunk, its rows for the 16-bit router and for 8-bit projections
        dict(name="norm prefill chunk", op="norm", rows=8192, d=2048, residual=True, normed=True, fp8=True, dtype="bfloat16"),
        # attention's output of a verify batch on its way into a projection
        dict(name="quantize verify batch", op="quantize", rows=33, d=4096, gated=False, dtype="bfloat16"),
        # the activation between a prefill chunk's two dense feed-forward products
        dict(name="quantize gated chunk", op="quantize", rows=8192, d=4096, gated=True, dtype="bfloat16"),
        # one request's projection
        dict(name="matmul verify step", op="matmul", rows=4, n=5120, k=2048, dtype="bfloat16"),
        # the vocabulary of a verify batch: every weight is read for 16 rows
        dict(name="matmul vocabulary", op="matmul", rows=16, n=131072, k=2048, dtype="float32"),
        # a prefill chunk through a dense projection
        dict(name="matmul prefill chunk", op="matmul", rows=8192, n=8192, k=4096, dtype="bfloat16"),
        # a decode batch's routes: half of the experts have one row or two
        dict(name="grouped decode batch", op="grouped", groups=512, rows=320, n=1024, k=2048, skew=0.5, dtype="bfloat16"),
        # a prefill chunk's routes, 160 rows an expert on average
        dict(name="grouped prefill chunk", op="grouped", groups=512, rows=81920, n=1024, k=2048, skew=0.2, dtype="bfloat16"),
        # the drafted tokens of one request against the model's logits
        dict(name="logprobs verify step", op="logprobs", rows=4, vocab=131072, tokens=1, top=8, masked=0.0, dtype="float32"),
        # a batch under a grammar that forbids much, an odd vocabulary
        dict(name="logprobs masked batch", op="logprobs", rows=127, vocab=100003, tokens=3, top=20, masked=0.6, dtype="float32"),
        # a prompt's tokens scored
        dict(name="logprobs prompt", op="logprobs", rows=2048, vocab=131072, tokens=1, top=5, masked=0.0, dtype="bfloat16"),
    ]


def draw(rng):
    def spread(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    op = rng.choice(("norm", "quantize", "matmul", "matmul", "grouped", "logprobs"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    if op == "norm":
        fp8 = rng.random() < 0.6
        d = 16 * spread(4, 512) if fp8 else spread(64, 8192)
        return dict(op=op, rows=min(spread(1, 8192), (1 << 24) // d), d=d, residual=rng.random() < 0.7,
                    normed=not fp8 or rng.random() < 0.5, fp8=fp8, dtype=dtype)
    if op == "quantize":
        d = 16 * spread(4, 512)
        return dict(op=op, rows=min(spread(1, 8192), (1 << 24) // d), d=d, gated=rng.random() < 0.5, dtype=dtype)
    if op == "matmul":
        n, k = spread(64, 16384), 16 * spread(8, 512)
        return dict(op=op, rows=max(1, min(spread(1, 8192), (1 << 36) // (n * k))), n=n, k=k, dtype=dtype)
    if op == "grouped":
        groups, n, k = spread(2, 512), spread(64, 2048), 16 * spread(8, 128)
        return dict(op=op, groups=groups, rows=max(1, min(spread(4, 65536), 160 * groups)), n=n, k=k,
                    skew=round(rng.uniform(0.0, 1.0), 2), dtype=dtype)
    vocab = spread(500, 160000)
    return dict(op=op, rows=min(spread(1, 2048), (1 << 27) // vocab), vocab=vocab, tokens=rng.randint(1, 5), top=rng.randint(0, 20),
                masked=rng.choice((0.0, 0.0, 0.3, 0.9)), dtype=dtype)


def blocks(n):
    return -(-n // BLOCK)


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("norm", "quantize"):
        size, values = TYPES[case["dtype"]].itemsize, rows * case["d"]
        fp8 = values + 4 * rows * blocks(case["d"])
        if op == "quantize":
            return dict(bytes=values * size * (2 if case["gated"] else 1) + fp8, flops=values * (8 if case["gated"] else 2))
        reads = 1 + case["residual"]
        writes = case["residual"] + case["normed"]
        return dict(bytes=values * size * (reads + writes) + 2 * case["d"] + (fp8 if case["fp8"] else 0), flops=6 * values)
    if op == "logprobs":
        size = TYPES[case["dtype"]].itemsize
        return dict(bytes=rows * (case["vocab"] * size + case["tokens"] * 12 + 8 + case["top"] * 8), flops=5 * rows * case["vocab"])
    n, k = case["n"], case["k"]
    row_bytes = rows * (k + 4 * blocks(k) + n * TYPES[case["dtype"]].itemsize)
    weights = 1
    if op == "grouped":
        weights = sum(c > 0 for c in counts_of(case))
    return dict(bytes=row_bytes + weights * (n * k + 4 * blocks(n) * blocks(k)), flops=2 * rows * n * k)


def counts_of(case):
    """Rows of each group: shares exp(-skew z) of them, z going round the groups; some groups have none."""
    groups, rows, skew = case["groups"], case["rows"], case["skew"]
    share = [math.exp(-2.0 * skew * ((g * 7919) % groups) / groups) for g in range(groups)]
    total, counts, run, given = sum(share), [], 0.0, 0
    for s in share:
        run += s
        upto = int(rows * run / total + 0.5)
        counts.append(upto - given)
        given = upto
    # every seventh group gives its rows to the one behind it
    for g in range(0, groups - 1, 7):
        counts[g + 1] += counts[g]
        counts[g] = 0
    return counts


# the magnitudes of the E4M3 codes 0 .. 126, and the borders between neighbours
MAGNITUDES = [(c % 8) / 512 if c < 8 else (1 + (c % 8) / 8) * 2.0 ** (c // 8 - 7) for c in range(127)]
BORDERS = [(a + b) / 2 for a, b in zip(MAGNITUDES, MAGNITUDES[1:])]


def e4m3(v):
    """Values as E4M3, to nearest even, at most 448.  In 64 bits: a quotient next to a border would be rounded onto it."""
    borders = torch.tensor(BORDERS, dtype=torch.float64, device=v.device)
    size = v.double().abs()
    code = torch.bucketize(size, borders)
    on = size == borders[code.clamp(max=125)]
    code = code + (on & (code % 2 == 1))
    return torch.where(v < 0, code + 128, code).to(torch.uint8).view(torch.float8_e4m3fn)


def quantized(v):
    """Codes and scales of the rows v (32 bits)."""
    rows, d = v.shape
    b = torch.nn.functional.pad(v, (0, blocks(d) * BLOCK - d)).view(rows, -1, BLOCK)
    most = b.abs().amax(-1)
    scales = most / torch.full_like(most, 448.0)  # by a tensor: a number's reciprocal would be multiplied, one rounding more
    codes = e4m3(torch.where(scales[..., None] > 0, b.double() / scales[..., None].double(), 0.0))
    return codes.view(rows, -1)[:, :d].contiguous(), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, dtype = case["op"], case["rows"], TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def hidden(*shape):
        # a hidden state: a few channels are far larger than the others
        loud = 1.0 + 15.0 * (torch.rand(shape[-1], generator=gen, device="cuda") < 0.01)
        return normal(*shape) * loud

    s = dict(case=case)
    if op == "norm":
        s["x"], s["weight"] = hidden(rows, case["d"]).to(dtype), (1.0 + 0.2 * normal(case["d"])).to(torch.bfloat16)
        s["residual"] = (4.0 * hidden(rows, case["d"])).to(dtype) if case["residual"] else None
        if own:
            import routed_moe_decode_gb300 as moe
            s["own"] = moe.RmsNorm(s["weight"], eps=1e-6)
    elif op == "quantize":
        s["x"] = hidden(rows, case["d"] * (2 if case["gated"] else 1)).to(dtype)
    elif op in ("matmul", "grouped"):
        n, k = case["n"], case["k"]
        s["x"], xs = quantized(hidden(rows, k))
        s["x_scales"] = xs.t().contiguous().t()  # as the norm and the quantiser lay them out: a block's rows together
        lead = (case["groups"],) if op == "grouped" else ()
        w = torch.randn(*lead, n, k, generator=gen, device="cuda", dtype=torch.float16) * 100.0
        s["w"] = w.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        spread = torch.rand(*lead, blocks(n), blocks(k), generator=gen, device="cuda")
        s["w_scales"] = (0.5 + spread) / (100.0 * math.sqrt(k))
        if op == "grouped":
            counts = counts_of(case)
            s["most"] = max(counts)
            s["offsets"] = torch.tensor([0] + counts, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
        if own:
            import routed_moe_decode_gb300 as moe
            s["own"] = moe.Fp8Linear(s["w"], s["w_scales"])
            s["rows"] = moe.Fp8Rows(s["x"], s["x_scales"])
    else:
        vocab = case["vocab"]
        logits = 2.0 * normal(rows, vocab)
        if case["masked"]:
            logits.masked_fill_(torch.rand(rows, vocab, generator=gen, device="cuda") < case["masked"], -math.inf)
        # the model is sure of some rows' next token
        best = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
        sure = 8.0 + 10.0 * torch.rand(rows, generator=gen, device="cuda")
        at = torch.arange(rows, device="cuda")
        logits[at, best] = sure
        s["logits"] = logits.to(dtype)
        s["tokens"] = torch.randint(0, vocab, (rows, case["tokens"]), generator=gen, device="cuda").to(torch.int32)
        s["tokens"][:, 0] = best
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import routed_moe_decode_gb300 as moe
    case = s["case"]
    op = case["op"]
    if op == "norm":
        normed, residual, fp8 = s["own"](s["x"], residual=s["residual"], normed=case["normed"], quantize=case["fp8"])
        return dict(normed=normed, residual=residual, **(dict(codes=fp8.codes, scales=fp8.scales) if fp8 is not None else {}))
    if op == "quantize":
        fp8 = moe.quantize_rows(s["x"], gated=case["gated"])
        return dict(codes=fp8.codes, scales=fp8.scales)
    if op == "matmul":
        return dict(out=s["own"](s["rows"], dtype=TYPES[case["dtype"]]))
    if op == "grouped":
        return dict(out=s["own"](s["rows"], offsets=s["offsets"], dtype=TYPES[case["dtype"]]))
    return moe.token_logprobs(s["logits"], s["tokens"], top=case["top"])._asdict()


def widened(codes, scales, rows_of_scales):
    """The values that codes [..., N, K] stand for, in 32 bits; one row of scales for rows_of_scales rows of codes."""
    n, k = codes.shape[-2:]
    s = scales.repeat_interleave(rows_of_scales, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]
    return codes.float() * s


def run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        x, dtype = s["x"], s["x"].dtype
        h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(dtype)
        v = h.float()
        n = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
        out = dict(normed=n.to(dtype) if case["normed"] else None, residual=None if s["residual"] is None else h)
        if case["fp8"]:
            out["codes"], out["scales"] = quantized(n)
        return out
    if op == "quantize":
        v = s["x"].float()
        if case["gated"]:
            gate, up = v[:, :case["d"]], v[:, case["d"]:]
            v = gate / (1.0 + torch.exp(-gate)) * up
        codes, scales = quantized(v)
        return dict(codes=codes, scales=scales)
    if op == "matmul":
        out = widened(s["x"], s["x_scales"], 1) @ widened(s["w"], s["w_scales"], BLOCK).t()
        return dict(out=out.to(TYPES[case["dtype"]]))
    if op == "grouped":
        x = widened(s["x"], s["x_scales"], 1)
        first, last = s["offsets"][:-1].long(), s["offsets"][1:].long()
        slots = first[:, None] + torch.arange(s["most"], device=x.device)
        used = slots < last[:, None]
        padded = x[slots.clamp(max=x.shape[0] - 1)]
        product = torch.bmm(padded, widened(s["w"], s["w_scales"], BLOCK).transpose(1, 2))
        return dict(out=product[used].to(TYPES[case["dtype"]]))
    x = s["logits"].float()
    most = x.amax(-1, keepdim=True)
    e = torch.exp(x - most)
    total = e.sum(-1, keepdim=True)
    lse = (most + torch.log(total)).squeeze(-1)
    p = e / total
    entropy = lse - torch.where(p > 0, p * x, torch.zeros_like(p)).sum(-1)
    given = x.gather(1, s["tokens"].long()) - lse[:, None]
    out = dict(logprobs=given, lse=lse, entropy=entropy, top_ids=None, top_logprobs=None)
    if case["top"]:
        value, index = torch.sort(x, dim=-1, descending=True, stable=True)
        out["top_ids"] = index[:, :case["top"]].to(torch.int32)
        out["top_logprobs"] = value[:, :case["top"]] - lse[:, None]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64

    def codes_and_scales(v):
        rows, d = v.shape
        padded = torch.zeros(rows, blocks(d) * BLOCK, dtype=f64, device=v.device)
        padded[:, :d] = v
        padded = padded.view(rows, -1, BLOCK)
        scale = (padded.abs().max(-1).values / 448).float().double()
        q = padded / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
        q = q.clamp(-448, 448)
        # 4 significant bits, at least 2^-9 apart
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        q = torch.round(q / step) * step
        return q.view(rows, -1)[:, :d], scale

    if op == "norm":
        h = s["x"].to(f64)
        if s["residual"] is not None:
            h = (h + s["residual"].to(f64)).to(s["x"].dtype).to(f64)
        n = h * (h.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).rsqrt() * s["weight"].to(f64)
        out = dict(normed=n if case["normed"] else None, residual=h if s["residual"] is not None else None)
        if case["fp8"]:
            out["codes"], out["scales"] = codes_and_scales(n)
        return out
    if op == "quantize":
        v = s["x"].to(f64)
        if case["gated"]:
            v = v[:, :case["d"]] * torch.sigmoid(v[:, :case["d"]]) * v[:, case["d"]:]
        codes, scales = codes_and_scales(v)
        return dict(codes=codes, scales=scales)
    if op in ("matmul", "grouped"):
        rows, n, k = case["rows"], case["n"], case["k"]
        spans = [(0, rows, s["w"], s["w_scales"])]
        if op == "grouped":
            edges = s["offsets"].tolist()
            spans = [(a, b, s["w"][g], s["w_scales"][g]) for g, (a, b) in enumerate(zip(edges, edges[1:])) if b > a]
        out = torch.zeros(rows, n, dtype=f64, device="cuda")
        for a, b, w, ws in spans:
            ws = ws.to(f64).repeat_interleave(BLOCK, 0)[:n]
            for j in range(blocks(k)):
                cut = slice(j * BLOCK, (j + 1) * BLOCK)
                part = s["x"][a:b, cut].to(f64) @ w[:, cut].to(f64).t()
                out[a:b] += part * s["x_scales"][a:b, j:j + 1].to(f64) * ws[:, j]
        return dict(out=out)
    out = []
    for row, tokens in zip(s["logits"], s["tokens"].long()):
        x = row.to(f64)
        lse = torch.logsumexp(x, 0)
        logp = x - lse
        entropy = -(logp.exp() * torch.where(logp > -math.inf, logp, torch.zeros_like(logp))).sum()
        got = [logp[tokens], lse, entropy]
        if case["top"]:
            got.append(logp.topk(case["top"]).values)
        out.append(got)
    given, lse, entropy, *best = (torch.stack(v) for v in zip(*out))
    return dict(logprobs=given, lse=lse, entropy=entropy, top_ids=None, top_logprobs=best[0] if best else None)
