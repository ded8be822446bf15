"""Timed cases of the operators around the routed-MoE layer in a speculative-decode serving step.

  route    scores of all experts (softmax or sigmoid), a selection bias, expert groups, top-k and
           renormalised weights;
  append   a step's K and V rows quantised into the pages of a 4-bit cache, and read back as the values
           that the pages hold;
  attend   attention of a step's query rows over that cache (grouped-query heads, causal, windowed or
           tree-masked within the step), with the log-sum-exp of every row;
  fork     sequences that share another's pages, and the pages that the next step writes made their own
           (copy on write) or newly allocated, on every layer of the cache;
  compact  the accepted tokens of a verified step moved together on every layer, the others' pages freed.

Cache page format (one page holds `page` tokens of one layer, `page` a multiple of 16):
  page     [kv heads][page / 16][tile]        tile: 16 tokens of one head, 18 D bytes (D = head size):
    K codes   [D / 32][16 tokens][16 bytes]   piece j: channels 32 j .. 32 j + 31, two to a byte
    V codes   [16 tokens][D / 2 bytes]        two channels to a byte, the even one in the low nibble
    K scales  [16 tokens][D / 16]             E4M3, one for 16 consecutive channels
    V scales  [16 tokens][D / 16]
A code is E2M1; the value is code * block scale * tensor scale.  A block of 16 values x is stored with the
scale s = E4M3(max|x| / (6 ts)) (at most 448) and the codes E2M1(x / (s ts)), both to nearest even.
"""
import math

import torch

own = False

# the magnitudes of the E2M1 codes 0..7
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # a verify step of one request: latency is all
        dict(name="route verify step", op="route", tokens=4, experts=512, k=10, groups=8, keep=4, score="sigmoid", dtype="float32"),
        # a prefill chunk: 8192 rows of 512 scores
        dict(name="route prefill chunk", op="route", tokens=8192, experts=512, k=10, groups=8, keep=4, score="sigmoid", dtype="float32"),
        # the K and V rows of 32 requests' verify steps, few wide heads
        dict(name="append verify step", op="append", seqs=32, rows=4, ragged=False, length=4096, heads=2, dim=256, page=64, ts=1.0, dtype="bfloat16"),
        # a prefill chunk of three prompts of different lengths
        dict(name="append prefill chunk", op="append", seqs=3, rows=2731, ragged=True, length=8192, heads=8, dim=128, page=64, ts=0.375, dtype="bfloat16"),
        # one request early in its answer: latency is all
        dict(name="attend one short sequence", op="attend", seqs=1, rows=1, ragged=False, length=777, heads=2, group=8, dim=256, page=64, mask="causal", window=0, dtype="bfloat16"),
        # verify steps of a batch of requests of very different lengths
        dict(name="attend verify batch", op="attend", seqs=32, rows=4, ragged=True, length=8192, heads=8, group=4, dim=128, page=64, mask="causal", window=0, dtype="bfloat16"),
        # draft trees of 16 tokens, narrow heads, an odd group
        dict(name="attend draft trees", op="attend", seqs=24, rows=16, ragged=True, length=6001, heads=4, group=7, dim=64, page=16, mask="tree", window=0, dtype="float16"),
        # single-token decode over long documents
        dict(name="attend long documents", op="attend", seqs=4, rows=1, ragged=False, length=131072, heads=8, group=8, dim=128, page=128, mask="causal", window=0, dtype="bfloat16"),
        # one prompt sampled four ways
        dict(name="fork one prompt", op="fork", layers=12, parents=1, children=4, length=1000, new=4, heads=2, dim=256, page=64),
        # a batch of prompts, eight branches each
        dict(name="fork batch of branches", op="fork", layers=48, parents=16, children=128, length=2048, new=5, heads=8, dim=128, page=64),
        # accepted paths of 8 requests' draft trees
        dict(name="compact few requests", op="compact", layers=12, seqs=8, rows=8, length=2000, heads=2, dim=256, page=64),
        # accepted paths of a full batch, every layer
        dict(name="compact full batch", op="compact", layers=48, seqs=64, rows=16, length=1024, heads=8, dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "append", "attend", "attend", "attend", "fork", "compact"))
    if op == "route":
        groups = rng.choice((1, 4, 8, 16))
        experts = groups * rng.choice([n for n in (8, 9, 12, 16, 20, 24, 32, 40, 64, 96, 128) if 32 <= n * groups <= 512])
        keep = rng.randint((groups + 1) // 2, groups)
        return dict(op=op, tokens=_log(rng, 1, 8192), experts=experts, k=rng.randint(1, min(10, keep * experts // groups)), groups=groups, keep=keep,
                    score=rng.choice(("sigmoid", "softmax")), dtype=rng.choice(("float32", "bfloat16")))
    heads, dim, page = rng.choice(((1, 256), (2, 256), (4, 128), (8, 128), (4, 64), (8, 64), (3, 128))) + (rng.choice((16, 32, 64, 128)),)
    if op == "append":
        rows = _log(rng, 1, 2731)
        seqs = max(1, min(_log(rng, 1, 128), 8192 // rows))
        return dict(op=op, seqs=seqs, rows=rows, ragged=rng.random() < 0.7, length=rows + _log(rng, 1, 4096), heads=heads, dim=dim, page=page,
                    ts=rng.choice((1.0, 0.375, 2.5)), dtype=rng.choice(("bfloat16", "float16")))
    if op == "attend":
        mask, group = rng.choice(("causal", "causal", "window", "tree")), rng.choice((1, 3, 4, 7, 8))
        rows = rng.choice((1, 1, 2, 4, 5, 8)) if mask != "tree" else rng.randint(2, 16)
        length = min(_log(rng, 1, 131072), 60_000_000 // (rows * heads * group))
        seqs = max(1, min(_log(rng, 1, 128), 500_000 // length, 60_000_000 // (length * rows * heads * group)))
        return dict(op=op, seqs=seqs, rows=rows, ragged=rng.random() < 0.7, length=length, heads=heads, group=group, dim=dim, page=page,
                    mask="tree" if mask == "tree" else "causal", window=_log(rng, 16, 8192) if mask == "window" else 0, dtype=rng.choice(("bfloat16", "float16")))
    if op == "fork":
        parents = _log(rng, 1, 16)
        return dict(op=op, layers=rng.randint(1, 48), parents=parents, children=parents * rng.randint(1, 8), length=_log(rng, 1, 2048), new=rng.randint(1, 8), heads=heads,
                    dim=dim, page=min(page, 64))
    layers = rng.randint(1, 48)
    return dict(op=op, layers=layers, seqs=min(_log(rng, 1, 256), 48 * 64 // layers), rows=rng.randint(2, 16), length=_log(rng, 16, 1024), heads=heads, dim=dim, page=min(page, 64))


# ---- inputs ----------------------------------------------------------------------------------------------


def _quantise(x, ts):
    """Codes (0..15) and block scales (uint8 E4M3 bits) of x [..., D] in 32 bits."""
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s8 = (b.abs().amax(-1) / (6.0 * ts)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s8.float() * ts).unsqueeze(-1)
    y = torch.where(d > 0, b / d, torch.zeros_like(b))
    a = y.abs()
    # ties at the midpoints go to the even code: the comparison with an even code below is strict
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8)
            + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    return (code | ((y < 0).to(torch.uint8) << 3)).reshape(x.shape), s8.view(torch.uint8)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _fields(pool, dim):
    """The four fields of the tiles of `pool` [..., tile bytes] as views."""
    c = 8 * dim
    return (pool[..., :c].unflatten(-1, (dim // 32, 16, 16)), pool[..., c:2 * c].unflatten(-1, (16, dim // 2)),
            pool[..., 2 * c:2 * c + dim].unflatten(-1, (16, dim // 16)), pool[..., 2 * c + dim:].unflatten(-1, (16, dim // 16)))


def _fill(pool, dim, gen, std):
    """Writes K and V drawn from N(0, std^2) with a few large channels into the pages of `pool` [pages, heads, tiles, bytes]."""
    pages, heads, tiles, _ = pool.shape
    big = 1.0 + 3.0 * (torch.rand(2, heads, 1, 1, dim, generator=gen, device="cuda") < 0.03)
    step = max(1, (1 << 25) // (heads * tiles * 16 * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        kc, vc, ks, vs = _fields(pool[p:p + n], dim)
        for j, (codes, scales) in enumerate(((kc, ks), (vc, vs))):
            x = torch.randn(n, heads, tiles, 16, dim, generator=gen, device="cuda") * (std * big[j])
            q, s = _quantise(x, 1.0)
            q = _packed(q)
            codes.copy_(q.unflatten(-1, (dim // 32, 16)).transpose(-3, -2) if j == 0 else q)
            scales.copy_(s)


def _counts(case, gen, n):
    """Rows of each sequence in the step, and their running sum."""
    most = case["rows"]
    rows = torch.full((n,), most, dtype=torch.int32, device="cuda")
    if case["ragged"]:  # from half the most to the most, in an order of the seed's
        rows = most - (torch.arange(n, device="cuda") * (most // 2 + 1) // n)[torch.randperm(n, generator=gen, device="cuda")].to(torch.int32)
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1:] = rows.cumsum(0)
    return rows, cu


def _handle(case, s):
    """The cache handle that a user's program keeps beside the tensors."""
    import routed_moe_decode_gb300 as moe
    return moe.Kv4Cache(layers=s["pool"].shape[0], pages=s["pool"].shape[1], kv_heads=case["heads"], head_dim=case["dim"], page_size=case["page"], seqs=s["table"].shape[0],
                        max_pages=s["table"].shape[1], pool=s["pool"], table=s["table"], lens=s["lens"], refs=s["refs"], k_scale=s["ts"], v_scale=s["ts"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "route":
        t, e, dt = case["tokens"], case["experts"], getattr(torch, case["dtype"])
        s["logits"] = (torch.randn(t, e, generator=gen, device="cuda") + 0.7 * torch.randn(e, generator=gen, device="cuda")).to(dt)
        s["bias"] = 0.1 * torch.randn(e, generator=gen, device="cuda") if case["score"] == "sigmoid" else None
        s["ids"] = torch.empty(t, case["k"], dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(t, case["k"], dtype=torch.float32, device="cuda")
        if own:
            import routed_moe_decode_gb300 as moe
            s["routing"] = moe.Routing(e, case["k"], score=case["score"], groups=case["groups"], keep_groups=case["keep"],
                                       group_score="top2" if case["score"] == "sigmoid" else "max", renormalise=True, scale=2.5)
        return s
    heads, dim, page, length = case["heads"], case["dim"], case["page"], case["length"]
    tile, tiles = 18 * dim, page // 16
    s["ts"] = case.get("ts", 1.0)
    s["lut"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    if case["op"] in ("append", "attend"):
        n, dt = case["seqs"], getattr(torch, case["dtype"])
        rows, cu = _counts(case, gen, n)
        lens = torch.randint((length + 1) // 2, length + 1, (n,), generator=gen, device="cuda", dtype=torch.int32) if case["ragged"] else \
            torch.full((n,), length, dtype=torch.int32, device="cuda")
        lens[0] = length
        s["lens"] = torch.maximum(lens, rows)
        longest = max(length, case["rows"])
        per = -(-longest // page)
        pages = n * per
        s["table"] = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).reshape(n, per)
        s["refs"] = torch.ones(pages, dtype=torch.int32, device="cuda")
        s["pool"] = torch.zeros(1, pages, heads * tiles * tile, dtype=torch.uint8, device="cuda")
        s["cu"], total = cu, int(cu[-1])
        s["longest"] = longest
        if case["op"] == "append":
            # K and V as the slices of a fused projection's output
            kv = (torch.randn(total, 2, heads, dim, generator=gen, device="cuda") * (1.0 + 3.0 * (torch.rand(2, heads, dim, generator=gen, device="cuda") < 0.03))).to(dt)
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
            s["read"] = (torch.empty(total, heads, dim, dtype=dt, device="cuda"), torch.empty(total, heads, dim, dtype=dt, device="cuda"))
        else:
            _fill(s["pool"].view(pages, heads, tiles, tile), dim, gen, 1.0)
            s["q"] = (1.5 * torch.randn(total, heads * case["group"], dim, generator=gen, device="cuda")).to(dt)
            s["scale"] = 1.0 / math.sqrt(dim)
            s["tree"] = None
            if case["mask"] == "tree":  # row i's ancestors: a parent among the rows before it, and so on up
                m = max(int(r) for r in rows.tolist())
                seen = torch.zeros(n, m, dtype=torch.int64, device="cuda")
                for i in range(m):
                    up = torch.randint(max(0, i - 4), i, (n, 1), generator=gen, device="cuda") if i else None
                    seen[:, i] = (seen.gather(1, up)[:, 0] if i else 0) | (1 << i)
                i = torch.arange(m, device="cuda")
                s["tree"] = seen[i[None, :] < rows[:, None]].contiguous()
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(total, heads * case["group"], dtype=torch.float32, device="cuda")
        if own:
            s["cache"] = _handle(case, s)
        return s
    # fork, compact: several layers; the last page is never handed out
    layers, n = case["layers"], case["parents"] if case["op"] == "fork" else case["seqs"]
    seqs = n + case.get("children", 0)
    new = case["new"] if case["op"] == "fork" else case["rows"]
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    lens[:n] = torch.randint((length + 1) // 2, length + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    lens[0] = length
    per = -(-(length + new) // page)
    own_pages = (lens + page - 1) // page
    pages = n * per + case.get("children", 0) * (2 + -(-new // page)) + 9
    perm = torch.randperm(pages - 1, generator=gen, device="cuda").to(torch.int32)[:n * per].reshape(n, per)
    used = torch.arange(per, device="cuda")[None, :] < own_pages[:n, None]
    s["table"] = torch.full((seqs, per), -1, dtype=torch.int32, device="cuda")
    s["table"][:n] = torch.where(used, perm, -1)
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s["refs"][perm[used].long()] = 1
    s["refs"][-1] = 1
    s["lens"] = lens
    s["pool"] = torch.randint(0, 256, (layers, pages, heads * tiles * tile), generator=gen, device="cuda", dtype=torch.uint8)
    if case["op"] == "fork":
        kids = case["children"]
        s["src"] = (torch.arange(kids, device="cuda", dtype=torch.int32) % n).contiguous()
        s["dst"] = torch.arange(n, seqs, device="cuda", dtype=torch.int32)
        s["new"] = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        s["new"][n:] = new
    else:
        s["base"] = lens.clone()
        s["new"] = torch.randint(1, new + 1, (seqs,), generator=gen, device="cuda", dtype=torch.int32)
        s["cu"] = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
        s["cu"][1:] = s["new"].cumsum(0)
        total = int(s["cu"][-1])
        s["keep"] = (torch.rand(total, generator=gen, device="cuda") < 0.4).to(torch.uint8)
        s["keep"][s["cu"][:-1].long()] = 1  # the first token of a step is always right
    if own:
        s["cache"] = _handle(case, s)
    return s


# ---- plain forms -----------------------------------------------------------------------------------------


def _plain_route(s):
    c = s["case"]
    x = s["logits"].float()
    t, e = x.shape
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
        key = score + s["bias"]
        g = key.reshape(t, c["groups"], -1).sort(dim=-1, descending=True, stable=True).values
        g = g[..., 0] + g[..., 1]
    else:
        p = torch.exp(x - x.amax(-1, keepdim=True))
        score, key = p / p.sum(-1, keepdim=True), x  # the softmax keeps the order of the logits
        g = key.reshape(t, c["groups"], -1).amax(-1)
    kept = g.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
    allowed = torch.zeros(t, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, kept, True)
    key = key.masked_fill(~allowed.repeat_interleave(e // c["groups"], 1), -math.inf)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, ids)
    return ids.to(torch.int32), 2.5 * w / w.sum(-1, keepdim=True)


def _places(s, page):
    """Sequence and position of every row of the step: the last rows of its sequence."""
    cu = s["cu"].long()
    r = torch.arange(s["rows_total"], device="cuda")
    seq = torch.searchsorted(cu[1:], r, right=True)
    pos = s["lens"].long()[seq] - (cu[seq + 1] - r)
    return seq, pos, s["table"].long()[seq, pos // page], pos % page // 16, pos % 16


def _values(s, codes, scales):
    """Packed codes [..., D / 2] and scales [..., D / 16] to values in 32 bits."""
    v = s["lut"][torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    f = scales.contiguous().view(torch.float8_e4m3fn).float() * s["ts"]
    return (v.unflatten(-1, (-1, 16)) * f.unsqueeze(-1)).flatten(-2)


def _plain_append(s):
    c = s["case"]
    heads, dim, page = c["heads"], c["dim"], c["page"]
    s["rows_total"] = s["k"].shape[0]
    _, _, pid, tile, slot = _places(s, page)
    kc, vc, ks, vs = _fields(s["pool"][0].view(-1, heads, page // 16, 18 * dim), dim)
    h = torch.arange(heads, device="cuda")[None, :]
    pid, tile, slot = pid[:, None], tile[:, None], slot[:, None]
    q, sc = _quantise(s["k"], s["ts"])
    kc[pid, h, tile, :, slot] = _packed(q).unflatten(-1, (dim // 32, 16))
    ks[pid, h, tile, slot] = sc
    q, sc = _quantise(s["v"], s["ts"])
    vc[pid, h, tile, slot] = _packed(q)
    vs[pid, h, tile, slot] = sc
    return (_values(s, kc[pid, h, tile, :, slot].flatten(-2), ks[pid, h, tile, slot]).to(s["k"].dtype),
            _values(s, vc[pid, h, tile, slot], vs[pid, h, tile, slot]).to(s["v"].dtype))


def _cached(s):
    """K and V of every sequence, padded: [seqs, heads, tokens, D] in 32 bits."""
    c = s["case"]
    heads, dim, page = c["heads"], c["dim"], c["page"]
    t = s["pool"][0].view(-1, heads, page // 16, 18 * dim)[s["table"].long()]  # [seqs, pages, heads, tiles, bytes]
    t = t.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seqs, heads, tiles, bytes]
    kc, vc, ks, vs = _fields(t, dim)
    k = _values(s, kc.transpose(-3, -2).flatten(-2), ks).flatten(2, 3)
    return k, _values(s, vc, vs).flatten(2, 3)


def _plain_attend(s):
    c = s["case"]
    heads, group, dim, m = c["heads"], c["group"], c["dim"], c["rows"]
    k, v = _cached(s)
    n, _, tokens, _ = k.shape
    cu, lens = s["cu"].long(), s["lens"].long()
    rows = cu[1:] - cu[:-1]
    i = torch.arange(m, device="cuda")
    at = (cu[:-1, None] + torch.minimum(i[None, :], rows[:, None] - 1))  # [seqs, m], short steps repeat a row
    q = s["q"].float()[at].reshape(n, m, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(n, heads, m * group, dim)
    score = (q @ k.transpose(-1, -2)) * s["scale"]
    j = torch.arange(tokens, device="cuda")[None, None, :]
    first = (lens - rows)[:, None, None]  # of the step's tokens
    pos = first + i[None, :, None]
    see = j <= pos
    if c["window"]:
        see = see & (j > pos - c["window"])
    if s["tree"] is not None:
        bit = (j - first).clamp(0, 63)
        see = ((s["tree"][at][:, :, None] >> bit) & 1).bool() & (j < lens[:, None, None])
        see = see | (j < first)
    see = see[:, None, :, None, :].expand(n, heads, m, group, tokens).reshape(n, heads, m * group, tokens)
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = torch.log(total) + top
    seq = torch.searchsorted(cu[1:], torch.arange(s["q"].shape[0], device="cuda"), right=True)
    row = torch.arange(s["q"].shape[0], device="cuda") - cu[seq]
    back = lambda x: x.reshape(n, heads, m, group, -1).permute(0, 2, 1, 3, 4)[seq, row].flatten(1, 2)  # noqa: E731
    return back(out).to(s["q"].dtype), back(lse)[..., 0]


def _plain_trim(s, to, who):
    """Cuts the sequences where `who` is true to `to` tokens; pages that no sequence points at any more are free."""
    page = s["case"]["page"]
    to = torch.where(who, torch.minimum(to, s["lens"]), s["lens"])
    j = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    drop = (j >= ((to + page - 1) // page)[:, None]) & (s["table"] >= 0)
    s["refs"].scatter_add_(0, s["table"].clamp(min=0).long().flatten(), -drop.flatten().to(torch.int32))
    s["table"].masked_fill_(drop, -1)
    s["lens"].copy_(to)


def _plain_reserve(s):
    """Room for new[s] more tokens of every sequence: shared pages that will be written are copied, further ones taken, lowest first."""
    page, table, refs, new = s["case"]["page"], s["table"], s["refs"], s["new"]
    lens, last = s["lens"], s["refs"].shape[0] - 1
    have, want = (lens + page - 1) // page, (lens + new + page - 1) // page
    tail = table.gather(1, (have - 1).clamp(min=0).long()[:, None])[:, 0]
    copies = (new > 0) & (lens % page != 0) & (refs[tail.clamp(min=0).long()] > 1)
    need = copies.to(torch.int32) + (want - have)
    start = need.cumsum(0) - need
    free = (refs != 0).to(torch.int32).sort(dim=-1, stable=True).indices.to(torch.int32)
    copy_to = torch.where(copies, free[start.clamp(max=last).long()], last)
    copy_from = torch.where(copies, tail, last)
    refs.scatter_add_(0, copy_from.long(), -copies.to(torch.int32))
    refs.scatter_add_(0, copy_to.long(), copies.to(torch.int32))
    s["pool"][:, copy_to.long()] = s["pool"][:, copy_from.long()]
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (j >= have[:, None]) & (j < want[:, None])
    at = (start + copies.to(torch.int32))[:, None] + (j - have[:, None])
    got = free[at.clamp(0, last).long()]
    refs.scatter_add_(0, torch.where(fresh, got, last).long().flatten(), fresh.flatten().to(torch.int32))
    table.copy_(torch.where(fresh, got, torch.where(copies[:, None] & (j == have[:, None] - 1), copy_to[:, None], table)))
    lens.add_(new)


def _plain_fork(s):
    _plain_trim(s, torch.zeros_like(s["lens"]), torch.zeros_like(s["lens"], dtype=torch.bool).scatter_(0, s["dst"].long(), True))
    rows = s["table"][s["src"].long()]
    s["table"][s["dst"].long()] = rows
    s["lens"][s["dst"].long()] = s["lens"][s["src"].long()]
    s["refs"].scatter_add_(0, rows.clamp(min=0).long().flatten(), (rows >= 0).flatten().to(torch.int32))
    _plain_reserve(s)
    return s["table"], s["lens"], s["refs"], s["pool"]


def _plain_compact(s):
    c = s["case"]
    heads, dim, page = c["heads"], c["dim"], c["page"]
    everyone = torch.ones_like(s["lens"], dtype=torch.bool)
    _plain_trim(s, s["base"], everyone)
    _plain_reserve(s)
    s["rows_total"] = s["keep"].shape[0]
    seq, pos, pid, tile, slot = _places(s, page)
    cu, keep = s["cu"].long(), s["keep"].long()
    run = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), keep.cumsum(0)))
    kept = run[cu[1:]] - run[cu[:-1]]  # of each sequence
    r = torch.arange(s["rows_total"], device="cuda")
    rank = run[:-1] - run[cu[:-1]][seq]
    # the row that comes to stand at each row's place: the kept ones in order, then every place keeps what it has
    source = torch.where(r - cu[:-1][seq] < kept[seq], 0, r)
    source = source.scatter_add(0, cu[:-1][seq] + torch.where(keep > 0, rank, 0), torch.where(keep > 0, r, 0))
    kc, vc, ks, vs = _fields(s["pool"].view(c["layers"], -1, heads, page // 16, 18 * dim), dim)
    h = torch.arange(heads, device="cuda")[None, :]
    put, get = [(pid[i][:, None], h, tile[i][:, None], slot[i][:, None]) for i in (r, source)]
    kc[:, put[0], put[1], put[2], :, put[3]] = kc[:, get[0], get[1], get[2], :, get[3]]
    vc[:, put[0], put[1], put[2], put[3]] = vc[:, get[0], get[1], get[2], get[3]]
    ks[:, put[0], put[1], put[2], put[3]] = ks[:, get[0], get[1], get[2], get[3]]
    vs[:, put[0], put[1], put[2], put[3]] = vs[:, get[0], get[1], get[2], get[3]]
    _plain_trim(s, s["lens"] - ((cu[1:] - cu[:-1]) - kept).to(torch.int32), everyone)
    return s["table"], s["lens"], s["refs"], s["pool"]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"route": _plain_route, "append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact}[op](s)
    if op == "route":
        s["routing"].route(s["logits"], s["bias"], s["ids"], s["weights"])
        return s["ids"], s["weights"]
    cache = s["cache"]
    if op == "append":
        cache.append(0, s["k"], s["v"], s["cu"])
        return cache.read(0, s["cu"], out=s["read"])
    if op == "attend":
        return cache.attend(0, s["q"], s["cu"], max_rows=c["rows"], scale=s["scale"], window=c["window"], tree=s["tree"], out=s["out"], lse=s["lse"])
    if op == "fork":
        cache.fork(s["src"], s["dst"])
        cache.reserve(s["new"])
    else:
        cache.trim(s["base"])
        cache.reserve(s["new"])
        cache.compact(s["keep"], s["cu"], max_rows=c["rows"])
    return s["table"], s["lens"], s["refs"], s["pool"]


# ---- work and 64-bit results -----------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "route":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["tokens"] * (case["experts"] * size + case["k"] * 8) + case["experts"] * 4, "flops": 8 * case["tokens"] * case["experts"]}
    heads, dim, page = case["heads"], case["dim"], case["page"]
    token = heads * (dim + dim // 8)  # K and V of a token in 4 bits with their scales
    if op in ("append", "attend"):
        rows = case["seqs"] * case["rows"] * (0.75 if case["ragged"] else 1.0)
        if op == "append":  # in, quantised, read back, out
            return {"bytes": rows * (2 * 2 * heads * dim * 2 + 2 * token), "flops": rows * heads * dim * 2 * 8}
        seen = case["length"] * (0.75 if case["ragged"] else 1.0)
        if case["window"]:
            seen = min(seen, case["window"] + case["rows"])
        q = rows * heads * case["group"]
        return {"bytes": case["seqs"] * seen * token + q * (2 * 2 * dim + 4), "flops": 4 * q * seen * dim}
    if op == "fork":  # a shared last page is read and written on every layer
        tables = (case["parents"] + case["children"]) * (-(-case["length"] // page)) * 4 * 3
        return {"bytes": case["children"] * case["layers"] * 2 * page * token + tables, "flops": 0}
    moved = case["seqs"] * 0.2 * case["rows"]  # accepted tokens that change their place
    return {"bytes": moved * case["layers"] * 2 * token + case["seqs"] * (-(-case["length"] // page)) * 8, "flops": 0}


def _exact_quantise(x, ts):
    """The values that the blocks of x [..., D] are held as, from the definition, in 64 bits."""
    b = x.double().reshape(*x.shape[:-1], -1, 16)
    a = (b.abs().amax(-1) / (6.0 * ts)).clamp(max=448.0)
    # E4M3: 3 bits after the leading one, steps of 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    scale = ((a / step).round() * step * ts).unsqueeze(-1)
    y = torch.where(scale > 0, b / scale, torch.zeros_like(b))
    m = y.abs()
    half = torch.exp2(torch.floor(torch.log2(m.clamp(min=1.0))) - 1.0)  # E2M1: one bit after the leading one, steps of 1/2 below 1
    return ((m / half).round() * half).clamp(max=6.0).mul(torch.sign(y)).mul(scale).reshape(x.shape)


def _exact_values(s, seq, tokens):
    """K and V [heads, tokens, D] of one sequence in 64 bits, code by code from the page format."""
    c = s["case"]
    heads, dim, page = c["heads"], c["dim"], c["page"]
    t = torch.arange(tokens, device="cuda")
    base = s["table"][seq].long()[t // page]
    raw = s["pool"][0].view(-1, heads, page // 16, 18 * dim)[base, :, t % page // 16].transpose(0, 1)  # [heads, tokens, bytes]
    ch, slot = torch.arange(dim, device="cuda"), (t % 16)[:, None]
    places = ((ch // 32 * 256 + ch % 32 // 2) + slot * 16, 8 * dim + slot * (dim // 2) + ch // 2)
    found = []
    for j, place in enumerate(places):
        nib = raw.gather(2, place.expand(heads, tokens, dim)).long() >> (ch % 2 * 4) & 15
        mag, expo = nib & 1, nib >> 1 & 3
        v = torch.where(expo > 0, (1.0 + 0.5 * mag.double()) * torch.exp2(expo.double() - 1.0), 0.5 * mag.double())
        b = raw.gather(2, (16 * dim + j * dim + slot * (dim // 16) + ch // 16).expand(heads, tokens, dim)).long()
        e, f = b >> 3 & 15, (b & 7).double()
        sc = torch.where(e > 0, (1.0 + f / 8.0) * torch.exp2(e.double() - 7.0), f * 2.0 ** -9)
        found.append(torch.where(nib > 7, -v, v) * sc * s["ts"])
    return found


def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "append":
        return _exact_quantise(s["k"], s["ts"]), _exact_quantise(s["v"], s["ts"])
    if op == "route":
        x = s["logits"].double()
        t, e = x.shape
        score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
        key = score + s["bias"].double() if s["bias"] is not None else x
        g = key.reshape(t, case["groups"], -1)
        g = g.topk(2, -1).values.sum(-1) if case["score"] == "sigmoid" else g.amax(-1)
        place = (g[:, :, None] < g[:, None, :]).sum(-1) + ((g[:, :, None] == g[:, None, :]) & torch.ones(case["groups"], case["groups"], device="cuda").tril(-1).bool()).sum(-1)
        key = torch.where((place < case["keep"]).repeat_interleave(e // case["groups"], 1), key, torch.full_like(key, -math.inf))
        w = score.gather(1, key.argsort(dim=-1, descending=True, stable=True)[:, :case["k"]])
        return None, 2.5 * w / w.sum(-1, keepdim=True)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    heads, group, dim = case["heads"], case["group"], case["dim"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    if sum(4.0 * (cu[b + 1] - cu[b]) * heads * group * dim * lens[b] for b in range(case["seqs"])) > 4e12:
        return None
    for b in range(case["seqs"]):
        n, first = cu[b + 1] - cu[b], lens[b] - (cu[b + 1] - cu[b])
        k, v = _exact_values(s, b, lens[b])
        q = s["q"][cu[b]:cu[b + 1]].double().reshape(n, heads, group, dim)
        j = torch.arange(lens[b], device="cuda")
        for i in range(n):
            see = j <= first + i
            if case["window"]:
                see = see & (first + i - j < case["window"])
            if s["tree"] is not None:
                see = (j < first) | ((j >= first) & (s["tree"][cu[b] + i] >> (j - first).clamp(0, 63) & 1).bool())
            score = torch.einsum("hgd,htd->hgt", q[i], k[:, see]) * s["scale"]
            lse[cu[b] + i] = torch.logsumexp(score, -1).reshape(-1)
            out[cu[b] + i] = torch.einsum("hgt,htd->hgd", torch.softmax(score, -1), v[:, see]).reshape(heads * group, dim)
    return out, lse
