"""The 4-bit K/V cache on the GPU against the plain 64-bit implementation (tests/kv4_plain.py)."""
import numpy as np
import pytest
import torch

import kv4_plain as P
from gpu_helpers import BF16_HALF_ULP_REL

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_moe_decode_gb300 as m
    return m


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def make_cache(moe, lens, heads, D, page, layers=1, extra_pages=3, max_pages=None, k_scale=1.0, v_scale=1.0, seed=0,
               fill=True):
    """A cache whose sequences hold `lens` tokens of random K and V in pages of random order, and the
    same as numpy arrays.  Bytes that belong to no token are 0x7f (scales there are NaN)."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int32)
    need = [-(-int(n) // page) for n in lens]
    per = max_pages or max(max(need), 1)
    pages = sum(need) + extra_pages
    table = np.full((len(lens), per), -1, dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    order = rng.permutation(pages)[:sum(need)]
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    refs[order] = 1
    nbytes = heads * (page // 16) * 18 * D
    pool = np.full((layers, pages, nbytes), 0x7f, dtype=np.uint8)
    if fill:
        for layer in range(layers):
            for s, n in enumerate(lens):
                for t in range(0, int(n), 16):
                    for h in range(heads):
                        kv = rng.standard_normal((2, 16, D)) * np.where(rng.random(D) < 0.05, 4.0, 1.0)
                        (kc, ks), (vc, vs) = (P.quantise(x, 1.0) for x in kv)
                        m = min(16, int(n) - t)
                        tile = P.tile_at(pool[layer], table, s, t, h, heads, D, page)
                        new = [np.full_like(c, 15) for c in (kc, vc)] + [np.full_like(c, 0x7f) for c in (ks, vs)]
                        for a, b in zip(new, (kc, vc, ks, vs)):
                            a[:m] = b[:m]
                        tile[:] = P.make_tile(*new)
    cache = moe.Kv4Cache(layers, pages, heads, D, page, len(lens), per, pool=dev(pool, torch.uint8), table=dev(table),
                         lens=dev(lens), refs=dev(refs), k_scale=k_scale, v_scale=v_scale)
    return cache, pool, table, lens.copy(), refs


def cu_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def check_attend(moe, lens, rows, heads, group, D, page, dtype="bf16", window=0, trees=None, scale=None, q_std=1.0,
                 k_scale=1.0, v_scale=1.0, strided=False, max_rows=None, layers=1, layer=0, seed=0, cache=None):
    cache, pool, table, lens, _ = cache or make_cache(moe, lens, heads, D, page, layers=layers, k_scale=k_scale,
                                                      v_scale=v_scale, seed=seed)
    rng = np.random.default_rng(seed + 1)
    cu, total, hq = cu_of(rows), int(sum(rows)), heads * group
    dt = DT[dtype]
    if strided:  # the queries as a slice of a wider projection, heads further apart than head_dim
        wide = torch.randn((total, hq + 3, D + 8), generator=torch.Generator().manual_seed(seed)).to(dt).cuda() * q_std
        q = wide[:, 1:hq + 1, :D]
    else:
        q = (dev(rng.standard_normal((total, hq, D)), torch.float32) * q_std).to(dt)
    lse = torch.full((total, hq), 7.0, dtype=torch.float32, device="cuda")
    out = torch.full((total, hq, D), 7.0, dtype=dt, device="cuda")
    tree = None if trees is None else dev(trees, torch.int64)
    cache.attend(layer, q, dev(cu), max_rows=max_rows or max(max(rows), 1), scale=scale, window=window, tree=tree, out=out,
                 lse=lse)
    assert cache.status() == 0
    got, got_lse, qd = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    scale = D ** -0.5 if scale is None else scale
    half = BF16_HALF_ULP_REL if dtype == "bf16" else 2.0 ** -11
    tiny = 2.0 ** -134 if dtype == "bf16" else 2.0 ** -25  # half the spacing of the smallest outputs
    for s in range(len(lens)):
        n, first = int(rows[s]), int(lens[s]) - int(rows[s])
        for h in range(heads):
            k, v = P.kv_of(pool[layer], table, s, int(lens[s]), h, heads, D, page, k_scale, v_scale)
            for r in range(n):
                see = P.visible(int(lens[s]), first, r, window, None if trees is None else trees[cu[s] + r])
                for j in range(group):
                    at = (cu[s] + r, h * group + j)
                    ref, ref_lse, spread, qk, vmax = P.attend_row(qd[at], k, v, see, scale)
                    N = int(see.sum())
                    # FP32 scores: D products summed, error at most D 2^-23 of sum |q k|; exp2 to 2^-21; p
                    # rounded to FP16 (2^-11, and 2^-25 where it is subnormal; the largest p is at
                    # least 1); FP32 sums over N tokens, 16 a step
                    z = D * 2.0 ** -23 * qk
                    sums = (N / 16 + 64) * 2.0 ** -22
                    bound = spread * (2.0 ** -11 + 2 * z + 2.0 ** -20 + sums) + N * 2.0 ** -25 * vmax
                    bound = bound + np.abs(ref) * half * 1.01 + bound * half + tiny
                    err = np.abs(got[at] - ref)
                    assert (err <= bound).all(), (s, h, r, j, float((err / bound).max()))
                    if N == 0:
                        assert got_lse[at] == -np.inf and (got[at] == 0).all()
                    else:
                        assert abs(got_lse[at] - ref_lse) <= z + sums + 2.0 ** -20 + abs(ref_lse) * 2.0 ** -22, (s, h, r, j)
    return got


# ---- attention ----

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 129, 300])
def test_attend_one_token(moe, D, page, length):
    check_attend(moe, [length], [1], heads=2, group=3, D=D, page=page, seed=length)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group,rows", [(1, 1), (1, 5), (4, 4), (7, 3), (8, 1), (8, 2), (16, 4), (5, 13), (12, 64)])
def test_attend_groups_and_rows(moe, D, group, rows):
    check_attend(moe, [rows + 70, rows + 1, rows + 17], [rows, rows, max(rows // 2, 1)], heads=2, group=group, D=D, page=32,
                 seed=group * 100 + rows)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_ragged_batch(moe, D, dtype):
    lens = [1, 700, 33, 5, 64, 257, 0, 16, 1000]
    rows = [1, 4, 2, 3, 1, 4, 0, 0, 2]
    check_attend(moe, lens, rows, heads=3, group=4, D=D, page=64, dtype=dtype, seed=5)


@pytest.mark.parametrize("window", [1, 7, 16, 40, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_window(moe, D, window):
    check_attend(moe, [200, 31, 3], [5, 3, 2], heads=2, group=4, D=D, page=16, window=window, seed=window)


def test_attend_rows_that_see_nothing(moe):
    # more rows than tokens: the first rows lie before the sequence's start; and an empty sequence
    check_attend(moe, [3, 0, 20], [6, 2, 1], heads=2, group=4, D=128, page=32)
    # tree rows without a bit and without a prefix
    check_attend(moe, [4, 3], [4, 3], heads=2, group=2, D=64, page=16, trees=[0, 1, 0, 0xf, 0, 2, 0])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_trees(moe, D):
    rng = np.random.default_rng(3)
    rows, lens = [16, 1, 64, 7, 33], [130, 1, 64, 300, 40]
    trees = []
    for n in rows:
        for i in range(n):
            bits = int(rng.integers(0, 2 ** 62)) & ((1 << (i + 1)) - 1) | (1 << i)
            trees.append(bits - 2 ** 64 if bits >> 63 else bits)
    trees[3] = -1  # every bit, the sign bit too: every token of the step
    check_attend(moe, lens, rows, heads=2, group=3, D=D, page=32, trees=np.array(trees, dtype=np.int64))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_strided_queries_layers_and_scales(moe, D):
    check_attend(moe, [150, 90], [3, 4], heads=2, group=4, D=D, page=32, strided=True, layers=3, layer=2, k_scale=0.37,
                 v_scale=12.5, scale=0.21, seed=9)


def test_attend_peaked_and_flat_scores(moe):
    # scores of hundreds, where one token takes all, and of 0; queries far from 1
    check_attend(moe, [400], [4], heads=2, group=4, D=128, page=64, q_std=60.0)
    check_attend(moe, [400], [4], heads=2, group=4, D=128, page=64, q_std=0.0)
    check_attend(moe, [400], [4], heads=2, group=4, D=128, page=64, q_std=1e-20)
    check_attend(moe, [400], [4], heads=2, group=4, D=128, page=64, q_std=1e20, scale=1e-20)


def test_attend_tile_hint_does_not_matter(moe):
    # max_rows only chooses the tile: fewer rows than there are, or more, are computed all the same
    for hint in (1, 2, 64, 1000):
        check_attend(moe, [300, 120], [9, 5], heads=2, group=4, D=128, page=64, max_rows=hint)


def test_attend_long_split_over_many_ctas_is_deterministic(moe):
    cache = make_cache(moe, [6000, 50], 1, 64, 128, seed=2)
    a = check_attend(moe, None, [2, 1], 1, 8, 64, 128, cache=cache)
    b = check_attend(moe, None, [2, 1], 1, 8, 64, 128, cache=cache)
    assert np.array_equal(a, b)


def test_attend_repeated_calls_same_bits(moe):
    cache, *_ = make_cache(moe, [9000, 30, 4000], 2, 64, 64, seed=4)
    q = torch.randn((9, 16, 64), device="cuda").to(torch.bfloat16)
    cu = dev([0, 4, 5, 9])
    first = cache.attend(0, q, cu, max_rows=4)
    for _ in range(20):
        assert torch.equal(first, cache.attend(0, q, cu, max_rows=4))
    assert cache.status() == 0


def test_attend_bad_page_is_reported_and_skipped(moe):
    cache, pool, table, lens, _ = make_cache(moe, [100, 40], 2, 64, 16, seed=6)
    cache.table[0, 2] = 10 ** 6
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    out = cache.attend(0, q, dev([0, 1, 2]), max_rows=1)
    assert torch.isfinite(out.float()).all()
    assert cache.status() == moe.KV4_BAD_PAGE and cache.status() == 0


def test_attend_on_another_stream_and_in_a_graph(moe):
    cache, *_ = make_cache(moe, [500, 77], 2, 128, 64, seed=8)
    q = torch.randn((4, 8, 128), device="cuda").to(torch.bfloat16)
    cu = dev([0, 2, 4])
    want = cache.attend(0, q, cu, max_rows=2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(want)
    with torch.cuda.stream(side):
        cache.attend(0, q, cu, max_rows=2, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(0, q, cu, max_rows=2, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_results_made_on_another_stream(moe):
    # the current stream is busy and then writes into memory it has freed: a call on another stream, which makes its own
    # results, is not disturbed by either
    cache, *_ = make_cache(moe, [500, 77], 2, 128, 64, seed=8)
    q = torch.randn((4, 8, 128), device="cuda").to(torch.bfloat16)
    cu = dev([0, 2, 4])
    want, held = cache.attend(0, q, cu, max_rows=2).clone(), [t.clone() for t in cache.read(0, cu, rows=4)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = [torch.empty_like(t) for t in (want, *held)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    for t in junk:
        t.fill_(7.0)
    del junk, t
    out = cache.attend(0, q, cu, max_rows=2, stream=side)
    got = cache.read(0, cu, rows=4, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for a, b in zip(got, held):
        assert torch.equal(a, b)
    assert cache.status() == 0


# Blocks of many rows (a step's rows times query heads per K/V head).

@pytest.mark.parametrize("D,group,dtype", [(64, 4, "bf16"), (64, 7, "fp16"), (128, 4, "fp16"), (128, 1, "bf16"), (256, 3, "bf16")])
@pytest.mark.parametrize("window", [0, 1, 70, 2 ** 31 - 1])
def test_attend_chunks_of_a_prompt(moe, D, group, dtype, window):
    # several blocks a head, blocks that end inside 64 tokens, steps that a block does not see, a short step beside them
    check_attend(moe, [700, 150, 0, 1203, 64], [150, 150, 0, 40, 1], heads=2, group=group, D=D, page=48, dtype=dtype,
                 window=window, seed=window % 97 + D)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_many_rows_that_see_nothing(moe, D):
    # more rows than tokens, an empty sequence, tree rows without a bit
    check_attend(moe, [30, 0, 5], [90, 41, 44], heads=1, group=3, D=D, page=16)
    check_attend(moe, [30, 0, 5], [90, 41, 44], heads=1, group=3, D=D, page=16, window=4)
    trees = np.zeros(100, dtype=np.int64)
    trees[[3, 63, 70]] = 5
    check_attend(moe, [64, 36], [64, 36], heads=2, group=2, D=D, page=32, trees=trees)


@pytest.mark.parametrize("D,group", [(64, 7), (128, 5), (256, 9)])
def test_attend_trees_of_many_heads(moe, D, group):
    rng = np.random.default_rng(D)
    rows, lens = [16, 64, 5], [3000, 64, 191]
    trees = [(int(rng.integers(0, 2 ** 62)) & ((1 << (i + 1)) - 1)) | (1 << i) for n in rows for i in range(n)]
    trees = [t - 2 ** 64 if t >> 63 else t for t in trees]
    check_attend(moe, lens, rows, heads=2, group=group, D=D, page=16, dtype="fp16", trees=np.array(trees, dtype=np.int64))


def test_attend_many_rows_scores_and_strides(moe):
    for D in (64, 128, 256):
        check_attend(moe, [900], [12], heads=1, group=6, D=D, page=64, q_std=60.0)  # references that rise on the way
        check_attend(moe, [300], [12], heads=1, group=6, D=D, page=64, q_std=1e-20)
        check_attend(moe, [150, 190], [30, 24], heads=2, group=4, D=D, page=32, strided=True, layers=3, layer=2, k_scale=0.37,
                     v_scale=12.5, scale=-0.21, seed=9)


def test_attend_many_rows_of_many_sequences(moe):
    rng = np.random.default_rng(0)
    rows = rng.integers(0, 4, 300)
    check_attend(moe, rows + rng.integers(0, 90, 300), rows, heads=1, group=16, D=128, page=16, max_rows=3)


@pytest.mark.parametrize("group", [1, 16])  # few and many rows
@pytest.mark.parametrize("seqs", [31, 32, 33, 256, 257])
def test_attend_numbers_of_sequences(moe, seqs, group):
    rng = np.random.default_rng(seqs)
    rows = rng.integers(0, 4, seqs)
    rows[-1] = 2
    check_attend(moe, rows + rng.integers(0, 70, seqs), rows, heads=1, group=group, D=128, page=16, max_rows=3, seed=seqs)


@pytest.mark.parametrize("D,group,dtype", [(64, 1, "fp16"), (64, 12, "bf16"), (64, 24, "fp16"), (64, 40, "fp16"), (128, 1, "bf16"),
                                           (128, 12, "fp16"), (128, 40, "fp16"), (256, 1, "fp16"), (256, 12, "fp16"),
                                           (256, 40, "bf16")])
def test_attend_small_p_beside_a_large_one(moe, D, group, dtype):
    # every row's first token has a score 25.5 (in powers of two) above the others', and a value of 0: the output is what
    # the many small p give.  As many items as there are parts of the work, so that they are cut in few places
    seqs, heads, N, page = 40, 64, 320, 64
    cache = moe.Kv4Cache(1, seqs * N // page, heads, D, page, seqs, N // page, v_scale=1000.0)
    cache.reserve(dev([N] * seqs))
    k = torch.zeros((seqs, N, heads, D), dtype=torch.bfloat16, device="cuda")
    v = torch.full((seqs, N, heads, D), 6000.0, dtype=torch.bfloat16, device="cuda")
    k[:, 0], v[:, 0] = 6.0, 0.0
    cache.append(0, k.view(-1, heads, D), v.view(-1, heads, D), dev(N * np.arange(seqs + 1)))
    q = torch.ones((seqs, heads * group, D), dtype=DT[dtype], device="cuda")
    lse = torch.empty((seqs, heads * group), dtype=torch.float32, device="cuda")
    scale = 25.5 * np.log(2.0) / (6 * D)
    out, lse = cache.attend(0, q, dev(np.arange(seqs + 1)), max_rows=1, scale=scale, lse=lse)
    assert cache.status() == 0
    scale = float(np.float32(scale))
    small = (N - 1) * np.exp(-scale * 6 * D)
    want, want_lse = 6000.0 * small / (1 + small), scale * 6 * D + np.log1p(small)
    # p in FP16: 2^-11, and 2^-25 against a largest p of at least 2^7; the score in FP32 (18 natural units, as are its
    # factor's roundings), exp2 to 2^-21, sums of 320 tokens; the output's own rounding
    half = BF16_HALF_ULP_REL if dtype == "bf16" else 2.0 ** -11
    rel = 2.0 ** -11 + 4 * 18 * 2.0 ** -23 + 2.0 ** -20 + (N / 16 + 64) * 2.0 ** -22
    bound = want * rel + (N - 1) * 2.0 ** -25 * 2.0 ** -7 * 6000.0 + want * half * 1.01
    assert (out.double() - want).abs().max() <= bound, (float((out.double() - want).abs().max()), bound)
    assert (lse.double() - want_lse).abs().max() <= 4 * 18 * 2.0 ** -23 + 2.0 ** -20 + (N / 16 + 64) * 2.0 ** -22


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_scores_of_any_size(moe, D):
    # references far from 0, where their own spacing is above 1: finite, and the tokens of the largest score
    cache = moe.Kv4Cache(1, 8, 1, D, 64, 1, 8)
    n = 500
    cache.reserve(dev([n]))
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[:, 0, 0] = torch.arange(n, device="cuda") % 7 - 3.0          # held as 0, +-1.03, +-2.06, +-3
    v = (torch.arange(n, device="cuda") % 7 - 3.0)[:, None, None].expand(n, 1, D).to(torch.bfloat16).contiguous()
    cache.append(0, k, v, dev([0, n]))
    for group in (1, 40):
        for size in (1e3, 1e5, 1e6, 3e7):
            q = torch.zeros((1, group, D), dtype=torch.bfloat16, device="cuda")
            q[..., 0] = size
            q[:, ::2, 0] = -size
            out = cache.attend(0, q, dev([0, 1]), max_rows=1, scale=1.0).float()
            # scores are at least 900 apart: only the tokens of the largest count
            assert (out[:, 1::2] == 3).all() and (out[:, ::2] == -3).all(), (group, size)
    assert cache.status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_many_rows_same_bits_and_rows_apart(moe, D):
    cache, *_ = make_cache(moe, [5000, 30, 2000], 2, D, 64, seed=4)
    q = torch.randn((50, 16, D), device="cuda").to(torch.bfloat16)
    cu = dev([0, 20, 40, 50])
    first = cache.attend(0, q, cu, max_rows=20)
    for _ in range(20):
        assert torch.equal(first, cache.attend(0, q, cu, max_rows=20))
    # a row of NaN and one of infinities spoil no other
    q[3, 5] = float("nan")
    q[45, 0] = float("inf")
    other = cache.attend(0, q, cu, max_rows=20)
    spoiled = torch.zeros((50, 16), dtype=torch.bool, device="cuda")
    spoiled[3, 5] = spoiled[45, 0] = True
    assert torch.equal(first[~spoiled], other[~spoiled]) and not torch.isfinite(other[3, 5].float()).any()
    assert cache.status() == 0


@pytest.mark.parametrize("D,group", [(64, 8), (64, 16), (64, 32), (64, 40), (128, 8), (128, 16), (128, 40), (256, 8), (256, 16),
                                     (256, 40)])
def test_attend_rows_do_not_depend_on_their_neighbours(moe, D, group):
    # one row of a head has scores that rise by far more than the others' in the middle of the sequence: the others'
    # bits stay.  So many heads that a part of the work is several steps long
    n, heads, page = 6400, 64, 128
    cache = moe.Kv4Cache(1, n // page, heads, D, page, 1, n // page)
    cache.reserve(dev([n]))
    g = torch.Generator(device="cuda").manual_seed(D + group)
    k, v = (torch.randn((n, heads, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache.append(0, k, v, dev([0, n]))
    q = torch.randn((1, heads, group, D), generator=g, device="cuda").to(torch.bfloat16)
    cu, at = dev([0, 1]), torch.arange(heads, device="cuda")
    first = cache.attend(0, q.view(1, -1, D), cu, max_rows=1).view(heads, group, D)
    for row in (0, 5):
        token = (97 * at + 150) % n
        other = q.clone()
        other[0, :, row] = 4 * k[token, at]
        got = cache.attend(0, other.view(1, -1, D), cu, max_rows=1).view(heads, group, D)
        apart = torch.arange(group, device="cuda") != row
        assert torch.equal(first[:, apart], got[:, apart]), row
        assert (got[:, row].float() - v[token, at].float()).abs().max() < 1
    assert cache.status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_many_rows_bad_page_and_stale_tokens(moe, D):
    lens, page = [300, 100], 32
    cache, pool, table, _, _ = make_cache(moe, lens, 2, D, page, seed=6)
    q = torch.randn((60, 16, D), device="cuda").to(torch.bfloat16)
    cu = dev([0, 30, 60])
    want = cache.attend(0, q, cu, max_rows=30)
    # the unused end of a sequence's last page holds NaN scales: no difference
    tile = 18 * D
    last = int(table[1, 3])
    cache.pool.view(1, -1, 2, page // 16, tile)[0, last, :, 1, 16 * D:] = 0xff
    cache.pool.view(1, -1, 2, page // 16, tile)[0, last, :, 0, 16 * D:].view(2, 2, 16, D // 16)[:, :, 4:] = 0xff
    assert torch.equal(want, cache.attend(0, q, cu, max_rows=30))
    cache.table[0, 2] = 10 ** 6
    out = cache.attend(0, q, cu, max_rows=30)
    assert torch.isfinite(out.float()).all() and torch.equal(out[30:], want[30:])
    assert cache.status() == moe.KV4_BAD_PAGE and cache.status() == 0


@pytest.mark.parametrize("D,group", [(64, 3), (64, 24), (128, 8), (128, 24), (256, 2), (256, 20)])
def test_attend_long_sequences(moe, D, group):
    # two steps of 2 rows over 140001 and 70003 tokens, against the values that the cache gives back, in 64 bits
    lens, page, rows = [140001, 70003], 128, 2
    pages = [-(-n // page) for n in lens]
    cache = moe.Kv4Cache(1, sum(pages), 1, D, page, 2, max(pages))
    cache.reserve(dev(lens))
    g = torch.Generator(device="cuda").manual_seed(D)
    total, cu_all = sum(lens), dev([0, lens[0], sum(lens)])
    k, v = (torch.randn((total, 1, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache.append(0, k, v, cu_all)
    k, v = (t[:, 0].double() for t in cache.read(0, cu_all, rows=total))  # at most 6 bits a value: exact in BF16
    q = (2 * torch.randn((2 * rows, group, D), generator=g, device="cuda")).to(torch.bfloat16)
    lse = torch.empty((2 * rows, group), dtype=torch.float32, device="cuda")
    out, lse = cache.attend(0, q, dev([0, rows, 2 * rows]), max_rows=rows, lse=lse)
    assert cache.status() == 0
    for s, first in enumerate((0, lens[0])):
        for r in range(rows):
            N = lens[s] - rows + r + 1
            ks, vs, qs = k[first:first + N], v[first:first + N], q[s * rows + r].double()
            z = qs @ ks.T * D ** -0.5
            p = z.softmax(-1)
            want, spread = p @ vs, p @ vs.abs()
            # the terms of check_attend, with the largest p at least 2^7 where p is rounded to FP16
            qk = (qs.abs() @ ks.abs().T).max() * D ** -0.5
            score, sums = D * 2.0 ** -23 * qk, (N / 16 + 64) * 2.0 ** -22
            bound = spread * (2.0 ** -11 + 2 * score + 2.0 ** -20 + sums) + N * 2.0 ** -32 * vs.abs().max()
            bound = bound + want.abs() * BF16_HALF_ULP_REL * 1.01 + bound * BF16_HALF_ULP_REL
            assert ((out[s * rows + r].double() - want).abs() <= bound).all()
            exact = z.logsumexp(-1)
            assert ((lse[s * rows + r].double() - exact).abs() <= score + sums + 2.0 ** -20 + exact.abs() * 2.0 ** -22).all()


# ---- append and read ----

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,page,ts", [(1, 16, 1.0), (3, 48, 0.375), (8, 128, 2.5)])
def test_append_and_read(moe, D, dtype, heads, page, ts):
    lens, rows = [40, 1, 17, 300, 0], [5, 1, 17, 130, 0]
    cache, pool, table, lens, _ = make_cache(moe, lens, heads, D, page, layers=2, k_scale=ts, v_scale=2 * ts, fill=False)
    cu, total = cu_of(rows), sum(rows)
    rng = np.random.default_rng(D + heads)
    dt = DT[dtype]
    x = rng.standard_normal((total, 2, heads, D)) * np.exp2(rng.integers(-6, 7, (total, 2, heads, 1)))
    x[1] = 0.0
    x[2, :, :, :16] = 0.0
    kv = dev(x, torch.float64).to(dt)  # K and V interleaved: strided rows
    k, v = kv[:, 0], kv[:, 1]
    cache.append(1, k, v, dev(cu))
    assert cache.status() == 0
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    want_k, want_v = [P.values(*P.quantise(a, t), t) for a, t in ((kn, ts), (vn, 2 * ts))]
    after = cache.pool.cpu().numpy()
    assert np.array_equal(after[0], pool[0])  # the other layer is untouched
    touched = np.zeros_like(pool[1], dtype=bool)
    for s, n in enumerate(rows):
        for i in range(n):
            pos = int(lens[s]) - n + i
            for h in range(heads):
                tile = P.tile_at(after[1], table, s, pos, h, heads, D, page)
                kc, vc, ks, vs = (f[pos % 16] for f in P.tile_fields(tile, D))
                assert np.array_equal(P.values(kc, ks, ts), want_k[cu[s] + i, h])
                assert np.array_equal(P.values(vc, vs, 2 * ts), want_v[cu[s] + i, h])
                mark = P.tile_at(touched, table, s, pos, h, heads, D, page)
                mark[:8 * D].reshape(D // 32, 16, 16)[:, pos % 16] = True
                mark[8 * D:16 * D].reshape(16, D // 2)[pos % 16] = True
                mark[16 * D:17 * D].reshape(16, D // 16)[pos % 16] = True
                mark[17 * D:].reshape(16, D // 16)[pos % 16] = True
    assert np.array_equal(after[1][~touched], pool[1][~touched])
    gk, gv = cache.read(1, dev(cu), rows=total, dtype=dt)
    for got, want in ((gk, want_k), (gv, want_v)):
        assert torch.equal(got.cpu(), torch.tensor(want).float().to(dt))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_and_read_rows_aligned_to_16_bytes_only(moe, D):
    heads, n = 3, 40
    cu = dev([0, n])
    caches = [make_cache(moe, [n + 7], heads, D, 48, fill=False)[0] for _ in range(2)]
    g = torch.Generator().manual_seed(D)
    wide = torch.randn((2, n, heads, D + 8), generator=g).to(torch.bfloat16).cuda()
    k, v = wide[0, :, :, 8:], wide[1, :, :, 8:]  # 16 bytes past a row's start, heads 16 bytes further apart
    assert k.data_ptr() % 32 == 16
    caches[0].append(0, k, v, cu)
    caches[1].append(0, k.contiguous(), v.contiguous(), cu)
    assert torch.equal(caches[0].pool, caches[1].pool)
    want = caches[0].read(0, cu, rows=n)
    room = torch.full((2, n * heads * D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = tuple(r[8:8 + n * heads * D].view(n, heads, D) for r in room)
    assert out[0].data_ptr() % 32 == 16
    caches[0].read(0, cu, out=out)
    for a, b, r in zip(out, want, room):
        assert torch.equal(a, b) and (r[:8] == 7).all() and (r[8 + n * heads * D:] == 7).all()
    assert caches[0].status() == 0


def test_append_ties_go_to_even(moe):
    # every tie of the code grid under a scale of 1 (largest value 6), and ties of the scale itself
    x = np.zeros((3, 1, 64))
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x[0, 0, :15] = ties + [-t for t in ties] + [6.0]
    x[1, 0, 0] = 6 * 1.0625  # halfway between the scales 1 and 1.125: to 1
    x[1, 0, 16] = 6 * 1.1875  # halfway between 1.125 and 1.25: to 1.25
    x[2, 0, 0] = 2.0 ** -10 * 6  # half the smallest scale: to 0
    cache, *_ = make_cache(moe, [3], 1, 64, 16, fill=False)
    t = dev(x, torch.float64).to(torch.bfloat16)
    cache.append(0, t, t, dev([0, 3]))
    k, v = cache.read(0, dev([0, 3]), rows=3)
    want = P.values(*P.quantise(t.double().cpu().numpy(), 1.0), 1.0)
    assert list(want[0, 0, :7]) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert want[1, 0, 0] == 6.0 and want[1, 0, 16] == 7.5 and want[2, 0, 0] == 0.0
    for got in (k, v):
        assert np.array_equal(got.double().cpu().numpy(), want)


def held_one():
    """The value that a block of ones is held as (the scale 1/6 is rounded to 1.375 / 8)."""
    one = P.values(*P.quantise(np.ones(16), 1.0), 1.0)
    assert (one == 6 * 1.375 / 8).all()
    return float(one[0])


def test_append_nonfinite(moe):
    cache, *_ = make_cache(moe, [2], 1, 64, 16, fill=False)
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[0, 0, 4], x[0, 0, 20] = float("inf"), float("-inf"), float("nan")
    cache.append(0, x, torch.ones_like(x), dev([0, 2]))
    k, v = cache.read(0, dev([0, 2]), rows=2)
    assert cache.status() == moe.KV4_NONFINITE
    k = k.float().cpu()
    assert k[0, 0, 3] == 2688 and k[0, 0, 4] == -2688 and k[0, 0, 0] == 0  # 1 is below half the smallest step at scale 448
    one = held_one()
    assert k[0, 0, 20] == 0 and k[0, 0, 21] == one and (k[1] == one).all() and (v.float() == one).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ts", [2.0 ** -13, 0.001, 2.0 ** -60, 2.0 ** -100, 1e-30, 2.0 ** 60, 2.0 ** 100])
def test_append_far_from_the_tensor_scale(moe, dtype, ts):
    # finite values whose quotient by the scale leaves FP32, or all but does: the code keeps their sign
    ts = float(np.float32(ts))
    top = torch.finfo(DT[dtype]).max
    x = np.zeros((4, 1, 64))
    x[0, 0, :6] = top, -top, top / 2, -top / 3, 1.0, -1.0
    x[1, 0, :3] = -top, 0.5 * top, -1e-4
    x[2, 0, 16:20] = -1.0, 0.25, 1e-4, -1e-3
    x[3, 0, :2] = -448 * 6 * ts * np.array([1.0, 0.5])
    x = np.clip(x, -top, top)
    cache, *_ = make_cache(moe, [4], 1, 64, 16, k_scale=ts, v_scale=ts, fill=False)
    t = dev(x, torch.float64).to(DT[dtype])
    cache.append(0, t, -t, dev([0, 4]))
    assert cache.status() == 0
    for got, sign in zip(cache.read(0, dev([0, 4]), rows=4, dtype=DT[dtype]), (1.0, -1.0)):
        want = P.values(*P.quantise(sign * t.double().cpu().numpy(), ts), ts)
        assert np.array_equal(got.double().cpu().numpy(), torch.tensor(want).float().to(DT[dtype]).double().numpy())


def test_append_outside_the_sequence_is_reported(moe):
    cache, pool, *_ = make_cache(moe, [2, 5], 1, 64, 16, fill=False)
    x = torch.ones((8, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache.table[1, 0] = 99
    cache.append(0, x, x, dev([0, 4, 8]))  # two rows before the start of sequence 0; a page that is none
    assert cache.status() == moe.KV4_BAD_PAGE
    k, _ = cache.read(0, dev([0, 4, 8]), rows=8)
    assert (k[:2] == 0).all() and (k[2:4] == held_one()).all() and (k[4:] == 0).all()


def test_offsets_past_32_bits(moe):
    # two layers of 2.4 GB: the last pages of the last layer lie past 2^32 bytes
    heads, D, page, pages = 8, 256, 64, 16400
    cache = moe.Kv4Cache(2, pages, heads, D, page, 3, 4)
    assert cache.page_bytes * pages > 2 ** 31 and cache.page_bytes * pages * 2 > 2 ** 32
    cache.refs[:pages - 6] = 1
    cache.reserve(dev([70, 40, 0]))
    assert cache.table[0, :2].tolist() == [pages - 6, pages - 5] and cache.table[1, 0] == pages - 4
    cu = dev([0, 70, 110, 110])
    kv = torch.randn((110, 2, heads, D), device="cuda").to(torch.bfloat16)
    cache.append(1, kv[:, 0], kv[:, 1], cu)
    k, v = cache.read(1, cu, rows=110)
    for got, x in ((k, kv[:, 0]), (v, kv[:, 1])):
        want = P.values(*P.quantise(x[::29].double().cpu().numpy(), 1.0), 1.0)
        assert np.array_equal(got[::29].double().cpu().numpy(), want)
    q = torch.randn((110, heads, D), device="cuda").to(torch.bfloat16)
    out = cache.attend(1, q, cu, max_rows=70).double()
    see = torch.ones(70, 70, dtype=torch.bool, device="cuda").tril()
    z = torch.einsum("rhd,thd->hrt", q[:70].double(), k[:70].double()) * D ** -0.5
    want = torch.einsum("hrt,thd->rhd", z.masked_fill(~see, -float("inf")).softmax(-1), v[:70].double())
    assert (out[:70] - want).abs().max() <= 4 * 2.0 ** -8 + 4 * 2.0 ** -10  # values up to 4: BF16's half unit, p's rounding
    cache.fork(dev([1]), dev([2]))
    cache.reserve(dev([0, 0, 1]))  # the shared page is copied on both layers
    assert cache.table[2, 0] == pages - 3
    for layer in range(2):
        assert torch.equal(cache.pool[layer, pages - 3], cache.pool[layer, pages - 4])
    assert cache.status() == 0


# ---- pages ----

def same(cache, plain):
    assert np.array_equal(cache.table.cpu().numpy(), plain.table)
    assert np.array_equal(cache.lens.cpu().numpy(), plain.lens)
    assert np.array_equal(cache.refs.cpu().numpy(), plain.refs)
    assert np.array_equal(cache.pool.cpu().numpy(), plain.pool)


def random_cache(moe, lens, heads, D, page, layers, extra, max_pages, seed):
    cache, pool, table, lens, refs = make_cache(moe, lens, heads, D, page, layers=layers, extra_pages=extra, max_pages=max_pages,
                                                seed=seed, fill=False)
    rng = np.random.default_rng(seed)
    pool[:] = rng.integers(0, 256, pool.shape, dtype=np.uint8)
    cache.pool.copy_(dev(pool, torch.uint8))
    return cache, P.PlainPages(pool, table, lens, refs, heads, D, page)


@pytest.mark.parametrize("D,heads,page", [(64, 3, 16), (128, 2, 48), (256, 1, 32)])
@pytest.mark.parametrize("seed", range(4))
def test_pages_random_steps(moe, D, heads, page, seed):
    rng = np.random.default_rng(seed)
    n = 9
    cache, plain = random_cache(moe, rng.integers(0, 70, n), heads, D, page, 3, 40, 12, seed)
    for step in range(6):
        if step % 2 == 0:
            dst = rng.choice(n, 3, replace=False)
            src = rng.choice([s for s in range(n) if s not in dst], 3)
            cache.fork(dev(src), dev(dst))
            plain.fork(src, dst)
            same(cache, plain)
        new = rng.integers(-1, 9, n)
        cache.reserve(dev(new))
        plain.reserve(new)
        same(cache, plain)
        assert not plain.no_page and cache.status() == 0
        rows = np.maximum(new, 0)
        cu = cu_of(rows)
        keep = (rng.random(max(int(cu[-1]), 1)) < 0.5).astype(np.uint8)
        cache.compact(dev(keep, torch.uint8), dev(cu), max_rows=8)
        plain.compact(keep, cu)
        same(cache, plain)
        to = plain.lens - rng.integers(0, 20, n) * (rng.random(n) < 0.3)
        cache.trim(dev(to))
        plain.trim(to)
        same(cache, plain)
    assert cache.status() == 0
    cache.trim(dev(np.zeros(n)))
    assert (cache.refs == 0).all() and (cache.table == -1).all() and (cache.lens == 0).all()


def test_reserve_out_of_pages(moe):
    # 5 free pages of 16: sequence 0 takes two, 1 needs four and is refused, 2 (which needs none) still grows, 3 is
    # refused although one page would do; 4 has no room in its table
    cache, plain = random_cache(moe, [16, 32, 20, 16, 90], 1, 64, 16, 2, 5, 6, 1)
    new = [32, 64, 3, 1, 7]
    cache.reserve(dev(new))
    plain.reserve(new)
    same(cache, plain)
    assert plain.no_page and cache.status() == moe.KV4_NO_PAGE
    assert list(plain.lens) == [48, 32, 23, 16, 90]


def test_step_after_a_refused_reservation(moe):
    # 0 and 1 share a partly filled page and get no free one to copy it to, 2 grows inside its page, 3 has no room in
    # its table: a whole step leaves every byte of 0, 1 and 3 as it was, and does for 2 what it does without them
    lens, heads, D, page, layers = [21, 0, 18, 64], 2, 64, 16, 2
    cache, pool, table, lens, refs = make_cache(moe, lens, heads, D, page, layers=layers, extra_pages=0, max_pages=4, seed=3)
    cache.fork(dev([0]), dev([1]))
    before = [t.clone() for t in (cache.pool, cache.table, cache.lens, cache.refs)]
    rows, group = [3, 3, 3, 3], 4
    cu, keep = dev(cu_of(rows)), dev([0, 0, 1] * 4, torch.uint8)
    g = torch.Generator().manual_seed(7)
    k, v = (torch.randn((12, heads, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn((12, heads * group, D), generator=g).to(torch.bfloat16).cuda()

    def step(cache, only=None):
        new = dev([3 if only is None or s in only else 0 for s in range(4)])
        c, i = (cu, slice(0, 12)) if only is None else (dev([0, 0, 0, 3, 3]), slice(6, 9))
        cache.reserve(new)
        got = []
        for layer in range(layers):
            cache.append(layer, k[i], v[i], c)
            got += cache.read(layer, c, rows=q[i].shape[0])
            for hint in (3, 64):  # few rows a block, many rows a block
                lse = torch.full(q[i].shape[:2], 7.0, dtype=torch.float32, device="cuda")
                out = torch.full(q[i].shape, 7.0, dtype=torch.bfloat16, device="cuda")
                got += cache.attend(layer, q[i], c, max_rows=hint, out=out, lse=lse)
        cache.compact(keep[i], c, max_rows=3)
        return got

    got = step(cache)
    assert cache.status() == moe.KV4_NO_PAGE
    alone, *_ = make_cache(moe, lens, heads, D, page, layers=layers, extra_pages=0, max_pages=4, seed=3)
    want = step(alone, only=[2])
    assert alone.status() == 0
    out = torch.ones(12, dtype=torch.bool, device="cuda")
    out[6:9] = False
    for a, b in zip(got, want):
        assert torch.equal(a[6:9], b)
        assert (a[out] == (0 if a.dim() == 3 else -float("inf"))).all()
    assert cache.lens.tolist() == [21, 21, 19, 64] and torch.equal(cache.table, before[1]) and torch.equal(cache.refs, before[3])
    assert torch.equal(cache.pool, alone.pool)
    mine = table[2, :2]
    others = [p for p in range(cache.pool.shape[1]) if p not in mine]
    assert torch.equal(cache.pool[:, others], before[0][:, others])


def test_refused_sequences_take_part_again(moe):
    lens = [21, 0, 40]
    cache, _ = random_cache(moe, lens, 2, 64, 16, 2, 0, 4, 5)
    cache.fork(dev([0]), dev([1]))
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")

    def held(rows, seq):  # whether the sequence's rows are written and read
        cu = dev([0 if s <= seq else rows for s in range(4)])
        cache.append(1, x[:rows], x[:rows], cu)
        return bool((cache.read(1, cu, rows=rows)[0] == held_one()).all())

    cache.reserve(dev([2, 0, 0]))
    assert cache.status() == moe.KV4_NO_PAGE and not held(2, 0) and held(1, 2)
    cache.reserve(dev([0, 0, 3]))      # another sequence's reservation changes nothing for it
    assert not held(2, 0) and held(3, 2)
    cache.trim(dev([21, 21, 16]))      # two pages are free: its next reservation succeeds
    cache.reserve(dev([2, 0, 0]))
    assert held(2, 0) and cache.status() == 0
    cache.reserve(dev([0, 30, 0]))     # refused, then cut
    assert cache.status() == moe.KV4_NO_PAGE and not held(1, 1)
    cache.trim(dev([100, 16, 100]))
    bits = [cache.read(1, cu, rows=n)[0].view(torch.int16) for cu, n in ((dev([0, 0, 16, 16]), 16), (dev([0, 23, 23, 23]), 23))]
    assert torch.equal(bits[0], bits[1][:16]) and bits[0].any()  # the page that 0 and 1 share
    assert held(1, 2)
    cache.reserve(dev([0, 60, 0]))     # refused, then replaced by a fork
    assert cache.status() == moe.KV4_NO_PAGE
    cache.fork(dev([2]), dev([1]))
    assert (cache.read(1, dev([0, 0, 1, 2]), rows=2)[0] == held_one()).all() and cache.status() == 0


def test_reserve_shared_page_of_several_writers(moe):
    # the last page of a sequence shared by three, two of which write: both copy; then all three
    for writers in ([1, 2], [0, 1, 2]):
        cache, plain = random_cache(moe, [21, 0, 0, 5], 2, 64, 16, 2, 12, 4, 2)
        cache.fork(dev([0, 0]), dev([1, 2]))
        plain.fork([0, 0], [1, 2])
        new = [13 if s in writers else 0 for s in range(4)]
        cache.reserve(dev(new))
        plain.reserve(new)
        same(cache, plain)
        assert cache.status() == 0


def test_reserve_many_sequences_and_pages(moe):
    # more sequences than the allocation keeps in shared memory, pages over several rounds
    rng = np.random.default_rng(5)
    cache, plain = random_cache(moe, rng.integers(0, 20, 5000), 1, 64, 16, 1, 9000, 4, 3)
    new = rng.integers(0, 20, 5000)
    cache.reserve(dev(new))
    plain.reserve(new)
    same(cache, plain)
    assert cache.status() == 0


@pytest.mark.parametrize("kept", [[], [0], [0, 1, 2], [63], [5, 6, 7, 40], list(range(64)), list(range(0, 64, 2)), list(range(1, 64))])
def test_compact_patterns(moe, kept):
    cache, plain = random_cache(moe, [70, 64, 200], 2, 128, 16, 2, 4, 16, 4)
    keep = np.zeros(3 * 64, dtype=np.uint8)
    for s in range(3):
        keep[64 * s + np.array(kept, dtype=int)] = 1 + 100 * s  # any value but 0 keeps a row
    cu = [0, 64, 128, 192]
    cache.compact(dev(keep, torch.uint8), dev(cu), max_rows=64)
    plain.compact(keep, np.array(cu))
    same(cache, plain)
    assert cache.status() == 0


def test_fork_bad_sequences_are_reported(moe):
    cache, plain = random_cache(moe, [20, 0, 3], 1, 64, 16, 1, 4, 4, 1)
    cache.fork(dev([0, 7, 2]), dev([1, 0, 2]))
    plain.fork([0], [1])
    same(cache, plain)
    assert cache.status() == moe.KV4_BAD_SEQ


def test_another_current_device_is_refused(moe, monkeypatch):
    from routed_moe_decode_gb300 import _routing
    cache, *_ = make_cache(moe, [20, 30], 2, 64, 16)
    cu, q = dev([0, 1, 2]), torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    r = moe.Routing(16, 2)
    route = (torch.zeros((3, 16), device="cuda"), None, torch.zeros((3, 2), dtype=torch.int32, device="cuda"),
             torch.zeros((3, 2), device="cuda"))
    calls = [lambda: cache.append(0, q, q, cu), lambda: cache.read(0, cu, rows=2), lambda: cache.attend(0, q, cu, max_rows=1),
             lambda: cache.reserve(dev([0, 0])), lambda: cache.trim(dev([20, 30])), lambda: cache.fork(dev([0]), dev([1])),
             lambda: cache.compact(dev([1, 1], torch.uint8), cu, max_rows=1), cache.status, lambda: r.route(*route),
             lambda: moe.Kv4Cache(1, 4, 2, 64, 16, 2, 4, device="cuda:0")]
    before = [t.clone() for t in (cache.pool, cache.table, cache.lens, cache.refs)]
    monkeypatch.setattr(_routing, "_devices", 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)  # the tensors lie on device 0
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    monkeypatch.undo()
    for a, b in zip(before, (cache.pool, cache.table, cache.lens, cache.refs)):
        assert torch.equal(a, b)
    for call in calls:
        call()


def test_refusals(moe):
    with pytest.raises(moe.MoeError):
        moe.Kv4Cache(1, 4, 2, 96, 16, 2, 4)  # head size
    with pytest.raises(moe.MoeError):
        moe.Kv4Cache(1, 4, 2, 64, 24, 2, 4)  # page size
    with pytest.raises(moe.MoeError):
        moe.Kv4Cache(1, 4, 2, 64, 16, 2, 4, k_scale=0.0)
    with pytest.raises(ValueError):
        moe.Kv4Cache(1, 4, 2, 64, 16, 2, 4, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    cache, *_ = make_cache(moe, [20, 30], 2, 64, 16)
    cu = dev([0, 1, 2])
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (q.float(), q[..., :32], q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            cache.attend(0, bad, cu, max_rows=1)
    with pytest.raises(moe.MoeError):  # 5 query heads over 2
        cache.attend(0, torch.zeros((2, 5, 64), dtype=torch.bfloat16, device="cuda"), cu, max_rows=1)
    with pytest.raises(moe.MoeError):  # rows 4 elements off a 16-byte boundary
        wide = torch.zeros((2, 4, 72), dtype=torch.bfloat16, device="cuda")
        cache.attend(0, wide[..., 4:68], cu, max_rows=1)
    with pytest.raises(moe.MoeError):
        cache.attend(1, q, cu, max_rows=1)  # no such layer
    with pytest.raises(moe.MoeError):
        cache.attend(0, q, cu, max_rows=1, window=-1)
    tree = torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(moe.MoeError):
        cache.attend(0, q, cu, max_rows=1, window=4, tree=tree)
    with pytest.raises(moe.MoeError):
        cache.attend(0, q, cu, max_rows=65, tree=tree)
    with pytest.raises(ValueError):
        cache.attend(0, q, cu[:2], max_rows=1)
    with pytest.raises(ValueError):
        cache.attend(0, q, cu.long(), max_rows=1)
    with pytest.raises(ValueError):
        cache.append(0, q[:, :2], q[:1, :2], cu)
    with pytest.raises(ValueError):
        cache.reserve(dev([1, 2, 3]))
    with pytest.raises(moe.MoeError):
        cache.compact(torch.zeros(2, dtype=torch.uint8, device="cuda"), cu, max_rows=65)
    assert cache.attend(0, q[:0], dev([0, 0, 0]), max_rows=0).shape == (0, 4, 64)
    assert cache.status() == 0
