"""Host-side checks of the 4-bit cache and the grouped router that need no GPU: the headers'
functions are exported and bound, bad arguments are refused before anything is enqueued, sizes
are as documented, and the tests' plain implementation agrees with the golden tables."""
import ctypes
import os
import re

import numpy as np
import pytest

import kv4_plain as P
import __graft_entry__
from conftest import ROOT, read_golden


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    from routed_moe_decode_gb300 import _lib
    return _lib


def cache_args(L, **kw):
    a = L.Kv4Args()
    v = dict(pool=0x100000, table=0x200000, lens=0x300000, refs=0x400000, workspace=0x500000, workspace_bytes=1 << 40,
             layers=2, pages=8, kv_heads=2, head_dim=128, page_size=64, seqs=4, max_pages=4, k_scale=1.0, v_scale=1.0)
    v.update(kw)
    for n, x in v.items():
        setattr(a, n, x)
    return ctypes.byref(a)


def test_header_functions_are_exported_and_bound(L):
    text = open(os.path.join(ROOT, "include", "moe_kv4.h")).read()
    names = set(re.findall(r"^MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text, flags=re.M))
    assert len(names) >= 12
    lib = ctypes.CDLL(L.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert names <= set(L.SIGNATURES)


def test_cache_sizes(L):
    lib = L.lib()
    assert lib.moe_kv4_check(cache_args(L)) == 0
    assert lib.moe_kv4_page_bytes(cache_args(L)) == 2 * 4 * 18 * 128
    assert lib.moe_kv4_page_bytes(cache_args(L, head_dim=64, page_size=16, kv_heads=1)) == 18 * 64
    ws = lib.moe_kv4_workspace_bytes(cache_args(L))
    assert ws > 0 and ws % 256 == 0
    for kw, rc in ((dict(head_dim=96), -2), (dict(page_size=24), -2), (dict(page_size=2048), -2), (dict(seqs=1 << 17), -2),
                   (dict(kv_heads=0), -1), (dict(pages=0), -1), (dict(layers=-1), -1), (dict(max_pages=0), -1),
                   (dict(k_scale=0.0), -1), (dict(v_scale=float("nan")), -1), (dict(v_scale=float("inf")), -1)):
        assert lib.moe_kv4_check(cache_args(L, **kw)) == rc, kw
        assert lib.moe_kv4_workspace_bytes(cache_args(L, **kw)) == 0
    assert lib.moe_kv4_check(None) == -1


def test_cache_calls_refuse_bad_arguments(L):
    lib, ok = L.lib(), cache_args(L)
    p = 0x600000
    append = [0, p, 256, 128, p, 256, 128, 0, p, 4, None]
    attend = [0, p, 512, 128, 4, 0, p, 4, 1, 0.1, 0, None, p, None, None]

    def with_(args, i, v):
        return args[:i] + [v] + args[i + 1:]

    for i, v in ((0, -1), (0, 2), (1, None), (1, p + 2), (2, 100), (3, 4), (4, None), (5, 7), (7, 5), (8, None), (8, p + 2), (9, -1)):
        assert lib.moe_kv4_append(ok, *with_(append, i, v)) == L.MOE_ERR_INVALID_ARG, (i, v)
    for i, v in ((0, 9), (1, None), (1, p + 8), (2, 4), (3, 12), (4, 3), (4, 0), (5, 2), (6, None), (7, -1), (8, -1),
                 (9, float("nan")), (10, -1), (11, p + 4), (12, None), (12, p + 8), (13, p + 2)):
        assert lib.moe_kv4_attend(ok, *with_(attend, i, v)) == L.MOE_ERR_INVALID_ARG, (i, v)
    tree = with_(attend, 11, p)
    assert lib.moe_kv4_attend(ok, *with_(tree, 10, 8)) == L.MOE_ERR_UNSUPPORTED  # window and tree
    assert lib.moe_kv4_attend(ok, *with_(tree, 8, 65)) == L.MOE_ERR_UNSUPPORTED  # more rows than a tree's bits
    assert lib.moe_kv4_attend(ok, *with_(attend, 7, (1 << 31) - 1)) == L.MOE_ERR_UNSUPPORTED
    # nothing to do is no error, whatever the other pointers are
    assert lib.moe_kv4_append(ok, *with_(with_(append, 9, 0), 1, None)) == 0
    assert lib.moe_kv4_attend(ok, *with_(with_(attend, 7, 0), 1, None)) == 0
    assert lib.moe_kv4_read(ok, 0, None, None, 0, p, 4, None) == 0
    assert lib.moe_kv4_read(ok, 0, p + 2, None, 0, p, 4, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_kv4_fork(ok, None, None, 0, None) == 0
    assert lib.moe_kv4_fork(ok, p, p, 5, None) == L.MOE_ERR_INVALID_ARG  # more than there are sequences
    assert lib.moe_kv4_reserve(ok, None, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_kv4_trim(ok, p + 1, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_kv4_compact(ok, p, p, 4, 65, None) == L.MOE_ERR_UNSUPPORTED
    assert lib.moe_kv4_compact(ok, None, p, 4, 4, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_kv4_read_status(ok, 1, None, None) == L.MOE_ERR_INVALID_ARG
    for kw, rc in ((dict(pool=0), -1), (dict(pool=0x100010), -1), (dict(table=0), -1), (dict(lens=2), -1), (dict(refs=0), -1),
                   (dict(workspace=0), -3), (dict(workspace=0x500010), -3), (dict(workspace_bytes=1024), -3)):
        assert lib.moe_kv4_append(cache_args(L, **kw), *append) == rc, kw
        assert lib.moe_kv4_reserve(cache_args(L, **kw), p, None) == rc, kw


def test_routing_refuses_bad_arguments(L):
    lib, p = L.lib(), 0x600000
    good = dict(E=64, k=4, softmax=0, groups=8, keep_groups=2, top2=1, renormalise=1, scale=1.0)

    def call(T=4, logits=p, stride=64, dtype=0, bias=None, ids=p, weights=p, **kw):
        r = L.RoutingArgs(**dict(good, **kw))
        return lib.moe_route_grouped(ctypes.byref(r), T, logits, stride, dtype, bias, ids, weights, None)

    assert call(T=0, logits=None, ids=None, weights=None) == 0
    for kw in (dict(T=-1), dict(logits=None), dict(logits=p + 2), dict(stride=63), dict(dtype=3), dict(dtype=-1), dict(ids=None),
               dict(weights=None), dict(bias=p + 1), dict(E=0), dict(k=0), dict(k=65), dict(groups=0), dict(groups=7),
               dict(keep_groups=0), dict(keep_groups=9), dict(k=17, keep_groups=2), dict(scale=float("nan")),
               dict(scale=float("inf"))):
        assert call(**kw) == L.MOE_ERR_INVALID_ARG, kw
    for kw in (dict(T=65537), dict(k=33, keep_groups=8), dict(E=2048, stride=2048), dict(groups=64, keep_groups=64)):
        assert call(**kw) == L.MOE_ERR_UNSUPPORTED, kw
    assert lib.moe_route_grouped(None, 4, p, 64, 0, None, p, p, None) == L.MOE_ERR_INVALID_ARG


def test_plain_tables_agree_with_the_golden_files():
    for row in read_golden("e2m1_values.txt"):
        code, value = int(row[0], 0), float(row[-1])
        assert P.values(np.full(16, code, dtype=np.uint8), np.array([0x38], dtype=np.uint8), 1.0)[0] == value
    for row in read_golden("e4m3_values.txt"):
        bits, value = int(row[0], 0), row[-1]
        got = P.e4m3_value(bits)
        assert np.isnan(got) if value.lower() == "nan" else got == float(value), row


def test_plain_tiles_round_trip():
    rng = np.random.default_rng(0)
    for D in (64, 128, 256):
        tile = rng.integers(0, 256, 18 * D, dtype=np.uint8)
        assert np.array_equal(P.make_tile(*P.tile_fields(tile, D)), tile)
        kc, vc, ks, vs = P.tile_fields(tile, D)
        # channel 37 of token 5: K in piece 1, byte 2 of its 16, high nibble; V in byte 18 of the token
        assert kc[5, 37] == tile[256 + 5 * 16 + 2] >> 4 and vc[5, 37] == tile[8 * D + 5 * D // 2 + 18] >> 4
        assert ks[5, 2] == tile[16 * D + 5 * D // 16 + 2] and vs[5, 2] == tile[17 * D + 5 * D // 16 + 2]


def test_plain_quantise_is_the_nearest():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 32)) * 3
    code, sb = P.quantise(x, 0.5)
    v = P.values(code, sb, 0.5)
    d = np.repeat(P.e4m3_value(sb) * 0.5, 16, axis=1)
    grid = np.concatenate([P.E2M1, -P.E2M1])
    best = np.abs(x[..., None] - grid * d[..., None]).min(-1)
    assert np.allclose(np.abs(x - v), best, rtol=0, atol=1e-12)


def test_scales_out_of_range_are_refused(L):
    # above 2^119 a block's factor (448 times the tensor scale) and then 6 times it are no floats, and values would be held as 0
    lib, p = L.lib(), 0x600000
    for kw in (dict(k_scale=2.0 ** 120), dict(v_scale=3e38)):
        assert lib.moe_kv4_check(cache_args(L, **kw)) == L.MOE_ERR_UNSUPPORTED, kw
        assert lib.moe_kv4_workspace_bytes(cache_args(L, **kw)) == 0
    assert lib.moe_kv4_check(cache_args(L, k_scale=2.0 ** 119, v_scale=2.0 ** -100)) == 0
    # the factor of the scores
    attend = [0, p, 512, 128, 4, 0, p, 4, 1, 1e30, 0, None, p, None, None]
    assert lib.moe_kv4_attend(cache_args(L, k_scale=1e20), *attend) == L.MOE_ERR_UNSUPPORTED
