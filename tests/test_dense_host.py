"""Host-side checks of the dense path in 8 bits that need no GPU: the header's functions are exported and bound, bad
arguments are refused before anything is enqueued, and the tests' plain implementation agrees with the golden table."""
import ctypes
import os
import re

import pytest
import torch

import dense_plain as P
import __graft_entry__
from conftest import ROOT, read_golden


@pytest.fixture(scope="module")
def L():
    __graft_entry__.build()
    from routed_moe_decode_gb300 import _lib
    return _lib


def test_header_functions_are_exported_and_bound(L):
    text = open(os.path.join(ROOT, "include", "moe_dense.h")).read()
    names = set(re.findall(r"^MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text, flags=re.M))
    assert len(names) == 5
    lib = ctypes.CDLL(L.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert names <= set(L.SIGNATURES)


def test_plain_codes_are_the_golden_table(L):
    table = {int(r[0], 0): float(r[1]) for r in read_golden("e4m3_values.txt") if r[1].lower() not in ("nan", "-nan")}
    for code, value in table.items():
        if code < 127:
            assert float(P.MAGNITUDES[code]) == value
    x = torch.randn(20000, dtype=torch.float64) * 60
    assert torch.equal(P.e4m3_codes(x.float().double()).to(torch.uint8).view(torch.float8_e4m3fn).float(),
                       x.float().clamp(-448, 448).to(torch.float8_e4m3fn).float())


P0 = 0x100000  # an address that is never used


def refused(L, fn, good, changes):
    """Each change (positions to values) of a good call is refused with its status; rows of 0 make the good one a call
    that does nothing."""
    f = getattr(L.lib(), fn)
    for change, rc in changes:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert f(*args, None) == rc, (fn, change)


def test_norm_refuses_bad_arguments(L):
    #       0  1  2    3  4   5    6  7   8    9   10 11 12    13  14   15  16   17 18  19   20  21 22
    good = [4, 1, 256, 1, P0, 256, 0, P0, 256, P0, 1, 0, 1e-6, P0, 256, 2 * P0, 256, 0, P0, 256, P0, 1, 4]
    INV, UNS = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    refused(L, "moe_rms_norm", good, [
        ({0: 0}, L.MOE_OK), ({1: 0}, L.MOE_OK), ({0: -1}, INV), ({1: -1}, INV), ({2: 0}, INV), ({3: 3}, INV), ({3: -1}, INV),
        ({4: None}, INV), ({9: None}, INV), ({10: 7}, INV), ({12: -1.0}, INV), ({12: float("nan")}, INV),
        ({12: float("inf")}, INV), ({4: P0 + 1}, INV), ({7: P0 + 1}, INV), ({13: P0 + 1}, INV), ({15: P0 + 1}, INV),
        ({20: P0 + 2}, INV), ({9: P0 + 1}, INV),
        ({7: None}, INV),                       # residual_out without a residual
        ({7: None, 13: None, 15: None, 18: None, 20: None}, INV),  # nothing to write
        ({20: None}, INV), ({18: None}, INV),   # codes and scales go together
        ({15: P0}, INV),                        # normed in residual_out's place
        ({19: 255}, INV), ({0: 1 << 20, 1: 1 << 20}, UNS), ({2: 1 << 25, 19: 1 << 25}, UNS),
        # rows of an output on top of each other
        ({14: 255}, INV), ({16: 0}, INV), ({21: 0}, INV), ({22: 0}, INV), ({22: 3}, INV), ({22: 1}, INV),
        ({1: 3, 6: 256, 5: 768, 17: 256, 16: 767, 7: None, 13: None, 18: None, 20: None}, INV),
        ({1: 3, 6: 256, 5: 768, 17: 1023, 16: 256, 7: None, 13: None, 18: None, 20: None}, INV)])


def test_quantize_refuses_bad_arguments(L):
    #       0  1    2  3  4   5    6   7    8   9  10
    good = [4, 256, 0, 1, P0, 256, P0, 256, P0, 1, 4]
    INV, UNS = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    refused(L, "moe_quantize_rows", good, [
        ({0: 0}, L.MOE_OK), ({0: -1}, INV), ({1: 0}, INV), ({3: 9}, INV), ({4: None}, INV), ({6: None}, INV), ({8: None}, INV),
        ({4: P0 + 1}, INV), ({8: P0 + 1}, INV), ({7: 200}, INV), ({0: 1 << 30, 1: 1 << 20, 7: 1 << 20}, UNS), ({1: 1 << 25}, UNS),
        ({9: 0}, INV), ({10: 0}, INV), ({10: 3}, INV), ({10: 1}, INV)])


def test_matmul_refuses_bad_arguments(L):
    #       0  1    2    3  4   5    6   7  8  9   10  11    12  13   14 15
    good = [4, 256, 256, 0, P0, 256, P0, 1, 4, P0, P0, None, P0, 256, 1, P0]
    INV, UNS = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    refused(L, "moe_fp8_matmul", good, [
        ({0: 0}, L.MOE_OK), ({0: -1}, INV), ({1: 0}, INV), ({2: 0}, INV), ({3: -1}, INV), ({14: 5}, INV), ({2: 250}, UNS),
        ({3: 1025, 11: P0}, UNS), ({4: None}, INV), ({6: None}, INV), ({9: None}, INV), ({10: None}, INV), ({12: None}, INV),
        ({15: None}, INV), ({3: 2}, INV), ({11: P0}, INV), ({4: P0 + 8}, INV), ({9: P0 + 8}, INV), ({12: P0 + 1}, INV),
        ({5: 240}, INV), ({5: 264}, INV), ({13: 255}, INV), ({3: 1024, 11: P0, 1: 1 << 22, 13: 1 << 22}, UNS)])
    lib = L.lib()
    assert lib.moe_selftest_fp8_matmul(*good, 2, 100, None) == INV
    assert lib.moe_selftest_fp8_matmul(*good, 0, -1, None) == INV


def test_logprobs_refuse_bad_arguments(L):
    #       0  1    2  3   4    5    6   7  8  9  10  11  12  13  14
    good = [4, 500, 0, P0, 500, 1.0, P0, 1, 1, 8, P0, P0, P0, P0, P0]
    INV, UNS = L.MOE_ERR_INVALID_ARG, L.MOE_ERR_UNSUPPORTED
    refused(L, "moe_token_logprobs", good, [
        ({0: 0}, L.MOE_OK), ({0: -1}, INV), ({1: 0}, INV), ({2: 3}, INV), ({3: None}, INV), ({3: P0 + 2}, INV), ({5: 0.0}, INV),
        ({5: -1.0}, INV), ({5: float("nan")}, INV), ({5: float("inf")}, INV), ({6: None}, INV), ({7: -1}, INV), ({7: 1025}, UNS),
        ({9: -1}, INV), ({9: 33}, UNS), ({9: 501}, INV), ({9: 0}, INV), ({10: P0 + 2}, INV), ({1: (1 << 30) + 1}, UNS)])


def test_status_refuses_bad_arguments(L):
    lib = L.lib()
    bits = ctypes.c_uint32(0)
    assert lib.moe_dense_read_status(None, 0, ctypes.byref(bits), None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_dense_read_status(P0 + 1, 0, ctypes.byref(bits), None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_dense_read_status(P0, 0, None, None) == L.MOE_ERR_INVALID_ARG


def test_tensors_of_the_host_are_refused(L):
    import routed_moe_decode_gb300 as moe
    codes = torch.zeros(4, 32, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        moe.Fp8Rows(codes, torch.zeros(4, 1))
    with pytest.raises(ValueError):
        moe.RmsNorm(torch.ones(32))
    with pytest.raises(ValueError):
        moe.Fp8Linear(codes, torch.zeros(1, 1))
    with pytest.raises(ValueError):
        moe.quantize_rows(torch.zeros(4, 32))
    with pytest.raises(ValueError):
        moe.token_logprobs(torch.zeros(4, 32), torch.zeros(4, dtype=torch.int32))


def test_logprobs_refuse_scales_far_from_one(L):
    good = [4, 500, 0, P0, 500, 1.0, P0, 1, 1, 8, P0, P0, P0, P0, P0]
    refused(L, "moe_token_logprobs", good, [({5: 2.0 ** -81}, L.MOE_ERR_UNSUPPORTED), ({5: 2.0 ** 81}, L.MOE_ERR_UNSUPPORTED)])
