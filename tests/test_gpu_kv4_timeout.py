"""The bounded waits of the attention over the 4-bit cache.

Both kernels wait on barriers in shared memory for copies, and the wide one for the work of other
warps and for products.  A wait that runs out ends the launch with MOE_KV4_TIMEOUT, after what is in
flight has landed.  The failure is an arrival that nothing makes, and limits so short that waits may give
up on work that is still under way; the next call on the same cache has to give the bits of a clean one.
"""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_moe_decode_gb300 as m
    return m


# few rows: the kernel that streams tiles by warps; many: the one with roles in warps of their own
@pytest.mark.parametrize("D,group", [(64, 1), (64, 3), (64, 8), (128, 1), (128, 4), (256, 1), (256, 4), (64, 40), (128, 40),
                                     (256, 40)])
def test_waits_that_run_out_end_the_call_and_leave_the_cache_usable(moe, D, group):
    seqs, heads, n, page, rows = 8, 8, 4096, 64, 4
    cache = moe.Kv4Cache(1, seqs * (n // page + 1), heads, D, page, seqs, n // page + 1)
    cache.reserve(torch.full((seqs,), n, dtype=torch.int32, device="cuda"))
    kv = torch.randn((seqs * n, 2, heads, D), device="cuda").to(torch.bfloat16)
    starts = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    cache.append(0, kv[:, 0], kv[:, 1], starts * n)
    q = torch.randn((seqs * rows, heads * group, D), device="cuda").to(torch.bfloat16)
    cu = starts * rows
    want = cache.attend(0, q, cu, max_rows=rows)
    assert cache.status() == 0
    out = torch.empty_like(want)
    other = torch.empty(1 << 26, dtype=torch.float32, device="cuda")  # twice the L2 cache
    # a limit that no wait reaches changes nothing
    assert torch.equal(moe.selftest_kv4_attend(cache, 0, q, cu, rows, out, 0, 1 << 32), want) and cache.status() == 0
    for stuck, limit in ((1, 1 << 20), (1, 0), (0, 0), (0, 300), (0, 1000), (0, 3000)):
        other.fill_(1.0)  # the tiles come from memory
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        moe.selftest_kv4_attend(cache, 0, q, cu, rows, out, stuck, limit)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 5.0
        status = cache.status()
        assert status == moe.KV4_TIMEOUT or (status == 0 and not stuck), (stuck, limit, status)
        if status == 0:
            assert torch.equal(out, want)
        assert torch.equal(cache.attend(0, q, cu, max_rows=rows), want) and cache.status() == 0


def test_selftest_refuses_bad_arguments(moe):
    cache = moe.Kv4Cache(1, 4, 1, 64, 16, 1, 4)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    for stuck, limit in ((0, -1), (2, 1), (-1, 1)):
        with pytest.raises(moe.MoeError):
            moe.selftest_kv4_attend(cache, 0, q, torch.zeros(2, dtype=torch.int32, device="cuda"), 1, torch.empty_like(q), stuck, limit)
