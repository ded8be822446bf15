"""The products' bounded waits: an arrival that nothing makes and limits that end in the middle of the work make them run
out, without a GPU fault; the launch completes with its status bit, and the next product has a clean one's bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_moe_decode_gb300 as m
    return m


# rows, n, k, groups: the kernel of few rows (one CTA a tile, parts of k in clusters, 128-row tiles), that of many, groups
CASES = [(4, 40000, 512, 0), (4, 512, 4096, 0), (100, 1024, 512, 0), (600, 2048, 1024, 0), (2500, 700, 272, 0), (64, 256, 512, 32),
         (900, 512, 512, 6)]


@pytest.mark.parametrize("rows,n,k,groups", CASES)
def test_waits_run_out(moe, rows, n, k, groups):
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    x = moe.quantize_rows(torch.randn(rows, k, generator=g, device="cuda"))
    lead = (groups,) if groups else ()
    codes = (torch.randn(*lead, n, k, generator=g, device="cuda") * 50).to(torch.float8_e4m3fn)
    scales = torch.rand(*lead, -(-n // 128), -(-k // 128), generator=g, device="cuda")
    linear = moe.Fp8Linear(codes, scales)
    offsets = torch.arange(groups + 1, device="cuda").mul(rows).div(groups, rounding_mode="floor").to(torch.int32) if groups else None
    clean = linear(x, offsets=offsets)
    torch.cuda.synchronize()
    assert linear.status() == 0
    out = torch.empty_like(clean)
    for stuck, limit in ((1, 1 << 20), (0, 0), (0, 3000), (1, 0)):
        moe.selftest_fp8_matmul(linear, x, out, stuck=stuck, wait_limit_cycles=limit, offsets=offsets)
        torch.cuda.synchronize()
        bits = linear.status()
        assert bits & ~moe.DENSE_TIMEOUT == 0
        if stuck:  # without, what a wait is for may come within the hardware's own try
            assert bits == moe.DENSE_TIMEOUT
        again = linear(x, offsets=offsets)
        torch.cuda.synchronize()
        assert linear.status() == 0 and torch.equal(again, clean)
