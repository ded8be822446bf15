"""The dense path in 8 bits against plain 64-bit implementations (tests/dense_plain.py)."""
import math

import pytest
import torch

import dense_plain as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # half a step of FP32, relative
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import routed_moe_decode_gb300 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *shape, dtype=FP32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def half_step(ref, dtype):
    """Half a step of `dtype` at `ref`, subnormal values included."""
    tiny = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}[dtype]
    return ref.abs() * (torch.finfo(dtype).eps / 2) + tiny


def codes_of(rows):
    return rows.codes.contiguous().view(torch.uint8).long()


def equal_codes(got, want):
    """Equal codes, +0 and -0 being the same."""
    fold = lambda c: torch.where(c == 128, torch.zeros_like(c), c)  # noqa: E731
    return torch.equal(fold(got), fold(want))


def check_quantized(rows, n, rel):
    """Rows in 8 bits against the 64-bit values n that they hold, computed with the relative error `rel`."""
    _, scales = P.quantize(n)
    s = rows.scales.double()
    assert ((s - scales.double()).abs() <= scales.double() * (rel + 2 * U) + 2.0 ** -149).all()
    v = P.values(rows.codes, rows.scales)
    se = s.repeat_interleave(128, -1)[:, :n.shape[1]]
    # a code is off by half a step, 2^-4 of the value or 2^-10 of the scale; the quotient by rel and the scale's error
    bound = torch.maximum(n.abs() * 2.0 ** -4, se * 2.0 ** -10) * (1 + 1e-5) + n.abs() * (2 * rel + 4 * U)
    assert ((v - n).abs() <= bound).all(), float(((v - n).abs() - bound).max())


# ---- norm ----

# factor: sums of squares (a chain of 8, one of a row's steps, shuffles) below 60 roundings of positive sums, halved by the
# root, and four more; h * w, 1 + w, the last product
NORM_REL = 40 * U

NORMS = [(1, 1), (3, 7), (5, 64), (17, 128), (33, 120), (4, 256), (9, 500), (6, 512), (3, 1000), (8, 1024), (5, 1030), (2, 2048),
         (3, 2047), (700, 2048), (2, 4096), (3, 5000), (2, 8192), (3, 8193), (2, 20000), (1, 65536)]


@pytest.mark.parametrize("rows,d", NORMS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_norm(moe, rows, d, dtype):
    g = gen(rows * 100003 + d)
    x, r = rand(g, rows, d, dtype=dtype), rand(g, rows, d, dtype=dtype, scale=3.0)
    wtype = {BF16: FP32, FP16: FP16, FP32: BF16}[dtype]
    w = (1 + rand(g, d, scale=0.2)).to(wtype)
    for residual, one_plus, quantize in ((True, False, True), (False, True, False), (True, True, False), (False, False, True)):
        if quantize and d % 16 and d > 1030:
            continue
        norm = moe.RmsNorm(w, eps=1e-5, one_plus=one_plus)
        n, h, q = norm(x, residual=r if residual else None, quantize=quantize)
        want_h = (x.float() + r.float()).to(dtype) if residual else x
        if residual:
            assert torch.equal(h, want_h)
        else:
            assert h is None
        want = P.rms_norm(want_h, w, 1e-5, one_plus)
        assert ((n.double() - want).abs() <= half_step(want, dtype) * (1 + 2.0 ** -8) + want.abs() * NORM_REL).all()
        if quantize:
            check_quantized(q, want, NORM_REL)
        else:
            assert q is None


def test_norm_strides_heads_and_places(moe):
    g = gen(1)
    qkv = rand(g, 37, 12, 96, dtype=BF16)
    w = rand(g, 96, dtype=BF16)
    before = qkv.clone()
    # query heads of a fused projection, in place; then the same with rows in 8 bits
    q = qkv[:, 2:10]
    want = P.rms_norm(q, w, 1e-6, True)
    norm = moe.RmsNorm(w, one_plus=True)
    n, _, fp8 = norm(q, normed=q, quantize=True)
    assert n.data_ptr() == q.data_ptr()
    assert ((q.double() - want).abs() <= half_step(want, BF16) * (1 + 2.0 ** -8) + want.abs() * NORM_REL).all()
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 10:], before[:, 10:])
    check_quantized(fp8, want.reshape(37 * 8, 96), NORM_REL)
    # unaligned rows and odd strides
    buf = rand(g, 19, 203, dtype=FP16)
    x = buf[:, 1:201]
    w2 = rand(g, 200)
    n, _, _ = moe.RmsNorm(w2)(x)
    want = P.rms_norm(x, w2, 1e-6, False)
    assert ((n.double() - want).abs() <= half_step(want, FP16) * (1 + 2.0 ** -8) + want.abs() * NORM_REL).all()
    # the sum in the residual's place, the norm in x's; long rows are read twice
    for d in (2048, 12000, 333):
        x, r, w3 = rand(g, 5, d, dtype=BF16), rand(g, 5, d, dtype=BF16), rand(g, d)
        h = (x.float() + r.float()).to(BF16)
        want = P.rms_norm(h, w3, 1e-6, False)
        n, ro, _ = moe.RmsNorm(w3)(x, residual=r, residual_out=r, normed=x)
        assert ro.data_ptr() == r.data_ptr() and torch.equal(r, h)
        assert ((x.double() - want).abs() <= half_step(want, BF16) * (1 + 2.0 ** -8) + want.abs() * NORM_REL).all()
        # without its sum written
        x, r = rand(g, 5, d, dtype=BF16), rand(g, 5, d, dtype=BF16)
        want = P.rms_norm((x.float() + r.float()).to(BF16), w3, 1e-6, False)
        n, ro, _ = moe.RmsNorm(w3)(x, residual=r, residual_out=False, normed=r)
        assert ro is None and ((r.double() - want).abs() <= half_step(want, BF16) * (1 + 2.0 ** -8) + want.abs() * NORM_REL).all()


def test_norm_zeros_infinities_and_refusals(moe):
    w = torch.ones(256, device="cuda")
    norm = moe.RmsNorm(w, eps=0.0)
    x = torch.zeros(4, 256, device="cuda")
    x[1], x[2, 7], x[3, 200] = 1.0, math.inf, math.nan
    n, _, q = moe.RmsNorm(w)(x, quantize=True)
    assert (n[0] == 0).all() and (q.scales[0] == 0).all() and (q.codes[0].float() == 0).all()
    assert torch.isnan(n[2, 7]) and torch.isnan(n[3]).all()
    assert torch.isnan(q.scales[3]).all() and torch.isfinite(q.scales[:2]).all()
    assert torch.isnan(norm(x)[0][0]).all()  # 0 / 0 without an eps
    y = rand(gen(1), 4, 256)
    with pytest.raises(ValueError):
        norm(y[:, ::2])
    with pytest.raises(ValueError):
        norm(y.double())
    with pytest.raises(ValueError):
        norm(y, residual_out=y)
    with pytest.raises(ValueError):
        norm(y, residual=y.half())
    with pytest.raises(ValueError):
        norm(y.view(2, 2, 256), residual=y.view(2, 2, 256))
    with pytest.raises(ValueError):
        norm(y, quantize=moe.Fp8Rows.empty(3, 256))
    with pytest.raises(ValueError):  # in x's place with other strides
        big = rand(gen(2), 8, 256)
        norm(big[:4], normed=big[::2])
    for bad in (dict(normed=y[:1].clone().expand(4, 256)), dict(residual=y, residual_out=y[:1].clone().expand(4, 256))):
        with pytest.raises(moe.MoeError):  # rows on top of each other
            norm(y, **bad)
    with pytest.raises(moe.MoeError):
        norm(y, normed=False)
    with pytest.raises(moe.MoeError):
        h = torch.empty_like(y)
        norm(y, residual=y, residual_out=h, normed=h)
    e = torch.empty(0, 256, device="cuda")
    assert norm(e)[0].shape == (0, 256)


@pytest.mark.parametrize("d", [1, 64, 100, 250, 512, 1000, 1030, 2048, 4096, 5000, 8192, 20000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_norm_of_rows_whose_squares_leave_fp32(moe, d, dtype):
    """Rows of every size that the type has, alone and beside ordinary ones of the same warp: the norm is of size 1."""
    g = gen(d)
    sizes = [1e30, 1.0, 1e-30, 1e18, 1e19, 3e37, 1e-18, 1e-20, 1e-23, 1e-36, 3e-39, 1e-40, 1e-10, 1.0, 1e25, 3e-38, 2.0 ** -133]
    x = torch.stack([rand(g, d) * 1.0 for _ in sizes]).clamp(-8, 8) * torch.tensor(sizes, device="cuda")[:, None]
    x[1::4, d // 2] *= 2.0 ** -40  # far below the rest of its row
    x[:, 0] = torch.tensor(sizes, device="cuda")  # no row of zeros
    x = x.to(dtype)
    r = (x.flip(1).float() * 0.5).to(dtype)
    w = (1 + rand(g, d, scale=0.2)).to(FP32)
    for eps in (0.0, 1e-6, 1e-42, 1e-30):
        norm = moe.RmsNorm(w, eps=eps)
        eps32 = float(torch.tensor(eps, dtype=FP32))
        for residual, quantize, place in ((False, False, False), (True, True, False), (False, True, True), (True, False, True)):
            if quantize and d % 16 and d > 1030:
                continue
            a, b = x.clone(), r.clone()
            h = (x.float() + r.float()).to(dtype) if residual else x
            want = P.rms_norm(h, w, eps32, False)
            n, ro, q = norm(a, residual=b if residual else None, residual_out=None if residual and not place else False,
                            normed=a if place else True, quantize=quantize)
            assert ro is None or torch.equal(ro, h)
            # the scaled row's products round as often as the others'; without a scale, an h * w below FP32's normal values is off by
            # 2^-150, times the factor
            mean = h.double().square().mean(-1, keepdim=True) + eps32
            plain = mean >= 2.0 ** -126
            low = torch.where(plain, 2.0 ** -150 / mean.sqrt(), torch.zeros_like(mean))
            assert ((n.double() - want).abs() <= half_step(want, dtype) * (1 + 2.0 ** -8) + want.abs() * NORM_REL + low).all()
            if quantize:
                keep = ~plain[:, 0] | (h.double().abs().amax(-1) >= 2.0 ** -110)
                check_quantized(moe.Fp8Rows(q.codes[keep], q.scales[keep]), want[keep], NORM_REL)


@pytest.mark.parametrize("d", [100, 256, 2048, 9000])
def test_norm_of_infinite_rows(moe, d):
    """h / sqrt(infinity): 0 for what is finite and NaN for the infinities, block by block in 8 bits."""
    x = rand(gen(d), 5, d) + 3.0
    x[1, 70], x[3, 5] = math.inf, -math.inf
    n, _, q = moe.RmsNorm(torch.ones(d, device="cuda"))(x, quantize=True)
    assert torch.isfinite(n[0::2]).all() and torch.isfinite(q.scales[0::2]).all()
    for row, at in ((1, 70), (3, 5)):
        rest = torch.arange(d, device="cuda") != at
        assert torch.isnan(n[row, at]) and (n[row, rest] == 0).all()
        assert torch.isnan(q.scales[row, 0]) and (q.scales[row, 1:] == 0).all() and (q.codes[row].float() == 0).all()


# ---- quantised rows ----

@pytest.mark.parametrize("rows,d", [(1, 1), (1, 16), (3, 100), (5, 128), (2, 136), (33, 4096), (7, 1000), (4, 131), (300, 640)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_quantize(moe, rows, d, dtype):
    g = gen(d + rows)
    x = rand(g, rows, d, dtype=dtype)
    x[rows // 2] *= 1000.0
    q = moe.quantize_rows(x)
    codes, scales = P.quantize(x.double())
    # quotients are exact: the same codes bit by bit
    assert torch.equal(q.scales, scales)
    assert equal_codes(codes_of(q), codes)


def test_quantize_every_ratio_of_16_bit_values(moe):
    """Quotients on and next to the borders between codes: every pair of 8-bit significands and a few exponents."""
    sig = torch.arange(128, 256, device="cuda", dtype=FP32)
    rows = []
    for exp in (0, -1, -3, -6, -8, -9, -10):
        block = torch.empty(128, 128, device="cuda")
        block[:, :] = sig[None, :] * 2.0 ** exp
        rows.append(block)
    x = torch.cat(rows)
    top = sig.repeat(len(rows)) * 2.0
    x = torch.cat([top[:, None], x[:, :127]], dim=1)
    x2 = torch.cat([top[:, None], torch.cat(rows)[:, 1:]], dim=1)
    for y in (x, x2, -x, x * 2.0 ** -60, x * 2.0 ** -100, x * 2.0 ** -125, x * 2.0 ** 100):
        q = moe.quantize_rows(y.to(BF16))
        codes, scales = P.quantize(y.to(BF16).double())
        assert torch.equal(q.scales, scales)
        assert equal_codes(codes_of(q), codes)


def test_quantize_small_and_large(moe):
    x = torch.zeros(7, 256, device="cuda")
    x[0, 3] = 2.0 ** -149
    x[1] = rand(gen(1), 256) * 1e-40
    x[2] = 3.4e38
    x[3, :128] = rand(gen(2), 128)
    x[3, 5], x[4, 130], x[5, 0] = math.inf, math.nan, -math.inf
    x[4, :128], x[6, 255] = 1.0, -7.0
    q = moe.quantize_rows(x)
    for row in (0, 1, 2, 6):
        codes, scales = P.quantize(x[row:row + 1].double())
        assert torch.equal(q.scales[row:row + 1], scales)
        assert equal_codes(codes_of(q)[row:row + 1], codes)
    assert torch.isnan(q.scales[3, 0]) and torch.isnan(q.scales[4, 1]) and torch.isnan(q.scales[5, 0])
    assert q.scales[3, 1] == 0 and q.scales[4, 0] == torch.tensor(1 / 448.0) and (codes_of(q)[3, :128] == 0).all()


@pytest.mark.parametrize("rows,d", [(1, 16), (3, 100), (65, 512), (4, 131)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_quantize_gated(moe, rows, d, dtype):
    g = gen(d * 3 + rows)
    x = rand(g, rows, 2 * d, dtype=dtype, scale=4.0)
    x[0, 0], x[0, 1 % d] = 95.0, -95.0
    q = moe.quantize_rows(x, gated=True)
    a, b = x[:, :d].double(), x[:, d:].double()
    want = a / (1 + torch.exp(-a)) * b
    # the exponential to 2 units (4 halves), the sum, the quotient, the product
    check_quantized(q, want, 8 * U)
    with pytest.raises(ValueError):
        moe.quantize_rows(x[:, :-1], gated=True)


def test_quantize_gates_far_below_zero(moe):
    """exp(gate) is no normal FP32 value below -87.34: such gates count as 0, those above do not."""
    x = torch.ones(3, 256, device="cuda")
    x[0, :128], x[1, :128], x[2, :128] = -87.5, -200.0, -87.0
    q = moe.quantize_rows(x, gated=True)
    assert (q.scales[:2] == 0).all() and (q.codes[:2].float() == 0).all()
    check_quantized(moe.Fp8Rows(q.codes[2:], q.scales[2:]), torch.full((1, 128), -87.0 * math.exp(-87.0), dtype=torch.float64, device="cuda"), 8 * U)


def test_quantize_strides_and_places(moe):
    g = gen(5)
    x = rand(g, 20, 300, dtype=BF16)
    a = moe.quantize_rows(x[::2, 4:204])
    codes, scales = P.quantize(x[::2, 4:204].double())
    assert torch.equal(a.scales, scales) and equal_codes(codes_of(a), codes)
    store = torch.zeros(10, 208, dtype=torch.uint8, device="cuda")
    out = moe.Fp8Rows(store.view(torch.float8_e4m3fn)[:, :200], torch.zeros(10, 5, device="cuda")[:, ::3])
    b = moe.quantize_rows(x[::2, 4:204], out=out)
    assert b is out and torch.equal(out.scales, scales) and equal_codes(codes_of(out), codes)
    assert (store[:, 200:] == 0).all()


# ---- products ----

def make_rows(moe, g, rows, k):
    return moe.quantize_rows(rand(g, rows, k) * torch.exp(rand(g, k)))


def make_weight(g, *shape):
    n, k = shape[-2:]
    codes = (rand(g, *shape) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (0.5 + torch.rand(*shape[:-2], -(-n // 128), -(-k // 128), generator=g, device="cuda")) / 100
    return codes, scales


def check_product(out, x, codes, scales):
    """A block's sum of 128 products is formed 32 at a time in wider registers, each sum off by at most one step (2^-23) of
    its largest term for every term: 2^-18 of the sum of magnitudes; a scale, a product and an addition a block more."""
    xv, wv = P.values(x.codes, x.scales), P.weight_values(codes, scales)
    want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    blocks = -(-codes.shape[-1] // 128)
    bound = size * (2.0 ** -18 + (blocks + 3) * U) + half_step(want, out.dtype)
    assert ((out.double() - want).abs() <= bound).all(), float(((out.double() - want).abs() / bound).max())


PRODUCTS = [(1, 1, 16), (1, 128, 128), (4, 100, 144), (4, 5120, 2048), (16, 257, 1040), (17, 128, 512), (31, 300, 80), (32, 640, 4096), (33, 129, 256),
            (64, 1000, 512), (100, 384, 2064), (128, 2048, 256), (129, 128, 128), (200, 513, 400), (256, 256, 512), (257, 300, 1024),
            (500, 100, 208), (1000, 513, 272), (1024, 1024, 1024), (2049, 2304, 512), (4000, 4100, 304)]


@pytest.mark.parametrize("rows,n,k", PRODUCTS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_product(moe, rows, n, k, dtype):
    g = gen(rows + 7 * n + 11 * k)
    x = make_rows(moe, g, rows, k)
    codes, scales = make_weight(g, n, k)
    linear = moe.Fp8Linear(codes, scales)
    out = linear(x, dtype=dtype)
    assert out.dtype is dtype and linear.status() == 0
    check_product(out, x, codes, scales)
    assert torch.equal(out, linear(x, dtype=dtype))


def test_product_of_one_hot_rows_is_the_weight(moe):
    """Each value of a weight comes back exactly, so rows, channels and scales meet where they should."""
    g = gen(3)
    n, k = 300, 272
    codes, scales = make_weight(g, n, k)
    one = torch.eye(k, device="cuda")
    x = moe.quantize_rows(one)  # 1 = 448 * fl(1 / 448)
    want = P.weight_values(codes, scales).t() * (448.0 * float(x.scales.max()))
    for rows in (k, 20, 100):
        part = moe.Fp8Rows(x.codes[:rows], x.scales[:rows])
        out = moe.Fp8Linear(codes, scales)(part, dtype=FP32)
        assert ((out.double() - want[:rows]).abs() <= want[:rows].abs() * 4 * U).all()


@pytest.mark.parametrize("rows", [50, 700])
def test_product_strides_types_and_places(moe, rows):
    g = gen(4)
    n, k = 200, 160
    wide = (rand(g, rows, 320) * 50).to(torch.float8_e4m3fn)
    x = moe.Fp8Rows(wide[:, 128:288], torch.rand(rows, 6, generator=g, device="cuda")[:, 1:5:3])
    codes, scales = make_weight(g, n, k)
    linear = moe.Fp8Linear(codes, scales)
    base = linear(x, dtype=FP32)
    check_product(base, x, codes, scales)
    for dtype in (BF16, FP16):
        check_product(linear(x, dtype=dtype), x, codes, scales)
    for off, width in ((0, 208), (1, 203), (4, 260)):
        for dtype in (BF16, FP32):
            store = torch.full((rows, width + off), 7.0, device="cuda", dtype=dtype)
            out = linear(x, out=store[:, off:off + n])
            check_product(out, x, codes, scales)
            assert (store[:, :off] == 7).all() and (store[:, off + n:] == 7).all()
    # every other row of a larger array
    x2 = moe.Fp8Rows(wide[::2, 128:288], x.scales[::2])
    assert torch.equal(linear(x2, dtype=FP32), base[::2])


@pytest.mark.parametrize("groups", [0, 2])
def test_product_of_one_row_of_any_stride(moe, groups):
    g = gen(5)
    n, k = 200, 160
    codes, scales = make_weight(g, *((groups,) if groups else ()), n, k)
    linear = moe.Fp8Linear(codes, scales)
    x = make_rows(moe, g, 1, k)
    offsets = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda") if groups else None
    want = linear(x, offsets=offsets, dtype=FP32)
    for stride in (1, 7, k, k + 8, 1 << 41):
        one = moe.Fp8Rows(x.codes.as_strided((1, k), (stride, 1)), x.scales.as_strided((1, 2), (stride, x.scales.stride(1))))
        out = torch.zeros(1, n, device="cuda").as_strided((1, n), (stride, 1))
        assert torch.equal(linear(one, offsets=offsets, out=out), want)


def test_norm_of_one_row_in_place_whatever_its_stride(moe):
    g = gen(6)
    w = torch.ones(256, device="cuda")
    norm = moe.RmsNorm(w)
    for shape in ((1, 256), (3, 1, 256), (1, 3, 256)):
        x = rand(g, *shape)
        want = norm(x)[0]
        other = x.as_strided(shape, tuple(999 if n == 1 else s for n, s in zip(shape, x.stride())))
        assert norm(x, normed=other)[0] is other and torch.equal(x, want)
    empty = torch.empty(0, 512, device="cuda")
    assert norm(empty[:, :256], normed=torch.empty(0, 256, device="cuda"))[0].shape == (0, 256)


def test_product_nan_rows_stay_alone(moe):
    g = gen(6)
    v = rand(g, 40, 512)
    v[3, 100] = math.nan
    v[17, 511] = math.inf
    x = moe.quantize_rows(v)
    codes, scales = make_weight(g, 256, 512)
    out = moe.Fp8Linear(codes, scales)(x)
    bad = torch.isnan(out).all(-1)
    assert bad.nonzero().flatten().tolist() == [3, 17] and torch.isfinite(out[~bad]).all()


def test_product_refusals(moe):
    g = gen(8)
    codes, scales = make_weight(g, 64, 256)
    linear = moe.Fp8Linear(codes, scales)
    x = make_rows(moe, g, 4, 256)
    with pytest.raises(ValueError):
        linear(make_rows(moe, g, 4, 128))
    with pytest.raises(ValueError):
        linear(x, dtype=torch.float64)
    with pytest.raises(ValueError):
        linear(x, out=torch.empty(4, 65, device="cuda"))
    with pytest.raises(ValueError):
        linear(x, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moe.Fp8Linear(codes, scales[:, :1].contiguous())
    with pytest.raises(ValueError):
        moe.Fp8Linear(codes.t(), scales)
    with pytest.raises(moe.MoeError):
        moe.Fp8Linear(codes[:, :250].contiguous(), scales)
    with pytest.raises(moe.MoeError):  # rows 250 bytes apart
        linear(moe.Fp8Rows(torch.zeros(4 * 264, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).view(4, 264)[:, :256],
                           x.scales))
    assert linear(make_rows(moe, g, 4, 256)).shape == (4, 64)
    empty = moe.Fp8Rows(x.codes[:0], x.scales[:0])
    assert linear(empty).shape == (0, 64)


# ---- products of groups ----

GROUPS = [([5], 128, 128), ([0, 3, 0, 0, 7, 1], 200, 272), ([1] * 40, 130, 512), ([0, 0, 0], 128, 128), ([300, 2, 0, 257, 90], 300, 144),
          ([16, 17, 31, 32, 33, 64, 128, 129], 256, 256), ([1000, 0, 600], 140, 384), ([40] * 100, 128, 128),
          ([0] * 500 + [9] + [0] * 522 + [1], 64, 64)]


@pytest.mark.parametrize("counts,n,k", GROUPS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_grouped_product(moe, counts, n, k, dtype):
    g = gen(sum(counts) + n + k)
    rows = sum(counts)
    extra = 5  # rows behind the last group, and 2 before the first: left as they were
    x = make_rows(moe, g, rows + 2 + extra, k)
    codes, scales = make_weight(g, len(counts), n, k)
    linear = moe.Fp8Linear(codes, scales)
    edges = [2]
    for c in counts:
        edges.append(edges[-1] + c)
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    out = torch.full((rows + 2 + extra, n), 7.0, dtype=dtype, device="cuda")
    assert linear(x, offsets=offsets, out=out) is out
    assert linear.status() == 0
    assert (out[:2] == 7).all() and (out[rows + 2:] == 7).all()
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        if b > a:
            check_product(out[a:b], moe.Fp8Rows(x.codes[a:b], x.scales[a:b]), codes[i], scales[i])


@pytest.mark.parametrize("rows", [20, 1000])
def test_grouped_product_of_no_rows(moe, rows):
    g = gen(14)
    x = make_rows(moe, g, rows, 128)
    linear = moe.Fp8Linear(*make_weight(g, 3, 128, 128))
    for at in (0, 7, rows):
        out = torch.full((rows, 128), 7.0, device="cuda")
        linear(x, offsets=torch.full((4,), at, dtype=torch.int32, device="cuda"), out=out)
        assert (out == 7).all() and linear.status() == 0


def test_grouped_product_bad_offsets(moe):
    """Offsets out of range or decreasing are cut, set a status bit and touch nothing outside."""
    g = gen(12)
    x = make_rows(moe, g, 20, 128)
    codes, scales = make_weight(g, 4, 128, 128)
    linear = moe.Fp8Linear(codes, scales)
    for edges, spans in (([0, 5, 5, 25, 30], [(0, 0, 5), (2, 5, 20)]), ([-4, 6, 8, 8, 20], [(0, 0, 6), (1, 6, 8), (3, 8, 20)]),
                         ([0, 5, 3, 3, 2], [(0, 0, 5)])):
        store = torch.full((24, 128), 7.0, device="cuda")
        linear(x, offsets=torch.tensor(edges, dtype=torch.int32, device="cuda"), out=store[2:22])
        assert linear.status() == moe.DENSE_BAD_OFFSETS and linear.status() == 0
        rest = torch.ones(24, dtype=torch.bool, device="cuda")
        for i, a, b in spans:
            check_product(store[2 + a:2 + b], moe.Fp8Rows(x.codes[a:b], x.scales[a:b]), codes[i], scales[i])
            rest[2 + a:2 + b] = False
        assert (store[rest] == 7).all()
    with pytest.raises(ValueError):
        linear(x)
    with pytest.raises(ValueError):
        linear(x, offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        linear(x, offsets=torch.zeros(5, dtype=torch.int64, device="cuda"))


def spans_of(edges, rows):
    """(group, first row, end) by the header's rule for offsets out of order."""
    end, spans = 0, []
    for i, (a, b) in enumerate(zip(edges, edges[1:])):
        a, b = max(min(max(a, 0), rows), end), min(max(b, 0), rows)
        if b > a:
            spans.append((i, a, b))
            end = b
    return spans


@pytest.mark.parametrize("rows,edges", [(20, [0, 10, 5, 15]), (20, [3, 18, 0, 19, 1, 40]), (1000, [0, 600, 100, 900, 200, 1000]),
                                        (900, [0, 900] * 5), (700, [0, 700] * 512 + [0]), (64, [30, 20, 40, 10, 64])])
def test_grouped_product_overlapping_offsets(moe, rows, edges):
    """Offsets that decrease give no row to two groups: the first group that has it multiplies it, every time."""
    g = gen(rows)
    n, k = 136, 144
    x = make_rows(moe, g, rows, k)
    codes, scales = make_weight(g, len(edges) - 1, n, k)
    linear = moe.Fp8Linear(codes, scales)
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    outs = []
    for _ in range(3):
        out = torch.full((rows, n), 7.0, device="cuda")
        linear(x, offsets=offsets, out=out)
        assert linear.status() == moe.DENSE_BAD_OFFSETS
        outs.append(out)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    for i, a, b in spans_of(edges, rows):
        check_product(outs[0][a:b], moe.Fp8Rows(x.codes[a:b], x.scales[a:b]), codes[i], scales[i])
        rest[a:b] = False
    assert (outs[0][rest] == 7).all() and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_grouped_rows_do_not_depend_on_the_others(moe):
    """A group's rows have the bits of the same rows alone under the same kernel (order of sums fixed by k alone)."""
    g = gen(13)
    x = make_rows(moe, g, 48, 512)
    codes, scales = make_weight(g, 3, 256, 512)
    linear = moe.Fp8Linear(codes, scales)
    a = linear(x, offsets=torch.tensor([0, 20, 20, 48], dtype=torch.int32, device="cuda"))
    b = linear(x, offsets=torch.tensor([3, 20, 41, 48], dtype=torch.int32, device="cuda"), out=torch.zeros_like(a))
    assert torch.equal(a[3:20], b[3:20]) and torch.equal(a[41:], b[41:])


# ---- log probabilities ----

def check_logprobs(got, logits, tokens, top, scale):
    want = P.logprobs(logits, tokens.view(tokens.shape[0], -1), top, scale)
    for i, (given, lse, ent, ids, tops, spread) in enumerate(want):
        def near(a, b, tol):
            if math.isnan(b) or math.isinf(b):
                assert (math.isnan(a) and math.isnan(b)) or a == b, (i, a, b)
            else:
                assert abs(a - b) <= tol, (i, a, b, tol)
        # 61 additions in a row of sums of positive terms, exponentials to 2^-22 and their arguments to 2^-23 of at
        # most 40: below 1e-5 of the sum; FP32 results
        near(float(got.lse[i]), lse, 1e-5 + 4 * U * abs(lse))
        near(float(got.entropy[i]), ent, 2e-5 * (1 + spread))
        for a, b in zip(got.logprobs[i].view(-1).tolist(), given):
            near(a, b, 1e-5 + 4 * U * (abs(b) + abs(lse)))
        if top:
            assert got.top_ids[i].tolist() == ids
            for a, b in zip(got.top_logprobs[i].tolist(), tops):
                near(a, b, 1e-5 + 4 * U * (abs(b) + abs(lse)))


@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 3), (3, 17), (5, 100), (4, 1000), (3, 4099), (2, 20000), (1, 131072), (130, 997), (700, 64)])
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
def test_logprobs(moe, rows, vocab, dtype):
    g = gen(vocab + rows)
    logits = rand(g, rows, vocab, dtype=dtype, scale=3.0)
    for n, top, scale in ((1, min(vocab, 8), 1.0), (3, 0, 0.7), (40, min(vocab, 32), 2.5), (2, 1, 1.0)):
        tokens = torch.randint(0, vocab, (rows, n), generator=g, device="cuda").to(torch.int32)
        got = moe.token_logprobs(logits, tokens, top=top, scale=scale)
        assert (got.top_ids is None) == (top == 0)
        check_logprobs(got, logits, tokens, top, scale)


@pytest.mark.parametrize("rows", [2, 700])
def test_logprobs_of_a_large_vocabulary(moe, rows):
    """Many steps a thread: one CTA a row where there are many rows, parts of a cluster where there are few."""
    g = gen(rows)
    vocab = 400003
    logits = rand(g, rows, vocab, dtype=BF16, scale=2.0)
    logits[0, ::2] = logits[0, 1]
    tokens = torch.randint(0, vocab, (rows, 2), generator=g, device="cuda").to(torch.int32)
    got = moe.token_logprobs(logits, tokens, top=32)
    few = [0, rows - 1]
    check_logprobs(moe.TokenLogprobs(*(t[few] for t in got)), logits[few], tokens[few], 32, 1.0)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_logprobs_of_many_short_rows(moe, dtype):
    """A CTA takes several rows, of every alignment; among them rows of masks, equal logits and NaN."""
    g = gen(79)
    rows, vocab = 1900, 2503
    logits = rand(g, rows, vocab + 3, dtype=dtype, scale=2.0)[:, 1:vocab + 1]
    logits[3::11] = -math.inf
    logits[5::13] = 0.25
    logits[7::17, ::2] = -math.inf
    logits[9::19, 100:700] = math.nan
    tokens = torch.randint(0, vocab, (rows, 40), generator=g, device="cuda").to(torch.int32)
    for top in (0, 3, 32):
        got = moe.token_logprobs(logits, tokens, top=top)
        check_logprobs(got, logits, tokens, top, 1.0)
        again = moe.token_logprobs(logits, tokens, top=top)
        for a, b in zip(got, again):
            assert a is None and b is None or torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_logprobs_masks_ties_and_bad_tokens(moe):
    g = gen(77)
    inf = math.inf
    v = 9000
    logits = rand(g, 10, v, scale=2.0)
    logits[0] = -inf                       # nothing left
    logits[1] = -inf
    logits[1, 4321] = -3.0                 # one left
    logits[2] = 1.5                        # all equal
    logits[3, ::2] = -inf
    logits[4] = torch.arange(v, device="cuda") * 1e-3   # every value a new best
    logits[5] = -torch.arange(v, device="cuda") * 1e-3
    logits[6, 77] = math.nan
    logits[7, 5] = inf
    logits[8] = torch.finfo(FP32).min
    logits[9, 100:140] = 9.0               # more ties than places
    tokens = torch.tensor([[0, 1, -1, v]] * 10, dtype=torch.int32, device="cuda")
    tokens[1, 0] = 4321
    for dtype in (FP32, BF16, FP16):
        x = logits.to(dtype)
        for top in (0, 5, 32):
            check_logprobs(moe.token_logprobs(x, tokens, top=top), x, tokens, top, 1.0)
    zero = torch.zeros(2, 50, device="cuda")
    zero[:, 1::2] = -0.0
    got = moe.token_logprobs(zero, tokens[:2], top=32)
    assert got.top_ids.tolist() == [list(range(32))] * 2
    big = torch.full((1, 300), 1e38, device="cuda")  # finite, but not times the scale
    got = moe.token_logprobs(big, tokens[:1], top=2, scale=5.0)
    assert math.isnan(got.lse[0]) and math.isnan(got.entropy[0]) and torch.isnan(got.logprobs).all() and got.top_ids.tolist() == [[0, 1]]
    got = moe.token_logprobs(-big, tokens[:1], top=2, scale=5.0)
    assert got.lse[0] == -inf and got.entropy[0] == 0 and (got.logprobs == -inf).all()
    few = torch.full((1, 5000), -inf, device="cuda")
    few[0, [4000, 17, 2500]] = torch.tensor([1.0, 1.0, 2.0], device="cuda")
    got = moe.token_logprobs(few, tokens[:1], top=6)
    assert got.top_ids.tolist() == [[2500, 17, 4000, 0, 1, 2]]


@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
def test_logprobs_of_large_logits_with_a_scale(moe, dtype, rows):
    """Rows whose scaled logits FP32 does not hold exactly: nothing but masks of any kind, and differences far below their size."""
    lowest = torch.finfo(dtype).min
    v, large = 5003, min(1e10, -lowest)
    g = gen(79 + rows)
    kinds = [torch.full((v,), lowest), torch.full((v,), -large), torch.full((v,), large), torch.full((v,), lowest),
             torch.full((v,), -large), torch.randint(0, 20, (v,), generator=torch.Generator().manual_seed(rows)) - 1e7]
    kinds[3][torch.tensor([17, 2500, 4999])] = torch.tensor([0.25, -1.0, 2.0])
    kinds[4][4321] = 3.0
    if dtype is not FP32:
        kinds.pop()  # their steps are larger than 1 there
    x = torch.stack(kinds).to(dtype).cuda()
    if rows > 1:
        x = x[torch.randint(0, len(kinds), (rows,), generator=g, device="cuda")]
    tokens = torch.randint(0, v, (x.shape[0], 3), generator=g, device="cuda").to(torch.int32)
    tokens[:, 0] = 2500
    for scale in (0.699999988079071044921875, 1.2999999523162841796875):  # values of FP32
        for i in range(x.shape[0] if rows == 1 else 0):  # a row in parts of a cluster
            one(moe, x[i:i + 1], tokens[i:i + 1], scale)
        one(moe, x, tokens, scale)


def one(moe, x, tokens, scale):
    got = moe.token_logprobs(x, tokens, top=4, scale=scale)
    seen = {}
    for i, row in enumerate(x):
        key = (row[0].item(), row[2500].item(), row[4321].item())
        if key not in seen:
            seen[key] = P.logprobs(row[None], torch.arange(x.shape[1])[None], 4, scale)[0]
        lps, lse, ent, ids, tops, spread = seen[key]
        if lse < -torch.finfo(FP32).max:  # FP32 has -infinity for all of them
            assert got.lse[i] == -math.inf and got.entropy[i] == 0 and (got.logprobs[i] == -math.inf).all()
            continue
        # the sums as in check_logprobs; the difference of two logits, its product and one addition round to FP32
        assert abs(float(got.lse[i]) - lse) <= 1e-5 + 4 * U * abs(lse)
        assert abs(float(got.entropy[i]) - ent) <= 2e-5 * (1 + spread)
        for a, b in zip(got.logprobs[i].tolist() + got.top_logprobs[i].tolist(), [lps[t] for t in tokens[i].tolist()] + tops):
            if b < -(2 - 2.0 ** -24) * 2.0 ** 127:  # its nearest FP32 value (the lowest mask times 1.3 is -4.4e38)
                b = -math.inf
            assert a == b or abs(a - b) <= 1e-5 + 4 * U * abs(b), (i, a, b)
        assert got.top_ids[i].tolist() == ids


@pytest.mark.parametrize("rows", [2, 800])
def test_logprobs_of_nan_beside_values_whose_scaled_ones_are_minus_infinity(moe, rows):
    for dtype in (FP32, BF16):
        x = torch.full((rows, 3001), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        x[0, 77], x[1] = math.nan, math.nan
        tokens = torch.zeros(rows, 2, dtype=torch.int32, device="cuda")
        for top in (0, 3):
            got = moe.token_logprobs(x, tokens, top=top, scale=5.0)
            for t in got:
                if t is not None and t.dtype is FP32:
                    assert torch.isnan(t[:2]).all() and not torch.isnan(t[2:]).any()
            assert (got.lse[2:] == -math.inf).all() and (got.entropy[2:] == 0).all()


def check_sure(got, x, tokens, scale, steps):
    """Rows in which one token has nearly all the probability, by relative errors.  With x = scale * (logit - largest) and r the sum
    of exp(x) over the other tokens: lse - max = log1p(r) is the sure token's log probability (negated), entropy = log1p(r) +
    sum exp(x) |x| / (1 + r).  A term's exponent has three roundings (the difference, scale * log2(e), their product), in parts that add up to
    |x|: 3 U |x| of the term, so that of r 3 U times the mean of |x| under the terms, that of the entropy with |x| times the terms as
    weights.  Every exponential (of the term; of its thread's, warp's and part's largest; of a step that finds a larger one) is
    good to 4 U; additions one after the other: 10 in a step, one a step, 15 in joins; logarithm, quotient and product 6."""
    f = x.double()
    most, at = f.max(-1)
    d = (f - most[:, None]) * scale
    d[torch.arange(len(x)), at] = -math.inf
    e = d.exp()
    size = torch.where(e > 0, -d, torch.zeros_like(d))
    r = e.sum(-1)
    mean, mean2 = (e * size).sum(-1) / r, (e * size * size).sum(-1) / (e * size).sum(-1)
    want = -torch.log1p(r)
    entropy = torch.log1p(r) + (e * size).sum(-1) / (1 + r)
    terms = 10 + 15 + 4 * 4 + 6 + 6 * steps
    sure = got.logprobs[:, 0].double()
    assert (tokens[:, 0] == at).all() and (got.top_ids is None or (got.top_ids[:, 0] == at).all())
    assert ((sure - want).abs() <= -want * U * (3 * mean + terms)).all(), float(((sure - want) / want).abs().max())
    assert got.top_logprobs is None or torch.equal(got.top_logprobs[:, 0], got.logprobs[:, 0])
    assert ((got.entropy.double() - entropy).abs() <= entropy * U * (3 * torch.maximum(mean, mean2) + terms)).all(), \
        float(((got.entropy.double() - entropy) / entropy).abs().max())
    # the others: a difference, its product and one addition
    other = (f.gather(1, tokens[:, 1:].long()) - most[:, None]) * scale + want[:, None]
    assert ((got.logprobs[:, 1:].double() - other).abs() <= 4 * U * other.abs() + 1e-5 * r[:, None].clamp(max=1)).all()
    lse = most * scale + torch.log1p(r)
    assert ((got.lse.double() - lse).abs() <= 4 * U * lse.abs() + 1e-5 * r).all()


RESTS = [10.0 ** -(i / 2) for i in range(0, 17)]  # 1 to 1e-8


@pytest.mark.parametrize("rows,vocab,steps", [(2, 60, 1), (1, 131072, 4), (5, 50001, 2), (300, 3001, 2), (640, 20011, 6), (640, 70001, 18)])
@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
def test_logprobs_of_sure_tokens(moe, dtype, rows, vocab, steps):
    """One CTA for each row, several rows a CTA, parts of a cluster; the sure token anywhere, outside all vectors too."""
    g = gen(vocab)
    for turn, (top, scale) in enumerate(((0, 1.0), (3, 1.0), (20, 0.699999988079071044921875), (0, 2.5))):
        x = rand(g, rows, vocab + 9, dtype=dtype)[:, 1 + turn:1 + turn + vocab]
        targets = torch.tensor([RESTS[i % len(RESTS)] for i in range(turn, turn + rows)], dtype=torch.float64, device="cuda")
        total = (x.double() * scale).exp().sum(-1)
        sure = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        edge = torch.tensor([0, vocab - 1, 1, vocab - 2], device="cuda")
        sure[::3] = edge[torch.arange(len(sure[::3]), device="cuda") % 4]
        x[torch.arange(rows, device="cuda"), sure] = ((total / targets).log() / scale).to(dtype)
        tokens = torch.randint(0, vocab, (rows, 3), generator=g, device="cuda")
        tokens = torch.cat([sure[:, None], torch.where(tokens == sure[:, None], (tokens + 1) % vocab, tokens)], 1).to(torch.int32)
        got = moe.token_logprobs(x, tokens, top=top, scale=scale)
        check_sure(got, x, tokens, scale, steps)
        again = moe.token_logprobs(x, tokens, top=top, scale=scale)
        assert torch.equal(got.entropy, again.entropy) and torch.equal(got.logprobs, again.logprobs)


@pytest.mark.parametrize("rows", [3, 900])
def test_logprobs_of_sure_tokens_with_few_others(moe, rows):
    """Everything else masked but one token, or all of it: the rest is one term, or nothing."""
    vocab = 40009
    g = gen(rows)
    for mask in (-math.inf, torch.finfo(FP32).min, -1e10):
        x = torch.full((rows, vocab), mask, device="cuda")
        pair = torch.stack([torch.randperm(vocab, generator=g, device="cuda")[:2] for _ in range(rows)])
        at = torch.arange(rows, device="cuda")
        x[at, pair[:, 0]] = 3.25
        x[at, pair[:, 1]] = 3.25 - torch.linspace(0.5, 18.5, rows, device="cuda")
        for top in (0, 2):
            check_sure(moe.token_logprobs(x, pair.to(torch.int32), top=top), x, pair, 1.0, 10)
        x[at, pair[:, 1]] = mask
        for top in (0, 1):
            got = moe.token_logprobs(x, pair.to(torch.int32), top=top)
            assert (got.logprobs[:, 0] == 0).all() and (got.entropy == 0).all() and (got.lse == 3.25).all()
            assert top == 0 or ((got.top_logprobs == 0).all() and torch.equal(got.top_ids[:, 0], pair[:, 0].to(torch.int32)))
    # two of the same: each has a half
    x[at, pair[:, 1]] = 3.25
    for top in (0, 2):
        got = moe.token_logprobs(x, pair.to(torch.int32), top=top)
        assert ((got.logprobs.double() + math.log(2)).abs() <= 8 * U).all() and ((got.entropy.double() - math.log(2)).abs() <= 8 * U).all()


def test_logprobs_strides(moe):
    g = gen(78)
    for dtype in (FP32, BF16):
        buf = rand(g, 12, 5013, dtype=dtype)
        tokens = torch.randint(0, 5000, (6, 8), generator=g, device="cuda").to(torch.int32)
        for off in range(5):
            x = buf[::2, off:off + 5001 - off]
            check_logprobs(moe.token_logprobs(x, tokens[:, 2:5], top=3), x, tokens[:, 2:5], 3, 1.0)
        flat = moe.token_logprobs(buf[:6], tokens[:, 0].contiguous(), top=3)
        assert flat.logprobs.shape == (6,)
        strided = moe.token_logprobs(buf[:6], tokens[:, 0], top=3)
        assert torch.equal(flat.logprobs, strided.logprobs)


def test_logprobs_refusals(moe):
    x = torch.zeros(4, 100, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: moe.token_logprobs(x.t(), t), lambda: moe.token_logprobs(x, t.long()), lambda: moe.token_logprobs(x, t[:3]),
                lambda: moe.token_logprobs(x.double(), t), lambda: moe.token_logprobs(x, t.cpu())):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(top=33), dict(top=-1), dict(scale=0.0), dict(scale=math.inf)):
        with pytest.raises(moe.MoeError):
            moe.token_logprobs(x, t, **kw)
    with pytest.raises(moe.MoeError):
        moe.token_logprobs(x[:, :8], t, top=9)
    assert moe.token_logprobs(x[:0], t[:0], top=2).top_ids.shape == (0, 2)
