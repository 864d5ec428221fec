"""8-bit linear: rows, scales and codes exactly, the product against the integer sums in 64 bits."""
import pytest

from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F16, F32 = R.FLOATS


def _svdq():
    from bit_rank_compensated_b200 import svdq

    return svdq


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _acts(M, K, dtype, seed, scale=1.0):
    g = _gen(seed)
    X = torch.randn(M, K, generator=g, device="cuda") * scale
    X[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 30
    return X.to(dtype)


def _codes(M, K, seed):
    return torch.randint(-127, 128, (M, K), generator=_gen(seed), device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("dtype", R.FLOATS)
@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("M,K", [(1, 16), (3, 48), (257, 64), (5, 1040), (64, 2560), (2, 12288), (9, 4112), (1, 131072), (33, 20000)])
def test_quantize_rows_exactly(M, K, smooth, dtype):
    svdq = _svdq()
    X = _acts(M, K, dtype, 1)
    col = (torch.rand(K, generator=_gen(2), device="cuda") + 0.1) if smooth else None
    xq, scale = svdq.i8_quantize_rows(X, col)
    q, s = R.quantize_rows(X, col)
    assert torch.equal(xq, q) and torch.equal(scale, s)


@pytest.mark.parametrize("dtype", R.FLOATS)
def test_quantize_ties_zeros_and_extremes(dtype):
    """Every quotient k + 1/2 is a tie (max 127 or 254 times a power of two): to even. Rows of zeros, of the
    type's smallest and largest values; infinities and NaNs stay in their row."""
    svdq = _svdq()
    f = torch.finfo(dtype)
    k = torch.arange(-127, 128, device="cuda").float()
    row = torch.zeros(512, device="cuda")
    row[:255], row[255:510] = k, (k - 0.5).clamp(-127, 127)
    rows = [row, 0.5 * row, torch.zeros_like(row), torch.full_like(row, f.smallest_normal * f.eps), torch.full_like(row, -f.max),
            torch.linspace(-1, 1, 512, device="cuda") * f.max]
    X = torch.stack(rows + [row, row, row]).to(dtype)
    X[6, 100], X[7, 511], X[8, 0] = float("inf"), float("nan"), float("-inf")
    xq, scale = svdq.i8_quantize_rows(X)
    q, s = R.quantize_rows(X)
    assert torch.equal(xq, q) and torch.equal(scale.view(torch.int32)[:6], s.view(torch.int32)[:6])
    assert bool(scale[6:].isnan().all()) and not bool(xq[6:].any()) and float(scale[2]) == 0
    wq, ws = svdq.i8_quantize_rows(_acts(32, 512, F32, 3))
    Y = svdq.i8_gemm(xq, scale, wq, ws)
    assert bool(Y[6:].isnan().all()) and not bool(Y[2].any()) and bool(Y[:4].isfinite().all())


@pytest.mark.parametrize("dtype,bits", [(BF16, 8), (F16, 11)])
@pytest.mark.parametrize("wide", [False, True])
def test_quantize_every_16_bit_quotient(dtype, bits, wide):
    """Every significand of a maximum with every value of the eight binades below it (whose quotients reach 1/2),
    positive and negative: all borders that 16-bit values can come near to, and all ties. As 32-bit rows too."""
    svdq = _svdq()
    n = 2 ** (bits - 1)
    sig = torch.arange(n, 2 * n, device="cuda").float() / n
    values = torch.cat([sig * 2.0 ** -e for e in range(9)])  # n values in each of [1, 2), [1/2, 1), ..
    for top in sig.split(128):
        X = torch.minimum(values[None], top[:, None])  # what is above the maximum becomes it
        X = torch.cat([X, -X], 1)
        X = torch.nn.functional.pad(X, (0, -X.shape[1] % 16)).to(F32 if wide else dtype)
        for part in X.split(4096, 1):
            part = torch.cat([part, top[:, None].to(part.dtype), torch.zeros(len(top), 15, device="cuda", dtype=part.dtype)], 1)
            xq, scale = svdq.i8_quantize_rows(part)
            q, s = R.quantize_rows(part)
            assert torch.equal(xq, q) and torch.equal(scale, s)


@pytest.mark.parametrize("dtype", R.FLOATS)
@pytest.mark.parametrize("K,at,wide", [(512, 1, 515), (64, 3, 100), (1040, 8, 2096)])
def test_quantize_strided_rows(dtype, K, at, wide):
    svdq = _svdq()
    X = _acts(21, wide, dtype, 5)[:, at:at + K]
    xq, scale = svdq.i8_quantize_rows(X)
    q, s = R.quantize_rows(X)
    assert torch.equal(xq, q) and torch.equal(scale, s)


# tokens, output channels, columns: single tokens, a few, tile edges on every side, long K
SHAPES = [
    (1, 16, 16), (1, 256, 512), (1, 4096, 4096), (1, 1040, 12288), (2, 512, 1040), (3, 96, 64), (4, 4112, 2048), (5, 272, 4096),
    (7, 1536, 1536), (8, 2064, 528), (9, 512, 512), (15, 160, 1024), (16, 4096, 2560), (17, 640, 16), (31, 48, 8192),
    (33, 256, 144), (63, 1024, 1024), (64, 128, 4096), (65, 528, 272), (100, 3200, 1504), (127, 256, 640), (128, 512, 12288),
    (129, 4096, 512), (200, 272, 2064), (255, 1040, 128), (256, 256, 256), (257, 272, 144), (333, 5120, 2560),
    (512, 768, 1040), (777, 2064, 336), (1024, 1024, 4096), (1300, 4608, 1536), (2202, 528, 1536),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,bias", [(BF16, True), (F16, False), (F32, True)])
def test_product(M, N, K, dtype, bias):
    svdq = _svdq()
    xq, wq = _codes(M, K, 10), _codes(N, K, 11)
    xs = torch.rand(M, generator=_gen(12), device="cuda") * 1e-2
    ws = torch.rand(N, generator=_gen(13), device="cuda") * 1e-3
    b = torch.randn(N, generator=_gen(14), device="cuda") if bias else None
    Y = svdq.i8_gemm(xq, xs, wq, ws, b, dtype=dtype)
    y, err = R.i8_product(xq, xs, wq, ws, b)
    R.assert_within(Y, y, R.allowed(y, dtype, err))
    assert torch.equal(Y, svdq.i8_gemm(xq, xs, wq, ws, b, dtype=dtype))
    assert svdq.last_device_error() == 0


@pytest.mark.parametrize("M", [1, 4, 40, 300])
def test_sums_are_exact_integers(M):
    """Unit scales and 32-bit outputs: sums below 2^24 come out as they are, the largest ones of the longest K too
    (within their rounding to fp32)."""
    svdq = _svdq()
    N = 64
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    xq, wq = _codes(M, 912, 20), _codes(N, 912, 21)
    Y = svdq.i8_gemm(xq, one(M), wq, one(N), dtype=F32)
    assert torch.equal(Y.double(), xq.double() @ wq.double().t())
    K = 131072
    xq = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    wq[1::2] = -127
    wq[2] = torch.arange(K, device="cuda") % 2 * 254 - 127
    Y = svdq.i8_gemm(xq, one(M), wq, one(N), dtype=F32)
    assert torch.equal(Y, (xq.double() @ wq.double().t()).float())


@pytest.mark.parametrize("M,N,K,dtype,smooth", [(1, 512, 1024, BF16, True), (6, 272, 528, F16, False),
                                                (140, 1040, 2064, F32, True), (600, 512, 1536, BF16, False),
                                                (1, 48, 16, F32, False), (2, 96, 496, F16, True), (3, 528, 2560, F32, True),
                                                (4, 1040, 4112, BF16, False), (5, 4096, 9216, F16, True),
                                                (8, 272, 12288, BF16, True), (8, 64, 1040, F32, False), (1, 32, 65536, BF16, True)])
def test_linear_forward(M, N, K, dtype, smooth):
    """From floating rows to floating rows; the weight quantized by the same rows' quantizer under the inverse smoothing."""
    svdq = _svdq()
    X = _acts(M, K, dtype, 30)
    W = torch.randn(N, K, generator=_gen(31), device="cuda") * 0.02
    lam = (torch.rand(K, generator=_gen(32), device="cuda") + 0.5) if smooth else None
    b = torch.randn(N, generator=_gen(33), device="cuda")
    wq, ws = svdq.i8_quantize_rows(W, lam)
    inv = None if lam is None else 1 / lam
    Y = svdq.i8_linear_forward(X, wq, ws, b, col_scale=inv)
    q, s = R.quantize_rows(X, inv)
    y, err = R.i8_product(q, s, wq, ws, b)
    R.assert_within(Y, y, R.allowed(y, dtype, err))
    # q s is within s / 2 of each value (and the fp32 scale and smoothing within a few U of theirs), so the product
    # is within sum_k(s_m / 2 |w| + s_n / 2 |x| + s_m s_n / 4) of the unquantized one
    full = X.double() @ W.double().t() + b.double()
    xa = (X.double() if inv is None else X.double() * inv.double()).abs()
    wa = (W.double() if lam is None else W.double() * lam.double()).abs()
    hx, hw = s.double()[:, None] / 2, ws.double()[None] / 2
    assert bool(((y - full).abs() <= (hx * wa.sum(1) + xa.sum(1, keepdim=True) * hw + K * hx * hw) * (1 + 1e-4)
                 + 8 * R.U * (xa @ wa.t())).all())


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 40])
@pytest.mark.parametrize("dtype", R.FLOATS)
def test_few_tokens_and_many_give_the_same_bits(M, dtype):
    """The quantizer and the product are exact, so a token's output does not depend on how many come with it, nor on
    whether its rows are given as int8 or as (strided, unaligned) floating ones."""
    svdq = _svdq()
    X = _acts(40, 1100, dtype, 60)[:, 3:3 + 1040]
    wq, ws = _codes(272, 1040, 61), torch.rand(272, generator=_gen(62), device="cuda") * 1e-3
    col = torch.rand(1040, generator=_gen(63), device="cuda") + 0.5
    every = svdq.i8_gemm(*svdq.i8_quantize_rows(X, col), wq, ws, dtype=dtype)
    assert torch.equal(svdq.i8_linear_forward(X[:M], wq, ws, col_scale=col), every[:M])
    assert torch.equal(svdq.i8_linear_forward(X[:M].contiguous(), wq, ws, col_scale=col), every[:M])
    assert torch.equal(svdq.i8_gemm(*svdq.i8_quantize_rows(X[:M], col), wq, ws, dtype=dtype), every[:M])


def test_few_tokens_special_rows():
    """Zeros, infinities and NaNs among few tokens: as among many."""
    svdq = _svdq()
    X = _acts(4, 512, BF16, 65)
    X[0], X[2, 7], X[3, 500] = 0, float("inf"), float("nan")
    wq, ws = _codes(48, 512, 66), torch.ones(48, device="cuda")
    b = torch.arange(48, device="cuda").float()
    Y = svdq.i8_linear_forward(X, wq, ws, b)
    assert torch.equal(Y[0].float(), b) and bool(Y[1].isfinite().all()) and bool(Y[2:].isnan().all())


def test_no_rows_and_caller_buffers():
    svdq = _svdq()
    wq, ws = _codes(64, 128, 40), torch.ones(64, device="cuda")
    assert svdq.i8_gemm(_codes(0, 128, 41), torch.ones(0, device="cuda"), wq, ws).shape == (0, 64)
    assert svdq.i8_linear_forward(torch.zeros(0, 128, device="cuda"), wq, ws).shape == (0, 64)
    X = _acts(50, 128, BF16, 42)
    want = svdq.i8_linear_forward(X, wq, ws)
    # rows behind the last one keep what they held; a used workspace changes nothing
    Y = torch.full((70, 64), 7.0, dtype=BF16, device="cuda")
    xq = torch.full((70, 128), 9, dtype=torch.int8, device="cuda")
    xs = torch.full((70,), 5.0, device="cuda")
    space = torch.full((max(16, svdq.i8_workspace_bytes(50, 64, 128)),), 0xA5, dtype=torch.uint8, device="cuda")
    svdq.i8_linear_forward(X, wq, ws, xq=xq[:50], x_scale=xs[:50], Y=Y[:50], workspace=space)
    assert torch.equal(Y[:50], want)
    assert bool((Y[50:] == 7).all()) and bool((xq[50:] == 9).all()) and bool((xs[50:] == 5).all())
