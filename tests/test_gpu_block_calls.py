"""Calls of the operators around the projections that their documentation allows, at the ends of its ranges and
from programs other than one thread on one stream."""
import pytest

from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F16, F32 = R.FLOATS


def _svdq():
    from bit_rank_compensated_b200 import svdq

    return svdq


def _normal(*shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2147480000])
@pytest.mark.parametrize("M", [1, 2, 5, 700, 4608])
def test_one_group_for_all_rows_whatever_its_size(M, rows):
    """rows_per_group near 2^31 is one group: the bits that rows_per_group = M gives, and nothing outside the outputs."""
    svdq = _svdq()
    K = 512
    X, dY, w = _normal(M, K, seed=1, dtype=BF16), _normal(M, K, seed=2, dtype=BF16), _normal(2, K, seed=3)
    _, mean, rstd = svdq.layer_norm(X, stats=True)
    assert torch.equal(svdq.layer_norm(X, w, w, rows_per_group=rows), svdq.layer_norm(X, w[0], w[0], rows_per_group=M))
    want = svdq.layer_norm_backward(dY, X, mean, rstd, w[0], rows_per_group=M)
    got = svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=rows)
    assert torch.equal(got[0], want[0])
    for g, v in zip(got[1:], want[1:]):
        assert torch.equal(g[:1], v) and not bool(g[1:].any())
    # into a buffer of the caller's, between rows that are to stay
    import ctypes

    lib = svdq.load()
    a = svdq.NormAffineStruct(w.data_ptr(), None, K, 0, 2, 2, rows, 0.0)
    need = lib.svdq_layer_norm_workspace_bytes(M, K, 2, rows)
    space = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    out = torch.full((6, K), 7.0, device="cuda")
    st = lib.svdq_layer_norm_backward(dY.data_ptr(), K, X.data_ptr(), K, 0, M, K, ctypes.addressof(a), mean.data_ptr(),
                                      rstd.data_ptr(), None, 0, out[2:].data_ptr(), None, space.data_ptr(), need,
                                      torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(out[2:4], got[1]) and bool((out[:2] == 7).all()) and bool((out[4:] == 7).all())
    assert svdq.last_device_error() == 0


# ---------------------------------------------------------------- host threads
class Worker:
    """A host thread that makes calls when it is told to."""

    def __init__(self):
        import concurrent.futures

        self.pool = concurrent.futures.ThreadPoolExecutor(max_workers=1)

    def __call__(self, f):
        return self.pool.submit(f).result(timeout=120)


def _norm_call(svdq, dtype, K):
    X, w = _normal(9, K, seed=10, dtype=dtype), _normal(K, seed=11)
    return lambda: [svdq.layer_norm(X, w, w)]


def _int8_norm_call(svdq, dtype, K):
    X, w = _normal(9, K, seed=12, dtype=dtype), _normal(K, seed=13)
    return lambda: list(svdq.i8_layer_norm_quantize(X, w, w))


def _gradient_call(svdq, dtype, K):
    X, dY = _normal(9, K, seed=14, dtype=dtype), _normal(9, K, seed=15, dtype=dtype)
    _, mean, rstd = svdq.layer_norm(X[:, :64].contiguous(), stats=True)
    return lambda: list(svdq.layer_norm_backward(dY, X, mean, rstd))


def _quantize_call(svdq, dtype, K):
    X = _normal(9, K, seed=16, dtype=dtype)
    return lambda: list(svdq.i8_quantize_rows(X))


def _few_call(svdq, dtype, K):
    X = _normal(7, K, seed=17, dtype=dtype)
    wq, ws = svdq.i8_quantize_rows(_normal(64, K, seed=18, dtype=dtype))
    return lambda: [svdq.i8_linear_forward(X, wq, ws)]


@pytest.mark.parametrize("call,dtype,large,small", [
    (_norm_call, F32, 16384, 12288), (_norm_call, F16, 16384, 12800), (_int8_norm_call, BF16, 16384, 12800),
    (_gradient_call, BF16, 8192, 6144), (_gradient_call, F32, 8192, 6144), (_gradient_call, F16, 16384, 12288),
    (_quantize_call, F32, 16384, 12288), (_few_call, BF16, 12288, 8192), (_few_call, F32, 12288, 8192),
])
def test_two_threads_with_rows_of_different_lengths(call, dtype, large, small):
    """Two host threads use one kernel with more and with less shared memory in turn: neither takes from the other
    what its launches need."""
    svdq = _svdq()
    a, b = Worker(), Worker()
    more, less = call(svdq, dtype, large), call(svdq, dtype, small)
    first = a(more)
    for _ in range(3):
        other = b(less)
        for x, y in zip(a(more), first):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        for x, y in zip(b(less), other):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # and both at once
    futures = [w.pool.submit(lambda f=f: [f() for _ in range(20)]) for w, f in ((a, more), (b, less))]
    for got in (f.result(timeout=120) for f in futures):
        assert len(got) == 20
    torch.cuda.synchronize()
    assert svdq.last_device_error() == 0


# ---------------------------------------------------------------- rows far from zero
@pytest.mark.parametrize("dtype", R.FLOATS)
@pytest.mark.parametrize("K", [3, 97, 104, 777, 1000, 1153, 1920, 4096, 5120, 12288, 16383])
def test_a_constant_row_is_its_bias(K, dtype):
    """x - mean is 0 for every column, whatever K and the value: no rounding of the mean is left for rstd = eps^-1/2
    to make a thousand times larger. (The sum of K <= 16384 equal values is within 131 U of itself, so the first mean
    is off by j <= 131 steps of the value; x less it is exact, K j < 2^24 steps sum exactly, and their mean is j.)"""
    svdq = _svdq()
    values = [0.0, 1.0, -3.0, 0.1, 100.0, 1000.0, -1000.1, 1 / 3, 3e4, 1e-3] + ([1e6, 7654321.0, 3e9, -1e-9] if dtype != F16 else [])
    X = torch.tensor(values, device="cuda").to(dtype)[:, None].repeat(1, K)
    w, b = _normal(K, seed=20), _normal(K, seed=21)
    Y, mean, rstd = svdq.layer_norm(X, w, b, stats=True)
    assert torch.equal(Y, b.to(dtype).expand_as(Y))
    assert torch.equal(mean, X[:, 0].float())
    # the variance is 0 in exact arithmetic; what is subtracted as the first mean's error squared leaves 4 U of it at
    # most, beside eps
    left = 4 * R.U * (131 * R.U * X[:, 0].double()) ** 2 * 140
    assert bool(((rstd.double() * R.EPS ** 0.5 - 1).abs() <= 140 * R.U + left / R.EPS).all())
    assert not bool(svdq.layer_norm(X).any())
    if K % 16 == 0:
        xq, scale = svdq.i8_layer_norm_quantize(X)
        assert not bool(xq.any()) and not bool(scale.any())


# rows, columns, mean, deviation
FAR = [(5, 1920, 1000.0, 1e-2), (5, 777, 1000.0, 1.0), (3, 4096, -5e4, 1.0), (4, 1153, 30.0, 1e-3), (3, 12288, 300.0, 0.1),
       (3, 104, 1e4, 1e-1), (2, 16384, 100.0, 1e-3)]


@pytest.mark.parametrize("M,K,far,deviation", FAR)
def test_rows_far_from_zero(M, K, far, deviation):
    """With A = mean|x|: the first mean is within D = 131 U A; d = x - mean rounds once, its sum within 130 U sum|d|;
    so x - mean is within 134 U (mean|d|) + 4 U |d| of itself, where |d| <= |x - mean| + D, and no longer within
    130 U A. The variance is sum d^2 / K (140 U of it and of D^2) less the square of what was corrected."""
    svdq = _svdq()
    X = far + _normal(M, K, seed=30, scale=deviation)
    x = X.double()
    mu = x.mean(1, keepdim=True)
    c = x - mu
    rs = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + R.EPS)
    D = 131 * R.U * x.abs().mean(1, keepdim=True)
    off = 134 * R.U * (c.abs().mean(1, keepdim=True) + D) + 4 * R.U * (c.abs() + D)
    rel = 150 * R.U * (1 + (D * rs) ** 2)
    Y, mean, rstd = svdq.layer_norm(X, stats=True)
    R.assert_within(rstd[:, None], rs, rel * rs)
    R.assert_within(mean[:, None], mu, off.amax(1, keepdim=True) + R.U * mu.abs())
    R.assert_within(Y, c * rs, rs * off * (1 + rel) + (rel + 4 * R.U) * (c * rs).abs())


def test_other_threads_run_while_a_call_waits():
    """A call that waits in the library (for memory, for a full launch queue) leaves the interpreter to the other
    threads. In the place of the library's functions, a C function that sleeps as many microseconds as xq has rows."""
    import ctypes
    import threading
    import time

    svdq = _svdq()
    native, lib, libc = svdq._native(), svdq.load(), ctypes.CDLL(None)
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    own = [address(getattr(lib, "svdq_" + name)) for name in svdq._BOUND]
    fakes = dict(i8_workspace_bytes=address(libc.usleep), i8_gemm=address(lib.svdq_version))
    xq = torch.zeros(400000, 16, dtype=torch.int8, device="cuda")
    wq, xs, ws = xq[:16], torch.zeros(400000, device="cuda"), torch.zeros(16, device="cuda")
    Y = torch.empty(400000, 16, dtype=BF16, device="cuda")
    turns, stop = [], threading.Event()

    def count():
        while not stop.is_set():
            turns.append(time.perf_counter())
            time.sleep(0.002)

    other = threading.Thread(target=count)
    try:
        native.bind(*(fakes.get(name, at) for name, at in zip(svdq._BOUND, own)))
        other.start()
        start = time.perf_counter()
        got = native.i8_gemm(xq, xs, wq, ws, None, Y, 0, None)
        end = time.perf_counter()
    finally:
        native.bind(*own)
        stop.set()
        other.join()
    assert isinstance(got, int) and got == lib.svdq_version()  # (what the fake returned as a status)
    assert end - start >= 0.4
    assert sum(start + 0.05 < t < end - 0.05 for t in turns) >= 10


def test_a_flag_without_a_truth_value_is_an_error():
    svdq = _svdq()
    X, st = _normal(4, 64, seed=40), torch.zeros(4, device="cuda")
    flag = torch.ones(2)  # "Boolean value of Tensor with more than one value is ambiguous"
    q, pos = X.unflatten(1, (2, 32)), torch.zeros(4, 1, dtype=torch.int64, device="cuda")
    for f in (lambda: svdq.layer_norm(X, stats=flag), lambda: svdq.layer_norm_backward(X, X, st, st, need_dX=flag),
              lambda: svdq.rope_axes_apply(q, None, pos, svdq.RopeAxes((16,)), inverse=flag)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            f()


# ---------------------------------------------------------------- few tokens
@pytest.mark.parametrize("N,K", [(272, 1024), (272, 1040), (272, 2048), (272, 4112), (64, 8208), (9472, 1552), (9488, 1536),
                                 (9488, 1552)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_tokens_by_every_way(N, K, dtype):
    """Rows quantized where they are multiplied, rows quantized before, tokens left to the tensor cores: the sums are
    exact and the codes the same, so a token's output does not depend on the way."""
    svdq = _svdq()
    X = _normal(9, K, seed=50, dtype=dtype)
    col = _normal(K, seed=51).abs() + 0.5
    wq, ws = svdq.i8_quantize_rows(_normal(N, K, seed=52, dtype=BF16))
    b = _normal(N, seed=53)
    every = svdq.i8_linear_forward(X, wq, ws, b, col_scale=col)
    q, s = R.quantize_rows(X, col)
    y, err = R.i8_product(q, s, wq, ws, b)
    R.assert_within(every, y, R.allowed(y, dtype, err))
    for M in range(1, 9):
        assert torch.equal(svdq.i8_linear_forward(X[:M], wq, ws, b, col_scale=col), every[:M])
        assert torch.equal(svdq.i8_gemm(q[:M], s[:M], wq, ws, b, dtype=dtype), every[:M])
    assert svdq.last_device_error() == 0


@pytest.mark.parametrize("M", [1, 8, 9])
def test_as_many_channels_as_an_int_counts(M):
    """N = 2^31 - 16: a tile's or task's size added to it passes 31 bits. Weight rows of zeros but at the ends."""
    svdq = _svdq()
    N, K, ends = 2 ** 31 - 16, 16, 400
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("about 90 GB of device memory")
    try:
        xq = torch.randint(-127, 128, (M, K), generator=torch.Generator("cuda").manual_seed(60), device="cuda", dtype=torch.int8)
        wq = torch.zeros(N, K, dtype=torch.int8, device="cuda")
        for part in (wq[:ends], wq[-ends:]):
            part.copy_(torch.randint(-127, 128, (ends, K), generator=torch.Generator("cuda").manual_seed(61), device="cuda"))
        xs, ws = torch.rand(M, device="cuda") + 0.5, torch.ones(N, device="cuda")
        Y = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
        svdq.i8_gemm(xq, xs, wq, ws, Y=Y)
        for at in (slice(0, ends), slice(N - ends, N)):
            y, err = R.i8_product(xq, xs, wq[at], ws[at], None)
            R.assert_within(Y[:, at], y, R.allowed(y, BF16, err))
        for m in range(M):
            for part in Y[m, ends:N - ends].split(2 ** 29):
                assert int(torch.count_nonzero(part)) == 0
    finally:
        xq = wq = xs = ws = Y = part = None
        torch.cuda.empty_cache()
    assert svdq.last_device_error() == 0


def test_lazily_negated_views_are_refused():
    """The imaginary part of a conjugated tensor is a view whose memory holds the other sign."""
    svdq = _svdq()
    z = torch.complex(_normal(4, 64, seed=70), _normal(4, 64, seed=71))
    assert z.conj().imag.is_neg()
    rows = z.imag.contiguous()
    negated = torch._neg_view(rows)
    assert negated.is_neg() and torch.equal(negated, -rows)
    q, pos, axes = negated.unflatten(1, (2, 32)), torch.zeros(4, 1, dtype=torch.int64, device="cuda"), svdq.RopeAxes((16,))
    one, w = torch.ones(4, device="cuda"), torch._neg_view(torch.ones(64, device="cuda"))
    for f in (lambda: svdq.layer_norm(negated), lambda: svdq.layer_norm(rows, w), lambda: svdq.layer_norm(rows, None, w),
              lambda: svdq.layer_norm(rows, Y=negated), lambda: svdq.layer_norm_backward(negated, rows, one, one),
              lambda: svdq.layer_norm_backward(rows, negated, one, one), lambda: svdq.i8_quantize_rows(negated),
              lambda: svdq.i8_quantize_rows(rows, w), lambda: svdq.i8_layer_norm_quantize(negated),
              lambda: svdq.rope_axes_apply(q, None, pos, axes), lambda: svdq.rope_axes_apply(q.resolve_neg(), q, pos, axes),
              lambda: svdq.rope_axes_table(torch._neg_view(pos.float()), axes)):
        with pytest.raises(ValueError, match="resolve_neg"):
            f()
    assert torch.equal(svdq.layer_norm(negated.resolve_neg()), -svdq.layer_norm(rows))


# ---------------------------------------------------------------- autograd
def test_calls_are_detached():
    svdq = _svdq()
    X = _normal(4, 64, seed=80).requires_grad_()
    w = _normal(64, seed=81).requires_grad_()
    q = X.unflatten(1, (2, 32))
    pos, axes = torch.zeros(4, 1, dtype=torch.int64, device="cuda"), svdq.RopeAxes((16,))
    wq, ws = svdq.i8_quantize_rows(_normal(16, 64, seed=82))
    for y in (svdq.layer_norm(X, w), svdq.rope_axes_apply(q, None, pos, axes)[0], svdq.i8_linear_forward(X, wq, ws)):
        assert not y.requires_grad


@pytest.mark.parametrize("M,groups", [(1, 1), (37, 3), (600, 2)])
def test_gradients_in_a_function_of_the_callers(M, groups):
    """Norm and rotation as one torch.autograd.Function, as the tuning of a block's norms makes it: the gradients of
    fp32 leaves against those of the formula under autograd in 64 bits, by the bounds of each call."""
    svdq = _svdq()
    K, heads, rows = 256, 2, -(-M // groups)
    pos, axes = torch.arange(M, device="cuda")[:, None] * 3, svdq.RopeAxes((32, 32))
    pos = torch.cat([pos, pos // 5], 1)

    class NormRotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, w, b):
            Y, mean, rstd = svdq.layer_norm(X, w, b, rows_per_group=rows, weight_offset=1.0, stats=True)
            ctx.save_for_backward(X, w, mean, rstd)
            return svdq.rope_axes_apply(Y.unflatten(1, (heads, K // heads)), None, pos, axes)[0]

        @staticmethod
        def backward(ctx, dq):
            X, w, mean, rstd = ctx.saved_tensors
            dY = svdq.rope_axes_apply(dq.contiguous(), None, pos, axes, inverse=True)[0].flatten(1)
            return svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=rows, weight_offset=1.0)

    leaves = [_normal(M, K, seed=90), _normal(groups, K, seed=91, scale=0.3), _normal(groups, K, seed=92, scale=0.3)]
    dq = _normal(M, heads, K // heads, seed=93)
    own = [t.clone().requires_grad_() for t in leaves]
    got = torch.autograd.grad(NormRotate.apply(*own), own, dq)
    x, w, b = [t.double().requires_grad_() for t in leaves]
    d = x - x.mean(1, keepdim=True)
    xhat = d / torch.sqrt((d * d).mean(1, keepdim=True) + R.EPS)
    row = torch.arange(M, device="cuda") // rows
    y = (xhat * (1 + w[row]) + b[row]).unflatten(1, (heads, K // heads))
    cos, sin, angle = R.cos_sin(pos, (32, 32), 10000.0, False)
    u, v = y[..., 0:128:2], y[..., 1:128:2]
    turned = torch.stack([u * cos[:, None] - v * sin[:, None], v * cos[:, None] + u * sin[:, None]], -1).flatten(-2)
    want = torch.autograd.grad(turned, (x, w, b), dq.double())
    # the rotation back is within e |u| + |v| of each pair, and goes linearly through the norm's gradient; the
    # statistics are within 140 U of theirs, which the gradient takes with a factor of its own size
    e = 2.0 ** -22 + 2.0 ** -50 * float(angle.abs().max()) + 3 * R.U
    dy, _ = R.rope(dq, cos, sin, angle, False, True)
    dy = dy.flatten(1)
    off = e * dq.double().abs().unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1).flatten(1)
    with torch.no_grad():
        mean, rstd = x.mean(1), 1 / torch.sqrt((d * d).mean(1) + R.EPS)
        _, bounds = R.layer_norm_backward(dy, leaves[0], mean, rstd, leaves[1], rows, groups, 1.0)
        wa, r, xa = 1 + w.abs()[row], rstd[:, None], xhat.abs()
        g, gdy = off * wa, dy.abs() * wa
        stat = 300 * R.U * (1 + (x.abs().mean(1, keepdim=True) * r))
        more = r * (g + g.mean(1, keepdim=True) + xa * (g * xa).mean(1, keepdim=True))
        more = more + stat * r * (gdy + gdy.mean(1, keepdim=True) + (1 + xa) * (gdy * (1 + xa)).mean(1, keepdim=True)) * 3
        grouped = lambda t: torch.zeros(groups, K, dtype=torch.float64, device="cuda").index_add(0, row, t)  # noqa: E731
        R.assert_within(got[0], want[0], R.allowed(want[0], F32, bounds[0] + more))
        R.assert_within(got[1], want[1], bounds[1] + grouped(off * xa + stat * dy.abs() * (1 + xa)) + 1e-30)
        R.assert_within(got[2], want[2], bounds[2] + grouped(off) + 1e-30)
