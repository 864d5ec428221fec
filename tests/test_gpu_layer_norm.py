"""Layer norm with a weight and a bias for each group of rows: forward, int8 form and gradient against
the definitions in 64 bits, at the sizes, strides and groups where they can go wrong."""
import pytest

from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F16, F32 = R.FLOATS


def _svdq():
    from bit_rank_compensated_b200 import svdq

    return svdq


def _normal(*shape, seed, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dtype)


# rows, columns, groups, rows per group (0: shared out), type of X, type of the parameters
CASES = [
    (1, 1, 1, 0, F32, F32), (1, 8, 1, 0, BF16, BF16), (3, 7, 1, 0, F16, F32), (5, 64, 2, 0, BF16, F32),
    (33, 128, 5, 7, BF16, BF16), (17, 333, 3, 0, F32, F16), (64, 512, 1, 0, F16, F16), (9, 1000, 4, 3, BF16, F32),
    (130, 1024, 2, 0, F32, BF16), (65, 1153, 1, 0, BF16, BF16), (41, 1536, 6, 8, BF16, F32), (12, 2056, 2, 0, F16, F32),
    (300, 4096, 2, 0, BF16, BF16), (7, 5120, 1, 0, F32, F32), (19, 6144, 3, 7, F16, BF16), (5, 9000, 1, 0, BF16, F32),
    (11, 12288, 2, 0, BF16, BF16), (3, 16384, 1, 0, F32, F32), (2, 16383, 2, 0, BF16, F32), (700, 96, 700, 1, BF16, F32),
]


def _inputs(M, K, groups, rows, dtype, params, seed):
    X = _normal(M, K, seed=seed, dtype=dtype, scale=1.5) + _normal(M, 1, seed=seed + 1, dtype=dtype)
    w = _normal(groups, K, seed=seed + 2, dtype=params, scale=0.3)
    b = _normal(groups, K, seed=seed + 3, dtype=params, scale=0.3)
    return X, w, b, rows or -(-M // groups)


@pytest.mark.parametrize("M,K,groups,rows,dtype,params", CASES)
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_forward(M, K, groups, rows, dtype, params, offset):
    svdq = _svdq()
    X, w, b, per = _inputs(M, K, groups, rows, dtype, params, 10)
    Y, mean, rstd = svdq.layer_norm(X, w, b, rows_per_group=rows, weight_offset=offset, stats=True)
    y, _, mu, rs, err = R.layer_norm(X, w, b, per, offset)
    R.assert_within(Y, y, R.allowed(y, dtype, err))
    R.assert_within(mean, mu, 130 * R.U * X.double().abs().mean(1) + 2.0 ** -149)
    R.assert_within(rstd, rs, (140 * R.U + 130 * R.U * X.double().abs().mean(1) * rs) * rs)
    # without statistics, and each call again: the same bits
    assert torch.equal(Y, svdq.layer_norm(X, w, b, rows_per_group=rows, weight_offset=offset))


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("K", [256, 777])
def test_forward_without_weight_or_bias(weight, bias, K):
    svdq = _svdq()
    X, w, b, _ = _inputs(20, K, 1, 0, BF16, F32, 30)
    w, b = (w[0] if weight else None), (b[0] if bias else None)
    Y = svdq.layer_norm(X, w, b, weight_offset=0.5)
    y, _, _, _, err = R.layer_norm(X, w, b, 20, 0.5)
    R.assert_within(Y, y, R.allowed(y, BF16, err))


@pytest.mark.parametrize("dtype", R.FLOATS)
@pytest.mark.parametrize("K,offset,wide", [(512, 0, 520), (512, 1, 515), (768, 3, 771), (100, 4, 301), (2048, 8, 4096)])
def test_strided_rows_and_views(dtype, K, offset, wide):
    """Rows that are sections of wider ones, at every alignment; what lies between them stays as it was."""
    svdq = _svdq()
    M = 37
    buf, out = _normal(M, wide + 8, seed=50, dtype=dtype), _normal(M, wide + 8, seed=51, dtype=dtype)
    mod = _normal(2, 2 * K + 2 * offset, seed=52, dtype=BF16, scale=0.2)
    shift, scale = mod[:, offset:offset + K], mod[:, offset + K:offset + 2 * K]
    X, Y = buf[:, offset:offset + K], out[:, offset:offset + K]
    kept = out.clone()
    svdq.layer_norm(X, scale, shift, weight_offset=1.0, Y=Y)
    y, xhat, mean, rstd, err = R.layer_norm(X, scale, shift, 19, 1.0)
    R.assert_within(Y, y, R.allowed(y, dtype, err))
    kept[:, offset:offset + K] = Y
    assert torch.equal(kept, out)
    dY = _normal(M, wide + 8, seed=53, dtype=dtype)[:, offset:offset + K]
    mean, rstd = mean.float(), rstd.float()
    (dx, dw, db), (dxe, dwe, dbe) = R.layer_norm_backward(dY, X, mean, rstd, scale, 19, 2, 1.0)
    got = svdq.layer_norm_backward(dY, X, mean, rstd, scale, weight_offset=1.0, dX=Y)
    assert got[0] is Y
    R.assert_within(Y, dx, R.allowed(dx, dtype, dxe))
    R.assert_within(got[1], dw, dwe + 1e-30)
    R.assert_within(got[2], db, dbe + 1e-30)
    kept[:, offset:offset + K] = Y
    assert torch.equal(kept, out)


def test_in_place():
    svdq = _svdq()
    X, w, b, _ = _inputs(50, 1536, 1, 0, BF16, F32, 60)
    dY = _normal(50, 1536, seed=64, dtype=BF16)
    want, mean, rstd = svdq.layer_norm(X, w, b, stats=True)
    dX, dw, db = svdq.layer_norm_backward(dY, X, mean, rstd, w)
    for target in (dY.clone(), X.clone()):
        x, dy = (X, target) if target.data_ptr() != X.data_ptr() and torch.equal(target, dY) else (target, dY)
        got = svdq.layer_norm_backward(dy, x, mean, rstd, w, dX=target)
        assert torch.equal(target, dX) and torch.equal(got[1], dw) and torch.equal(got[2], db)
    assert svdq.layer_norm(X, w, b, Y=X) is X
    assert torch.equal(X, want)


def test_constant_rows_and_far_means():
    """A row of one value has no variance (rstd = eps^-1/2); a mean far from zero costs bits of x - mean."""
    svdq = _svdq()
    X = torch.full((4, 4096), 3.0, device="cuda")
    X[1] = 0
    X[2] = 1000 + _normal(4096, seed=70)
    X[3] = -5e4 + 100 * _normal(4096, seed=71)
    Y, mean, rstd = svdq.layer_norm(X, stats=True)
    y, _, mu, rs, err = R.layer_norm(X, None, None, 4, 0.0)
    R.assert_within(Y, y, R.allowed(y, F32, err))
    assert torch.equal(Y[:2], torch.zeros_like(Y[:2]))
    assert float((rstd[0] - 1e3).abs()) < 1e-3


def test_infinite_and_nan_rows_stay_in_their_row():
    svdq = _svdq()
    X = _normal(6, 640, seed=80, dtype=BF16)
    clean = svdq.layer_norm(X)
    X[1, 5], X[4, 639] = float("nan"), float("inf")
    Y = svdq.layer_norm(X)
    keep = [0, 2, 3, 5]
    assert torch.equal(Y[keep], clean[keep]) and bool(Y[[1, 4]].isnan().all())
    xq, s = svdq.i8_layer_norm_quantize(X)
    assert bool(s[[1, 4]].isnan().all()) and not bool(xq[[1, 4]].any()) and bool(s[keep].isfinite().all())


@pytest.mark.parametrize("M,K,groups,rows,dtype,params", CASES)
def test_backward(M, K, groups, rows, dtype, params):
    svdq = _svdq()
    X, w, _, per = _inputs(M, K, groups, rows, dtype, params, 90)
    dY = _normal(M, K, seed=95, dtype=dtype)
    _, _, mean, rstd, _ = R.layer_norm(X, w, None, per, 1.0)
    mean, rstd = mean.float(), rstd.float()
    want, bounds = R.layer_norm_backward(dY, X, mean, rstd, w, per, groups, 1.0)
    dX, dw, db = svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=rows, weight_offset=1.0)
    R.assert_within(dX, want[0], R.allowed(want[0], dtype, bounds[0]))
    R.assert_within(dw, want[1], bounds[1] + 1e-30)
    R.assert_within(db, want[2], bounds[2] + 1e-30)
    # each output alone, and a workspace of the caller's that held something else: the same bits
    space = torch.full((max(16, svdq.load().svdq_layer_norm_workspace_bytes(M, K, groups, per)),), 0xFF,
                       dtype=torch.uint8, device="cuda")
    only = [svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=rows, weight_offset=1.0, need_dX=i == 0,
                                     need_dweight=i == 1, need_dbias=i == 2, workspace=space)[i] for i in range(3)]
    assert torch.equal(only[0], dX) and torch.equal(only[1], dw) and torch.equal(only[2], db)


def test_backward_of_empty_groups():
    """Groups behind the last row get zeros, whatever the buffers held; no rows at all do too."""
    svdq = _svdq()
    X, w, _, _ = _inputs(5, 320, 4, 3, BF16, F32, 100)
    dY = _normal(5, 320, seed=104, dtype=BF16)
    _, mean, rstd = svdq.layer_norm(X, stats=True)
    _, dw, db = svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=3)
    assert not bool(dw[2:].any()) and not bool(db[2:].any()) and bool(db[:2].any(1).all())
    none = svdq.layer_norm_backward(dY[:0], X[:0], mean[:0], rstd[:0], w, rows_per_group=3)
    assert none[0].shape == (0, 320) and not bool(none[1].any()) and not bool(none[2].any())
    assert svdq.layer_norm(X[:0]).shape == (0, 320)


def test_backward_of_many_groups_without_rows():
    """More groups than a grid has rows, most of them behind the last row."""
    svdq = _svdq()
    X, w, _, _ = _inputs(1000, 40, 70000, 100, BF16, F32, 130)
    dY = _normal(1000, 40, seed=134, dtype=BF16)
    _, _, mean, rstd, _ = R.layer_norm(X, w, None, 100, 0.0)
    mean, rstd = mean.float(), rstd.float()
    _, dw, db = svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=100)
    want, bounds = R.layer_norm_backward(dY, X, mean, rstd, w[:10], 100, 10, 0.0)
    R.assert_within(dw[:10], want[1], bounds[1] + 1e-30)
    R.assert_within(db[:10], want[2], bounds[2] + 1e-30)
    assert not bool(dw[10:].any()) and not bool(db[10:].any())


@pytest.mark.parametrize("K", [96, 97, 100, 1000, 1024])
def test_backward_of_far_constant_rows(K):
    """mean * rstd overflows, x - mean does not: nothing of that comes from beside the row."""
    svdq = _svdq()
    X = torch.full((3, K), 1e35, device="cuda")
    dY = _normal(3, K, seed=140)
    mean, rstd = X[:, 0].clone(), torch.full((3,), 1e6, device="cuda")
    dX, dw, db = svdq.layer_norm_backward(dY, X, mean, rstd)
    want, bounds = R.layer_norm_backward(dY, X, mean, rstd, None, 3, 1, 0.0)
    R.assert_within(dX, want[0], R.allowed(want[0], F32, bounds[0]))
    assert not bool(dw.any())
    R.assert_within(db, want[2], bounds[2] + 1e-30)


def test_backward_against_differences():
    """dX, dweight and dbias against central differences of the forward pass in fp32."""
    svdq = _svdq()
    M, K, h = 6, 40, 1e-2
    X, w, b, _ = _inputs(M, K, 2, 3, F32, F32, 110)
    dY = _normal(M, K, seed=114)
    _, mean, rstd = svdq.layer_norm(X, w, b, rows_per_group=3, stats=True)
    grads = svdq.layer_norm_backward(dY, X, mean, rstd, w, rows_per_group=3)
    loss = lambda x, w_, b_: (svdq.layer_norm(x, w_, b_, rows_per_group=3).double() * dY.double()).sum()  # noqa: E731
    for t, g in zip((X, w, b), grads):
        for i in range(0, t.numel(), 17):
            old = t.view(-1)[i].item()
            v = []
            for step in (h, -h):
                t.view(-1)[i] = old + step
                v.append(float(loss(X, w, b)))
            t.view(-1)[i] = old
            # truncation h^2 / 6 times a third derivative of a few units, plus fp32 noise of the loss / h
            assert abs((v[0] - v[1]) / (2 * h) - float(g.view(-1)[i])) < 5e-3 * (1 + abs(float(g.view(-1)[i])))


@pytest.mark.parametrize("M,K,groups,rows,dtype,params", [c for c in CASES if c[1] % 16 == 0])
def test_int8_form(M, K, groups, rows, dtype, params):
    """Codes are those of the 64-bit value, except where it lies within the fp32 error of a border."""
    svdq = _svdq()
    X, w, b, per = _inputs(M, K, groups, rows, dtype, params, 120)
    xq, scale = svdq.i8_layer_norm_quantize(X, w, b, rows_per_group=rows, weight_offset=1.0)
    y, _, _, _, err = R.layer_norm(X, w, b, per, 1.0)
    top = y.abs().amax(1)
    terr = err.amax(1)
    R.assert_within(scale, top / 127, terr / 127 + 2 * R.U * top / 127)
    t = 127 * y / top[:, None]
    terr = (127 * err / top[:, None]) + 127 * (terr / top)[:, None] + 2.0 ** -14
    off = (xq.double() - t).abs()
    assert bool((off <= 0.5 + terr).all())
    assert bool((xq.double().abs().amax(1) == 127).all())
