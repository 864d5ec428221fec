"""Rotary positions with several axes: table and rotation against the definition in 64 bits."""
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


def _normal(*shape, seed, dtype):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


def _pos(M, axes, seed, dtype=torch.int64, far=200):
    p = torch.randint(-far, far + 1, (M, axes), generator=_gen(seed), device="cuda")
    return p.to(dtype) if dtype != F32 else p + 0.25


@pytest.mark.parametrize("M,pairs,shared,dtype,far", [
    (1, (64,), False, torch.int64, 100), (300, (8, 28, 28), False, torch.int32, 4000), (77, (16, 24, 24), True, torch.int64, 10 ** 7),
    (5, (1, 1, 1, 1), True, F32, 50), (1000, (3, 37), False, F32, 3000), (2, (256,), True, torch.int32, 2 ** 31 - 1),
    (129, (128, 64, 64), False, torch.int64, 2 ** 40),
])
def test_table(M, pairs, shared, dtype, far):
    svdq = _svdq()
    pos = _pos(M, len(pairs), 1, dtype, far)
    got = svdq.rope_axes_table(pos, svdq.RopeAxes(pairs, theta=10000.0, shared_ladder=shared))
    cos, sin, angle = R.cos_sin(pos, pairs, 10000.0, shared)
    if far < 2 ** 40:
        R.assert_within(got[..., 0], cos, R.turn_error(angle))
        R.assert_within(got[..., 1], sin, R.turn_error(angle))
    else:  # a far angle has lost its last bits in 64 bits too: what stays is a rotation
        R.assert_within((got.double() ** 2).sum(-1), torch.ones_like(cos), 2.0 ** -21 + 0 * cos)


def test_table_is_the_fused_projections():
    """The axes of the fused QKV stage's workloads (16, 56 and 56 columns) give the table that it is fed."""
    svdq = _svdq()
    from synth import rope_table

    m = torch.arange(700, device="cuda")
    j = (m - 77).clamp_min(0)
    pos = torch.stack([0 * m, torch.where(m < 77, 0, j // 64), torch.where(m < 77, 0, j % 64)], 1)
    got = svdq.rope_axes_table(pos, svdq.RopeAxes((8, 28, 28)))
    want = torch.from_numpy(rope_table(700, n_text=77)).cuda()
    assert float((got - want).abs().max()) <= 2.0 ** -22 + 2.0 ** -24  # the bound above, and the table's own rounding


# tokens, Q heads, K heads, columns, pairs, halves, shared, inverse
CASES = [
    (1, 1, 0, 2, (1,), False, False, False), (1, 32, 8, 128, (16, 24, 24), True, True, False),
    (3, 4, 4, 64, (8, 12, 12), False, False, False), (37, 24, 24, 128, (8, 28, 28), False, False, False),
    (130, 3, 1, 96, (8, 16, 16), False, True, True), (65, 8, 2, 80, (40,), True, False, True),
    (50, 2, 2, 80, (3, 17), True, True, False), (17, 5, 5, 256, (32, 48, 48), True, False, False),
    (9, 1, 1, 512, (64, 64, 64, 64), False, True, False), (11, 2, 1, 70, (5, 6), False, False, True),
    (11, 2, 1, 70, (5, 6), True, False, False), (4, 7, 3, 6, (1, 1), False, False, False), (700, 2, 2, 128, (64,), True, True, True),
    (23, 16, 16, 96, (1, 2, 3), False, False, False), (23, 16, 16, 96, (1, 2, 3), True, False, True), (5, 100, 1, 64, (32,), False, False, False),
]


def _check(svdq, q, k, pos, pairs, halves, shared, inverse, q_out=None, k_out=None):
    axes = svdq.RopeAxes(pairs, theta=500.0, shared_ladder=shared, halves=halves)
    q0, k0 = q.clone(), None if k is None else k.clone()
    got = svdq.rope_axes_apply(q, k, pos, axes, inverse=inverse, q_out=q_out, k_out=k_out)
    cos, sin, angle = R.cos_sin(pos, pairs, 500.0, shared)
    for x, y in zip((q0, k0), got):
        if x is None:
            assert y is None
            continue
        want, err = R.rope(x, cos, sin, angle, halves, inverse)
        R.assert_within(y, want, R.allowed(want, x.dtype, err))
        P = 2 * sum(pairs)
        assert torch.equal(y[..., P:], x[..., P:])
    return got


@pytest.mark.parametrize("M,hq,hk,D,pairs,halves,shared,inverse", CASES)
@pytest.mark.parametrize("dtype", R.FLOATS)
def test_apply(M, hq, hk, D, pairs, halves, shared, inverse, dtype):
    svdq = _svdq()
    q = _normal(M, hq, D, seed=1, dtype=dtype)
    k = _normal(M, hk, D, seed=2, dtype=dtype) if hk else None
    _check(svdq, q, k, _pos(M, len(pairs), 3), pairs, halves, shared, inverse)


@pytest.mark.parametrize("dtype", R.FLOATS)
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("at,D,pad", [(0, 128, 0), (1, 128, 3), (8, 64, 8), (5, 72, 1)])
def test_views_in_place_and_orders(dtype, halves, at, D, pad):
    """Sections of packed rows at every alignment, head-major tensors, positions by axis, in place: the rest stays."""
    svdq = _svdq()
    M, H, pairs = 29, 3, (D // 8, D // 8)
    buf = _normal(M, at + 3 * H * D + pad, seed=4, dtype=dtype)
    q, k = buf[:, at:at + H * D].unflatten(1, (H, D)), buf[:, at + H * D:at + 2 * H * D].unflatten(1, (H, D))
    pos = _pos(2, M, 5).t()  # [M, 2] stored by axis
    want = _check(svdq, q, k, pos, pairs, halves, False, False)
    hm = _normal(H, M, D, seed=6, dtype=dtype).transpose(0, 1)  # head-major storage
    _check(svdq, hm, None, pos, pairs, halves, True, True)
    out = torch.full((H, M, D), 3.0, dtype=dtype, device="cuda").transpose(0, 1)
    _check(svdq, q, None, pos, pairs, halves, False, False, q_out=out)
    assert torch.equal(out, want[0])
    kept = buf.clone()
    axes = svdq.RopeAxes(pairs, theta=500.0, halves=halves)
    svdq.rope_axes_apply(q, k, pos, axes, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    kept[:, at:at + 2 * H * D] = buf[:, at:at + 2 * H * D]
    assert torch.equal(kept, buf)


def test_inverse_undoes_and_is_the_gradient():
    """In fp32 the inverse returns the input within the roundings of both; <dy, R x> = <R^-1 dy, x>."""
    svdq = _svdq()
    axes = svdq.RopeAxes((8, 28, 28))
    pos = _pos(100, 3, 7)
    q, k = _normal(100, 6, 128, seed=8, dtype=F32), _normal(100, 2, 128, seed=9, dtype=F32)
    y = svdq.rope_axes_apply(q, k, pos, axes)
    back = svdq.rope_axes_apply(*y, pos, axes, inverse=True)
    for x, z in zip((q, k), back):
        pair = x.double().unflatten(-1, (-1, 2)).abs().sum(-1).repeat_interleave(2, -1)
        R.assert_within(z, x.double(), 4 * (2.0 ** -22 + 4 * R.U) * pair)
    dy = _normal(100, 6, 128, seed=10, dtype=F32)
    dq, _ = svdq.rope_axes_apply(dy, None, pos, axes, inverse=True)
    a, b = (dy.double() * y[0].double()).sum(), (dq.double() * q.double()).sum()
    assert abs(float(a - b)) < 1e-5 * float((dy.double() * y[0].double()).abs().sum())


def test_far_positions_and_no_tokens():
    svdq = _svdq()
    pairs = (4, 6, 6)
    pos = _pos(40, 3, 11, torch.int64, 10 ** 8)
    q = _normal(40, 2, 32, seed=12, dtype=BF16)
    _check(svdq, q, None, pos, pairs, False, False, False)
    axes = svdq.RopeAxes(pairs)
    q_out, k_out = svdq.rope_axes_apply(q[:0], q[:0], pos[:0], axes)
    assert q_out.shape == k_out.shape == (0, 2, 32)
    assert svdq.rope_axes_table(pos[:0], axes).shape == (0, 16, 2)


def test_special_values_pass_through():
    """Zeros keep their place, NaN and infinities stay in their pair."""
    svdq = _svdq()
    q = torch.zeros(3, 2, 64, dtype=BF16, device="cuda")
    q[0, 0, 5], q[2, 1, 40] = float("nan"), float("inf")
    y, _ = svdq.rope_axes_apply(q, None, _pos(3, 1, 13), svdq.RopeAxes((16,)))
    bad = ~y.isfinite()
    assert bool(bad[0, 0, 4:6].all()) and bool(bad[2, 1, 40]) and int(bad.sum()) <= 3
    y = y.float().nan_to_num(0.0, 0.0, 0.0)
    assert not bool(y.any())


@pytest.mark.parametrize("dtype", R.FLOATS)
def test_shared_heads_of_an_input(dtype):
    """A head given for several by expansion (stride 0): each output is that head's."""
    svdq = _svdq()
    q = _normal(7, 1, 64, seed=14, dtype=dtype)
    pos, axes = _pos(7, 1, 15), svdq.RopeAxes((32,))
    want, _ = svdq.rope_axes_apply(q, None, pos, axes)
    got, k = svdq.rope_axes_apply(q.expand(7, 5, 64), q.expand(7, 3, 64), pos.expand(7, 1), axes)
    assert torch.equal(got, want.expand(7, 5, 64)) and torch.equal(k, want.expand(7, 3, 64))
