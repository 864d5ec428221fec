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
