"""Host-side behaviour of the entry points around the projections, without a GPU: refusals come before any
device query (the fake addresses are never dereferenced), and a GPU the kernels were not built for gets
the architecture error."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
DEV = 0x7F0000000000
BF16, F16, F32, I32, I64 = range(5)


@pytest.fixture(scope="module")
def lib():
    import os

    from bit_rank_compensated_b200 import build, svdq

    if not os.path.exists(svdq.LIB_PATH):
        build.build()
    return svdq.load()


@pytest.fixture
def unsupported(lib):
    """No call gets past the architecture check, so nothing is ever launched on the fake addresses."""
    assert lib.svdq_test_override_capability(9, 0) == OK
    yield
    assert lib.svdq_test_override_capability(-1, 0) == OK


def _affine(**kw):
    from bit_rank_compensated_b200.svdq import NormAffineStruct

    d = dict(weight=DEV, bias=DEV, weight_stride=64, bias_stride=64, dtype=F32, groups=2, rows_per_group=50, weight_offset=0.0)
    return NormAffineStruct(**{**d, **kw})


def _norm(lib, **kw):
    d = dict(X=DEV, xs=64, dtype=BF16, M=100, K=64, af=_affine(), eps=1e-6, Y=DEV, ys=64, mean=DEV, rstd=DEV)
    d.update(kw)
    return lib.svdq_layer_norm(d["X"], d["xs"], d["dtype"], d["M"], d["K"], d["af"] and ctypes.addressof(d["af"]), d["eps"],
                               d["Y"], d["ys"], d["mean"], d["rstd"], None)


def _backward(lib, **kw):
    d = dict(dY=DEV, dys=64, X=DEV, xs=64, dtype=F16, M=100, K=64, af=_affine(), mean=DEV, rstd=DEV, dX=DEV, dxs=64, dw=DEV,
             db=DEV, ws=DEV, wsb=1 << 30)
    d.update(kw)
    return lib.svdq_layer_norm_backward(d["dY"], d["dys"], d["X"], d["xs"], d["dtype"], d["M"], d["K"],
                                        d["af"] and ctypes.addressof(d["af"]), d["mean"], d["rstd"], d["dX"], d["dxs"], d["dw"],
                                        d["db"], d["ws"], d["wsb"], None)


def _quantize(lib, **kw):
    d = dict(X=DEV, xs=64, dtype=BF16, M=100, K=64, col=DEV, xq=DEV, s=DEV)
    d.update(kw)
    return lib.svdq_i8_quantize_rows(d["X"], d["xs"], d["dtype"], d["M"], d["K"], d["col"], d["xq"], d["s"], None)


def _norm_quantize(lib, **kw):
    d = dict(X=DEV, xs=64, dtype=BF16, M=100, K=64, af=_affine(), eps=1e-6, xq=DEV, s=DEV)
    d.update(kw)
    return lib.svdq_i8_layer_norm_quantize(d["X"], d["xs"], d["dtype"], d["M"], d["K"], d["af"] and ctypes.addressof(d["af"]),
                                           d["eps"], d["xq"], d["s"], None)


def _gemm(lib, **kw):
    d = dict(xq=DEV, s=DEV, M=100, wq=DEV, ws=DEV, bias=DEV, N=64, K=64, Y=DEV, dtype=BF16, space=DEV, bytes=1 << 40)
    d.update(kw)
    return lib.svdq_i8_gemm(d["xq"], d["s"], d["M"], d["wq"], d["ws"], d["bias"], d["N"], d["K"], d["Y"], d["dtype"], d["space"],
                            d["bytes"], None)


def _linear(lib, **kw):
    d = dict(X=DEV, xs=64, dtype=BF16, M=100, col=None, wq=DEV, ws=DEV, bias=None, N=64, K=64, xq=DEV, s=DEV, Y=DEV, space=DEV,
             bytes=1 << 40)
    d.update(kw)
    return lib.svdq_i8_linear_forward(d["X"], d["xs"], d["dtype"], d["M"], d["col"], d["wq"], d["ws"], d["bias"], d["N"], d["K"],
                                      d["xq"], d["s"], d["Y"], d["space"], d["bytes"], None)


def _axes(**kw):
    from bit_rank_compensated_b200.svdq import RopeAxesStruct

    d = dict(n_axes=2, pairs=(8, 24, 0, 0), shared_ladder=0, halves=0, theta=1e4)
    return RopeAxesStruct(**{**d, **kw})


def _pos(**kw):
    from bit_rank_compensated_b200.svdq import PositionsStruct

    return PositionsStruct(**{**dict(data=DEV, dtype=I64, token_stride=2, axis_stride=1), **kw})


def _h(**kw):
    from bit_rank_compensated_b200.svdq import HeadsStruct

    return HeadsStruct(**{**dict(data=DEV, heads=4, token_stride=256, head_stride=64), **kw})


def _at(s):
    return None if s is None else ctypes.addressof(s)


def _table(lib, **kw):
    d = dict(pos=_pos(), M=100, axes=_axes(), table=DEV)
    d.update(kw)
    return lib.svdq_rope_axes_table(_at(d["pos"]), d["M"], _at(d["axes"]), d["table"], None)


def _apply(lib, **kw):
    d = dict(q=_h(), qo=_h(), k=_h(heads=2), ko=_h(heads=2), dtype=BF16, M=100, D=64, pos=_pos(), axes=_axes(), inverse=0)
    d.update(kw)
    return lib.svdq_rope_axes_apply(_at(d["q"]), _at(d["qo"]), _at(d["k"]), _at(d["ko"]), d["dtype"], d["M"], d["D"],
                                    _at(d["pos"]), _at(d["axes"]), d["inverse"], None)


CALLS = {f.__name__: f for f in (_norm, _backward, _quantize, _norm_quantize, _gemm, _linear, _table, _apply)}

INVALID_ARGS = [
    *[(c, dict(M=-1)) for c in CALLS],
    *[(c, dict(dtype=t)) for c in ("_norm", "_backward", "_quantize", "_norm_quantize", "_gemm", "_linear", "_apply") for t in (-1, I32, I64, 9)],
    *[(c, dict(K=0)) for c in ("_norm", "_backward", "_quantize", "_norm_quantize", "_gemm", "_linear")],
    *[(c, dict(X=None)) for c in ("_norm", "_backward", "_quantize", "_norm_quantize", "_linear")],
    *[(c, dict(xs=63)) for c in ("_norm", "_backward", "_quantize", "_norm_quantize", "_linear")],
    *[(c, dict(K=16400, xs=16400, ys=16400, dys=16400, dxs=16400)) for c in ("_norm", "_backward", "_norm_quantize")],
    *[(c, dict(K=131088, xs=131088)) for c in ("_quantize", "_gemm", "_linear")],
    *[(c, dict(K=56)) for c in ("_quantize", "_norm_quantize", "_gemm", "_linear")],
    *[(c, dict(N=n)) for c in ("_gemm", "_linear") for n in (0, -16, 24)],
    *[(c, {p: None}) for c, ps in (("_norm", ["Y"]), ("_backward", ["dY", "mean", "rstd", "ws"]), ("_quantize", ["xq", "s"]),
                                  ("_norm_quantize", ["xq", "s"]), ("_gemm", ["xq", "s", "wq", "ws", "Y"]),
                                  ("_linear", ["xq", "s", "wq", "ws", "Y"]), ("_table", ["pos", "axes", "table"]),
                                  ("_apply", ["q", "qo", "k", "ko", "pos", "axes"])) for p in ps],
    ("_norm", dict(ys=63)), ("_norm", dict(eps=-1e-6)), ("_norm", dict(eps=float("nan"))), ("_norm_quantize", dict(eps=float("inf"))),
    ("_backward", dict(dys=63)), ("_backward", dict(dxs=63)), ("_backward", dict(wsb=16)),
    *[(c, dict(af=a)) for c in ("_norm", "_backward", "_norm_quantize") for a in ("dtype=3", "groups=0", "groups=1", "rows_per_group=0",
                                                                                "rows_per_group=49", "weight_stride=63", "bias_stride=0")],
    *[(c, dict(axes=a)) for c in ("_table", "_apply") for a in ("n_axes=0", "n_axes=5", "pairs=(0,8,0,0)", "pairs=(200,200,0,0)",
                                                              "pairs=(2**30,2**30,0,0)", "theta=0.0", "theta=-1.0",
                                                              "theta=float('inf')", "theta=float('nan')", "shared_ladder=2", "halves=-1")],
    *[(c, dict(pos=a)) for c in ("_table", "_apply") for a in ("data=None", "dtype=0", "dtype=1", "dtype=7")],
    ("_apply", dict(D=63)), ("_apply", dict(D=62)), ("_apply", dict(D=0)), ("_apply", dict(D=1024)), ("_apply", dict(inverse=2)),
    *[("_apply", {p: a}) for p in ("q", "qo", "k", "ko") for a in ("heads=0", "heads=3", "data=None", "heads=10**6")],
    # outputs whose heads overlap
    *[("_apply", {p: a}) for p in ("qo", "ko") for a in ("token_stride=63", "head_stride=8", "token_stride=0", "head_stride=0",
                                                        "token_stride=64", "token_stride=100,head_stride=100")],
]


def _made(name, v):
    make = {"af": _affine, "axes": _axes, "pos": _pos, "q": _h, "qo": _h, "k": _h, "ko": _h}.get(name)
    if make is None or not isinstance(v, str):
        return v
    base = dict(heads=2) if name in ("k", "ko") else {}
    return make(**{**base, **eval(f"dict({v})")})  # noqa: S307


@pytest.mark.parametrize("call,kw", INVALID_ARGS, ids=lambda v: str(v))
def test_invalid_arguments(lib, unsupported, call, kw):
    assert CALLS[call](lib, **{k: _made(k, v) for k, v in kw.items()}) == INVALID


MISALIGNED_ARGS = [
    *[(c, {p: DEV + 1}) for c, ps in (("_norm", ["X", "Y", "mean", "rstd"]), ("_backward", ["dY", "X", "dX", "mean", "rstd", "dw", "db"]),
                                     ("_quantize", ["X", "col", "s"]), ("_norm_quantize", ["X", "s"]),
                                     ("_gemm", ["s", "ws", "bias"]), ("_linear", ["X", "col", "s", "ws", "bias"])) for p in ps],
    *[(c, {p: DEV + 8}) for c, ps in (("_backward", ["ws"]), ("_quantize", ["xq"]), ("_norm_quantize", ["xq"]),
                                     ("_gemm", ["xq", "wq", "Y", "space"]), ("_linear", ["xq", "wq", "Y", "space"])) for p in ps],
    *[(c, dict(af=a)) for c in ("_norm", "_backward", "_norm_quantize") for a in (f"weight={DEV + 2}", f"bias={DEV + 1},dtype=0")],
    ("_table", dict(table=DEV + 4)), ("_table", dict(pos=f"data={DEV + 4}")), ("_apply", dict(pos=f"data={DEV + 2},dtype=3")),
    *[("_apply", {p: f"data={DEV + 1}"}) for p in ("q", "qo", "k", "ko")],
]


@pytest.mark.parametrize("call,kw", MISALIGNED_ARGS, ids=lambda v: str(v))
def test_misaligned_pointers(lib, unsupported, call, kw):
    assert CALLS[call](lib, **{k: _made(k, v) for k, v in kw.items()}) == MISALIGNED


def test_valid_calls_reach_the_architecture_check(lib, unsupported):
    for f in CALLS.values():
        assert f(lib) == UNSUPPORTED, f.__name__
    optional = [("_norm", dict(af=None, mean=None, rstd=None)), ("_norm", dict(X=DEV + 2, Y=DEV + 6, xs=65)),
                ("_norm", dict(af=_affine(weight=None, bias=None, weight_stride=0))), ("_norm", dict(M=0, X=None, Y=None)),
                ("_backward", dict(dw=None, db=None, ws=None, wsb=0)), ("_backward", dict(dX=None)), ("_backward", dict(af=None)),
                ("_quantize", dict(col=None)), ("_quantize", dict(M=0, X=None, xq=None, s=None)), ("_gemm", dict(bias=None)),
                ("_linear", dict(col=DEV, bias=DEV)), ("_apply", dict(k=None, ko=None)),
                ("_apply", dict(q=_h(head_stride=0), k=_h(heads=2, token_stride=0, head_stride=0))),
                ("_apply", dict(qo=_h(token_stride=64, head_stride=6400), ko=_h(heads=2, token_stride=64, head_stride=6400))), ("_apply", dict(M=1, pos=_pos(token_stride=0))),
                ("_table", dict(axes=_axes(n_axes=4, pairs=(64, 64, 64, 64))))]
    for name, kw in optional:
        assert CALLS[name](lib, **kw) == UNSUPPORTED, (name, kw)


def test_workspace_sizes(lib):
    assert lib.svdq_i8_workspace_bytes(0, 64, 64) == 0 and lib.svdq_i8_workspace_bytes(8, 24, 64) == 0
    assert lib.svdq_layer_norm_workspace_bytes(0, 64, 1, 1) == 0 and lib.svdq_layer_norm_workspace_bytes(8, 1 << 20, 1, 8) == 0
    for M, N, K in ((1, 4096, 4096), (77, 272, 8192), (4608, 12288, 4096)):
        assert lib.svdq_i8_workspace_bytes(M, N, K) % 16 == 0


def test_calls_fail_loudly_without_the_compiled_binding(lib, monkeypatch):
    import sys

    import bit_rank_compensated_b200 as package
    import torch
    from bit_rank_compensated_b200 import svdq

    monkeypatch.setattr(svdq, "_binding", None)
    monkeypatch.delattr(package, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "bit_rank_compensated_b200._binding", None)
    with pytest.raises(RuntimeError, match="_binding.so"):
        svdq.layer_norm(torch.zeros(2, 2))


def test_host_tensors_are_refused(lib):
    import torch
    from bit_rank_compensated_b200 import svdq

    x, q = torch.zeros(4, 32), torch.zeros(4, 2, 16)
    i8, one = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    axes = svdq.RopeAxes((4, 4))
    for f in (lambda: svdq.layer_norm(x), lambda: svdq.layer_norm_backward(x, x, one, one), lambda: svdq.i8_quantize_rows(x),
              lambda: svdq.i8_layer_norm_quantize(x), lambda: svdq.i8_gemm(i8, one, i8, one), lambda: svdq.i8_linear_forward(x, i8, one),
              lambda: svdq.rope_axes_table(torch.zeros(4, 2), axes), lambda: svdq.rope_axes_apply(q, None, torch.zeros(4, 2), axes),
              lambda: svdq.layer_norm(None), lambda: svdq.RopeAxes((0,)), lambda: svdq.RopeAxes((300,))):
        with pytest.raises(ValueError):
            f()
