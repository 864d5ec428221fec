"""The operators around the projections together, as a block calls them: norm -> int8 rows -> int8 QKV ->
rotation, the table -> fused 4-bit QKV, captured graphs, streams, and what the binding refuses."""
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


class Block:
    """Two samples' tokens through a modulated norm, an int8 QKV projection and the rotation of Q and K."""

    def __init__(self, svdq, M, dtype, seed=0, heads=2):
        self.svdq, self.heads, self.K = svdq, heads, 256 * heads
        K, N = self.K, 3 * heads * 128
        self.X = _normal(M, K, seed=seed, dtype=dtype)
        mod = _normal(2, 2 * K, seed=seed + 1, dtype=BF16, scale=0.2)
        self.shift, self.scale = mod[:, :K], mod[:, K:]
        self.wq, self.ws = svdq.i8_quantize_rows(_normal(N, K, seed=seed + 2, scale=0.02))
        self.b = _normal(N, seed=seed + 3, scale=0.1)
        self.pos = torch.stack([torch.arange(M, device="cuda"), torch.arange(M, device="cuda") % 7], 1)
        self.axes = svdq.RopeAxes((24, 40))

    def __call__(self):
        s = self.svdq
        xq, xs = s.i8_layer_norm_quantize(self.X, self.scale, self.shift, weight_offset=1.0)
        Y = s.i8_gemm(xq, xs, self.wq, self.ws, self.b, dtype=self.X.dtype)
        D = self.heads * 128
        q, k = Y[:, :D].unflatten(1, (self.heads, 128)), Y[:, D:2 * D].unflatten(1, (self.heads, 128))
        s.rope_axes_apply(q, k, self.pos, self.axes, q_out=q, k_out=k)
        return Y

    def reference(self):
        M, D = self.X.shape[0], self.heads * 128
        y, *_ = R.layer_norm(self.X, self.scale, self.shift, -(-M // 2), 1.0)
        q, s = R.quantize_rows(y)
        Y, _ = R.i8_product(q, s, self.wq, self.ws, self.b)
        cos, sin, angle = R.cos_sin(self.pos, (24, 40), 10000.0, False)
        for i in range(2):
            v = Y[:, i * D:(i + 1) * D].unflatten(1, (self.heads, 128))
            v.copy_(R.rope(v, cos, sin, angle, False, False)[0])
        return Y


@pytest.mark.parametrize("M", [1, 2, 9, 130, 700])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_norm_linear_rotation(M, dtype):
    """The chain rounds to 16 bits twice (projection, rotation: two values each) and a code that lies at a border
    may fall to either side: within 4 half steps of the row's norm in the mean square."""
    block = Block(_svdq(), M, dtype)
    Y, ref = block(), block.reference()
    assert float((Y.double() - ref).norm() / ref.norm()) < 4 * R.half_step(dtype)
    assert block.svdq.last_device_error() == 0


def test_table_feeds_the_fused_projection():
    """The 4-bit QKV projection under a table made from position ids, against the same under the generator's table;
    and the unfused step on an int8 projection's output against the rotation after a plain RMS norm."""
    svdq = _svdq()
    from synth import rope_table

    heads, M, K = 2, 300, 256
    N = 3 * heads * 128
    X = _normal(M, K, seed=1, dtype=BF16)
    layer = svdq.prepare_weights(_normal(N, K, seed=2, scale=0.05), None, svdq.act_absmax(X), 16)
    bufs = svdq.quant_act_lora_down(X, layer)
    m = torch.arange(M, device="cuda")
    j = (m - 33).clamp_min(0)
    pos = torch.stack([0 * m, torch.where(m < 33, 0, j // 64), torch.where(m < 33, 0, j % 64)], 1)
    axes = svdq.RopeAxes((8, 28, 28))
    table = svdq.rope_axes_table(pos, axes)
    nq, nk = _normal(128, seed=3) + 1, _normal(128, seed=4) + 1
    Y = svdq.gemm_w4a4_lora_up_qk_norm_rope(*bufs, M, layer, heads, nq, nk, table)
    Z = svdq.gemm_w4a4_lora_up_qk_norm_rope(*bufs, M, layer, heads, nq, nk, torch.from_numpy(rope_table(M, n_text=33)).cuda())
    # tables within a few 2^-23 of each other: outputs within one step of bf16
    assert float((Y.double() - Z.double()).abs().max()) <= 2 * R.half_step(BF16) * float(Z.double().abs().max())
    assert float((Y != Z).double().mean()) < 1e-3

    wq, ws = svdq.i8_quantize_rows(_normal(N, K, seed=5, scale=0.05))
    P = svdq.i8_linear_forward(X, wq, ws)
    D = heads * 128
    want = P.double()
    cos, sin, angle = R.cos_sin(pos, (8, 28, 28), 10000.0, False)
    for i, w in enumerate((nq, nk)):
        v = want[:, i * D:(i + 1) * D].unflatten(1, (heads, 128))
        u = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.double()
        v.copy_(R.rope(u, cos, sin, angle, False, False)[0])
    svdq.qk_norm_rope(P, heads, nq, nk, table)
    assert float((P.double() - want).norm() / want.norm()) < 2 * R.half_step(BF16)
    assert svdq.last_device_error() == 0


def _training_step(svdq, s):
    """Norm, its gradient and the rotation's, as the tuning of a block's norms over a frozen layer runs them."""
    Y, mean, rstd = svdq.layer_norm(s["X"], s["w"], s["b"], stats=True)
    q = Y.unflatten(1, (4, 128))
    q, _ = svdq.rope_axes_apply(q, None, s["pos"], s["axes"])
    dq, _ = svdq.rope_axes_apply(q, None, s["pos"], s["axes"], inverse=True)
    return (q, *svdq.layer_norm_backward(dq.flatten(1), s["X"], mean, rstd, s["w"]))


def _training_inputs(svdq, M, seed):
    return {"X": _normal(M, 512, seed=seed, dtype=BF16), "w": _normal(3, 512, seed=seed + 1), "b": _normal(3, 512, seed=seed + 2),
            "pos": torch.arange(M, device="cuda")[:, None] + seed, "axes": svdq.RopeAxes((64,))}


def test_two_captured_graphs_replay_in_turn():
    """Two graphs with workspaces of their own, replayed on new inputs, in turn and on two streams at once: the
    eager calls' bits."""
    svdq = _svdq()
    kinds = []
    for M, seed in ((150, 0), (90, 40)):
        s = _training_inputs(svdq, M, seed)
        block = Block(svdq, M, BF16, seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _training_step(svdq, s), block()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [*_training_step(svdq, s), block()]
        kinds.append((s, block, g, out))
    streams = [torch.cuda.Stream() for _ in kinds]
    for round_ in range(3):
        for i, (s, block, _, _) in enumerate(kinds):
            s["X"].copy_(_normal(*s["X"].shape, seed=200 + 10 * round_ + i, dtype=BF16))
            block.X.copy_(_normal(*block.X.shape, seed=300 + 10 * round_ + i, dtype=BF16))
        torch.cuda.synchronize()
        for (_, _, g, _), st in zip(kinds, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, block, _, out in kinds:
            for x, y in zip(out, [*_training_step(svdq, s), block()]):
                assert torch.equal(x, y)
    assert svdq.last_device_error() == 0


def test_other_stream():
    """stream= runs the call, and what it allocates, on that stream."""
    svdq = _svdq()
    X = _normal(400, 1024, seed=5, dtype=BF16)
    wq, ws = svdq.i8_quantize_rows(_normal(512, 1024, seed=6))
    pos, axes = torch.arange(400, device="cuda")[:, None], svdq.RopeAxes((64,))
    dY = _normal(400, 1024, seed=7, dtype=BF16)
    Y, mean, rstd = svdq.layer_norm(X, stats=True)

    def all_of(**kw):
        q, k = svdq.rope_axes_apply(X.unflatten(1, (8, 128)), None, pos, axes, **kw)
        return [svdq.layer_norm(X, **kw), *svdq.layer_norm_backward(dY, X, mean, rstd, **kw), *svdq.i8_quantize_rows(X, **kw),
                *svdq.i8_layer_norm_quantize(X, **kw), svdq.i8_linear_forward(X, wq, ws, **kw),
                svdq.i8_gemm(*svdq.i8_quantize_rows(X, **kw), wq, ws, **kw), q, svdq.rope_axes_table(pos, axes, **kw)]

    want = all_of()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = all_of(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_more_than_32_bit_offsets():
    """Rows whose offsets in elements pass 2^31 (a strided view of a large buffer, touched at its ends)."""
    svdq = _svdq()
    M, K, stride = 3, 512, 2 ** 30 + 8
    buf = torch.empty(2 * stride + K, dtype=BF16, device="cuda")
    X = buf.as_strided((M, K), (stride, 1))
    X.copy_(_normal(M, K, seed=9, dtype=BF16))
    dense = X.contiguous()
    for f in (svdq.layer_norm, lambda t: svdq.i8_quantize_rows(t)[0], lambda t: svdq.i8_layer_norm_quantize(t)[0]):
        assert torch.equal(f(X), f(dense))
    pos, axes = torch.arange(M, device="cuda")[:, None], svdq.RopeAxes((32,))
    heads = lambda t: t.as_strided((M, 8, 64), (t.stride(0), 64, 1))  # noqa: E731
    assert torch.equal(svdq.rope_axes_apply(heads(X), None, pos, axes)[0], svdq.rope_axes_apply(heads(dense), None, pos, axes)[0])
    _, mean, rstd = svdq.layer_norm(dense, stats=True)
    for x, y in zip(svdq.layer_norm_backward(X, X, mean, rstd), svdq.layer_norm_backward(dense, dense, mean, rstd)):
        assert torch.equal(x, y)


def test_the_binding_refuses():
    """Shapes, types, strides and devices that do not fit are refused before anything is launched."""
    svdq = _svdq()
    X, cpu = _normal(4, 64, seed=1, dtype=BF16), torch.zeros(4, 64)
    q, pos, axes = X.unflatten(1, (2, 32)), torch.zeros(4, 1, dtype=torch.int64, device="cuda"), svdq.RopeAxes((16,))
    wq, ws = svdq.i8_quantize_rows(_normal(32, 64, seed=2))
    xq, xs = svdq.i8_quantize_rows(X)
    st = torch.zeros(4, device="cuda")
    w = torch.zeros(2, 64, device="cuda")
    bad = [
        lambda: svdq.layer_norm(cpu), lambda: svdq.layer_norm(X.t()), lambda: svdq.layer_norm(X.double()),
        lambda: svdq.layer_norm(X[None]), lambda: svdq.layer_norm(X[:1].expand(4, 64)),
        lambda: svdq.layer_norm(X, w[:, :32]), lambda: svdq.layer_norm(X, w.cpu()), lambda: svdq.layer_norm(X, w, w[:1]),
        lambda: svdq.layer_norm(X, w, w.half()), lambda: svdq.layer_norm(X, w, rows_per_group=1),
        lambda: svdq.layer_norm(X, Y=X.float()), lambda: svdq.layer_norm(X, Y=X[:2]),
        lambda: svdq.layer_norm_backward(X.float(), X, st, st), lambda: svdq.layer_norm_backward(X, X, st[:3], st),
        lambda: svdq.layer_norm_backward(X, X, st, st.double()), lambda: svdq.layer_norm_backward(X, X, st, st, w, groups=3),
        lambda: svdq.layer_norm_backward(X, X, st, st, groups=2, rows_per_group=1),
        lambda: svdq.i8_quantize_rows(X, st), lambda: svdq.i8_quantize_rows(X, xq=xq[:2]),
        lambda: svdq.i8_gemm(xq.float(), xs, wq, ws), lambda: svdq.i8_gemm(xq, xs[:2], wq, ws),
        lambda: svdq.i8_gemm(xq, xs, wq[:, :32], ws), lambda: svdq.i8_gemm(xq, xs, wq, ws[:16]),
        lambda: svdq.i8_gemm(xq, xs, wq, ws, dtype=torch.int32), lambda: svdq.i8_gemm(xq, xs, wq, ws, bias=ws.half()),
        lambda: svdq.i8_gemm(xq, xs, wq, ws, Y=torch.empty(4, 32, device="cuda")), lambda: svdq.i8_gemm(xq, xs, wq.cpu(), ws),
        lambda: svdq.i8_linear_forward(X, wq, ws, col_scale=st), lambda: svdq.RopeAxes(()), lambda: svdq.RopeAxes((1,) * 5),
        lambda: svdq.RopeAxes((0, 4)), lambda: svdq.rope_axes_table(pos.short(), axes),
        lambda: svdq.rope_axes_table(pos.expand(4, 2), axes), lambda: svdq.rope_axes_apply(q, None, pos[:2], axes),
        lambda: svdq.rope_axes_apply(q, q.half(), pos, axes), lambda: svdq.rope_axes_apply(q, q[:2], pos, axes),
        lambda: svdq.rope_axes_apply(q.transpose(1, 2), None, pos, axes), lambda: svdq.rope_axes_apply(X, None, pos, axes),
        lambda: svdq.rope_axes_apply(q, None, pos, axes, q_out=q[:, :1]), lambda: svdq.rope_axes_apply(q, None, pos.cpu(), axes),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    # what the library itself refuses comes as its error
    for f in (lambda: svdq.layer_norm(X, eps=-1.0), lambda: svdq.rope_axes_apply(q, None, pos, svdq.RopeAxes((17,))),
              lambda: svdq.i8_gemm(xq[:, :8].contiguous(), xs, wq[:, :8].contiguous(), ws),
              lambda: svdq.i8_quantize_rows(X[:, :40]), lambda: svdq.rope_axes_table(pos, svdq.RopeAxes((4,), theta=0.0))):
        with pytest.raises(svdq.SvdqError) as e:
            f()
        assert e.value.status == 1
