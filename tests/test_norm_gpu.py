"""Layer norm against a plain implementation in 64 bits.

Tolerances are worst cases of the arithmetic: u = 2^-24 for each fp32 operation, and the output type's half step."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24
SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 128), (17, 129), (33, 256), (70, 500), (64, 512), (20, 1000), (21, 1024), (9, 1537), (16, 2048),
          (7, 4095), (9, 4096), (5, 8192), (3, 8191), (4, 16384), (2, 16385), (3, 40000), (3000, 128), (1300, 600), (2500, 4)]


def close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, by up to {float(((got - want).abs() - tol).max())}"


def depth(n):
    """Additions that a value of a row's sum passes: a thread's own (32, or every 1024th column), then two trees of 5."""
    return (32 if n <= 16384 else n // 1024 + 1) + 12


def inputs(rows, cols, dtype, param, x_stride=0, dy_stride=0, seed=0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=(rand(rows, x_stride or cols) * 1.5 + shift).to(DT[dtype])[:, :cols], w=(1 + 0.2 * rand(cols)).to(DT[param]),
                b=rand(cols).to(DT[param]), dy=rand(rows, dy_stride or cols).to(DT[dtype])[:, :cols])


def reference(t, eps):
    """y, mean, rstd in 64 bits, and how far fp32 arithmetic may be off: of mean, rstd (relative) and h."""
    x, n = t["x"].double(), t["x"].shape[1]
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    mean_tol = (depth(n) + 2) * F32 * x.abs().mean(1, keepdim=True)
    var_tol = 2 * d.abs().mean(1, keepdim=True) * mean_tol + mean_tol ** 2 + (depth(n) + 6) * F32 * var
    rel = 0.5 * var_tol / (var + eps) + 6 * F32
    h = d * rstd
    return mean, rstd, h, mean_tol, rel, rstd * mean_tol + h.abs() * (rel + 3 * F32)


def check_fwd(t, p, weight=True, bias=True, **kw):
    eps = p.c.eps
    stats = torch.full((2, p.c.rows), float("nan"), device="cuda")
    w, b = t["w"] if weight else None, t["b"] if bias else None
    mean, rstd, h, mean_tol, rel, h_tol = reference(t, eps)
    y = B.csa_layernorm_fwd(p, t["x"], w, b, stats=stats, **kw)
    ww = w.double() if weight else torch.ones(p.c.cols, dtype=torch.float64, device="cuda")
    bb = b.double() if bias else torch.zeros(p.c.cols, dtype=torch.float64, device="cuda")
    want = h * ww + bb
    tol = h_tol * ww.abs() + 3 * F32 * ((h * ww).abs() + bb.abs())
    close(y, want, tol + U[y.dtype] * (want.abs() + tol), "y")
    close(stats[0], mean[:, 0], mean_tol[:, 0], "mean")
    close(stats[1], rstd[:, 0], rstd[:, 0] * rel[:, 0], "rstd")
    return y, stats


def check_bwd(t, p, stats, weight=True, need=(True, True, True), **kw):
    """Of the statistics that it is given."""
    w = t["w"] if weight else None
    dx, dw, db = B.csa_layernorm_bwd(p, t["dy"], t["x"], w, stats, *need, **kw)
    n, rows = p.c.cols, p.c.rows
    mean, rstd = stats[0].double()[:, None], stats[1].double()[:, None]
    h, dy = (t["x"].double() - mean) * rstd, t["dy"].double()
    a = dy * (w.double() if weight else 1.0)
    ma, mh = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    ma_tol, mh_tol = (depth(n) + 4) * F32 * a.abs().mean(1, keepdim=True), (depth(n) + 8) * F32 * (a * h).abs().mean(1, keepdim=True)
    if need[0]:
        want = rstd * (a - ma - h * mh)
        tol = rstd * (ma_tol + h.abs() * mh_tol + 8 * F32 * (a.abs() + ma.abs() + (h * mh).abs()))
        close(dx, want, tol + U[dx.dtype] * (want.abs() + tol) + 1e-38, "dx")
    # rows of a block, then the blocks': each thread adds at most a 64th of the rows, and the joins 80
    adds = rows // 64 + 84
    pt = U[DT["f32" if p.c.param_dtype == 0 else "bf16"]]
    if need[1]:
        want, tol = (dy * h).sum(0), adds * F32 * (dy * h).abs().sum(0)
        close(dw, want, tol + pt * (want.abs() + tol) + 1e-38, "dweight")
    if need[2]:
        want, tol = dy.sum(0), adds * F32 * dy.abs().sum(0)
        close(db, want, tol + pt * (want.abs() + tol) + 1e-38, "dbias")
    for out, wanted in zip((dx, dw, db), need):
        assert (out is not None) == wanted
    return dx, dw, db


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,param", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_norm(rows, cols, dtype, param):
    t = inputs(rows, cols, dtype, param, seed=rows + cols)
    p = B.LayerNormParams(rows, cols, dtype, param, eps=1e-5)
    _, stats = check_fwd(t, p)
    check_bwd(t, p, stats)


@pytest.mark.parametrize("rows,cols", [(40, 128), (11, 1000), (6, 4096), (3, 17000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("more", [8, 4, 1])
def test_strides(rows, cols, dtype, more):
    t = inputs(rows, cols, dtype, "f32", cols + more, cols + 3 * more)
    p = B.LayerNormParams(rows, cols, dtype, x_stride=cols + more, dy_stride=cols + 3 * more)
    _, stats = check_fwd(t, p)
    check_bwd(t, p, stats)


@pytest.mark.parametrize("need", [(True, False, False), (False, True, True), (False, False, True), (True, True, False), (False, False, False)])
@pytest.mark.parametrize("cols", [128, 777, 4096, 20000])
def test_outputs_and_parameters_left_out(need, cols):
    t = inputs(50, cols, "bf16", "f32")
    p = B.LayerNormParams(50, cols)
    _, stats = check_fwd(t, p, weight=False)
    check_fwd(t, p, bias=False)
    check_bwd(t, p, stats, weight=False, need=need)


@pytest.mark.parametrize("cols", [128, 130, 4096, 16384, 16400])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(cols, dtype):
    t = inputs(37, cols, dtype, "f32", seed=3)
    p = B.LayerNormParams(37, cols, dtype)
    y, stats = check_fwd(t, p)
    x = t["x"].clone()
    version = x._version
    assert B.csa_layernorm_fwd(p, x, t["w"], t["b"], out=x) is x and torch.equal(x, y) and x._version > version
    want = check_bwd(t, p, stats)
    for name in ("dy", "x"):
        args = {k: t[k].clone() for k in ("dy", "x")}
        got = B.csa_layernorm_bwd(p, args["dy"], args["x"], t["w"], stats, out=(args[name], None, None))
        assert got[0] is args[name] and all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_of_one_value_and_far_from_zero():
    t = inputs(64, 512, "f32", "f32", shift=1000.0)  # the variance is a thousandth of a millionth of the mean's square
    p = B.LayerNormParams(64, 512, "f32", eps=0.0)
    _, stats = check_fwd(t, p)
    check_bwd(t, p, stats)
    x = torch.full((3, 100), 2.5, device="cuda", dtype=torch.bfloat16)
    bias = torch.arange(100, device="cuda", dtype=torch.float32)
    y = B.csa_layernorm_fwd(B.LayerNormParams(3, 100), x, None, bias)
    assert torch.equal(y, bias.bfloat16().expand(3, 100))  # no variance: the bias alone


def test_infinities_stay_in_their_row():
    t = inputs(6, 300, "bf16", "f32")
    p = B.LayerNormParams(6, 300)
    y, _ = check_fwd(t, p)
    t["x"][2, 7], t["x"][4, 0] = float("inf"), float("nan")
    got = B.csa_layernorm_fwd(p, t["x"], t["w"], t["b"])
    assert bool(got[[2, 4]].isnan().any(1).all()) and torch.equal(got[[0, 1, 3, 5]], y[[0, 1, 3, 5]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1023), (1, 2047), (2, 1017), (3, 2041)])
def test_few_rows_after_many(rows, cols, dtype):
    """What other rows left in shared memory is in no sum: parts of a block that have no row of their own add zeros."""
    many = inputs(2000, cols, dtype, "f32")
    many["x"] *= 1e15
    many["dy"] *= 1e15
    t, p, q = inputs(rows, cols, dtype, "f32", seed=1), B.LayerNormParams(rows, cols, dtype), B.LayerNormParams(2000, cols, dtype)
    ones = torch.ones(2, 2000, device="cuda")
    for _ in range(10):
        B.csa_layernorm_bwd(q, many["dy"], many["x"], many["w"], ones)
        _, stats = check_fwd(t, p)
        check_bwd(t, p, stats)


def test_no_rows():
    p = B.LayerNormParams(0, 24)
    x = torch.empty(0, 24, device="cuda", dtype=torch.bfloat16)
    stats = torch.empty(2, 0, device="cuda")
    assert B.csa_layernorm_fwd(p, x, stats=stats).shape == (0, 24)
    dx, dw, db = B.csa_layernorm_bwd(p, x, x, None, stats)
    assert dx.shape == (0, 24) and not bool(dw.any()) and not bool(db.any())


def test_same_bits_on_another_stream_and_captured():
    t = inputs(5000, 384, "bf16", "bf16")
    p = B.LayerNormParams(5000, 384, param_dtype="bf16")
    y, stats = check_fwd(t, p)
    want = check_bwd(t, p, stats)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(B.csa_layernorm_fwd(p, t["x"], t["w"], t["b"]), y)
        ws = torch.empty(p.bwd_workspace_bytes, dtype=torch.uint8, device="cuda")
        out = [torch.empty_like(o) for o in want]
        B.csa_layernorm_bwd(p, t["dy"], t["x"], t["w"], stats, workspace=ws, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            B.csa_layernorm_bwd(p, t["dy"], t["x"], t["w"], stats, workspace=ws, out=out)
        for o in out:
            o.fill_(7)
        graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    t2 = inputs(5000, 384, "bf16", "bf16", seed=9)
    t["dy"].copy_(t2["dy"])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, check_bwd(t, p, stats)))


@pytest.mark.parametrize("dtype,cols", [("f32", 40), ("f32", 513)])
def test_autograd_and_differences(dtype, cols):
    rows = 12
    t = inputs(rows, cols, dtype, "f32", seed=5)
    p = B.LayerNormParams(rows, cols, dtype, eps=1e-3)
    leaves = [t["x"].view(3, 4, cols).clone().requires_grad_(True), t["w"].clone().requires_grad_(True), t["b"].clone().requires_grad_(True)]
    y = B.csa_layernorm(*leaves, params=p)
    assert y.shape == (3, 4, cols)
    y.backward(t["dy"].view_as(y))

    def loss(x, w, b):
        d = x - x.mean(-1, keepdim=True)
        return ((d * ((d * d).mean(-1, keepdim=True) + 1e-3) ** -0.5 * w + b) * t["dy"].double().view(3, 4, cols)).sum()

    at = [v.detach().double() for v in leaves]
    g = torch.Generator(device="cuda").manual_seed(1)
    for i, leaf in enumerate(leaves):
        way = torch.randn(leaf.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        up, down = (loss(*[v + s * e * way if j == i else v for j, v in enumerate(at)]) for s in (1, -1))
        slope = float((leaf.grad.double() * way).sum())
        # differences: third derivatives times e^2 and 64-bit rounding; the gradient: some 100 fp32 roundings of terms
        assert abs(slope - float((up - down) / (2 * e))) <= 100 * F32 * float((leaf.grad.double() * way).abs().sum()) + 1e-7


def test_refusals():
    t = inputs(8, 64, "bf16", "f32")
    p = B.LayerNormParams(8, 64)
    stats = torch.empty(2, 8, device="cuda")
    with pytest.raises(ValueError):
        B.csa_layernorm_fwd(p, t["x"].float(), t["w"])
    with pytest.raises(ValueError):
        B.csa_layernorm_fwd(p, t["x"], t["w"].bfloat16())
    with pytest.raises(ValueError):
        B.csa_layernorm_fwd(p, t["x"].t().contiguous().t(), t["w"])
    with pytest.raises(ValueError):
        B.csa_layernorm_fwd(p, t["x"], t["w"], stats=stats[:, :7])
    with pytest.raises(ValueError):
        B.csa_layernorm_fwd(p, t["x"].cpu(), t["w"])
    with pytest.raises(ValueError):
        B.csa_layernorm_bwd(p, t["dy"], t["x"], t["w"], None)
    with pytest.raises(B.CSAError):
        B.csa_layernorm_bwd(p, t["dy"], t["x"], t["w"], stats, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        B.LayerNormParams(8, 64, dtype="f16")
