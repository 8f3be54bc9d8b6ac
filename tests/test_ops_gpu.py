"""The operators around the step (projections, rotary positions, AdamW) against plain implementations in 64 bits.

Tolerances are worst cases of the arithmetic: u(t) = finfo(t).eps / 2 is the largest relative error of rounding to t.
"""
import itertools
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def close(got, want, tol, what):
    """|got - want| <= tol elementwise (tol a tensor or a number), the largest excess named."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = int(((got - want).abs() - tol).nan_to_num(nan=float("inf")).flatten().argmax())
        t = tol.flatten()[i] if torch.is_tensor(tol) else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i}: {got.flatten()[i]} for "
                             f"{want.flatten()[i]}, allowed {t}")


# ------------------------------------------------------------------ projections

def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad64(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    k, c = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (z + c * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * c * z * z)


def product_tol(terms, count):
    """Worst case of an fp32 sum of `count` products whose magnitudes sum to `terms`: 2^-23 of them for each addition
    (tensor cores may truncate where they align), and the three-part products of fp32 values (2^-23)."""
    return (count + 8) * 2.0 ** -23 * terms


def linear_inputs(M, K, N, dtype, out, seed, x_stride=0, res_stride=0, dy_stride=0):
    g = gen(seed)

    def rows(m, n, stride, dt, scale=1.0):
        return randn(g, m, stride or n, dtype=dt, scale=scale)[:, :n]

    return dict(x=rows(M, K, x_stride, DT[dtype]), w=randn(g, N, K, dtype=DT[dtype], scale=K ** -0.5),
                bias=randn(g, N), res=rows(M, N, res_stride, DT[out]), dy=rows(M, N, dy_stride, DT[out]),
                z=randn(g, M, N, dtype=DT[dtype]))


def check_linear(M, K, N, dtype="bf16", out=None, act="none", bias=True, residual=False, alpha=1.0, preact=None,
                 x_stride=0, res_stride=0, dy_stride=0, seed=0, backward=True):
    out = out or dtype
    t = linear_inputs(M, K, N, dtype, out, seed, x_stride, res_stride, dy_stride)
    p = B.LinearParams(M, K, N, dtype, out, act, alpha, x_stride, res_stride, dy_stride)
    b = t["bias"] if bias else None
    r = t["res"] if residual else None
    z_out = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda") if preact else None
    y = B.csa_linear_fwd(p, t["x"], t["w"], b, r, preact=z_out)
    x, w = t["x"].double(), t["w"].double()
    z = alpha * (x @ w.t()) + (b.double() if bias else 0.0)
    z_tol = product_tol(abs(alpha) * (x.abs() @ w.abs().t()), K) + 4 * F32 * (z.abs() + (b.double().abs() if bias else 0))
    if preact:
        close(z_out, z, z_tol + U[DT[dtype]] * (z.abs() + z_tol), "preact")
    a = act64(z, act)
    # |act'| <= 1.13 carries z's error; the function itself is good to 2^-20 relative (exp of arguments up to |3 z|
    # to 2^-22, quotients), and to 2^-100 where exp overflows
    a_tol = 1.13 * z_tol + (2.0 ** -20) * (1 + z.abs()) * a.abs() + 1e-30 if act != "none" else z_tol
    want = a + r.double() if residual else a
    tol = a_tol + 2 * F32 * want.abs()
    close(y, want, tol + U[DT[out]] * (want.abs() + tol), "y")
    if not backward:
        return
    dx, dw, db = B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], t["z"] if act != "none" else None)
    z = t["z"].double()
    d = t["dy"].double() * (act_grad64(z, act) if act != "none" else 1.0)
    # act' is good to 2^-19 (1 + |z|) absolute: it is a sum of up to three terms of that relative error
    d_tol = (2.0 ** -19 * (1 + z.abs()) ** 2 * t["dy"].double().abs()) if act not in ("none", "relu") else torch.zeros_like(d)
    close(db, d.sum(0), d_tol.sum(0) + (M + 8) * F32 * d.abs().sum(0), "db")
    # dz is rounded to the values' type before the products where it is not a copy of dy
    e = d_tol + (U[DT[dtype]] * (d.abs() + d_tol) if act != "none" or out != dtype else 0.0)
    want, s = alpha * (d @ w), abs(alpha) * (d.abs() @ w.abs())
    tol = abs(alpha) * (e @ w.abs()) + product_tol(s, N)
    close(dx, want, tol + U[DT[dtype]] * (want.abs() + tol) + 1e-37, "dx")
    want, s = alpha * (d.t() @ x), abs(alpha) * (d.abs().t() @ x.abs())
    tol = abs(alpha) * (e.t() @ x.abs()) + product_tol(s, M)
    close(dw, want, tol + U[DT[dtype]] * (want.abs() + tol) + 1e-37, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 2048, 136), (2, 40, 8), (3, 7, 5), (5, 257, 129), (8, 64, 64), (9, 72, 264),
                                   (16, 512, 1000), (17, 1023, 33), (31, 96, 777), (64, 128, 256), (100, 200, 300),
                                   (127, 65, 255), (128, 64, 256), (129, 64, 257), (300, 1024, 640), (513, 1000, 520)])
def test_linear_sizes(M, K, N, dtype):
    check_linear(M, K, N, dtype, seed=M + K + N)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("M,K,N", [(4, 264, 200), (150, 264, 200), (150, 133, 77)])
def test_linear_epilogue(M, K, N, act, dtype, out):
    for i, (bias, residual, preact) in enumerate(itertools.product([False, True], repeat=3)):
        check_linear(M, K, N, dtype, out, act, bias, residual, alpha=0.375, preact=preact, seed=i, backward=bias and residual)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("K", [200, 600])
def test_linear_epilogue_of_large_tiles(K, dtype, out):
    """Tiles of 256 x 256 with 16 and with 8 epilogue warps, the last ones partly filled, rows on 16 bytes only."""
    check_linear(4200, K, 4104, dtype, out, act="silu", residual=True, alpha=0.5, preact=True, seed=6)


@pytest.mark.parametrize("xs,rs,ds", [(80, 0, 0), (0, 112, 120), (72, 104, 136), (67, 99, 101), (65, 0, 97)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 70])
def test_linear_strides(M, xs, rs, ds, dtype):
    check_linear(M, 64, 96, dtype, act="silu", residual=True, preact=True, x_stride=xs, res_stride=rs, dy_stride=ds)


@pytest.mark.parametrize("M,K,N", [(4096, 64, 64), (20000, 256, 64), (16384, 512, 136), (64, 8192, 512), (40, 4096, 8192),
                                   (2048, 2048, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_long_axes(M, K, N, dtype):
    """Long sums (split over CTAs where the tiles are few) and many tiles."""
    check_linear(M, K, N, dtype, act="gelu_tanh", residual=True, seed=1)


def test_linear_without_rows():
    p = B.LinearParams(0, 32, 16)
    w = torch.randn(16, 32, device="cuda").bfloat16()
    x, dy = w.new_empty(0, 32), w.new_empty(0, 16)
    assert B.csa_linear_fwd(p, x, w).shape == (0, 16)
    dx, dw, db = B.csa_linear_bwd(p, dy, x, w)
    assert dx.shape == (0, 32) and not dw.any() and not db.any()


def test_linear_residual_in_place():
    for M in (3, 200):
        t = linear_inputs(M, 72, 48, "bf16", "bf16", 3)
        p = B.LinearParams(M, 72, 48, activation="relu")
        want = B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], t["res"])
        got = t["res"].clone()
        assert B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], got, out=got) is got
        assert torch.equal(got, want)


@pytest.mark.parametrize("M,K,N", [(12, 200, 77), (300, 64, 1003), (3000, 128, 2053), (2600, 600, 2056), (40, 8192, 49)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_residual_in_place_of_odd_rows(M, K, N, dtype):
    """Rows off the 16-byte boundaries, whose vectors hold other rows' ends; tiles of every kind and a cut k axis."""
    t = linear_inputs(M, K, N, dtype, dtype, 8)
    p = B.LinearParams(M, K, N, dtype, activation="gelu_tanh")
    want = B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], t["res"])
    for _ in range(3):
        got = t["res"].clone()
        B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], got, out=got)
        assert torch.equal(got, want)


def test_linear_writes_its_rows_only():
    """Outputs inside larger buffers: nothing before or behind them is written."""
    for M, K, N in ((5, 40, 56), (130, 136, 200), (131, 77, 33)):
        for dtype in ("bf16", "f32"):
            t = linear_inputs(M, K, N, dtype, dtype, 4)
            p = B.LinearParams(M, K, N, dtype, activation="silu")
            outs = []
            for n, dt in ((M * N, DT[dtype]), (M * N, DT[dtype]), (M * K, DT[dtype]), (N * K, DT[dtype]), (N, torch.float32)):
                buf = torch.full((n + 256,), 7.0, dtype=dt, device="cuda")
                outs.append((buf, buf[128:128 + n], n))
            y, z, dx, dw, db = (o[1] for o in outs)
            B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], out=y, preact=z)
            B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], z, out=(dx, dw, db))
            for buf, _, n in outs:
                assert bool((buf[:128] == 7).all()) and bool((buf[128 + n:] == 7).all())


def test_linear_nan_and_infinity_stay_in_their_rows():
    for M in (4, 200):
        for dtype in ("bf16", "f32"):
            t = linear_inputs(M, 96, 80, dtype, dtype, 5)
            p = B.LinearParams(M, 96, 80, dtype)
            clean = B.csa_linear_fwd(p, t["x"], t["w"])
            t["x"][1, 5], t["x"][2, 95] = float("nan"), float("inf")
            y = B.csa_linear_fwd(p, t["x"], t["w"])
            assert bool(y[1].isnan().all()) and not bool(y[2].isfinite().any())
            keep = [i for i in range(M) if i not in (1, 2)]
            assert torch.equal(y[keep], clean[keep])


def test_linear_largest_fp32_values():
    """Finite values that the nearest bf16 number would overflow."""
    top = torch.finfo(torch.float32).max
    x = torch.zeros(20, 16, device="cuda")
    x[:, 3] = torch.tensor([top, -top, 3.395e38, 3.3895e38, 3.38e38] * 4, device="cuda")
    w = torch.zeros(24, 16, device="cuda")
    w[:, 3] = torch.linspace(-0.9, 0.9, 24, device="cuda")
    y = B.csa_linear_fwd(B.LinearParams(20, 16, 24, "f32"), x, w)
    want = x.double() @ w.double().t()
    close(y, want, product_tol(want.abs(), 1), "y")
    dw = B.csa_linear_bwd(B.LinearParams(20, 16, 24, "f32"), torch.full((20, 24), 2.0 ** -6, device="cuda"), x, w, need_dx=False)[1]
    close(dw, x.double().sum(0).expand(24, 16) * 2.0 ** -6, product_tol(x.double().abs().sum(0) * 2.0 ** -6, 20), "dw")


def test_linear_the_same_bits_again_and_from_two_streams():
    t = linear_inputs(700, 512, 264, "bf16", "bf16", 6)
    p = B.LinearParams(700, 512, 264, activation="gelu_tanh")
    first = (B.csa_linear_fwd(p, t["x"], t["w"]), *B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], t["z"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((B.csa_linear_fwd(p, t["x"], t["w"]), *B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], t["z"])))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(first, g))
    B.csa_check_device_status()


def test_linear_autograd_against_differences():
    """The whole chain by central differences in fp32 values: f = sum(y * c) moves by its gradient."""
    M, K, N = 24, 33, 17
    t = linear_inputs(M, K, N, "f32", "f32", 7)
    p = B.LinearParams(M, K, N, "f32", activation="gelu_tanh", alpha=0.5)
    leaves = [t[k].clone().requires_grad_(True) for k in ("x", "w", "bias", "res")]
    c = t["dy"]
    (B.csa_linear(*leaves, params=p) * c).sum().backward()

    def f(v):
        z = 0.5 * (v[0] @ v[1].t()) + v[2]
        return ((act64(z, "gelu_tanh") + v[3]) * c.double()).sum()

    v = [x.detach().double() for x in leaves]
    g = gen(8)
    for i in range(4):
        d = torch.randn(v[i].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        up, down = ([x + s * h * d if k == i else x for k, x in enumerate(v)] for s in (1, -1))
        want = float((f(up) - f(down)) / (2 * h))
        got = float((leaves[i].grad.double() * d).sum())
        # differences are off by h^2 / 6 of the third derivative (order one here), gradients by fp32 sums of M K N terms
        scale = float((leaves[i].grad.double().abs() * d.abs()).sum())
        assert abs(got - want) <= 1e-4 * scale, (i, got, want)


def test_linear_gradients_of_views_and_only_those_asked_for():
    M, K, N = 40, 24, 16
    t = linear_inputs(M, K, N, "bf16", "bf16", 9)
    p = B.LinearParams(M, K, N, activation="silu")
    x = t["x"].reshape(2, 20, K).clone().requires_grad_(True)
    res = t["res"].reshape(2, 20, N).clone().requires_grad_(True)
    y = B.csa_linear(x, t["w"], None, res, params=p)
    y.backward(t["dy"])
    assert x.grad.shape == x.shape and torch.equal(res.grad, t["dy"].view(2, 20, N))
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    B.csa_linear_fwd(p, t["x"], t["w"], preact=z)
    dx, dw, db = B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], z, need_dw=False, need_db=False)
    assert dw is None and db is None and torch.equal(dx.view(x.shape), x.grad)
    full = B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], z)
    assert torch.equal(B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], z, need_dx=False, need_db=False)[1], full[1])
    assert torch.equal(B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], z, need_dx=False, need_dw=False)[2], full[2])


# ------------------------------------------------------------------ rotary positions

def rope64(x, positions, inv_freq, sections, offset, rot, interleaved, inverse):
    """The rotation in 64 bits, angles reduced exactly: position times frequency as a 53-bit integer over 2^k."""
    import numpy as np
    f = inv_freq.cpu().numpy()
    pos = positions.cpu().numpy()
    out = x.double().clone()
    pair = 0
    for axis, n in enumerate(sections):
        for i in range(pair, pair + n):
            turns = []
            num, den = float(f[i] / (2 * math.pi)).as_integer_ratio()
            for p in pos[axis]:
                t = int(p) * num
                turns.append((t - (t // den) * den) / den)
            ang = torch.from_numpy(np.array(turns)).to(x.device)[:, None] * (2 * math.pi)
            c, s = torch.cos(ang), torch.sin(ang) * (-1 if inverse else 1)
            ia, ib = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + rot // 2 + i)
            a, b = x[:, :, ia].double(), x[:, :, ib].double()
            out[:, :, ia], out[:, :, ib] = a * c - b * s, a * s + b * c
        pair += n
    return out


def check_rope(rows, heads, dim, rot, offset=0, sections=None, dtype="bf16", interleaved=False, inverse=False, far=1 << 20,
               pos64=False, seed=0, xs=(0, 0), ys=(0, 0)):
    g = gen(seed)
    sections = sections or [rot // 2]
    x = randn(g, rows, heads, dim, dtype=DT[dtype])
    if xs != (0, 0):
        buf = randn(g, rows * xs[0] + heads * xs[1], dtype=DT[dtype])
        x = buf.as_strided((rows, heads, dim), (xs[0], xs[1], 1))
    pos = torch.randint(-far // 4, far, (len(sections), rows), generator=g, device="cuda",
                        dtype=torch.int64 if pos64 else torch.int32)
    f = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(1, rot // 2))
    p = B.RopeParams(rows, heads, dim, dtype, rot, offset, sections, interleaved, inverse, pos64, *xs, *ys)
    out = None
    if ys != (0, 0):
        out = torch.full((rows * ys[0] + heads * ys[1],), 7.0, dtype=DT[dtype], device="cuda").as_strided(
            (rows, heads, dim), (ys[0], ys[1], 1))
    out = B.csa_rope(p, x, pos, f, out)
    want = rope64(x, pos, f, sections, offset, rot, interleaved, inverse)
    # cosine and sine: the angle as a 32-bit fraction rounded to 24 bits (2^-24 of it, pi at most) and two units of the
    # functions, below 2^-21 in all; the frequency's own fraction is off by 2^-53 relative, times the position
    mag = x.double().abs().amax(-1, keepdim=True) * 2
    tol = mag * (2.0 ** -21 + far * 2.0 ** -52) + 3 * F32 * mag
    rotated = torch.zeros(dim, dtype=torch.bool, device="cuda")
    rotated[offset:offset + rot] = True
    tol = torch.where(rotated, tol + U[DT[dtype]] * (want.abs() + tol), torch.zeros_like(tol))
    close(out, want, tol, "rope")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,heads,dim,rot,offset,sections", [
    (1, 1, 2, 2, 0, None), (1, 64, 128, 64, 0, [16, 8, 8]), (3, 5, 7, 4, 3, [1, 1]), (7, 3, 24, 16, 4, [2, 3, 1, 2]),
    (33, 64, 192, 64, 128, [12, 10, 10]), (1000, 1, 128, 64, 0, None), (260, 1, 72, 72, 0, [36, 0]), (65, 9, 40, 24, 16, None),
    (50, 128, 64, 64, 0, [8, 8, 8, 8]), (300, 2, 1024, 1024, 0, None), (11, 2, 20, 10, 6, [3, 2]), (4, 3, 16, 0, 8, [0]),
    (2000, 4, 64, 12, 52, [6])])
def test_rope_shapes(rows, heads, dim, rot, offset, sections, dtype, interleaved):
    for inverse in (False, True):
        check_rope(rows, heads, dim, rot, offset, sections, dtype, interleaved, inverse, seed=rows + dim)


@pytest.mark.parametrize("far,pos64", [(1 << 30, False), (1 << 30, True), (1 << 40, True), (16, True)])
def test_rope_far_positions(far, pos64):
    # at 2^40 the frequency's own 53 bits leave 2^-12 of an angle: the tolerance follows
    check_rope(40, 2, 64, 64, dtype="f32", far=far, pos64=pos64, seed=2)


def test_rope_extreme_positions_are_exact_rotations():
    """The most negative and the largest position: |(a, b)| is kept."""
    for pos64 in (False, True):
        info = torch.iinfo(torch.int64 if pos64 else torch.int32)
        pos = torch.tensor([[info.min, info.max, 0, -1]], dtype=torch.int64 if pos64 else torch.int32, device="cuda")
        x = randn(gen(3), 4, 2, 32)
        f = 10000.0 ** (-torch.arange(16, dtype=torch.float64, device="cuda") / 16)
        out = B.csa_rope(B.RopeParams(4, 2, 32, "f32", positions_64=pos64), x, pos, f)
        n = lambda t: t[..., :16].double() ** 2 + t[..., 16:].double() ** 2  # noqa: E731
        close(n(out), n(x), 2.0 ** -20 * n(x), "norms")
        assert torch.equal(out[2], x[2])                      # position 0 turns nothing


@pytest.mark.parametrize("xs,ys", [((640, 80), (0, 0)), ((0, 0), (700, 64)), ((64, 64 * 50), (64, 64 * 50)),
                                   ((521, 65), (67, 67 * 50))])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rope_strides(xs, ys, dtype):
    """Padded rows and heads, heads outermost, odd strides."""
    check_rope(50, 8, 64, 32, 16, [4, 12], dtype, xs=xs, ys=ys)


def test_rope_in_place_and_copies():
    g = gen(4)
    for dtype, rot, off in ((torch.bfloat16, 64, 32), (torch.float32, 20, 7)):
        x = randn(g, 70, 6, 128, dtype=dtype)
        x[3, 2, 0], x[4, 1, 127] = float("nan"), float("inf")       # outside the rotation: copied as they are
        pos = torch.randint(0, 5000, (1, 70), device="cuda", dtype=torch.int32)
        f = 1000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / rot)
        p = B.RopeParams(70, 6, 128, dtype, rot, off)
        out = B.csa_rope(p, x, pos, f)
        assert bool(out[3, 2, 0].isnan()) and out[4, 1, 127] == float("inf")
        y = x.clone()
        assert B.csa_rope(p, y, pos, f, out=y) is y
        assert torch.equal(y.nan_to_num(1.0), out.nan_to_num(1.0))


def test_rope_gradient_is_the_inverse_rotation():
    g = gen(5)
    x = randn(g, 30, 4, 48).requires_grad_(True)
    pos = torch.randint(0, 100000, (2, 30), device="cuda", dtype=torch.int32)
    f = 100.0 ** (-torch.arange(16, dtype=torch.float64, device="cuda") / 16)
    p = B.RopeParams(30, 4, 48, "f32", 32, 8, [10, 6])
    c = randn(g, 30, 4, 48)
    (B.csa_rotary(x, pos, f, p) * c).sum().backward()
    want = rope64(c, pos, f, [10, 6], 8, 32, False, True)
    close(x.grad, want, 2.0 ** -20 * c.double().abs().amax(-1, keepdim=True), "gradient")


def test_rope_without_rows():
    p = B.RopeParams(0, 4, 32)
    out = B.csa_rope(p, torch.empty(0, 4, 32, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(1, 0, dtype=torch.int32, device="cuda"), torch.ones(16, dtype=torch.float64, device="cuda"))
    assert out.shape == (0, 4, 32)


# ------------------------------------------------------------------ AdamW

HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.98, eps=1e-6, weight_decay=0.05)


def scales(n):
    return -(-n // 256)


def adamw_tensors(sizes, param, grad, eight, master, seed, guard=64):
    """Buffers with guard elements behind every tensor; a tensor starts 16-byte aligned."""
    g = gen(seed)
    cols = {k: [] for k in ("param", "grad", "m", "v")}
    if eight:
        cols.update(m_scale=[], v_scale=[])
    if master:
        cols["master"] = []
    bufs = {k: [] for k in cols}

    def put(key, x):
        buf = torch.cat([x.flatten().float(), torch.full((guard,), 5.0, device="cuda")]).to(x.dtype) if x.dtype != torch.float8_e4m3fn \
            else torch.cat([x.view(torch.uint8).flatten(), torch.full((guard,), 5, dtype=torch.uint8, device="cuda")]).view(x.dtype)
        bufs[key].append(buf)
        cols[key].append(buf[:x.numel()])

    for n in sizes:
        w = randn(g, n, scale=0.05)
        put("param", w.to(DT[param]))
        if master:
            put("master", w)
        put("grad", randn(g, n, dtype=DT[grad], scale=1e-2))
        m, r = randn(g, n, scale=3e-3), randn(g, n, scale=3e-3).abs() + 1e-4
        if n > 600:
            m[256:512], r[256:512] = 0, 0            # a block whose state is zero
        if eight:
            for k, x in (("m", m), ("v", r)):
                pad = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
                top = pad.abs().amax(1) / 448
                put(k + "_scale", top)
                put(k, (pad / top.clamp_min(1e-30)[:, None]).flatten()[:n].to(torch.float8_e4m3fn))
        else:
            put("m", m)
            put("v", r * r)
    return cols, bufs


def state64(t):
    n = t["param"].numel()
    w = (t["master"] if "master" in t else t["param"]).double()
    if "m_scale" in t:
        blk = torch.arange(n, device="cuda") // 256
        return w, t["m"].double() * t["m_scale"].double()[blk], (t["v"].double() * t["v_scale"].double()[blk]) ** 2
    return w, t["m"].double(), t["v"].double()


def step64(t, step, gs, lr, beta1, beta2, eps, weight_decay):
    w, m, v = state64(t)
    g = t["grad"].double() * gs
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    upd = (m / (1 - beta1 ** step)) / ((v / (1 - beta2 ** step)).sqrt() + eps)
    return w - lr * weight_decay * w - lr * upd, m, v, upd, g


def check_adamw(sizes, param="bf16", grad="bf16", eight=False, master=False, step=3, gs=None, seed=0, device_scalars=False):
    cols, bufs = adamw_tensors(sizes, param, grad, eight, master, seed)
    rows = [{k: c[i] for k, c in cols.items()} for i in range(len(sizes))]
    want = [step64(t, step, 1.0 if gs is None else gs, **HYPER) for t in rows]
    before = [state64(t) for t in rows]
    table = B.AdamWTensors(**cols)
    scalar = torch.tensor(gs, device="cuda") if gs is not None else None
    h = dict(HYPER)
    if device_scalars:
        h["lr"] = torch.tensor(HYPER["lr"], device="cuda")
        step = torch.tensor(step, device="cuda")
    B.csa_adamw(table, step, grad_scale=scalar, **h)
    lr = HYPER["lr"]
    for t, (w, m, v, upd, g), (w0, m0, v0) in zip(rows, want, before):
        # moments: three roundings each of the terms; the decoded 8-bit values add two (scale, square)
        em = 4 * F32 * (0.9 * m0.abs() + g.abs() * 0.1)
        ev = 8 * F32 * v
        # the update: its moments' errors, the corrections (2^-21 with device scalars), root, quotient
        eu = upd.abs() * 2.0 ** -20 + em / (v.sqrt() + 1e-12)
        ew = 4 * F32 * (w0.abs() + lr * upd.abs()) + lr * eu * (20 if step == 1 else 8)
        if "master" in t:
            close(t["master"], w, ew, "master")
        close(t["param"], w, ew + U[t["param"].dtype] * (w.abs() + ew), "param")
        if not eight:
            close(t["m"], m, em + F32 * m.abs(), "m")
            close(t["v"], v, ev, "v")
            continue
        n, blk = w.numel(), torch.arange(w.numel(), device="cuda") // 256
        for key, y, ey in (("m", m, em), ("v", v.sqrt(), ev / (2 * v.sqrt() + 1e-30))):
            top = torch.zeros(scales(n), dtype=torch.float64, device="cuda").scatter_reduce_(0, blk, y.abs(), "amax")
            etop = torch.zeros(scales(n), dtype=torch.float64, device="cuda").scatter_reduce_(0, blk, ey, "amax")
            close(t[key + "_scale"], top / 448, (etop + 4 * F32 * top) / 448, key + "_scale")
            # half a step of e4m3 (2^-4 relative, 2^-10 of a scale below the smallest normal), a whole one for the
            # root that is raised to the smallest code
            sc = t[key + "_scale"].double()[blk]
            half = torch.maximum(2.0 ** -4 * y.abs(), (2.0 ** -9 if key == "v" else 2.0 ** -10) * sc)
            close(t[key].double() * sc, y, half * (1 + 2.0 ** -18) + ey, key)
        assert bool(((t["v"].double() > 0) == (v > 0)).all())
    for key, list_ in bufs.items():
        for buf, c in zip(list_, cols[key]):
            tail = buf[c.numel():]
            tail = tail.view(torch.uint8) if tail.dtype == torch.float8_e4m3fn else tail
            assert bool((tail == 5).all()), f"{key}: written behind its end"


@pytest.mark.parametrize("param,grad,master", [("bf16", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True),
                                               ("f32", "f32", False), ("f32", "bf16", False)])
@pytest.mark.parametrize("eight", [False, True])
def test_adamw_types_and_sizes(param, grad, master, eight):
    check_adamw([1, 7, 8, 255, 256, 257, 1000, 4096, 4097, 20000, 65537], param, grad, eight, master)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("device_scalars", [False, True])
@pytest.mark.parametrize("step,gs", [(1, None), (2, 0.25), (100000, 1.0)])
def test_adamw_steps_and_scales(step, gs, eight, device_scalars):
    check_adamw([300, 5000], "f32", "bf16", eight, False, step, gs, seed=step, device_scalars=device_scalars)


def test_adamw_many_tensors_of_mixed_types():
    """More tensors than one launch takes, in every combination of types, and tensors of no elements."""
    g = gen(1)
    cols = {k: [] for k in ("param", "grad", "m", "v", "m_scale", "v_scale", "master")}
    for i in range(1000):
        n = [0, 3, 300, 513][i % 4]
        eight, pt, gt = bool(i & 4), (torch.float32, torch.bfloat16)[i >> 3 & 1], (torch.float32, torch.bfloat16)[i >> 4 & 1]
        cols["param"].append(randn(g, n, dtype=pt))
        cols["grad"].append(randn(g, n, dtype=gt))
        z = B.AdamWTensors.zero_state([cols["param"][-1]], eight)
        for k in ("m", "v", "m_scale", "v_scale"):
            cols[k].append(z[k][0] if k in z else None)
        cols["master"].append(cols["param"][-1].float().clone() if i % 7 == 0 else None)
    start = [p.double() for p in cols["param"]]
    B.csa_adamw(B.AdamWTensors(**cols), 1, lr=0.01, weight_decay=0.0)
    for p, p0, gr in zip(cols["param"], start, cols["grad"]):
        # the first step from zero moments is lr g / (|g| + eps): the gradient's sign
        d = gr.double()
        want = p0 - 0.01 * d / (d.abs() + 1e-8)
        close(p, want, U[p.dtype] * (want.abs() + 0.01) + 1e-6, "first step")


def test_adamw_skips_on_found_inf():
    cols, _ = adamw_tensors([1000], "bf16", "bf16", True, True, 2)
    before = {k: c[0].clone() for k, c in cols.items()}
    table = B.AdamWTensors(**cols)
    flag = torch.ones((), device="cuda")
    B.csa_adamw(table, 1, found_inf=flag)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    assert all(same(before[k], c[0]) for k, c in cols.items())
    flag.zero_()
    B.csa_adamw(table, 1, found_inf=flag)
    assert not same(before["m"], cols["m"][0])


def test_adamw_nan_gradient_stays_in_its_element():
    for eight in (False, True):
        cols, _ = adamw_tensors([600], "f32", "f32", eight, False, 3)
        cols["grad"][0][10] = float("nan")
        B.csa_adamw(B.AdamWTensors(**cols), 1)
        assert bool(cols["param"][0][10].isnan()) and int(cols["param"][0].isnan().sum()) == 1
        assert int(cols["m"][0].float().isnan().sum()) == 1 and int(cols["v"][0].float().isnan().sum()) == 1


def test_adamw_overlapping_buffers_refused():
    buf = torch.zeros(1000, device="cuda")
    a, b = buf[:600], buf[400:1000]
    z = B.AdamWTensors.zero_state([a, b])
    g = [torch.ones_like(a), torch.ones_like(b)]
    with pytest.raises(ValueError, match="overlap"):
        B.AdamWTensors(param=[a, b], grad=g, **z)
    with pytest.raises(ValueError, match="f32 or bf16"):
        B.AdamWTensors(param=[a.half()], grad=[g[0]], m=[z["m"][0]], v=[z["v"][0]])
    with pytest.raises(ValueError, match="m_scale"):
        e = B.AdamWTensors.zero_state([a], True)
        B.AdamWTensors(param=[a], grad=[g[0]], m=e["m"], v=e["v"], m_scale=[e["m_scale"][0][:1]], v_scale=e["v_scale"])


def test_adamw_captured_with_device_scalars():
    """A captured step replayed with another step count and rate equals the eager ones."""
    sizes = [700, 4100]
    for eight in (False, True):
        one, _ = adamw_tensors(sizes, "bf16", "bf16", eight, True, 4)
        two = {k: [t.clone() for t in c] for k, c in one.items()}
        step, lr = torch.ones((), dtype=torch.int64, device="cuda"), torch.tensor(1e-3, device="cuda")
        ta, tb = B.AdamWTensors(**one), B.AdamWTensors(**two)
        B.csa_adamw(ta, step, lr)
        B.csa_adamw(tb, step, lr)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            B.csa_adamw(ta, step, lr)
        for k in (2, 3, 4):
            step.fill_(k)
            lr.fill_(1e-3 / k)
            graph.replay()
            B.csa_adamw(tb, step, lr)
        torch.cuda.synchronize()
        for k in one:
            for a, b in zip(one[k], two[k]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_linear_long_sums_keep_their_bits():
    """fp32 results of long sums.  The tensor core cuts off, at most 2^-23 of the accumulator for each 16 k.  Three-part
    products start anew every 64 k (4 cuts at full size, the parts left out another 2^-23), bf16 ones every 512 k (32
    cuts); the pieces are added in fp32, whose roundings do not add up in one direction."""
    g = gen(10)
    for dtype, bound in (("f32", 6 * 2.0 ** -23), ("bf16", 33 * 2.0 ** -23)):
        for M, K, N in ((40, 65536, 200), (300, 20000, 136)):
            x, w = randn(g, M, K, dtype=DT[dtype]), randn(g, N, K, dtype=DT[dtype], scale=K ** -0.5)
            y = B.csa_linear_fwd(B.LinearParams(M, K, N, dtype, "f32"), x, w).double()
            want = x.double() @ w.double().t()
            assert float((y - want).norm() / want.norm()) <= bound
    x, dy = randn(g, 60000, 100), randn(g, 60000, 72)      # a gradient's sum over the rows
    dw = B.csa_linear_bwd(B.LinearParams(60000, 100, 72, "f32"), dy, x, None, need_dx=False, need_db=False)[1].double()
    want = dy.double().t() @ x.double()
    assert float((dw - want).norm() / want.norm()) <= 6 * 2.0 ** -23


def test_linear_captured_with_other_inputs():
    """Captured calls with workspaces of their own, replayed in turn on new inputs."""
    graphs = []
    for k, (M, act) in enumerate(((200, "silu"), (3, "none"), (513, "relu"))):
        t = linear_inputs(M, 136, 72, "bf16", "bf16", 20 + k)
        p = B.LinearParams(M, 136, 72, activation=act)
        B.csa_linear_fwd(p, t["x"], t["w"])
        B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], t["z"])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y = B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], t["res"])
            grads = B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], t["z"])
        graphs.append((graph, p, t, (y, *grads)))
    for seed in (30, 40):
        for k, (graph, p, t, _) in enumerate(graphs):
            for name, v in linear_inputs(p.c.rows, 136, 72, "bf16", "bf16", seed + k).items():
                t[name].copy_(v)
            graph.replay()
        torch.cuda.synchronize()
        for graph, p, t, got in graphs:
            want = (B.csa_linear_fwd(p, t["x"], t["w"], t["bias"], t["res"]), *B.csa_linear_bwd(p, t["dy"], t["x"], t["w"], t["z"]))
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_takes_slices_of_a_larger_gradient():
    """The gradient of a concatenation is a slice that need not start on 16 bytes; a bias of another shape."""
    g = gen(50)
    x, w, b = (randn(g, *s).requires_grad_(True) for s in ((6, 8), (9, 8), (1, 9)))
    p = B.LinearParams(6, 8, 9, "f32")
    head = torch.ones(5, 9, device="cuda")
    torch.cat([head, B.csa_linear(x, w, b, params=p)]).square().sum().backward()
    x64, w64 = x.detach().double(), w.detach().double()
    d = 2 * (x64 @ w64.t() + b.detach().double())                # the gradient of y, off by what y is off by, doubled
    e = 2 * product_tol(x64.abs() @ w64.abs().t() + b.detach().double().abs(), 9)
    ones = torch.ones(1, 6, device="cuda", dtype=torch.float64)
    for name, got, left, right, err in (("dx", x.grad, d, w64, e @ w64.abs()), ("dw", w.grad, d.t(), x64, e.t() @ x64.abs()),
                                        ("db", b.grad, ones, d, ones @ e)):
        close(got, left @ right, err + product_tol(left.abs() @ right.abs() + err, 9), name)
    r = B.RopeParams(3, 1, 6, "f32")
    v = randn(g, 3, 1, 6).requires_grad_(True)
    pos, f = torch.arange(3, device="cuda", dtype=torch.int32)[None], torch.ones(3, device="cuda", dtype=torch.float64)
    weight = randn(g, 4, 1, 6)
    (torch.cat([v.detach()[:1], B.csa_rotary(v, pos, f, r)]) * weight).sum().backward()
    assert torch.equal(v.grad, B.csa_rope(r.inverted(), weight[1:].clone(), pos, f))


def test_adamw_step_on_the_device_below_one_counts_as_one():
    g = gen(51)
    sides = []
    for first in (0, 1):
        w = [randn(gen(52), 300)]
        t = B.AdamWTensors(w, [randn(gen(53), 300)], **B.AdamWTensors.zero_state(w))
        B.csa_adamw(t, torch.tensor(first, device="cuda"))
        sides.append(w[0])
    assert torch.equal(*sides) and bool(sides[0].isfinite().all())


def test_offsets_beyond_32_bits():
    """More than 2^31 elements in an operand, an output or a workspace: the first and the last rows."""
    g = gen(60)
    bf = torch.bfloat16
    # y, z, dy and dz of 264000 x 8200
    M, K, N, T = 264000, 64, 8200, 40
    x, w = randn(g, M, K, dtype=bf), randn(g, N, K, dtype=bf)
    p = B.LinearParams(M, K, N, activation="relu")
    z = torch.empty(M, N, dtype=bf, device="cuda")
    y = B.csa_linear_fwd(p, x, w, preact=z)
    dx = B.csa_linear_bwd(p, y, x, w, z, need_dw=False)[0]
    w64 = w.double()
    for rows in (slice(0, T), slice(M - T, M)):
        want = x[rows].double() @ w64.t()
        tol = product_tol(x[rows].double().abs() @ w64.abs().t(), K)
        close(z[rows], want, tol + U[bf] * (want.abs() + tol), "z")
        close(y[rows], want.clamp(min=0), tol + U[bf] * (want.abs() + tol), "y")
        d = y[rows].double() * (z[rows] > 0)                     # exact in bf16
        want, tol = d @ w64, product_tol(d.abs() @ w64.abs(), N)
        close(dx[rows], want, tol + U[bf] * (want.abs() + tol), "dx")
    del y, z, dx
    # weights of 1050000 x 2056 and a few rows
    N, K = 1050000, 2056
    w = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16)
    x = randn(g, 3, K, dtype=torch.bfloat16)
    y = B.csa_linear_fwd(B.LinearParams(3, K, N, out_dtype="f32"), x, w)
    last = w[-50:].double()
    close(y[:, -50:], x.double() @ last.t(), product_tol(x.double().abs() @ last.abs().t(), K), "y of the last weights")
    del w, y
    # rotary positions on 2^31 + some values
    rows, heads, dim = 262150, 64, 128
    x = torch.randn(rows, heads, dim, generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (1, rows), generator=g, device="cuda", dtype=torch.int32)
    f = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    out = B.csa_rope(B.RopeParams(rows, heads, dim), x, pos, f)
    assert torch.equal(out[-20:], B.csa_rope(B.RopeParams(20, heads, dim), x[-20:].clone(), pos[:, -20:].contiguous(), f))
    del x, out
    # a tensor of 2^31 + 2^16 + 77 weights with 8-bit state
    n, t = (1 << 31) + (1 << 16) + 77, (1 << 16) + 77
    state = lambda w: B.AdamWTensors.zero_state(w, eight_bit=True)  # noqa: E731
    w = [torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)]
    gr = [torch.randn(n, generator=g, device="cuda", dtype=torch.bfloat16)]
    small, sg = [w[0][-t:].clone()], [gr[0][-t:].clone()]
    big = B.AdamWTensors(w, gr, **state(w))
    B.csa_adamw(big, 1)
    ref = B.AdamWTensors(small, sg, **state(small))
    B.csa_adamw(ref, 1)
    assert torch.equal(w[0][-t:], small[0])
    for name in ("m", "v"):
        assert torch.equal(big.tensors[name][0].view(torch.uint8)[-t:], ref.tensors[name][0].view(torch.uint8))


def test_wrong_tensors_refused_by_the_bindings():
    p = B.LinearParams(16, 32, 24)
    x, w = torch.zeros(16, 32, device="cuda").bfloat16(), torch.zeros(24, 32, device="cuda").bfloat16()
    for bad in (dict(x=x.float()), dict(x=x[:8]), dict(x=x.cpu()), dict(weight=w.t()), dict(weight=w.cpu()), dict(bias=torch.zeros(24, device="cuda").bfloat16()),
                dict(residual=torch.zeros(16, 24, device="cuda")), dict(out=torch.empty(16, 23, device="cuda").bfloat16()),
                dict(workspace=torch.empty(8, dtype=torch.uint8)), dict(preact=torch.empty(16, 24, device="cuda"))):
        args = dict(x=x, weight=w)
        args.update(bad)
        with pytest.raises(ValueError):
            B.csa_linear_fwd(p, args.pop("x"), args.pop("weight"), **args)
    with pytest.raises(ValueError):   # an activation's gradient needs its argument
        B.csa_linear_bwd(B.LinearParams(16, 32, 24, activation="relu"), torch.zeros(16, 24, device="cuda").bfloat16(), x, w)
    r = B.RopeParams(4, 2, 16)
    y, pos, f = torch.zeros(4, 2, 16, device="cuda").bfloat16(), torch.zeros(1, 4, device="cuda", dtype=torch.int32), torch.ones(8, device="cuda", dtype=torch.float64)
    for bad in (dict(x=y.float()), dict(positions=pos.long()), dict(positions=pos[:, :3]), dict(inv_freq=f.float()), dict(x=y.transpose(0, 1)),
                dict(out=y.float())):
        args = dict(x=y, positions=pos, inv_freq=f)
        args.update(bad)
        with pytest.raises(ValueError):
            B.csa_rope(r, **args)
    z = B.AdamWTensors.zero_state([x])
    t = B.AdamWTensors([x], [x.clone()], **z)
    with pytest.raises(ValueError):
        B.csa_adamw(t, torch.ones((), device="cuda"))                     # a step count is int64
    with pytest.raises(ValueError):
        t.set_grads([x[:3]])
    with pytest.raises(B.CSAError):
        B.csa_adamw(t, 0)
