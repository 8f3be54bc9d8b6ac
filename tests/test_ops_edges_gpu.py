"""The operators around the step where they can go wrong: kernels close behind one another, ends of buffers, infinities,
sums over very many rows, gradients that share memory.

Tolerances are worst cases of the arithmetic, as in test_ops_gpu.py: u(t) = finfo(t).eps / 2.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
DT = {"bf16": BF, "f32": F32}
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def test_products_close_behind_one_another():
    """Products of every tile shape in one stream with nothing between them: each starts on the SMs that its predecessor
    leaves, with barriers in the same places of shared memory."""
    g = gen(1)
    calls = []
    for M, K, N, dt, out in ((2048, 1024, 2048, "bf16", "bf16"), (1024, 512, 1024, "bf16", "bf16"), (512, 2048, 512, "bf16", "f32"),
                             (300, 512, 640, "f32", "f32"), (64, 256, 512, "bf16", "bf16"), (4096, 64, 4096, "bf16", "bf16")):
        t = BF if dt == "bf16" else F32
        p = B.LinearParams(M, K, N, dt, out)
        x, w = randn(g, M, K, dtype=t), randn(g, N, K, dtype=t, scale=K ** -0.5)
        ws = torch.empty(max(1, p.fwd_workspace_bytes), dtype=torch.uint8, device="cuda")
        first = B.csa_linear_fwd(p, x, w, workspace=ws)
        want = x.double() @ w.double().t()
        assert float((first.double() - want).norm() / want.norm()) <= U[first.dtype] + (K // 16 + 8) * 2.0 ** -23
        calls.append((p, x, w, ws, first, torch.empty_like(first)))
    torch.cuda.synchronize()
    for r in range(60):
        for p, x, w, ws, _, y in calls if r % 2 else calls[::-1]:
            B.csa_linear_fwd(p, x, w, workspace=ws, out=y)
    for *_, first, y in calls:
        assert torch.equal(first, y)
    B.csa_check_device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(129, 77, 33), (40, 1001, 8), (33, 9, 1001), (300, 65, 771)])
def test_arguments_that_end_inside_a_vector(M, K, N, dtype):
    """Arguments whose last value is the last of a buffer of which only they are defined: what lies behind them is NaN in
    one run and 7 in another, which changes nothing."""
    t = BF if dtype == "bf16" else F32
    g = gen(M + K + N)
    p = B.LinearParams(M, K, N, dtype, activation="silu")

    def put(x, behind):
        buf = torch.full((x.numel() + 64,), behind, dtype=x.dtype, device="cuda")
        v = buf[:x.numel()].view(x.shape)
        v.copy_(x)
        return v

    args = [randn(g, M, K, dtype=t), randn(g, N, K, dtype=t), randn(g, N), randn(g, M, N, dtype=t), randn(g, M, N, dtype=t),
            randn(g, M, N, dtype=t)]
    got = []
    for behind in (7.0, float("nan")):
        x, w, b, res, dy, z = (put(a, behind) for a in args)
        got.append((B.csa_linear_fwd(p, x, w, b, res), *B.csa_linear_bwd(p, dy, x, w, z)))
    for a, b in zip(*got):
        assert bool(a.isfinite().all()) and torch.equal(a, b)


def test_autograd_sees_what_the_calls_write():
    """A graph kept over an optimizer step, or over a call that writes to one of its tensors, refuses its backward pass."""
    g = gen(3)
    p = B.LinearParams(24, 16, 16, "f32")
    x, w = randn(g, 24, 16).requires_grad_(True), randn(g, 16, 16).requires_grad_(True)
    y = B.csa_linear(x, w, params=p)
    state = B.AdamWTensors.zero_state([w])
    B.csa_adamw(B.AdamWTensors([w.detach()], [torch.ones(16, 16, device="cuda")], **state), 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    r = B.RopeParams(24, 1, 16, "f32")
    pos, f = torch.arange(24, device="cuda", dtype=torch.int32)[None], torch.ones(8, device="cuda", dtype=torch.float64)
    dy = randn(g, 24, 16)
    for write in (lambda t: B.csa_rope(r, t, pos, f, out=t), lambda t: B.csa_linear_fwd(p, dy, w.detach(), residual=t, out=t),
                  lambda t: B.csa_linear_fwd(p, dy, w.detach(), preact=t),
                  lambda t: B.csa_linear_bwd(p, dy, dy.clone(), w.detach(), out=(t, None, None))):
        x = randn(g, 24, 16)
        y = B.csa_linear(x, w, params=p)
        write(x)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    with torch.inference_mode():                 # tensors without a counter
        out = torch.empty(24, 16, device="cuda")
        assert B.csa_linear_fwd(p, dy, w.detach(), out=out) is out and B.csa_rope(r, out, pos, f, out=out) is out
    # an unchanged graph goes through
    B.csa_linear(randn(g, 24, 16), w, params=p).sum().backward()


# ------------------------------------------------------------------ AdamW with 8-bit moments over many steps

def held(t, i=0):
    """m and v that an 8-bit state stands for."""
    c = {k: t.tensors[k][i] for k in ("m", "v", "m_scale", "v_scale")}
    blk = torch.arange(c["m"].numel(), device="cuda") // 256
    return c["m"].double() * c["m_scale"].double()[blk], (c["v"].double() * c["v_scale"].double()[blk]) ** 2


def recurrences(beta2, steps, gradient, n=256 * 16):
    """An 8-bit and an fp32 state after the same gradients (gradient(step, out) writes them)."""
    w, grad = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    sides = [B.AdamWTensors([w.clone()], [grad], **B.AdamWTensors.zero_state([w], eight)) for eight in (True, False)]
    for t in range(steps):
        gradient(t, grad)
        for s in sides:
            B.csa_adamw(s, t + 1, beta1=0.9, beta2=beta2)
    return sides


@pytest.mark.parametrize("beta2,steps", [(0.95, 1500), (0.98, 1500), (0.99, 2000), (0.999, 6000)])
def test_adamw_8_bit_second_moments_follow_smaller_gradients(beta2, steps):
    """240 of each 256 gradients become ten times smaller after 300 steps; the held v has fp32's mean all the same.

    A held v is unbiased.  A step moves it by (1 - beta2) |g^2 / v - 1|, about 1 - beta2 of itself on average, through
    codes at most 27 % of v apart: a variance of 0.27 (1 - beta2) a step, of which 1 / (2 (1 - beta2)) steps remain, so
    0.14, and as much again for the scale's own moves.  A standard deviation of 0.5, over 3840 elements 0.8 % of the mean;
    5 % are six of them.  (Rounded to nearest, v stays up to 140 times too large.)"""
    g = gen(5)
    few = torch.arange(256 * 16, device="cuda") % 256 < 16
    size = torch.where(few, 1.0, 0.1)

    def gradient(t, out):
        out.normal_(generator=g)
        if t >= 300:
            out.mul_(size)

    eight, full = recurrences(beta2, steps, gradient)
    v, want = held(eight)[1], full.tensors["v"][0].double()
    # 256 of the unchanged ones: 3.1 % of the mean, six times that
    for part, most in ((few, 0.19), (~few, 0.05)):
        assert abs(float(v[part].mean() / want[part].mean()) - 1) <= most
    root = (v / want).sqrt()[~few]
    assert 0.85 <= float(root.median()) <= 1.1
    m, want = held(eight)[0], full.tensors["m"][0].double()
    assert float((m - want).norm() / want.norm()) <= 0.2


def test_adamw_8_bit_first_moments_follow_steady_gradients():
    """m goes all the way to a steady gradient that is up to 30 % off the one before (to nearest it stays where a tenth of
    what is missing is less than half a code).  Codes are at most an eighth of m apart: a scatter of 6 % about the
    gradient, that of an average over 200 steps, of which 10 each tell the same, 1.4 %; six times that for every element,
    over their mean less than 1 %."""
    g = gen(6)
    steady = randn(g, 256 * 16).abs() + 0.5
    steady[::256] = 6.0                                         # the largest of each block: the scale stays
    off = 1 + 0.3 * (2 * torch.rand(256 * 16, generator=g, device="cuda") - 1)
    off[::256] = 1.0
    sums = torch.zeros(256 * 16, device="cuda", dtype=torch.float64)
    w, grad = torch.zeros(256 * 16, device="cuda"), torch.empty(256 * 16, device="cuda")
    t = B.AdamWTensors([w], [grad], **B.AdamWTensors.zero_state([w], True))
    for k in range(500):
        torch.mul(steady, off if k < 150 else 1.0, out=grad)
        B.csa_adamw(t, k + 1, beta1=0.9, beta2=0.99)
        if k >= 300:
            sums += held(t)[0]
    off = sums / 200 / steady.double() - 1
    assert abs(float(off.mean())) <= 0.01 and float(off.abs().max()) <= 0.085


def test_adamw_8_bit_stochastic_codes_are_neighbours_and_unbiased():
    """One step from a known state: each code is next to the value it stands for, on either side of it as often as its
    place asks; sums over 100000 elements are within six standard deviations."""
    g = gen(7)
    n = 256 * 400
    w, grad = torch.zeros(n, device="cuda"), randn(g, n)
    t = B.AdamWTensors([w], [grad], **B.AdamWTensors.zero_state([w], True, seed=11))
    B.csa_adamw(t, 1, beta1=0.9, beta2=0.99)
    m, v = held(t)
    want_m = grad.double() * (1 - 0.9)
    want_v = grad.double() ** 2 * (1 - 0.99)
    blk = torch.arange(n, device="cuda") // 256
    for got, want, scale in ((m, want_m, t.tensors["m_scale"][0]), (v.sqrt(), want_v.sqrt(), t.tensors["v_scale"][0])):
        x = want.abs() / scale.double()[blk]
        step = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -6))) - 3)
        assert bool(((got.abs() / scale.double()[blk] - x).abs() <= step * (1 + 2.0 ** -16)).all())
    big = (want_m.abs() / t.tensors["m_scale"][0].double()[blk] > 2.0 ** -6)       # not raised to the smallest code
    for got, want in ((m.abs(), want_m.abs()), (v, want_v)):
        d = (got - want)[big]
        # the fp32 formula's own roundings of v, 2^-21, are one-sided at worst
        assert abs(float(d.sum())) <= 6 * float(d.norm()) + 2.0 ** -20 * float(want.sum())
        assert float(d.norm()) > 0.02 * float(want[big].norm())                    # and it is not to nearest
    # The random words of neighbouring elements, and of m and v of one, do not go together: "up" less its probability p has
    # the mean 0 for every element, and the mean square p (1 - p) <= 1/4, so products of two have at most 1/16.  (Signs alone
    # would not do for m and v of one: from a zero state their places p are the same, and E (2 p - 1)^2 = 1/3.)
    def less_p(x, up):
        lo = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -6))) - 3)
        return up.double() - (x / lo - torch.floor(x / lo))

    sm, sv = (t.tensors[k][0].double()[blk] for k in ("m_scale", "v_scale"))
    s = less_p(want_m.abs() / sm, m.abs() > want_m.abs())[big]
    lo = torch.exp2(torch.floor(torch.log2((want_v.sqrt() / sv).clamp_min(2.0 ** -6))) - 3)
    x = want_v.sqrt() / sv
    low = torch.floor(x / lo) * lo
    r = ((v > want_v).double() - (x - low) * (x + low) / (lo * (2 * low + lo)))[big]
    for a, b in ((s[1:], s[:-1]), (r[1:], r[:-1]), (s, r), (s[256:], s[:-256])):
        assert abs(float((a * b).mean())) <= 6 * 0.25 * a.numel() ** -0.5


def test_adamw_8_bit_stochastic_codes_are_the_same_every_time():
    """The same bits from the same seed, tensor and step, replayed from a graph too; others from another seed, step or place
    in the list."""
    g = gen(8)
    w0, grads = randn(g, 5000), [randn(g, 5000), randn(g, 5000)]

    def make(seed, count=1):
        w = [w0.clone() for _ in range(count)]
        return B.AdamWTensors(w, [grads[0]] * count, **B.AdamWTensors.zero_state(w, True, seed=seed))

    def codes(t, i=0):
        return torch.cat([t.tensors[k][i].view(torch.uint8) for k in ("m", "v")])

    step = torch.ones((), dtype=torch.int64, device="cuda")
    a, b, other, later, pair = make(3), make(3), make(4), make(3), make(3, 2)
    for t, k in ((a, 1), (b, step), (other, 1), (later, 2), (pair, 1)):
        B.csa_adamw(t, k)
    assert torch.equal(codes(a), codes(b)) and torch.equal(codes(a), codes(pair))
    for t in (codes(other), codes(later), codes(pair, 1)):
        assert not torch.equal(codes(a), t)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        B.csa_adamw(b, step)
    for k in (2, 3):
        step.fill_(k)
        graph.replay()
        B.csa_adamw(a, k)
        torch.cuda.synchronize()
        assert torch.equal(codes(a), codes(b))


def test_adamw_8_bit_nan_gradient_stays_in_its_element_when_stochastic():
    g = gen(9)
    w, grad = [randn(g, 600)], [randn(g, 600)]
    grad[0][10] = float("nan")
    t = B.AdamWTensors(w, grad, **B.AdamWTensors.zero_state(w, True))
    for k in (1, 2):
        B.csa_adamw(t, k)
        assert int(w[0].isnan().sum()) == int(t.tensors["m"][0].float().isnan().sum()) == int(t.tensors["v"][0].float().isnan().sum()) == 1


def test_adamw_8_bit_to_nearest_says_what_it_cannot_follow():
    g = gen(10)
    w, grad = [randn(g, 600)], [randn(g, 600)]
    s = B.AdamWTensors.zero_state(w, True)
    del s["seed"]
    t = B.AdamWTensors(w, grad, **s)
    with pytest.warns(UserWarning, match="beta2"):
        B.csa_adamw(t, 1)


@pytest.mark.parametrize("seed", [None, 1])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), 3e30, float("nan")])
def test_adamw_8_bit_infinite_moment_stays_in_its_element(bad, seed):
    """A gradient that is infinite, or whose square is: the other elements and their codes are those without it."""
    g = gen(12)
    w0, grad = randn(g, 700), randn(g, 700)
    grad[300] = 0.0
    sides = []
    for value in (0.0, bad):
        w, gr = [w0.clone()], [grad.clone()]
        gr[0][300] = value
        s = B.AdamWTensors.zero_state(w, True)
        s["seed"] = seed
        t = B.AdamWTensors(w, gr, **s)
        for k in (1, 2):
            B.csa_adamw(t, k, beta2=0.8)
        sides.append((w[0], *held(t)))
    other = torch.arange(700, device="cuda") != 300
    outside = other.clone()
    outside[256:512] = False
    for name, a, b in zip(("param", "m", "v"), *sides):
        # 3e30 is finite: its m takes its block's scale, and the block's other m their codes; v is infinite as before
        keep = outside if bad == 3e30 and name != "v" else other
        assert torch.equal(a[keep], b[keep]), name
    assert bool(sides[1][2][300].isnan())
    if bad != 3e30:
        assert bool(sides[1][1][300].isnan()) and bool(sides[1][0][300].isnan())


# ------------------------------------------------------------------ projections: long sums, infinities

def test_linear_bf16_gradients_of_a_million_rows():
    """Sums of 2^20 positive terms in as many tiles as the GPU runs at once, none of them too small (in one piece: 6e-3).
    The tensor core cuts products and sum off at the sum's last place, 2^-23 to 2^-24 of it: with the sum's and a product's
    for each 16 k at most 2^-22 of the sum, of the growing one half of that on average, over 65536 k 4.9e-4.  Roundings to
    bf16 (2^-8 at most, 1.2e-3 rms) go either way, six times their mean over 1536 outputs is 1.8e-4."""
    M, K, N = 1 << 20, 2048, 2048
    g = gen(20)
    x = torch.rand(M, K, generator=g, device="cuda", dtype=BF)
    dy = torch.rand(M, N, generator=g, device="cuda", dtype=BF)
    x[:, :48] *= 1 + torch.arange(48, device="cuda", dtype=BF) / 48          # sums of every place between two bf16 values
    p = B.LinearParams(M, K, N)
    dw = B.csa_linear_bwd(p, dy, x, None, need_dx=False, need_db=False)[1][:32, :48].double()
    want = torch.zeros(32, 48, device="cuda", dtype=torch.float64)
    for i in range(0, M, 1 << 16):
        want += dy[i:i + (1 << 16), :32].double().t() @ x[i:i + (1 << 16), :48].double()
    off = dw / want - 1
    assert float(off.abs().max()) <= 2.0 ** -8 * (1 + 2.0 ** -8) + 4.9e-4
    assert abs(float(off.mean())) <= 6.7e-4


@pytest.mark.parametrize("M,K,N", [(200, 70000, 4096), (8, 131080, 24), (300, 65544, 264)])
def test_linear_axes_longer_than_one_accumulator(M, K, N):
    """Cut axes forward and in dx (where the features are summed), with the epilogue behind the join."""
    g = gen(21)
    x, w, b, res = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF, scale=K ** -0.5), randn(g, N), randn(g, M, N, dtype=BF)
    y = B.csa_linear_fwd(B.LinearParams(M, K, N, activation="relu"), x, w, b, res)
    z = (x.float() @ w.float().t()).double() + b.double()
    want = z.clamp(min=0) + res.double()
    terms = x.double().norm() * w.double().norm() / (M * N) ** 0.5
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -8
    assert float((y.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) + 2.0 ** -12 * float(terms) * 6
    dx = B.csa_linear_bwd(B.LinearParams(M, N, K), x, None, w.t().contiguous().view(K, N), need_dw=False, need_db=False)[0]
    want = x.double() @ w.double().t()
    assert float((dx.double() - want).norm() / want.norm()) <= 2.0 ** -8


@pytest.mark.parametrize("M,K,N", [(64, 40, 128), (2048, 512, 1024), (1002, 33, 70), (16384, 256, 64)])
def test_linear_fp32_gradients_of_bf16_values_keep_their_bits(M, K, N):
    """dy of 1 + 2^-10 and -1 in turn along rows and columns: what is left of its sums is what bf16 would drop."""
    p = B.LinearParams(M, K, N, "bf16", "f32")
    sign = (torch.arange(M, device="cuda")[:, None] + torch.arange(N, device="cuda")) % 2
    dy = torch.where(sign == 0, 1 + 2.0 ** -10, -1.0)
    x, w = torch.ones(M, K, dtype=BF, device="cuda"), torch.ones(N, K, dtype=BF, device="cuda")
    dx, dw, db = B.csa_linear_bwd(p, dy, x, w)
    # every partial sum is a multiple of 2^-10 below 2^14: exact but for the one rounding
    assert torch.equal(dx, torch.full((M, K), N / 2 * 2.0 ** -10, device="cuda").to(BF))
    assert torch.equal(dw, torch.full((N, K), M / 2 * 2.0 ** -10, device="cuda").to(BF))
    assert torch.equal(db, torch.full((N,), M / 2 * 2.0 ** -10, device="cuda"))


@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_fp32_gradients_are_rounded_once(act):
    """With fp32 dy the bf16 gradients are as near the formula as its own rounding to bf16; dz's 2^-16, the activation's
    2^-19 and what the tensor core cuts off (below 2^-16 at these lengths) are beside that nothing: 1 % and 2^-15."""
    M, K, N = 3000, 264, 520
    g = gen(22)
    p = B.LinearParams(M, K, N, "bf16", "f32", act)
    x, w, z, dy = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF), randn(g, M, N, dtype=BF), randn(g, M, N)
    dx, dw, _ = B.csa_linear_bwd(p, dy, x, w, z if act != "none" else None)
    d = dy.double()
    if act == "silu":
        s = torch.sigmoid(z.double())
        d = d * s * (1 + z.double() * (1 - s))
    for got, want in ((dx, d @ w.double()), (dw, d.t() @ x.double())):
        best = float((want.to(BF).double() - want).norm())
        assert float((got.double() - want).norm()) <= 1.01 * best + 2.0 ** -15 * float(want.norm())


def test_linear_infinite_factors_of_fp32_gradients():
    """An infinite weight or x beside an fp32 dy: the infinity of the product's sign, as in a plain product."""
    g = gen(23)
    M, K, N = 40, 24, 16
    p = B.LinearParams(M, K, N, "bf16", "f32")
    x, w, dy = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF), randn(g, M, N)
    dy[:, 3] = torch.where(torch.arange(M, device="cuda") % 2 == 0, 1.0, -0.75)    # exact in bf16
    w[3, 5], x[7, 2] = float("inf"), float("-inf")
    dx, dw, _ = B.csa_linear_bwd(p, dy, x, w)
    assert torch.equal(dx[:, 5].float(), torch.where(dy[:, 3] > 0, float("inf"), float("-inf")))
    assert torch.equal(dw[:, 2].float(), torch.where(dy[7] > 0, float("-inf"), float("inf")))
    keep = [k for k in range(K) if k not in (2, 5)]
    assert bool(dx[:, keep].isfinite().all()) and bool(dw[:, keep].isfinite().all())


def same_kinds(got, want, what):
    """The same NaN, and infinities of the same sign, in the same places."""
    got, want = got.double(), want.double()
    assert torch.equal(got.isnan(), want.isnan()), what
    assert torch.equal(got.isinf(), want.isinf()), what
    at = want.isinf()
    assert torch.equal(got[at], want[at]), what


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("M", [1, 8, 9, 16, 40, 300])
def test_linear_infinities_are_those_of_plain_products(M, dtype, out):
    """Infinite values beside factors of either sign, 0 and infinite ones: the same answers whatever the number of rows."""
    K, N = 72, 40
    inf, t = float("inf"), DT[dtype]
    g = gen(30)
    x, w, dy = randn(g, M, K, dtype=t), randn(g, N, K, dtype=t), randn(g, M, N, dtype=DT[out])
    x[0, 3] = inf
    w[2, 3], w[5, 3], w[6, 3] = 0.0, inf, -inf
    if M > 1:
        x[M - 1, 70], x[M // 2, 9], x[M // 2, 11] = -inf, inf, -inf
        w[7, 9] = 0.0
        dy[1, 4], dy[M - 1, 4] = -inf, inf
        dy[1, 30] = float("nan")
    w[8, 1] = -inf
    x[0, 1] = 1.0 + 2.0 ** -7                                # its second part is 0
    y = B.csa_linear_fwd(B.LinearParams(M, K, N, dtype, out), x, w)
    same_kinds(y, x.double() @ w.double().t(), "y")
    dx, dw, db = B.csa_linear_bwd(B.LinearParams(M, K, N, dtype, out), dy, x, w)
    same_kinds(dx, dy.double() @ w.double(), "dx")
    same_kinds(dw, dy.double().t() @ x.double(), "dw")
    same_kinds(db, dy.double().sum(0), "db")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_relu_lets_no_infinite_gradient_pass(dtype):
    """Where z <= 0 the gradient is 0 for an infinite or undefined dy too."""
    M, K, N = 50, 24, 33
    g = gen(31)
    x, w, dy, z = (randn(g, *s, dtype=DT[dtype]) for s in ((M, K), (N, K), (M, N), (M, N)))
    z[3, 4], z[5, 6], z[7, 8], z[9, 10] = -1.0, 0.0, -2.0, 1.0
    p = B.LinearParams(M, K, N, dtype, activation="relu")
    dy[3, 4] = dy[5, 6] = dy[7, 8] = 0.0
    clean = B.csa_linear_bwd(p, dy, x, w, z)
    dy[3, 4], dy[5, 6], dy[7, 8] = float("inf"), float("-inf"), float("nan")
    for a, b in zip(clean, B.csa_linear_bwd(p, dy, x, w, z)):
        assert torch.equal(a, b)
    dy[9, 10] = float("inf")
    assert B.csa_linear_bwd(p, dy, x, w, z)[2][10] == float("inf")


def test_weights_and_positions_the_other_way_round_refused():
    """Contiguous tensors of the right number of values whose axes lie the other way round."""
    g = gen(40)
    x, w, dy = randn(g, 12, 32), randn(g, 24, 32), randn(g, 12, 24)
    p = B.LinearParams(12, 32, 24, "f32")
    y = B.csa_linear_fwd(p, x, w)
    assert torch.equal(B.csa_linear_fwd(p, x, w.flatten()), y)
    for bad in (w.t().contiguous(), w.view(48, 16)):
        with pytest.raises(ValueError, match="weight"):
            B.csa_linear_fwd(p, x, bad)
        with pytest.raises(ValueError, match="weight"):
            B.csa_linear_bwd(p, dy, x, bad)
    q = randn(g, 12, 2, 8)
    r = B.RopeParams(12, 2, 8, "f32", sections=[1, 1, 2])
    f = torch.ones(4, device="cuda", dtype=torch.float64)
    pos = torch.arange(36, device="cuda", dtype=torch.int32).view(3, 12)
    out = B.csa_rope(r, q, pos, f)
    assert torch.equal(B.csa_rope(r, q, pos.flatten(), f), out) and torch.equal(B.csa_rope(r, q, pos.view(3, 4, 3), f), out)
    with pytest.raises(ValueError, match="positions"):
        B.csa_rope(r, q, pos.t().contiguous(), f)
