"""The operators around the step used together: hidden states to updated indexer weights (IndexerTrainer)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_attention_indexer_tcgen05_gb300 import synth  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402
    from sparse_attention_indexer_tcgen05_gb300 import indexer, workload  # noqa: E402

HIDDEN = 192
SECTIONS = [8, 4, 4]


def case(layout, dtype, seed=5):
    kw = dict(batch=2, seqlen=200) if layout != "thd" else dict(batch=1, seqlen=400)
    cfg = synth.Config(name="trainer", layout=layout, dtype=dtype, ratio=4, heads=64, head_dim=64, idx_heads=64, idx_dim=128,
                       topk=24, window=16, seed=seed, **kw)
    d = workload.to_device(synth.generate(cfg))
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = d.params
    randn = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(p.value_dtype)  # noqa: E731
    weights = [randn(n, HIDDEN, scale=HIDDEN ** -0.5) for n in (64 * 128, 128, 64)]
    inputs = dict(x=randn(p.rows, HIDDEN), x_c=randn(p.compressed_rows, HIDDEN),
                  positions=torch.randint(0, 4000, (3, p.rows), generator=g, device="cuda", dtype=torch.int32),
                  key_positions=torch.randint(0, 4000, (3, p.compressed_rows), generator=g, device="cuda", dtype=torch.int32),
                  inv_freq=10000.0 ** (-torch.arange(16, dtype=torch.float64, device="cuda") / 16))
    return d, weights, inputs


def trainer(d, weights, **kw):
    args = dict(rot_dim=32, sections=SECTIONS, weight_scale=0.0884, lr=1e-3, weight_decay=0.01)
    args.update(kw)
    return indexer.IndexerTrainer(d.params, *[w.clone() for w in weights], **args)


def call(d, i):
    return (i["x"], i["x_c"], *d.teacher_side, i["positions"], i["key_positions"], i["inv_freq"])


@pytest.mark.parametrize("layout,dtype", [("bshd", "bf16"), ("sbhd", "f32"), ("thd", "bf16")])
def test_gradients_equal_autograds(layout, dtype):
    """The trainer's explicit chain and the autograd functions make the same calls: the same bits."""
    d, weights, i = case(layout, dtype)
    t = trainer(d, weights)
    loss, grads = t.gradients(*call(d, i))
    leaves = [w.clone().requires_grad_(True) for w in weights]
    q = B.csa_rotary(B.csa_linear(i["x"], leaves[0], params=t.p_q).view(-1, 64, 128), i["positions"], i["inv_freq"], t.r_q)
    k = B.csa_rotary(B.csa_linear(i["x_c"], leaves[1], params=t.p_k), i["key_positions"], i["inv_freq"], t.r_k)
    w = B.csa_linear(i["x"], leaves[2], params=t.p_w)
    _, ref = B.csa_indexer_loss(q, w, k, *d.teacher_side, d.params)
    ref.backward()
    # dk_idx is accumulated by atomics: its order, and so the last bits of what follows from it, may change
    assert abs(float(loss) - float(ref)) <= 1e-6 * abs(float(ref))
    for g, leaf in zip(grads, leaves):
        err = float((g.double() - leaf.grad.double()).norm() / leaf.grad.double().norm())
        assert err <= (2.0 ** -8 if dtype == "bf16" else 1e-5), err
    B.csa_check_device_status()


def test_projections_against_64_bits():
    d, weights, i = case("bshd", "f32")
    q, w, k = trainer(d, weights).project(i["x"], i["x_c"], i["positions"], i["key_positions"], i["inv_freq"])
    axis = torch.tensor([0] * 8 + [1] * 4 + [2] * 4, device="cuda")

    def rope(y, pos):
        ang = pos.t().double()[:, axis] * i["inv_freq"]
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        a, b = y[..., :16], y[..., 16:32]
        return torch.cat([a * c - b * s, a * s + b * c, y[..., 32:]], -1)

    x, xc = i["x"].double(), i["x_c"].double()
    wq, wk, ww = (t.double() for t in weights)
    for got, want, terms in (
            (q, rope((x @ wq.t()).view(-1, 64, 128), i["positions"]), (x.abs() @ wq.abs().t()).view(-1, 64, 128)),
            (k[:, None], rope((xc @ wk.t())[:, None], i["key_positions"]), (xc.abs() @ wk.abs().t())[:, None]),
            (w, 0.0884 * (x @ ww.t()), x.abs() @ ww.abs().t())):
        # HIDDEN additions and the parts of the products (2^-23 of the terms each), then a rotation that mixes two
        # values of a head with factors good to 2^-21
        tol = (HIDDEN + 8) * 2.0 ** -23 * 2 * terms.amax(-1, keepdim=True) + 2.0 ** -20 * want.abs().amax(-1, keepdim=True)
        assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("eight_bit", [False, True])
def test_loss_gradient_by_differences_and_a_step(eight_bit):
    """The directional derivative of the loss along a random direction of wq and ww, by central differences in fp32
    values, and the first AdamW step of those gradients, -lr g / (|g| + eps) - lr wd w."""
    d, weights, i = case("bshd", "f32", seed=9)
    t = trainer(d, weights, eps=1e-12, eight_bit=eight_bit)
    _, grads = t.gradients(*call(d, i))
    grads = [g.clone() for g in grads]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for which in (0, 2):
        v = torch.randn(weights[which].shape, generator=gen, device="cuda") * weights[which].abs().mean()
        h = 1e-3
        side = []
        for s in (1, -1):
            moved = [w + s * h * v if n == which else w for n, w in enumerate(weights)]
            side.append(float(trainer(d, moved).gradients(*call(d, i))[0]))
        want, got = (side[0] - side[1]) / (2 * h), float((grads[which].double() * v.double()).sum())
        # the selection is held by the sampled rows' margins only: a few rows may swap a key, each of them worth its
        # share of the loss; the rest is third order in h and the loss's own rounding (2^-24 / h of it)
        scale = float((grads[which].double().abs() * v.double().abs()).sum())
        assert abs(got - want) <= 0.02 * scale + 2.0 ** -20 / h * abs(side[0]), (which, got, want)
    t.step(*call(d, i))
    for w0, w1, g in zip(weights, (t.wq, t.wk, t.ww), grads):
        g = g.double()
        want = w0.double() - 1e-3 * 0.01 * w0.double() - 1e-3 * g / (g.abs() + 1e-12)
        # where |g| is far above eps and dk's order left its sign alone
        keep = g.abs() > 1e-4 * g.abs().max()
        assert bool(((w1.double() - want).abs() <= 2.0 ** -20 * 1e-3 + 2.0 ** -22 * w0.double().abs())[keep].all())
    assert int(t.step_count) == 1


def test_captured_steps_equal_eager_ones():
    """Steps replayed from a graph leave what eager steps leave (dk's atomics aside)."""
    d, weights, i = case("bshd", "bf16", seed=11)
    a, b = trainer(d, weights, eight_bit=False), trainer(d, weights, eight_bit=False)
    for t in (a, b):
        t.step(*call(d, i))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step(*call(d, i))
    for _ in range(3):
        a.step(*call(d, i))
        graph.replay()
    torch.cuda.synchronize()
    assert int(a.step_count) == int(b.step_count) == 4
    assert abs(float(a.loss) - float(b.loss)) <= 1e-3 * abs(float(a.loss))
    for wa, wb, w0 in zip((a.wq, a.wk, a.ww), (b.wq, b.wk, b.ww), weights):
        moved = float((wa.double() - w0.double()).norm())
        assert moved > 0 and float((wa.double() - wb.double()).norm()) <= 0.05 * moved
    B.csa_check_device_status()


def test_a_step_with_found_inf_leaves_everything():
    """Two steps of which the second is skipped equal the first alone, the step count included."""
    d, weights, i = case("bshd", "bf16", seed=13)
    t = trainer(d, weights, eight_bit=True)
    found = torch.zeros(1, device="cuda")
    t.step(*call(d, i), found_inf=found)
    kept = [x.clone().view(torch.uint8) for name, c in t.tensors.tensors.items() if name != "grad" for x in c]
    assert int(t.step_count) == 1
    found.fill_(float("inf"))
    t.step(*call(d, i), found_inf=found)
    after = [x.view(torch.uint8) for name, c in t.tensors.tensors.items() if name != "grad" for x in c]
    assert int(t.step_count) == 1 and all(torch.equal(a, b) for a, b in zip(kept, after))
    found.zero_()
    t.step(*call(d, i), found_inf=found)
    assert int(t.step_count) == 2 and not torch.equal(kept[0], t.wq.view(torch.uint8))


def test_wrong_weights_refused():
    d, weights, _ = case("bshd", "bf16")
    with pytest.raises(ValueError, match="wk"):
        indexer.IndexerTrainer(d.params, weights[0], weights[1][:64], weights[2])
    with pytest.raises(ValueError, match="ww"):
        indexer.IndexerTrainer(d.params, weights[0], weights[1], weights[2].float())
