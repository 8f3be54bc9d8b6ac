"""Layer norm and the vocabulary's losses used together: VocabTrainer, and the keys' norm in IndexerTrainer."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_indexer_trainer_gpu import HIDDEN, SECTIONS, call, case, trainer  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402
    from sparse_attention_indexer_tcgen05_gb300 import indexer, vocab  # noqa: E402

M, K, V, SLOTS = 300, 136, 1003, 9


def setup(dtype="f32", slots=SLOTS, labels=True, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    weights = [(rand(V, K) * 2 * K ** -0.5).to(dt), 1 + 0.1 * rand(K), 0.1 * rand(K)]
    targets = {}
    if labels:
        at = torch.randint(0, V, (M,), generator=g, device="cuda")
        targets["labels"] = torch.where(torch.rand(M, generator=g, device="cuda") < 0.2, -100, at)
    if slots:
        targets["teacher_ids"] = torch.rand(M, V, generator=g, device="cuda").topk(slots, 1).indices
        targets["teacher_logits"] = 2 * rand(M, slots)
        targets["teacher_lse"] = targets["teacher_logits"].logsumexp(1) + 0.1
    p = B.VocabLossParams(M, K, V, dtype, slots=slots, label_weight=0.6, teacher_weight=0.4, labels_64=True, ids_64=True, **kw)
    return p, weights, (rand(M, K) * 3 + 0.5).to(dt), targets


def make(p, weights, **kw):
    return vocab.VocabTrainer(p, *[w.clone() for w in weights], **{**dict(lr=1e-3, weight_decay=0.01), **kw})


@pytest.mark.parametrize("dtype,slots,labels", [("f32", SLOTS, True), ("bf16", 0, True), ("bf16", SLOTS, False)])
def test_gradients_equal_autograds(dtype, slots, labels):
    """The trainer's explicit chain and the autograd functions make the same calls: the same bits."""
    p, weights, x, targets = setup(dtype, slots, labels)
    t = make(p, weights)
    loss, dx, grads = t.gradients(x, **targets)
    leaves = [w.clone().requires_grad_(True) for w in weights]
    hidden = x.clone().requires_grad_(True)
    ref = B.csa_vocab_loss(B.csa_layernorm(hidden, *leaves[1:], params=t.norm), leaves[0], **targets, params=p)
    ref.backward()
    assert torch.equal(loss, ref) and torch.equal(dx, hidden.grad)
    assert all(torch.equal(g, leaf.grad) for g, leaf in zip(grads, leaves))
    assert torch.equal(t.evaluate(x, **targets), ref)
    B.csa_check_device_status()


def test_gradients_by_differences_and_a_step():
    """Along random directions of the hidden states and of each weight, against differences of the loss in 64 bits; then the
    first AdamW step of those gradients, -lr g / (|g| + eps) - lr wd w."""
    p, weights, x, targets = setup(alpha=0.8)
    t = make(p, weights, adam_eps=1e-12)
    _, dx, grads = t.gradients(x, **targets)
    dx, grads = dx.clone(), [g.clone() for g in grads]

    def loss(x, w, a, b):
        d = x - x.mean(1, keepdim=True)
        z = 0.8 * ((d * ((d * d).mean(1, keepdim=True) + 1e-5) ** -0.5 * a + b) @ w.t())
        logp = z.log_softmax(1)
        held = targets["labels"] >= 0
        first = -logp.gather(1, targets["labels"].clamp(min=0)[:, None])[held].sum() / held.sum()
        s = (targets["teacher_logits"].double() - targets["teacher_lse"].double()[:, None]).exp()
        return 0.6 * first + 0.4 * (s * (s.log() - logp.gather(1, targets["teacher_ids"]))).sum() / M

    at = [x.double(), *[w.double() for w in weights]]
    gen = torch.Generator(device="cuda").manual_seed(1)
    for i, g in enumerate([dx, *grads]):
        way, e = torch.randn(g.shape, generator=gen, device="cuda", dtype=torch.float64), 1e-5
        up, down = (float(loss(*[v + s * e * way if j == i else v for j, v in enumerate(at)])) for s in (1, -1))
        slope = float((g.double() * way).sum())
        # differences: e^2 times third derivatives and 64-bit rounding over e; gradients: some 300 fp32 roundings of their terms
        assert abs(slope - (up - down) / (2 * e)) <= 300 * 2.0 ** -24 * float((g.double() * way).abs().sum()) + 1e-6, i
    t.step(x, **targets)
    for w0, w1, g in zip(weights, (t.weight, t.norm_weight, t.norm_bias), grads):
        g = g.double()
        want = w0.double() - 1e-3 * 0.01 * w0.double() - 1e-3 * g / (g.abs() + 1e-12)
        keep = g.abs() > 1e-6 * g.abs().max()   # far above eps
        assert bool(((w1.double() - want).abs() <= 2.0 ** -20 * 1e-3 + 2.0 ** -22 * w0.double().abs())[keep].all())
    assert int(t.step_count) == 1


@pytest.mark.parametrize("eight_bit", [False, True])
def test_captured_steps_equal_eager_ones(eight_bit):
    p, weights, x, targets = setup("bf16", piece_rows=128)
    a, b = make(p, weights, eight_bit=eight_bit), make(p, weights, eight_bit=eight_bit)
    for t in (a, b):
        t.step(x, **targets)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step(x, **targets)
    for _ in range(3):
        a.step(x, **targets)
        graph.replay()
    assert int(a.step_count) == int(b.step_count) == 4 and torch.equal(a.loss, b.loss) and torch.equal(a.dx, b.dx)
    assert all(torch.equal(u, v) for u, v in zip((a.weight, a.norm_weight, a.norm_bias), (b.weight, b.norm_weight, b.norm_bias)))
    assert not torch.equal(a.weight, weights[0])


def test_a_step_with_found_inf_leaves_everything():
    p, weights, x, targets = setup("bf16")
    t = make(p, weights)
    t.step(x, found_inf=torch.ones(1, device="cuda"), **targets)
    assert int(t.step_count) == 0 and all(torch.equal(u, v) for u, v in zip((t.weight, t.norm_weight, t.norm_bias), weights))


def test_without_a_bias_and_wrong_weights():
    p, weights, x, targets = setup()
    t = vocab.VocabTrainer(p, weights[0].clone(), weights[1].clone())
    t.step(x, **targets)
    assert len(t.grads) == 2
    for bad in ((weights[0][:-1], weights[1], weights[2]), (weights[0], weights[1][:-1], None), (weights[0], weights[1], weights[2].bfloat16())):
        with pytest.raises(ValueError):
            vocab.VocabTrainer(p, *bad)
    with pytest.raises(ValueError):
        vocab.VocabTrainer(B.VocabLossParams(M, K, V, "f32", slots=SLOTS, x_stride=K + 8), *weights)


# ------------------------------------------------------------------ the keys' norm of the indexer

def key_norm(dtype=None):
    g = torch.Generator(device="cuda").manual_seed(3)
    pair = (1 + 0.1 * torch.randn(128, generator=g, device="cuda"), 0.1 * torch.randn(128, generator=g, device="cuda"))
    return pair if dtype is None else tuple(t.to(dtype) for t in pair)


@pytest.mark.parametrize("layout,dtype,param", [("bshd", "bf16", torch.float32), ("sbhd", "f32", torch.float32), ("thd", "bf16", torch.bfloat16)])
def test_indexer_with_a_key_norm_equals_autograds(layout, dtype, param):
    d, weights, i = case(layout, dtype)
    t = trainer(d, weights, key_norm=[w.clone() for w in key_norm(param)])
    loss, grads = t.gradients(*call(d, i))
    assert len(grads) == 5
    leaves = [w.clone().requires_grad_(True) for w in (*weights, *key_norm(param))]
    q = B.csa_rotary(B.csa_linear(i["x"], leaves[0], params=t.p_q).view(-1, 64, 128), i["positions"], i["inv_freq"], t.r_q)
    k = B.csa_layernorm(B.csa_linear(i["x_c"], leaves[1], params=t.p_k), leaves[3], leaves[4], params=t.norm)
    k = B.csa_rotary(k, i["key_positions"], i["inv_freq"], t.r_k)
    w = B.csa_linear(i["x"], leaves[2], params=t.p_w)
    _, ref = B.csa_indexer_loss(q, w, k, *d.teacher_side, d.params)
    ref.backward()
    # dk_idx is accumulated by atomics: its order, and so the last bits of what follows from it, may change
    ref = ref.detach()
    assert abs(float(loss) - float(ref)) <= 1e-6 * abs(float(ref))
    for g, leaf in zip(grads, leaves):
        err = float((g.double() - leaf.grad.double()).norm() / leaf.grad.double().norm())
        assert err <= (2.0 ** -8 if dtype == "bf16" else 1e-5), err
    # a step of 1e-3 is less than half of a bf16 spacing at 1 (2^-8): the master copy shows it
    held = [m if m is not None else w for m, w in zip(t.tensors.tensors["master"], t.tensors.tensors["param"])]
    before = [w.clone() for w in held]
    t.step(*call(d, i))
    assert len(held) == 5 and all(not torch.equal(a, b) for a, b in zip(before, held)) and int(t.step_count) == 1
    B.csa_check_device_status()


def test_indexer_without_a_key_norm_is_as_before():
    d, weights, i = case("bshd", "f32")
    t = trainer(d, weights)
    assert t.norm is None and len(t.grads) == 3 and HIDDEN and SECTIONS
    with pytest.raises(ValueError, match="key_norm"):
        indexer.IndexerTrainer(d.params, *weights, key_norm=(torch.ones(64, device="cuda"), None))
