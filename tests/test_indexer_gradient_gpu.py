"""The trainer's gradients against differences of its loss, along directions in which the loss does move."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from sparse_attention_indexer_tcgen05_gb300 import synth  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import indexer, workload  # noqa: E402

HIDDEN = 192


@pytest.mark.parametrize("layout", ["bshd", "thd"])
def test_gradients_against_differences_of_the_loss(layout):
    """v = sign(g) times random sizes: <g, v> is a mean of |g| and not of signs that cancel, so that a gradient of 0, of the
    other sign or half as large is far off.  Every key is selected (topk above their number), so that the loss has no
    jumps; it is smooth but for the kinks of the scores' ReLU, which a step crosses in proportion to its length.  The step
    moves the loss by about 0.5 % each way: the loss's own rounding (2^-20 of it: sums of fp32 rows) is 1e-4 of that; the
    second-order terms of the two sides cancel, and the kinks leave the step's own order: 3 %."""
    kw = dict(batch=2, seqlen=200) if layout == "bshd" else dict(batch=1, seqlen=400)
    cfg = synth.Config(name="gradient", layout=layout, dtype="f32", ratio=4, heads=64, head_dim=64, idx_heads=64, idx_dim=128,
                       topk=128, window=16, seed=3, **kw)
    d = workload.to_device(synth.generate(cfg))
    p, g = d.params, torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s, scale=1.0: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
    weights = [randn(n, HIDDEN, scale=HIDDEN ** -0.5) for n in (64 * 128, 128, 64)]
    x, x_c = randn(p.rows, HIDDEN), randn(p.compressed_rows, HIDDEN)
    pos = [torch.randint(0, 4000, (3, n), generator=g, device="cuda", dtype=torch.int32) for n in (p.rows, p.compressed_rows)]
    freq = 10000.0 ** (-torch.arange(16, dtype=torch.float64, device="cuda") / 16)

    def run(w):
        t = indexer.IndexerTrainer(p, *w, rot_dim=32, sections=[8, 4, 4], weight_scale=0.0884)
        loss, grads = t.gradients(x, x_c, *d.teacher_side, *pos, freq)
        return float(loss), [q.double() for q in grads]

    loss, grads = run(weights)
    assert loss > 0
    for which, name in enumerate(("wq", "wk", "ww")):
        v = torch.sign(grads[which]) * torch.rand(weights[which].shape, generator=g, device="cuda")
        got = float((grads[which] * v).sum())
        h = 0.005 * loss / got
        side = [run([w + (s * h * v).float() if n == which else w for n, w in enumerate(weights)])[0] for s in (1, -1)]
        want = (side[0] - side[1]) / (2 * h)
        assert abs(want) * h >= 100 * 2.0 ** -20 * loss, name              # the difference is no rounding
        assert abs(got - want) <= 0.03 * abs(want), (name, got, want)
