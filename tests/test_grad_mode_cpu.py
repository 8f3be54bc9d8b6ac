"""The autograd forms where autograd is off: nothing is made or kept for a backward pass, whatever the leaves ask for."""
import pytest

torch = pytest.importorskip("torch")

from test_losses_norm_autograd_cpu import B, leaves  # noqa: E402, F401

OFF = [torch.no_grad, torch.inference_mode]
LABELS = torch.tensor([1, 2, 3, 4, 5, 10])


@pytest.mark.parametrize("off", OFF)
@pytest.mark.parametrize("form", ["csa_vocab_loss", "apply"])
def test_losses_make_no_gradients(B, off, form):  # noqa: F811
    x, w = leaves((6, 8), (11, 8))
    p = B.VocabLossParams(6, 8, 11, "f32", labels_64=True)
    call = {"csa_vocab_loss": lambda *t: B.csa_vocab_loss(*t, LABELS, params=p),
            "apply": lambda *t: B.CSAVocabLoss.apply(*t, LABELS, None, None, None, p)}[form]
    B.made = None
    for leaf in ((x, w), (x.detach(), w), (x, w.detach())):
        with off():
            loss = call(*leaf)
        assert B.made is None and not loss.requires_grad
    with off():
        with torch.inference_mode(False), torch.enable_grad():   # on again within
            call(x, w.detach()).backward()
    assert B.made == (True, False) and x.grad is not None and w.grad is None


@pytest.mark.parametrize("off", OFF)
@pytest.mark.parametrize("form", ["csa_layernorm", "apply"])
def test_the_norm_keeps_no_statistics(B, monkeypatch, off, form):  # noqa: F811
    x, w, b = leaves((6, 8), (8,), (8,))
    p = B.LayerNormParams(6, 8, "f32")
    call = {"csa_layernorm": lambda: B.csa_layernorm(x, w, b, params=p), "apply": lambda: B.CSALayerNorm.apply(x, w, b, p)}[form]
    plain, kept = B.csa_layernorm_fwd, []

    def fwd(*args, stats=None, **kw):
        kept.append(stats)
        return plain(*args, stats=stats, **kw)

    monkeypatch.setattr(B, "csa_layernorm_fwd", fwd)
    with off():
        y = call()
    assert kept == [None] and not y.requires_grad
    z = call()
    assert kept[1] is not None and z.requires_grad and torch.equal(z, y)


@pytest.mark.parametrize("off", OFF)
@pytest.mark.parametrize("form", ["csa_linear", "apply"])
def test_a_projection_keeps_no_z(B, monkeypatch, off, form):  # noqa: F811
    x, w, b = leaves((6, 4), (5, 4), (5,))
    p = B.LinearParams(6, 4, 5, "f32", activation="silu")
    call = {"csa_linear": lambda: B.csa_linear(x, w, b, params=p), "apply": lambda: B.CSALinear.apply(x, w, b, None, p)}[form]
    kept = []

    def fwd(p, x, weight, bias=None, residual=None, preact=None, **_):
        kept.append(preact)
        return torch.nn.functional.silu(x @ weight.t() + bias)

    monkeypatch.setattr(B, "csa_linear_fwd", fwd)
    with off():
        y = call()
    assert kept == [None] and not y.requires_grad
    z = call()
    assert kept[1] is not None and z.requires_grad and torch.equal(z, y)
