"""The autograd forms of layer norm and the vocabulary's losses, over plain stand-ins for the kernels' calls."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def B(monkeypatch):
    from sparse_attention_indexer_tcgen05_gb300 import build
    build.build()
    from sparse_attention_indexer_tcgen05_gb300 import binding

    def norm_fwd(p, x, weight=None, bias=None, out=None, stats=None):
        d = x.reshape(-1, x.shape[-1])
        mean, var = d.mean(1), d.var(1, unbiased=False)
        if stats is not None:
            stats[0], stats[1] = mean, (var + p.c.eps) ** -0.5
        y = (d - mean[:, None]) * (var[:, None] + p.c.eps) ** -0.5
        return y * (1 if weight is None else weight) + (0 if bias is None else bias)

    def norm_bwd(p, dy, x, weight=None, stats=None, need_dx=True, need_dweight=True, need_dbias=True, **_):
        d, dy = x.reshape(-1, x.shape[-1]), dy.reshape(-1, x.shape[-1])
        h = (d - stats[0][:, None]) * stats[1][:, None]
        a = dy * (1 if weight is None else weight)
        dx = stats[1][:, None] * (a - a.mean(1, keepdim=True) - h * (a * h).mean(1, keepdim=True))
        return dx if need_dx else None, (dy * h).sum(0) if need_dweight else None, dy.sum(0) if need_dbias else None

    def loss_fwd(p, x, weight, labels=None, *_, **__):
        return torch.nn.functional.cross_entropy(x.reshape(-1, x.shape[-1]) @ weight.t(), labels)

    def loss_bwd(p, x, weight, labels=None, *_, need_dx=True, need_dw=True, **__):
        with torch.enable_grad():
            x, w = x.detach().reshape(-1, x.shape[-1]).requires_grad_(True), weight.detach().requires_grad_(True)
            loss = loss_fwd(p, x, w, labels)
            loss.backward()
        binding.made = (need_dx, need_dw)
        return loss.detach(), x.grad if need_dx else None, w.grad if need_dw else None

    for name, f in (("csa_layernorm_fwd", norm_fwd), ("csa_layernorm_bwd", norm_bwd), ("csa_vocab_loss_fwd", loss_fwd), ("csa_vocab_loss_bwd", loss_bwd)):
        monkeypatch.setattr(binding, name, f)
    return binding


def leaves(*shapes):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(*s, generator=g).requires_grad_(True) for s in shapes]


@pytest.mark.parametrize("with_params", [True, False])
def test_norm_gradients(B, with_params):
    x, w, b = leaves((2, 3, 8), (8,), (8,))
    p = B.LayerNormParams(6, 8, "f32", eps=1e-5)
    args = (w, b) if with_params else (None, None)
    g = torch.randn(2, 3, 8, generator=torch.Generator().manual_seed(2))
    B.csa_layernorm(x, *args, params=p).backward(g)
    ref = [t.detach().clone().requires_grad_(True) for t in (x, w, b)]
    torch.nn.functional.layer_norm(ref[0], (8,), *(ref[1:] if with_params else (None, None)), eps=1e-5).backward(g)
    for got, want in zip((x, w, b), ref):
        assert (got.grad is None) == (want.grad is None)
        if got.grad is not None:
            assert torch.allclose(got.grad, want.grad, atol=1e-5)


def test_loss_gradients_are_scaled_and_backward_may_run_twice(B):
    x, w = leaves((2, 3, 8), (11, 8))
    labels = torch.tensor([1, 2, 3, 4, 5, 10])
    p = B.VocabLossParams(6, 8, 11, "f32", labels_64=True)
    loss = B.csa_vocab_loss(x, w, labels, params=p)
    (3 * loss).backward(retain_graph=True)
    first = [x.grad.clone(), w.grad.clone()]
    (3 * loss).backward()
    ref = [t.detach().clone().requires_grad_(True) for t in (x, w)]
    (3 * torch.nn.functional.cross_entropy(ref[0].view(6, 8) @ ref[1].t(), labels)).backward()
    for got, once, want in zip((x, w), first, ref):
        assert once.shape == want.grad.shape and torch.allclose(once, want.grad, atol=1e-6) and torch.allclose(got.grad, 2 * once)


def test_only_the_gradients_that_are_needed_are_made(B):
    x, w = leaves((6, 8), (11, 8))
    labels = torch.tensor([1, 2, 3, 4, 5, 10])
    p = B.VocabLossParams(6, 8, 11, "f32", labels_64=True)
    B.csa_vocab_loss(x, w.detach(), labels, params=p).backward()
    assert B.made == (True, False) and x.grad is not None
    B.made = None
    B.csa_vocab_loss(x.detach(), w.detach(), labels, params=p)
    assert B.made is None     # the loss alone
