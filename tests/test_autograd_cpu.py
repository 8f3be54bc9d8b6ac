"""The autograd forms of the projections, over plain stand-ins for the two kernels' calls: what autograd does with the
tensors they return needs no GPU."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def B(monkeypatch):
    from sparse_attention_indexer_tcgen05_gb300 import build
    build.build()
    from sparse_attention_indexer_tcgen05_gb300 import binding

    def fwd(p, x, weight, bias=None, residual=None, preact=None, **_):
        y = x.reshape(-1, x.shape[-1]) @ weight.t()
        y = y + bias if bias is not None else y
        return y + residual.reshape(y.shape) if residual is not None else y

    def bwd(p, dy, x, weight, preact=None, need_dx=True, need_dw=True, need_db=True, **_):
        dy = dy.reshape(-1, dy.shape[-1])
        return (dy @ weight if need_dx else None, dy.t() @ x.reshape(-1, x.shape[-1]) if need_dw else None,
                dy.sum(0) if need_db else None)

    monkeypatch.setattr(binding, "csa_linear_fwd", fwd)
    monkeypatch.setattr(binding, "csa_linear_bwd", bwd)
    return binding


def leaves(*shapes):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(*s, generator=g).requires_grad_(True) for s in shapes]


@pytest.mark.parametrize("shape", [(6, 5), (2, 3, 5)])
def test_the_same_gradient_handed_in_again(B, shape):
    """The caller's own gradient buffer is neither kept as a .grad nor written."""
    x, w, res = leaves((6, 4), (5, 4), shape)
    p = B.LinearParams(6, 4, 5, "f32")
    y = B.csa_linear(x, w, None, res, params=p)
    g = torch.ones(6, 5)
    for n in (1, 2, 3, 4):
        y.backward(g, retain_graph=True)
        assert torch.equal(g, torch.ones(6, 5))
        assert torch.equal(res.grad, torch.full(shape, float(n)))
        assert torch.allclose(w.grad, n * x.detach().sum(0).expand(5, 4), rtol=1e-6)
    assert res.grad.data_ptr() != g.data_ptr()


@pytest.mark.parametrize("shape", [(6, 5), (2, 3, 5)])
def test_two_residuals_of_a_sum_have_gradients_of_their_own(B, shape):
    x, w, r1, r2 = leaves((6, 4), (5, 4), shape, shape)
    p = B.LinearParams(6, 4, 5, "f32")
    y = B.csa_linear(x, w, None, r1, params=p) + B.csa_linear(x, w, None, r2, params=p)
    y.backward(torch.ones(6, 5))
    r1.grad.mul_(3)
    assert torch.equal(r2.grad, torch.ones(shape)) and torch.equal(r1.grad, torch.full(shape, 3.0))


def test_the_input_as_its_own_residual(B):
    x, w = leaves((6, 5), (5, 5))
    p = B.LinearParams(6, 5, 5, "f32")
    g = torch.randn(6, 5, generator=torch.Generator().manual_seed(2))
    kept = g.clone()
    B.csa_linear(x, w, None, x, params=p).backward(g)
    assert torch.equal(g, kept)
    assert torch.allclose(x.grad, g + g @ w.detach(), rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("shape", [(6, 5), (2, 3, 5)])
def test_a_gradient_off_the_16_byte_boundary_or_strided(B, shape):
    x, w, res = leaves((6, 4), (5, 4), shape)
    p = B.LinearParams(6, 4, 5, "f32")
    y = B.csa_linear(x, w, None, res, params=p)
    for g in (torch.arange(31.0)[1:].view(6, 5), torch.arange(30.0).view(5, 6).t(), torch.ones(1, 1).expand(6, 5)):
        res.grad = None
        y.backward(g, retain_graph=True)
        assert torch.equal(res.grad, g.reshape(shape))


def test_frequencies_that_ask_for_a_gradient_refused(B, monkeypatch):
    """The rotation has no gradient for them: silence would leave them as they are."""
    monkeypatch.setattr(B, "csa_rope", lambda p, x, positions, inv_freq, out=None: x.clone())
    r = B.RopeParams(3, 1, 4, "f32")
    x, pos, f = torch.ones(3, 1, 4, requires_grad=True), torch.zeros(1, 3, dtype=torch.int32), torch.ones(2, dtype=torch.float64)
    B.csa_rotary(x, pos, f, r).sum().backward()
    assert torch.equal(x.grad, torch.ones(3, 1, 4))
    y = B.csa_rotary(x, pos, f.requires_grad_(True), r)
    with pytest.raises(ValueError, match="inv_freq"):
        y.sum().backward()
