"""Evaluation with the autograd forms: the launches and the memory of the forward calls."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_vocab_loss_gpu import inputs  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402


def launches(call):
    n = B.csa_kernel_launches()
    out = call()
    return B.csa_kernel_launches() - n, out


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("M,K,V,slots", [(300, 512, 16384, 0), (300, 64, 1000, 4), (5, 64, 1000, 0)])
def test_losses_of_leaves_that_ask_for_gradients(off, M, K, V, slots):
    t = inputs(M, K, V, slots=slots)
    x, w = t["x"].requires_grad_(True), t["weight"].requires_grad_(True)
    p = B.VocabLossParams(M, K, V, slots=slots, labels_64=True, ids_64=True)
    targets = [t[k] for k in ("labels", "teacher_ids", "teacher_logits", "teacher_lse")]
    want, loss = launches(lambda: B.csa_vocab_loss_fwd(p, x.detach(), w.detach(), *targets))
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with off():
        n, got = launches(lambda: B.csa_vocab_loss(x, w, *targets, params=p))
    assert n == want and torch.equal(got, loss)
    assert torch.cuda.max_memory_allocated() - before <= p.fwd_workspace_bytes + 4096   # nothing of dW's or dx's size
