"""Which targets a call of the vocabulary's losses takes, on a machine without a GPU: a call that passes the checks of its targets goes
on to that of its workspace."""
import pytest

from test_losses_norm_abi_cpu import B, _no_gpu, addr, run, vocab  # noqa: F401

INVALID, WORKSPACE = 1, 4


@pytest.mark.parametrize("back", [True, False])
def test_either_target_may_be_left_out(B, back):  # noqa: F811
    p = vocab(B)
    call = lambda **kw: run(B, p, back, n=0, **kw)  # noqa: E731
    assert call() == WORKSPACE and call(labels=None) == WORKSPACE and call(lse=None) == WORKSPACE
    assert call(ids=None, logits=None, lse=None) == WORKSPACE
    for gone in (("ids",), ("logits",), ("ids", "lse"), ("logits", "lse"), ("ids", "logits"), ("labels", "ids", "logits"),
                 ("labels", "ids", "logits", "lse"), ("labels", "ids"), ("labels", "logits")):
        assert call(**{k: None for k in gone}) == INVALID, gone
