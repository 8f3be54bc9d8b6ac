"""Layer norm and the vocabulary's losses on a machine without a GPU: sizes, refusals and fault injection; no compute call gets
past the host checks."""
import ctypes

import pytest

BIG = 1 << 50


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_tcgen05_gb300 import build
    build.build()
    from sparse_attention_indexer_tcgen05_gb300 import binding
    return binding


@pytest.fixture(autouse=True)
def _no_gpu():
    """These tests hand made-up device addresses to the library."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("passes made-up device addresses: run only where no GPU exists")


def addr(k):
    return 0x100000 * k


# ------------------------------------------------------------------ layer norm

def norm(B, **kw):
    return B.LayerNormParams(**{**dict(rows=100, cols=64), **kw})


def norm_fwd(B, p, x=addr(1), w=addr(2), b=addr(3), y=addr(4), stats=addr(5)):
    return B._lib.csa_layernorm_fwd(p.ref, x, w, b, y, stats, None)


def norm_bwd(B, p, dy=addr(1), x=addr(2), w=addr(3), stats=addr(4), dx=addr(5), dw=addr(6), db=addr(7), ws=addr(8), n=BIG):
    return B._lib.csa_layernorm_bwd(p.ref, dy, x, w, stats, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("field,value,status", [
    ("dtype", 5, 1), ("param_dtype", -1, 1), ("cols", 0, 1), ("rows", -1, 1), ("eps", -1.0, 1), ("eps", float("nan"), 1),
    ("x_stride", 63, 1), ("dy_stride", 63, 1), ("rows", 1 << 31, 2), ("cols", 0x7fff0001, 2), ("x_stride", 1 << 37, 2)])
def test_norm_params_refused(B, field, value, status):
    p = norm(B)
    setattr(p.c, field, value)
    assert p.bwd_workspace_bytes == 0
    assert norm_fwd(B, p) == status and norm_bwd(B, p) == status


def test_norm_pointers_refused(B):
    p = norm(B)
    assert norm_fwd(B, p, x=None) == 1 and norm_fwd(B, p, y=None) == 1 and norm_fwd(B, p, x=addr(1) + 8) == 3
    assert norm_fwd(B, p, stats=addr(5) + 2) == 3 and norm_fwd(B, p, w=addr(2) + 4) == 3
    assert norm_fwd(B, p, y=addr(2)) == 1 and norm_fwd(B, p, stats=addr(4)) == 1
    assert norm_fwd(B, norm(B, x_stride=72), y=addr(1)) == 1       # in place with another stride
    assert norm_bwd(B, p, dy=None) == 1 and norm_bwd(B, p, x=None) == 1 and norm_bwd(B, p, stats=None) == 1
    assert norm_bwd(B, p, ws=None) == 4 and norm_bwd(B, p, n=p.bwd_workspace_bytes - 1) == 4
    assert norm_bwd(B, p, dw=addr(5)) == 1 and norm_bwd(B, p, db=addr(6)) == 1 and norm_bwd(B, p, dx=addr(4)) == 1
    assert norm_bwd(B, p, dw=addr(2)) == 1 and norm_bwd(B, p, db=addr(1)) == 1
    assert norm_bwd(B, norm(B, dy_stride=72), dx=addr(1)) == 1 and norm_bwd(B, norm(B, x_stride=72), dx=addr(2)) == 1
    assert B._lib.csa_layernorm_fwd(None, addr(1), None, None, addr(2), None, None) == 1


def test_norm_workspace_grows_with_columns(B):
    assert norm(B, rows=0).bwd_workspace_bytes == 0
    sizes = [norm(B, rows=4096, cols=n).bwd_workspace_bytes for n in (1, 128, 129, 1024, 16384, 16385, 1 << 20)]
    assert all(s > 0 for s in sizes) and norm(B, rows=1, cols=128).bwd_workspace_bytes >= 1024


# ------------------------------------------------------------------ losses of a vocabulary

def vocab(B, **kw):
    return B.VocabLossParams(**{**dict(rows=100, features=64, vocab=1000, slots=4), **kw})


def run(B, p, back=True, x=addr(1), w=addr(2), labels=addr(3), ids=addr(4), logits=addr(5), lse=addr(6), loss=addr(7), rows=addr(8),
        dx=addr(9), dw=addr(10), ws=addr(11), n=BIG):
    t = B.csa_vocab_targets(labels, ids, logits, lse)
    if back:
        return B._lib.csa_vocab_loss_bwd(p.ref, x, w, ctypes.byref(t), loss, rows, dx, dw, ws, n, None)
    return B._lib.csa_vocab_loss_fwd(p.ref, x, w, ctypes.byref(t), loss, rows, ws, n, None)


@pytest.mark.parametrize("field,value,status", [
    ("dtype", 2, 1), ("features", 0, 1), ("vocab", 0, 1), ("slots", -1, 1), ("rows", -1, 1), ("piece_rows", -1, 1), ("labels_64", 2, 1),
    ("ids_64", -1, 1), ("reduction", 2, 1), ("alpha", 0.0, 1), ("alpha", float("inf"), 1), ("label_weight", -0.5, 1),
    ("teacher_weight", float("nan"), 1), ("x_stride", 63, 1), ("slots", 1025, 2), ("rows", 1 << 31, 2), ("vocab", 0x7fff0001, 2),
    ("features", 0x7fff0001, 2), ("x_stride", 1 << 37, 2)])
def test_vocab_params_refused(B, field, value, status):
    p = vocab(B)
    setattr(p.c, field, value)
    assert p.fwd_workspace_bytes == 0 and p.bwd_workspace_bytes == 0
    assert run(B, p) == status and run(B, p, back=False) == status


@pytest.mark.parametrize("back", [True, False])
def test_vocab_pointers_refused(B, back):
    p = vocab(B)
    call = lambda **kw: run(B, p, back, **kw)  # noqa: E731
    for name in ("x", "w", "ids", "logits", "loss"):
        assert call(**{name: None}) == 1, name
    assert call(x=addr(1) + 8) == 3 and call(labels=addr(3) + 2) == 3 and call(ids=addr(4) + 1) == 3 and call(loss=addr(7) + 2) == 3
    assert call(rows=addr(8) + 1) == 3 and call(lse=addr(6) + 2) == 3
    p.c.ids_64 = 1
    assert call(ids=addr(4) + 4) == 3
    need = p.bwd_workspace_bytes if back else p.fwd_workspace_bytes
    assert need > 0 and call(n=need - 1) == 4 and call(ws=None) == 4 and call(ws=addr(11) + 8) == 3
    assert call(loss=addr(1)) == 1 and call(rows=addr(5)) == 1 and call(rows=addr(7)) == 1
    if back:
        assert call(dx=addr(1)) == 1 and call(dw=addr(9)) == 1 and call(dw=addr(2)) == 1 and call(dx=addr(9) + 4) == 3
    # a teacher without slots; no target at all; slots without the teacher's side
    p = vocab(B, slots=0)
    assert run(B, p, back) == 1 and run(B, p, back, ids=None, logits=None, lse=None, labels=None) == 1
    assert B._lib.csa_vocab_loss_fwd(p.ref, addr(1), addr(2), None, addr(7), None, addr(11), BIG, None) == 1


def test_vocab_workspace(B):
    """The scores of a piece at most 4 GiB (or 256 rows), or of as many rows as the caller names."""
    base = vocab(B, rows=65536, features=4096, vocab=131072, slots=0)
    scores = 4 << 30
    held = base.bwd_workspace_bytes
    assert scores <= held <= scores + (131072 * 4096 * 4) + (2 << 30)         # and dW's fp32 sums
    assert vocab(B, rows=65536, features=4096, vocab=131072, slots=0, piece_rows=1024).bwd_workspace_bytes < held - scores // 2
    assert vocab(B, rows=0).bwd_workspace_bytes == 0
    assert vocab(B, rows=1, vocab=1 << 30, features=8, slots=0).bwd_workspace_bytes > 2 << 30
    assert vocab(B, dtype="f32").bwd_workspace_bytes > vocab(B).bwd_workspace_bytes


@pytest.mark.parametrize("site,status", [("workspace", 4), ("cuda", 5), ("unsupported", 2)])
def test_fault_injection(B, monkeypatch, site, status):
    monkeypatch.setenv("CSA_FAULT", site)
    assert norm_fwd(B, norm(B)) == status and norm_bwd(B, norm(B)) == status
    assert run(B, vocab(B)) == status and run(B, vocab(B), back=False) == status


def test_python_refusals(B):
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        B.csa_layernorm_fwd(norm(B, rows=4), x)
    with pytest.raises(ValueError):
        B.csa_vocab_loss_fwd(vocab(B, rows=4), x, x)
    with pytest.raises(ValueError):
        vocab(B, reduction="batch")
