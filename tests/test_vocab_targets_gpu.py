"""Labels of a call, or a trainer, that has room for a teacher's candidates: the teacher may be left out."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_vocab_loss_gpu import inputs  # noqa: E402
from test_vocab_trainer_gpu import make, setup  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,V,piece", [(300, 512, 16384, 0), (300, 512, 16384, 130), (200, 64, 1000, 0), (200, 64, 1000, 70), (5, 64, 1000, 0),
                                         (0, 64, 1000, 0)])
@pytest.mark.parametrize("slots", [3, 200])
def test_labels_alone_with_slots(M, K, V, piece, slots, dtype):
    """The bits of a call without slots, in the workspace of one with."""
    t = inputs(M, K, V, dtype)
    p, q = (B.VocabLossParams(M, K, V, dtype, slots=s, labels_64=True, ids_64=True, piece_rows=piece) for s in (slots, 0))
    rows = [torch.full((2, M), 7.0, device="cuda") for _ in range(2)]
    a, b = (B.csa_vocab_loss_bwd(s, t["x"], t["weight"], t["labels"], row_loss=r) for s, r in zip((p, q), rows))
    assert all(torch.equal(u, v) for u, v in zip((*a, rows[0]), (*b, rows[1])))
    a, b = (B.csa_vocab_loss_fwd(s, t["x"], t["weight"], t["labels"], row_loss=r) for s, r in zip((p, q), rows))
    assert torch.equal(a, b) and torch.equal(*rows)
    B.csa_check_device_status()


def test_a_trainer_takes_either_target():
    p, weights, x, targets = setup("bf16")
    t = make(p, weights)
    labels = {"labels": targets["labels"]}
    teacher = {k: v for k, v in targets.items() if k != "labels"}
    for some in (targets, labels, teacher, labels, targets):
        alone = make(B.VocabLossParams(p.c.rows, p.c.features, p.c.vocab, p.c.dtype, slots=p.c.slots if "teacher_ids" in some else 0,
                                       label_weight=p.c.label_weight, teacher_weight=p.c.teacher_weight, labels_64=True, ids_64=True),
                     [t.weight, t.norm_weight, t.norm_bias])
        want = [v.clone() for v in (lambda o: (o[0], o[1], *o[2]))(alone.gradients(x, **some))]
        loss, dx = t.step(x, **some)
        assert all(torch.equal(u, v) for u, v in zip((loss, dx, *t.grads), want))
    assert int(t.step_count) == 5


def test_a_teacher_in_part_or_no_target_refused():
    t = inputs(20, 64, 300, slots=3, lse=True)
    p = B.VocabLossParams(20, 64, 300, slots=3, labels_64=True, ids_64=True)
    for gone in (("teacher_ids",), ("teacher_logits",), ("teacher_ids", "teacher_logits"), ("labels", "teacher_ids", "teacher_logits", "teacher_lse"),
                 ("labels", "teacher_ids", "teacher_logits")):
        targets = {k: None if k in gone else t[k] for k in ("labels", "teacher_ids", "teacher_logits", "teacher_lse")}
        for call in (B.csa_vocab_loss_fwd, B.csa_vocab_loss_bwd):
            with pytest.raises(ValueError):
                call(p, t["x"], t["weight"], **targets)
