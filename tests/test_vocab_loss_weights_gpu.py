"""What all rows' targets weigh in the vocabulary's losses: a factor of the gradients' products, rounded with no value of dz.

A weight rounded with dz moves the whole gradient along itself by as much as the weight's rounding, up to 2^-8.  Of the roundings that
are made, the result's cancel along it (2^-8 over the square root of the 2^17 and more values here), and so do the exponentials' in
fp16.  dz's own do not where the values are alike: of targets with small p all 1 - p round the same way (5e-4 of the gradient where p
is near 2^-9).  So what is compared with is the product of dz rounded as it should be: without the weight."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_vocab_loss_gpu import check, inputs, near, reference  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402

NAMES = ("labels", "teacher_ids", "teacher_logits", "teacher_lse")


def along(got, want):
    """How much longer got is along want."""
    return float(((got.double() - want) * want).sum() / (want * want).sum())


def straight(t, p, weight, wl=1.0, wt=1.0, mean=True):
    """`weight`: the one that all rows share."""
    _, dx, dw = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **{k: t[k] for k in NAMES})
    dz = reference(t, 1.0, wl, wt, mean)["dz"]
    rounded = (dz / weight).bfloat16().double() * weight
    for got, product, name in ((dx, lambda d: d @ t["weight"].double(), "dx"), (dw, lambda d: d.t() @ t["x"].double(), "dw")):
        near(got, product(dz), 2.0 ** -8.3, name)   # two roundings of 2^-8 / sqrt(3)
        assert abs(along(got, product(rounded))) <= 2.0 ** -12, (name, along(got, product(rounded)))


# 1 / 3891 lies halfway between two bf16 values; the packed rows' sizes and those that are not packed
SIZES = [(3891, 64, 700), (3891, 512, 16384)]


def one_candidate(M, K, V, labels, seed=0):
    """A teacher of one candidate a row: its share is 1, and what it weighs is the largest part of dz."""
    t = inputs(M, K, V, slots=1, labels=labels, scale=0.5, seed=seed)
    t["teacher_ids"] = torch.randint(0, V, (M, 1), generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda")
    return t


@pytest.mark.parametrize("M,K,V", SIZES)
@pytest.mark.parametrize("mean", [True, False])
def test_a_teacher_alone(M, K, V, mean):
    t, wt = one_candidate(M, K, V, False), 1.0 if mean else 1.0039
    p = B.VocabLossParams(M, K, V, slots=1, ids_64=True, teacher_weight=wt, reduction="mean" if mean else "sum")
    straight(t, p, 1 / M if mean else p.c.teacher_weight, wt=p.c.teacher_weight, mean=mean)


@pytest.mark.parametrize("M,K,V", SIZES)
@pytest.mark.parametrize("mean", [True, False])
def test_a_teacher_beside_labels_that_are_all_absent(M, K, V, mean):
    t, wt = one_candidate(M, K, V, True), 1.0 if mean else 1.0039
    t["labels"].fill_(-100)
    p = B.VocabLossParams(M, K, V, slots=1, labels_64=True, ids_64=True, teacher_weight=wt, reduction="mean" if mean else "sum")
    straight(t, p, 1 / M if mean else p.c.teacher_weight, wt=p.c.teacher_weight, mean=mean)


@pytest.mark.parametrize("mean", [True, False])
def test_labels_beside_candidates_that_are_all_absent(mean):
    M, K, V = SIZES[0]
    t, wl = one_candidate(M, K, V, True), 1.0 if mean else 1.0039
    t["labels"].clamp_(min=0)
    t["teacher_ids"].fill_(-1)
    p = B.VocabLossParams(M, K, V, slots=1, labels_64=True, ids_64=True, label_weight=wl, reduction="mean" if mean else "sum")
    straight(t, p, 1 / M if mean else p.c.label_weight, wl=p.c.label_weight, mean=mean)


@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("bad", ["label", "candidate"])
def test_ids_outside_the_vocabulary_still_make_nan(bad, mean):
    """Of the only label, or the only candidate, of a batch, beside the other kind of target."""
    M, K, V = 40, 64, 300
    t = one_candidate(M, K, V, True)
    (t["labels"] if bad == "label" else t["teacher_ids"]).fill_(-1)
    (t["labels"] if bad == "label" else t["teacher_ids"][:, 0])[5] = V
    p = B.VocabLossParams(M, K, V, slots=1, labels_64=True, ids_64=True, reduction="mean" if mean else "sum")
    loss, dx, _ = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **{k: t[k] for k in NAMES})
    assert bool(loss.isnan()) and dx.isnan().any(dim=1).nonzero().flatten().tolist() == [5]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,V", [(300, 64, 1000), (300, 512, 16384)])
@pytest.mark.parametrize("lse", [True, False])
def test_a_teachers_gradients_differ_by_random_roundings_alone(M, K, V, lse, dtype):
    """The relative length of the whole gradient's error, which a common one of its values would show in."""
    t = inputs(M, K, V, dtype, slots=33, labels=False, lse=lse, seed=3)
    _, dx, dw, r = check(t, B.VocabLossParams(M, K, V, dtype, slots=33, ids_64=True))
    limit = 2.0 ** -8.3 if dtype == "bf16" else 4e-6   # two roundings of 2^-8 / sqrt(3); fp32: sums of random signs
    near(dx, r["dz"] @ t["weight"].double(), limit, "dx")
    near(dw, r["dz"].t() @ t["x"].double(), limit, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wl,wt", [(1e-39, 1.0), (1e-30, 1e10), (1.0, 1e-39), (1e10, 1e-30), (0.0, 0.7), (0.7, 0.0), (2.0 ** -126, 2.0 ** 20)])
@pytest.mark.parametrize("mean", [True, False])
def test_weights_far_apart(wl, wt, mean, dtype):
    """Of each other: the smaller one's share of the gradient vanishes, and nothing else does."""
    M, K, V = 300, 64, 700
    t = inputs(M, K, V, dtype, slots=5, seed=5)
    p = B.VocabLossParams(M, K, V, dtype, slots=5, labels_64=True, ids_64=True, label_weight=wl, teacher_weight=wt,
                          reduction="mean" if mean else "sum")
    loss, dx, dw = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **{k: t[k] for k in NAMES})
    r = reference(t, wl=p.c.label_weight, wt=p.c.teacher_weight, mean=mean)
    assert abs(float(loss) - float(r["loss"])) <= 1e-4 * abs(float(r["loss"]))
    limit = 2.0 ** -8.3 if dtype == "bf16" else 4e-6
    near(dx, r["dz"] @ t["weight"].double(), limit, "dx")
    near(dw, r["dz"].t() @ t["x"].double(), limit, "dw")
