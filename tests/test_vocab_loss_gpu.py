"""The vocabulary's losses (cross entropy with labels, distillation from top logits) against a plain implementation in 64 bits.

Tolerances are worst cases of the arithmetic: 2^-23 of the terms for each addition of a product's sum (tensor cores may cut off
where they align), 2^-24 for other fp32 operations, half a step for each rounding to fewer bits (fp16 2^-11, bf16 2^-8)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F32 = 2.0 ** -24


def close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = int(((got - want).abs() - tol).nan_to_num(nan=float("inf")).flatten().argmax())
        t = tol.flatten()[i] if torch.is_tensor(tol) and tol.numel() > 1 else tol
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i}: {got.flatten()[i]} for {want.flatten()[i]}, allowed {t}")


def product_tol(terms, count):
    return (count + 8) * 2.0 ** -23 * terms


def inputs(M, K, V, dtype="bf16", slots=0, labels=True, lse=False, seed=0, x_stride=0, scale=2.0, ids_64=True, labels_64=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t = {"weight": (rand(V, K) * scale * K ** -0.5).to(DT[dtype])}
    token = torch.randint(0, V, (M,), generator=g, device="cuda")
    x = torch.empty(M, x_stride or K, device="cuda", dtype=DT[dtype]).normal_(generator=g)
    x[:, :K] += t["weight"][token]
    t["x"] = x[:, :K]
    t["labels"] = t["teacher_ids"] = t["teacher_logits"] = t["teacher_lse"] = None
    if labels:
        skip = torch.rand(M, generator=g, device="cuda") < (0.3 if M > 2 else 0.0)
        t["labels"] = torch.where(skip, -100, token).to(torch.int64 if labels_64 else torch.int32)
    if slots:
        ids = torch.rand(M, V, generator=g, device="cuda").topk(slots, dim=1).indices if slots <= V else \
            torch.randint(0, V, (M, slots), generator=g, device="cuda")
        drop = torch.rand(M, slots, generator=g, device="cuda") < 0.2
        ids = torch.where(drop, -1, ids)
        if M > 3:
            ids[1] = -1                    # no candidates
            ids[2, 1:] = -7                # one
        t["teacher_ids"] = ids.to(torch.int64 if ids_64 else torch.int32)
        t["teacher_logits"] = rand(M, slots) * 3
        if lse:
            t["teacher_lse"] = t["teacher_logits"].double().logsumexp(1).float() + 0.2
    return t


def reference(t, alpha=1.0, wl=1.0, wt=1.0, mean=True):
    """z, p, lse, row losses, loss and dz in 64 bits; the teacher's shares."""
    x, w = t["x"].double(), t["weight"].double()
    M, V = x.shape[0], w.shape[0]
    z = alpha * (x @ w.t())
    lse = z.logsumexp(1)
    c, dz = torch.zeros(M, 1, dtype=torch.float64, device="cuda"), torch.zeros_like(z)
    label_rows, teacher_rows = torch.zeros(M, dtype=torch.float64, device="cuda"), torch.zeros(M, dtype=torch.float64, device="cuda")
    shares = ids = norm = None
    if t["labels"] is not None:
        held = t["labels"] >= 0
        at = t["labels"].clamp(min=0).long()[:, None]
        label_rows = torch.where(held, lse - z.gather(1, at)[:, 0], 0.0)
        each = held.double()[:, None] * wl / (max(1, int(held.sum())) if mean else 1)
        dz.scatter_add_(1, at, -each)
        c = c + each
    if t["teacher_ids"] is not None:
        held = t["teacher_ids"] >= 0
        ids = t["teacher_ids"].clamp(min=0).long()
        logits = t["teacher_logits"].double().masked_fill(~held, -math.inf)
        norm = t["teacher_lse"].double() if t["teacher_lse"] is not None else logits.logsumexp(1)
        shares = torch.where(logits > -math.inf, (logits - norm[:, None]).exp(), 0.0)
        teacher_rows = (torch.xlogy(shares, shares) - shares * (z.gather(1, ids) - lse[:, None])).sum(1)
        each = shares * wt / (max(1, int(held.any(1).sum())) if mean else 1)
        dz.scatter_add_(1, ids, -each)
        c = c + each.sum(1, keepdim=True)
    n1 = max(1, int((t["labels"] >= 0).sum())) if t["labels"] is not None and mean else 1
    n2 = max(1, int((t["teacher_ids"] >= 0).any(1).sum())) if t["teacher_ids"] is not None and mean else 1
    loss = wl * label_rows.sum() / n1 + wt * teacher_rows.sum() / n2
    p = (z - lse[:, None]).exp()
    return dict(z=z, p=p, lse=lse, label=label_rows, teacher=teacher_rows, loss=loss, dz=dz + c * p, c=c, shares=shares, ids=ids, n=(n1, n2),
                norm=norm[:, None].nan_to_num(neginf=0.0) if norm is not None else None)


def check(t, params, alpha=1.0, wl=1.0, wt=1.0, mean=True, need=(True, True), **kw):
    x, w = t["x"].double(), t["weight"].double()
    M, K, V = *x.shape, w.shape[0]
    r = reference(t, alpha, wl, wt, mean)
    targets = {k: t[k] for k in ("labels", "teacher_ids", "teacher_logits", "teacher_lse")}
    rows = torch.full((2, M), float("nan"), device="cuda")
    loss = B.csa_vocab_loss_fwd(params, t["x"], t["weight"], **targets, row_loss=rows)
    z_tol = product_tol(abs(alpha) * (x.abs() @ w.abs().t()), K) + 2 * F32 * r["z"].abs()
    # a sum of exponentials: the scores' errors weighted by p, each exponential's own (its argument and 2^-22), the additions
    lse_tol = (r["p"] * z_tol).sum(1) * 1.1 + (24 + V / 2048) * 2.0 ** -23 + (r["p"] * (r["z"] - r["z"].amax(1, keepdim=True)).abs()).sum(1) * 2.0 ** -23 \
        + 4 * F32 * r["lse"].abs()
    label_tol = torch.zeros_like(lse_tol)
    if t["labels"] is not None:
        at = t["labels"].clamp(min=0).long()[:, None]
        label_tol = torch.where(t["labels"] >= 0, lse_tol + z_tol.gather(1, at)[:, 0] + 2 * F32 * r["label"].abs(), 0.0)
    close(rows[0], r["label"], label_tol, "label losses")
    teacher_tol = torch.zeros_like(lse_tol)
    if r["shares"] is not None:
        s, S = r["shares"], r["shares"].shape[1]
        diff = (r["z"].gather(1, r["ids"]) - r["lse"][:, None])
        # exp(l - N): the argument is rounded to 2^-24 |l - N| = 2^-24 |log s|, N to 2^-24 |N| and the sum's error; logits that no
        # share comes from (-inf and such) enter neither
        s_rel = (S + 16 + 2 * r["norm"].abs() + s.clamp(min=1e-45).log().abs()) * 2.0 ** -23
        terms = s * (s.clamp(min=1e-300).log().abs() + diff.abs() + 1)
        teacher_tol = (s * (z_tol.gather(1, r["ids"]) + lse_tol[:, None]) + terms * (s_rel + (S / 32 + 10) * F32)).sum(1)
    close(rows[1], r["teacher"], teacher_tol, "teacher losses")
    loss_tol = (wl * label_tol.sum() / r["n"][0] + wt * teacher_tol.sum() / r["n"][1]) + 4 * F32 * \
        (wl * r["label"].abs().sum() / r["n"][0] + wt * r["teacher"].abs().sum() / r["n"][1])
    close(loss, r["loss"], loss_tol, "loss")

    loss2, dx, dw = B.csa_vocab_loss_bwd(params, t["x"], t["weight"], **targets, need_dx=need[0], need_dw=need[1], **kw)
    if M > 16:   # few rows' forward runs on kernels of its own
        assert torch.equal(loss2, loss)
    close(loss2, r["loss"], loss_tol, "loss of the backward")
    bf16 = params.value_dtype is torch.bfloat16
    # p: the scores' and lse's errors, the exponential's; kept in fp16 against its group's largest; c and tau are fp32
    p_tol = r["p"] * ((z_tol + lse_tol[:, None]) * 1.1 + (r["z"] - r["z"].amax(1, keepdim=True)).abs() * 2.0 ** -23 + 2.0 ** -20)
    if bf16:
        p_tol = p_tol + 2.0 ** -11 * r["p"] + 2.0 ** -24 * r["p"].amax(1, keepdim=True)
    dz_tol = r["c"] * p_tol + 8 * F32 * (r["c"] * r["p"] + r["dz"].abs())
    if r["shares"] is not None:
        each = r["shares"] * s_rel * wt / r["n"][1]
        dz_tol.scatter_add_(1, r["ids"], each)
        dz_tol += r["p"] * each.sum(1, keepdim=True)
    if bf16:
        dz_tol = dz_tol + U[torch.bfloat16] * (r["dz"].abs() + dz_tol)
    a = abs(alpha)
    if need[0]:
        want = alpha * (r["dz"] @ w)
        tol = a * (dz_tol @ w.abs()) + product_tol(a * (r["dz"].abs() @ w.abs()), V)
        close(dx, want, tol + U[dx.dtype] * (want.abs() + tol) + 1e-37, "dx")
    if need[1]:
        want = alpha * (r["dz"].t() @ x)
        tol = a * (dz_tol.t() @ x.abs()) + product_tol(a * (r["dz"].abs().t() @ x.abs()), M + 8)
        close(dw, want, tol + U[dw.dtype] * (want.abs() + tol) + 1e-37, "dw")
    return loss2, dx, dw, r


def near(got, want, most, what):
    err = float((got.double() - want).norm() / want.norm())
    assert err <= most, (what, err)


SHAPES = [(1, 8, 1), (1, 64, 2), (3, 7, 5), (37, 64, 64), (130, 72, 65), (257, 136, 127), (300, 512, 1000), (128, 1032, 129), (1000, 64, 5000),
          (64, 2056, 333), (5, 4104, 70000), (513, 40, 4097), (2, 128, 131075), (700, 200, 320)]


@pytest.mark.parametrize("M,K,V", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_labels(M, K, V, dtype):
    t = inputs(M, K, V, dtype, seed=M + K + V)
    loss, dx, dw, r = check(t, B.VocabLossParams(M, K, V, dtype, labels_64=True))
    assert B.csa_last_path() == "tcgen05"
    if V > 64 and M > 2:
        # random roundings: of dz, of the result (and fp16's), each 2^-8 / sqrt(3) at most; fp32: sums of random signs
        limit = 2.0 ** -8 if dtype == "bf16" else 4e-6
        near(dx, K ** 0 * (r["dz"] @ t["weight"].double()), limit, "dx")
        near(dw, r["dz"].t() @ t["x"].double(), limit, "dw")
    B.csa_check_device_status()


@pytest.mark.parametrize("M,K,V", SHAPES[2:])
@pytest.mark.parametrize("slots,lse", [(1, True), (5, False), (33, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_teacher(M, K, V, slots, lse, dtype):
    t = inputs(M, K, V, dtype, slots=slots, labels=False, lse=lse, seed=M + slots)
    check(t, B.VocabLossParams(M, K, V, dtype, slots=slots, ids_64=True))
    B.csa_check_device_status()


@pytest.mark.parametrize("labels_64,ids_64", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("M,K,V,slots", [(200, 96, 777, 40), (50, 64, 1300, 1024), (33, 32, 20, 64)])
def test_both(M, K, V, slots, mean, labels_64, ids_64):
    t = inputs(M, K, V, slots=slots, lse=mean, seed=4, labels_64=labels_64, ids_64=ids_64)
    if M > 5:   # the label among the candidates, and the same candidate more than once
        t["teacher_ids"][3, 0] = t["labels"][3] = 5
        t["teacher_ids"][4, :3] = 11
        t["labels"][4] = 11
    p = B.VocabLossParams(M, K, V, slots=slots, alpha=0.5, label_weight=0.3, teacher_weight=1.7, reduction="mean" if mean else "sum",
                          labels_64=labels_64, ids_64=ids_64)
    check(t, p, 0.5, 0.3, 1.7, mean)


@pytest.mark.parametrize("slots", [63, 64, 65, 127, 128, 129, 255, 256, 257, 512, 513, 1023, 1024])
@pytest.mark.parametrize("M,K,V", [(37, 32, 100), (30, 64, 1100), (20, 32, 70000)])
@pytest.mark.parametrize("labels", [True, False])
def test_many_candidates(M, K, V, slots, labels):
    """Around the numbers where targets are ordered in another way; columns named twice, by the label too, and slots without one."""
    t = inputs(M, K, V, slots=slots, labels=labels, seed=slots + V)
    if labels:
        t["teacher_ids"][3:9, slots // 2] = t["labels"][3:9]
        t["labels"][10], t["labels"][11] = 0, V - 1
    t["teacher_ids"][12:15, 5:20] = t["teacher_ids"][12:15, 5:6]
    check(t, B.VocabLossParams(M, K, V, slots=slots, labels_64=True, ids_64=True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,piece", [(300, 100), (300, 256), (513, 256), (70, 7), (1025, 1024)])
def test_pieces(M, piece, dtype):
    """Pieces of rows: a short last one, odd ones; the first rows' results do not depend on the cut."""
    K, V = 104, 1000
    t = inputs(M, K, V, dtype, slots=6, seed=M)
    whole = B.VocabLossParams(M, K, V, dtype, slots=6, labels_64=True, ids_64=True)
    cut = B.VocabLossParams(M, K, V, dtype, slots=6, labels_64=True, ids_64=True, piece_rows=piece)
    check(t, cut)
    targets = {k: t[k] for k in ("labels", "teacher_ids", "teacher_logits")}
    a, b = (B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **targets) for p in (whole, cut))
    assert torch.equal(a[0], b[0])
    for _ in range(2):
        assert all(torch.equal(u, v) for u, v in zip(b, B.csa_vocab_loss_bwd(cut, t["x"], t["weight"], **targets)))


@pytest.mark.parametrize("stride", [72, 80, 67, 65])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(stride, dtype):
    t = inputs(150, 64, 500, dtype, slots=3, seed=stride, x_stride=stride)
    check(t, B.VocabLossParams(150, 64, 500, dtype, slots=3, labels_64=True, ids_64=True, x_stride=stride))


@pytest.mark.parametrize("need", [(True, False), (False, True), (False, False)])
def test_outputs_left_out(need):
    t = inputs(150, 64, 500, slots=3)
    check(t, B.VocabLossParams(150, 64, 500, slots=3, labels_64=True, ids_64=True), need=need)


def test_first_and_last_columns():
    for V in (64, 65, 127, 128, 256, 257, 1000):
        t = inputs(20, 64, V, slots=4, seed=V)
        edge = torch.tensor([0, 63 % V, 64 % V, V - 1], device="cuda")
        t["teacher_ids"][:] = edge
        t["labels"][:] = edge.repeat(5)
        check(t, B.VocabLossParams(20, 64, V, slots=4, labels_64=True, ids_64=True))


def test_rows_without_targets():
    M, K, V = 40, 64, 300
    t = inputs(M, K, V)
    t["labels"].fill_(-1)
    p = B.VocabLossParams(M, K, V, labels_64=True)
    loss, dx, dw = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"])
    assert float(loss) == 0 and not bool(dx.any()) and not bool(dw.any())
    # scores that are not finite pass nothing either, where the row has no target
    t = inputs(M, K, V)
    t["labels"][7], t["labels"][8] = -100, 3
    want = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"])
    t["x"][7, 3] = float("inf")
    loss, dx, _ = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"], need_dw=False)
    assert torch.equal(loss, want[0]) and torch.equal(dx, want[1]) and not bool(dx[7].any())


@pytest.mark.parametrize("where", ["label", "candidate"])
def test_ids_outside_the_vocabulary(where):
    M, K, V = 40, 64, 300
    t = inputs(M, K, V, slots=3, seed=2)
    p = B.VocabLossParams(M, K, V, slots=3, labels_64=True, ids_64=True)
    t["labels"][5] = 1
    bad = 1 << 40 if where == "label" else V
    (t["labels"] if where == "label" else t["teacher_ids"].view(M, 3)[:, 1])[5] = bad
    rows = torch.zeros(2, M, device="cuda")
    targets = {k: t[k] for k in ("labels", "teacher_ids", "teacher_logits")}
    loss, dx, dw = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **targets, row_loss=rows)
    nan = rows.isnan()
    assert bool(loss.isnan()) and bool(dx[5].isnan().all()) and bool(dw.isnan().any())
    assert nan.sum() == 1 and bool(nan[0 if where == "label" else 1, 5])
    assert not bool(dx[:5].isnan().any()) and not bool(dx[6:].isnan().any())


def test_values_that_are_not_finite():
    M, K, V = 12, 64, 300
    t = inputs(M, K, V)
    t["labels"][:] = 4
    p = B.VocabLossParams(M, K, V, labels_64=True)
    t["x"][2, 0] = float("nan")
    t["x"][9, 0] = float("inf")
    rows = torch.zeros(2, M, device="cuda")
    loss, dx, _ = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"], row_loss=rows)
    assert bool(loss.isnan()) and rows[0].isnan().nonzero().flatten().tolist() == [2, 9]
    assert bool(dx[2].isnan().all()) and bool(dx[9].isnan().all()) and int(dx.isnan().any(1).sum()) == 2


def test_teacher_logits_at_their_limits():
    M, K, V = 6, 64, 500
    t = inputs(M, K, V, slots=4, labels=False)
    inf = float("inf")
    t["teacher_ids"][:] = torch.tensor([7, 3, 499, 0], device="cuda")
    t["teacher_logits"][:] = torch.tensor([[1.0, -inf, 0.5, -inf], [-inf, -inf, -inf, 2.0], [-3e38, 3.0, -3e38, 1.0],
                                           [80.0, 90.0, 100.0, -100.0], [-90.0, -95.0, -100.0, -inf], [0.0, 0.0, 0.0, 0.0]], device="cuda")
    check(t, B.VocabLossParams(M, K, V, slots=4, ids_64=True))
    t["teacher_logits"][5] = -inf   # candidates without a share: they count as a row, with a loss of 0
    rows = torch.full((2, M), 7.0, device="cuda")
    loss, dx, _ = B.csa_vocab_loss_bwd(B.VocabLossParams(M, K, V, slots=4, ids_64=True), t["x"], t["weight"], None, t["teacher_ids"],
                                       t["teacher_logits"], row_loss=rows)
    assert float(rows[1, 5]) == 0 and not bool(dx[5].any()) and abs(float(loss) * 6 - float(rows[1].sum())) < 1e-5 * float(rows[1].abs().sum())


# ------------------------------------------------------------------ rows without a target, packed away

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,V,slots,piece", [(700, 512, 16384, 0, 0), (700, 520, 16411, 5, 0), (513, 515, 16384, 3, 0), (1000, 512, 20001, 0, 300),
                                               (260, 1024, 16400, 70, 100)])
def test_packed_rows(M, K, V, slots, piece, dtype):
    t = inputs(M, K, V, dtype, slots=slots, seed=M + V)
    if slots:
        t["teacher_ids"][torch.rand(M, device="cuda") < 0.5] = -1
    p = B.VocabLossParams(M, K, V, dtype, slots=slots, labels_64=True, ids_64=True, piece_rows=piece)
    _, dx, dw, r = check(t, p)
    gone = (r["c"] == 0)[:, 0]
    assert bool(gone.any()) and not bool(dx[gone].any())
    B.csa_check_device_status()


@pytest.mark.parametrize("held", ["none", "one", "first", "last", "all", 64, 256, 257, 384])
@pytest.mark.parametrize("piece", [0, 128])
def test_how_many_rows_are_packed(held, piece):
    """No row, one, a block at either end, all, and numbers at the edges of tiles and of dW's stages."""
    M, K, V = 600, 512, 16384
    t = inputs(M, K, V, seed=1)
    full = t["labels"].clamp(min=0)
    keep = torch.zeros(M, dtype=torch.bool, device="cuda")
    if held == "one":
        keep[431] = True
    elif held == "first":
        keep[:300] = True
    elif held == "last":
        keep[-5:] = True
    elif held == "all":
        keep[:] = True
    elif held != "none":
        keep[torch.randperm(M, device="cuda")[:held]] = True
    t["labels"] = torch.where(keep, full, -100)
    check(t, B.VocabLossParams(M, K, V, labels_64=True, piece_rows=piece))
    B.csa_check_device_status()


@pytest.mark.parametrize("dtype,x_stride", [("bf16", 515), ("bf16", 520), ("bf16", 700), ("f32", 513), ("f32", 516)])
def test_packed_rows_with_strides(dtype, x_stride):
    t = inputs(300, 512, 16384, dtype, slots=2, x_stride=x_stride, seed=x_stride)
    check(t, B.VocabLossParams(300, 512, 16384, dtype, slots=2, labels_64=True, ids_64=True, x_stride=x_stride))


@pytest.mark.parametrize("need", [(True, False), (False, True)])
@pytest.mark.parametrize("piece", [0, 130])
def test_packed_rows_one_gradient(need, piece):
    t = inputs(300, 512, 16384)
    p = B.VocabLossParams(300, 512, 16384, labels_64=True, piece_rows=piece)
    want = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"])
    got = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"], need_dx=need[0], need_dw=need[1])
    for g, w, n in zip(got, want, (True, *need)):
        assert torch.equal(g, w) if n else g is None


def test_packed_rows_with_ids_outside_the_vocabulary():
    """Such a row is NaN and no other row's loss is; nothing is read or written there."""
    M, K, V = 300, 512, 16384
    t = inputs(M, K, V, slots=3)
    t["labels"][7], t["teacher_ids"][200, 1] = V, V + 5
    p = B.VocabLossParams(M, K, V, slots=3, labels_64=True, ids_64=True)
    rows = torch.empty(2, M, device="cuda")
    loss = B.csa_vocab_loss_fwd(p, t["x"], t["weight"], t["labels"], t["teacher_ids"], t["teacher_logits"], row_loss=rows)
    bad = rows.isnan()
    assert bool(loss.isnan()) and bool(bad[0, 7]) and bool(bad[1, 200]) and int(bad.sum()) == 2
    _, dx, _ = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"], t["teacher_ids"], t["teacher_logits"])
    assert dx.isnan().any(dim=1).nonzero().flatten().tolist() == [7, 200]
    B.csa_check_device_status()


def test_rows_that_are_packed_away_are_not_read():
    M, K, V = 600, 512, 16384
    t = inputs(M, K, V, seed=2)
    p = B.VocabLossParams(M, K, V, labels_64=True)
    want = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"])
    t["x"][t["labels"] < 0] = float("nan")
    got = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_packed_rows_captured_with_other_targets():
    """The number of packed rows is the device's: a replayed call takes that of the targets it finds."""
    M, K, V = 700, 512, 16384
    t = inputs(M, K, V, slots=4)
    p = B.VocabLossParams(M, K, V, slots=4, labels_64=True, ids_64=True, piece_rows=256)
    names = ("labels", "teacher_ids", "teacher_logits")
    ws = torch.empty(p.bwd_workspace_bytes, dtype=torch.uint8, device="cuda")
    out = tuple(torch.empty_like(o) for o in B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **{k: t[k] for k in names}))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **{k: t[k] for k in names}, workspace=ws, out=out)
    for share in (0.1, 0.9, 0.0, 1.0):
        other = inputs(M, K, V, slots=4, seed=int(share * 10) + 3)
        gone = torch.rand(M, device="cuda") >= share
        other["labels"][gone], other["teacher_ids"][gone] = -1, -1
        for k in ("x", "weight", *names):
            t[k].copy_(other[k])
        ws.fill_(255)
        graph.replay()
        want = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **{k: t[k] for k in names})
        assert all(torch.equal(a, b) for a, b in zip(out, want)), share
        if share:
            check(t, p)


def test_the_losses_weight_is_not_rounded_with_dz():
    """A weight halfway between two bf16 values: rounded with dz, whose largest parts it is, every gradient would be off by 2^-8 of
    itself.  The roundings that are made, of dz and of the result, are random: 2^-8 / sqrt(3) each at most."""
    M, K, V = 500, 64, 4000
    t = inputs(M, K, V, scale=0.5)
    p = B.VocabLossParams(M, K, V, label_weight=1.0039, reduction="sum", labels_64=True)
    _, dx, dw = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], t["labels"])
    r = reference(t, wl=p.c.label_weight, mean=False)
    near(dx, r["dz"] @ t["weight"].double(), 2.0 ** -8.6, "dx")
    near(dw, r["dz"].t() @ t["x"].double(), 2.0 ** -8.6, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    """Rows whose scores lie hundreds apart: most columns' exponentials vanish."""
    t = inputs(60, 64, 700, dtype, slots=4, scale=60.0)
    check(t, B.VocabLossParams(60, 64, 700, dtype, slots=4, labels_64=True, ids_64=True))
    check(t, B.VocabLossParams(60, 64, 700, dtype, slots=4, labels_64=True, ids_64=True, alpha=-1.5), alpha=-1.5)


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.randn(100, 64, device="cuda").bfloat16()
    p = B.VocabLossParams(0, 64, 100)
    labels = torch.empty(0, dtype=torch.int32, device="cuda")
    loss, dx, dw = B.csa_vocab_loss_bwd(p, x, w, labels)
    assert float(loss) == 0 and dx.shape == (0, 64) and not bool(dw.any())
    assert float(B.csa_vocab_loss_fwd(p, x, w, labels)) == 0


def test_same_bits_on_another_stream_and_captured():
    M, K, V, S = 400, 256, 3001, 5
    t = inputs(M, K, V, slots=S)
    p = B.VocabLossParams(M, K, V, slots=S, labels_64=True, ids_64=True, piece_rows=256)
    names = ("labels", "teacher_ids", "teacher_logits")
    targets = {k: t[k] for k in names}
    want = B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **targets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = torch.empty(p.bwd_workspace_bytes, dtype=torch.uint8, device="cuda")
        out = tuple(torch.empty_like(o) for o in want)
        B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **targets, workspace=ws, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **targets, workspace=ws, out=out)
        for o in out:
            o.fill_(7)
        ws.fill_(255)   # nothing of it is kept from call to call
        graph.replay()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    other = inputs(M, K, V, slots=S, seed=8)
    for k in ("x", "weight", *names):
        t[k].copy_(other[k])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, B.csa_vocab_loss_bwd(p, t["x"], t["weight"], **targets)))


@pytest.mark.parametrize("slots", [0, 7])
def test_autograd_and_differences(slots):
    M, K, V = 24, 40, 90
    t = inputs(M, K, V, "f32", slots=slots)
    p = B.VocabLossParams(M, K, V, "f32", slots=slots, alpha=0.7, labels_64=True, ids_64=True)
    x, w = t["x"].view(4, 6, K).clone().requires_grad_(True), t["weight"].clone().requires_grad_(True)
    targets = [t[k] for k in ("labels", "teacher_ids", "teacher_logits", "teacher_lse")]
    loss = B.csa_vocab_loss(x, w, *targets, params=p)
    (3.0 * loss).backward()
    g = torch.Generator(device="cuda").manual_seed(1)
    for leaf, key in ((x, "x"), (w, "weight")):
        way, e = torch.randn(t[key].shape, generator=g, device="cuda", dtype=torch.float64), 1e-5
        up, down = (float(reference({**t, key: t[key].double() + s * e * way}, 0.7)["loss"]) for s in (1, -1))
        grad = leaf.grad.double().view(way.shape)
        slope = float((grad * way).sum())
        # differences: e^2 times third derivatives, 64-bit rounding over e; gradients: some 200 fp32 roundings of their terms
        assert abs(slope - 3 * (up - down) / (2 * e)) <= 200 * F32 * float((grad * way).abs().sum()) + 1e-6
    with torch.no_grad():
        assert torch.equal(B.csa_vocab_loss(x, w, *targets, params=p), loss)


def test_refusals():
    t = inputs(8, 64, 100, slots=2)
    p = B.VocabLossParams(8, 64, 100, slots=2, labels_64=True, ids_64=True)
    q = B.VocabLossParams(8, 64, 100, labels_64=True)
    x, w, args = t["x"], t["weight"], (t["labels"], t["teacher_ids"], t["teacher_logits"])
    for bad in (lambda: B.csa_vocab_loss_fwd(p, x.float(), w, *args), lambda: B.csa_vocab_loss_fwd(p, x, w.t().contiguous(), *args),
                lambda: B.csa_vocab_loss_fwd(p, x, w, args[0].int(), *args[1:]), lambda: B.csa_vocab_loss_fwd(p, x, w, args[0], args[1].int(), args[2]),
                lambda: B.csa_vocab_loss_fwd(p, x, w, args[0], args[1]), lambda: B.csa_vocab_loss_fwd(q, x, w, *args),
                lambda: B.csa_vocab_loss_fwd(q, x, w), lambda: B.csa_vocab_loss_fwd(p, x, w, args[0], args[1], args[2].t().contiguous()),
                lambda: B.csa_vocab_loss_fwd(q, x, w, args[0][:7]), lambda: B.csa_vocab_loss_fwd(q, x[:, :32], w, args[0]),
                lambda: B.csa_vocab_loss_fwd(q, x, w, args[0].cpu()), lambda: B.VocabLossParams(8, 64, 100, reduction="none"),
                lambda: B.csa_vocab_loss_fwd(q, x, w, args[0], row_loss=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(B.CSAError):
        B.csa_vocab_loss_bwd(q, x, w, args[0], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.CSAError):
        B.csa_vocab_loss_bwd(q, x, w, args[0], out=(None, x, None))
