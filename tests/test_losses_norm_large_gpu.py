"""Layer norm and the vocabulary's losses where offsets pass 32 bits, and many rows of strides that no vector fits; tolerances as in
test_norm_gpu.py and test_vocab_loss_gpu.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_norm_gpu import F32, U, check_bwd, check_fwd, close, depth, inputs, reference  # noqa: E402
from test_vocab_loss_gpu import near  # noqa: E402

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402


@pytest.mark.parametrize("cols", [2056, 2049, 300])
def test_norm_of_more_values_than_32_bits_count(cols):
    rows = (1 << 31) // cols + 1000
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, dy = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w, b = torch.randn(cols, generator=g, device="cuda"), torch.randn(cols, generator=g, device="cuda")
    p = B.LayerNormParams(rows, cols, eps=1e-5)
    stats = torch.empty(2, rows, device="cuda")
    y = B.csa_layernorm_fwd(p, x, w, b, stats=stats)
    dx, dw, db = B.csa_layernorm_bwd(p, dy, x, w, stats)
    edge = (1 << 31) // cols   # the row of the element 2^31
    for part in (slice(0, 40), slice(edge // 2 - 20, edge // 2 + 20), slice(edge - 20, edge + 20), slice(rows - 40, rows)):
        mean, rstd, h, mean_tol, rel, h_tol = reference(dict(x=x[part]), 1e-5)
        want, tol = h * w.double() + b.double(), h_tol * w.double().abs() + 3 * F32 * ((h * w).abs() + b.abs())
        close(y[part], want, tol + U[y.dtype] * (want.abs() + tol), "y")
        close(stats[0, part], mean[:, 0], mean_tol[:, 0], "mean")
        close(stats[1, part], rstd[:, 0], rstd[:, 0] * rel[:, 0], "rstd")
        mean, rstd = stats[0, part].double()[:, None], stats[1, part].double()[:, None]
        h, a = (x[part].double() - mean) * rstd, dy[part].double() * w.double()
        ma, mh = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
        want = rstd * (a - ma - h * mh)
        tol = rstd * ((depth(cols) + 4) * F32 * a.abs().mean(1, keepdim=True) + h.abs() * (depth(cols) + 8) * F32 * (a * h).abs().mean(1, keepdim=True)
                      + 8 * F32 * (a.abs() + ma.abs() + (h * mh).abs()))
        close(dx[part], want, tol + U[dx.dtype] * (want.abs() + tol), "dx")
    sums = [torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(4)]
    for xs, ds, st in zip(x.split(65536), dy.split(65536), stats.t().split(65536)):
        h, d = (xs.double() - st[:, :1]) * st[:, 1:], ds.double()
        for s, v in zip(sums, (d * h, (d * h).abs(), d, d.abs())):
            s += v.sum(0)
    adds = rows // 64 + 84
    close(dw, sums[0], adds * F32 * sums[1], "dweight")
    close(db, sums[2], adds * F32 * sums[3], "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,x_more,dy_more", [(50021, 130, 3, 0), (50021, 129, 0, 1), (20011, 1000, 5, 2), (3001, 4096, 1, 8)])
def test_many_rows_of_strides_that_differ(rows, cols, x_more, dy_more, dtype):
    """x, dy and the result lie differently between 16-byte boundaries."""
    t = inputs(rows, cols, dtype, "f32", cols + x_more, cols + dy_more)
    p = B.LayerNormParams(rows, cols, dtype, x_stride=cols + x_more, dy_stride=cols + dy_more)
    _, stats = check_fwd(t, p)
    check_bwd(t, p, stats)


@pytest.mark.parametrize("M,K,V,piece", [(20011, 64, 131080, 0), (20011, 64, 131080, 20011), (4200, 520, 524300, 4200)])
def test_losses_of_more_scores_than_32_bits_count(M, K, V, piece):
    """A label and a candidate in the last columns of the last rows among them; kept scores beyond 2^31 elements in one piece."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x, w = torch.randn(M, K, generator=g, device="cuda").bfloat16(), (torch.randn(V, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
    labels, ids = torch.randint(0, V, (M,), generator=g, device="cuda"), torch.randint(0, V, (M, 2), generator=g, device="cuda")
    labels[torch.rand(M, generator=g, device="cuda") < 0.2] = -1
    labels[-1], ids[-1, 0], labels[-2], ids[-2, 1] = V - 1, V - 2, 0, V - 1
    logits = torch.randn(M, 2, generator=g, device="cuda")
    p = B.VocabLossParams(M, K, V, slots=2, labels_64=True, ids_64=True, piece_rows=piece)
    rows = torch.empty(2, M, device="cuda")
    loss, dx, dw = B.csa_vocab_loss_bwd(p, x, w, labels, ids, logits, row_loss=rows)
    held, shares = labels >= 0, logits.double().softmax(1)
    each, n = held.double() / held.sum(), float(M)
    want_dx, want_dw = [], torch.zeros(V, K, dtype=torch.float64, device="cuda")
    for first in range(0, M, 512):
        r = slice(first, min(M, first + 512))
        here, wd = torch.arange(r.stop - first, device="cuda"), w.double()
        logp = (x[r].double() @ wd.t()).log_softmax(1)
        want = torch.where(held[r], -logp[here, labels[r].clamp(min=0)], 0.0)
        # scores of K products below 2^6 in sum, 2^20 exponentials: 2^-13 covers each by far, and a wrong place is off by some units
        assert float((rows[0, r].double() - want).abs().max()) < 2.0 ** -13
        want = (shares[r] * (shares[r].log() - logp.gather(1, ids[r]))).sum(1)
        assert float((rows[1, r].double() - want).abs().max()) < 2.0 ** -13
        d = logp.exp_() * (each[r] + 1 / n)[:, None]
        d.index_put_((here, labels[r].clamp(min=0)), -each[r], accumulate=True)
        d.index_put_((here[:, None].expand(-1, 2), ids[r]), -shares[r] / n, accumulate=True)
        want_dx.append(d @ wd)
        want_dw += d.t() @ x[r].double()
    want_dx = torch.cat(want_dx)
    # two roundings of 2^-8 / sqrt(3), of dz and of the result, and fp16's of the exponentials
    near(dx, want_dx, 2.0 ** -8.2, "dx")
    near(dx[-40:], want_dx[-40:], 2.0 ** -8.2, "the last rows' dx")
    near(dw, want_dw, 2.0 ** -8.2, "dw")
    near(dw[-40:], want_dw[-40:], 2.0 ** -8.2, "the last columns' dw")
    B.csa_check_device_status()
