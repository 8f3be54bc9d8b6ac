"""Millions of rows over a small vocabulary: the time of a call grows as its rows do."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402


def call(M, K=8, V=64):
    g = torch.Generator(device="cuda").manual_seed(M)
    x, w = torch.randn(M, K, generator=g, device="cuda").bfloat16(), torch.randn(V, K, generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, V, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    p = B.VocabLossParams(M, K, V, slots=1)
    logits, ws = torch.zeros(M, 1, device="cuda"), torch.empty(p.fwd_workspace_bytes, dtype=torch.uint8, device="cuda")
    out, rows = torch.empty((), device="cuda"), torch.empty(2, M, device="cuda")
    run = lambda: B.csa_vocab_loss_fwd(p, x, w, None, ids, logits, row_loss=rows, workspace=ws, out=out)  # noqa: E731
    return run, (x, w, ids), (out, rows)


def best(run, tries=5):
    times = []
    for _ in range(tries):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        run()
        a.record()
        run()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def test_time_grows_as_rows_do():
    """Eight times the rows: eight times the work.  Were every block of rows to read what every other one counted, it would be 64
    times; the test allows twice the work."""
    few, many = (best(call(M)[0]) for M in (1 << 18, 1 << 21))
    assert many <= 16 * few, (few, many)


@pytest.mark.parametrize("M", [32768 + 8, 300001, 1 << 20])
def test_losses_of_many_rows(M):
    run, (x, w, ids), (out, rows) = call(M)
    run()
    logp = (x.double() @ w.double().t()).log_softmax(1)
    held = ids[:, 0] >= 0
    want = torch.where(held, -logp.gather(1, ids.clamp(min=0).long())[:, 0], 0.0)
    # a row: its scores of 8 products, 64 exponentials and their sum, each within some 2^-23 of values below 2^6
    assert float((rows[1].double() - want).abs().max()) <= 64 * 2.0 ** -23 * 4 and not bool(rows[0].any())
    assert abs(float(out) - float(want.sum() / held.sum())) <= 1e-5 * float(want.sum() / held.sum())
    first = out.clone()
    run()
    assert torch.equal(first, out)
