"""The operators around the step where they can go wrong: kernels close behind one another, ends of buffers, infinities,
sums over very many rows, gradients that share memory.

Tolerances are worst cases of the arithmetic, as in test_ops_gpu.py: u(t) = finfo(t).eps / 2.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_attention_indexer_tcgen05_gb300 import binding as B  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def test_products_close_behind_one_another():
    """Products of every tile shape in one stream with nothing between them: each starts on the SMs that its predecessor
    leaves, with barriers in the same places of shared memory."""
    g = gen(1)
    calls = []
    for M, K, N, dt, out in ((2048, 1024, 2048, "bf16", "bf16"), (1024, 512, 1024, "bf16", "bf16"), (512, 2048, 512, "bf16", "f32"),
                             (300, 512, 640, "f32", "f32"), (64, 256, 512, "bf16", "bf16"), (4096, 64, 4096, "bf16", "bf16")):
        t = BF if dt == "bf16" else F32
        p = B.LinearParams(M, K, N, dt, out)
        x, w = randn(g, M, K, dtype=t), randn(g, N, K, dtype=t, scale=K ** -0.5)
        ws = torch.empty(max(1, p.fwd_workspace_bytes), dtype=torch.uint8, device="cuda")
        first = B.csa_linear_fwd(p, x, w, workspace=ws)
        want = x.double() @ w.double().t()
        assert float((first.double() - want).norm() / want.norm()) <= U[first.dtype] + (K // 16 + 8) * 2.0 ** -23
        calls.append((p, x, w, ws, first, torch.empty_like(first)))
    torch.cuda.synchronize()
    for r in range(60):
        for p, x, w, ws, _, y in calls if r % 2 else calls[::-1]:
            B.csa_linear_fwd(p, x, w, workspace=ws, out=y)
    for *_, first, y in calls:
        assert torch.equal(first, y)
    B.csa_check_device_status()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(129, 77, 33), (40, 1001, 8), (33, 9, 1001), (300, 65, 771)])
def test_arguments_that_end_inside_a_vector(M, K, N, dtype):
    """Arguments whose last value is the last of a buffer of which only they are defined: what lies behind them is NaN in
    one run and 7 in another, which changes nothing."""
    t = BF if dtype == "bf16" else F32
    g = gen(M + K + N)
    p = B.LinearParams(M, K, N, dtype, activation="silu")

    def put(x, behind):
        buf = torch.full((x.numel() + 64,), behind, dtype=x.dtype, device="cuda")
        v = buf[:x.numel()].view(x.shape)
        v.copy_(x)
        return v

    args = [randn(g, M, K, dtype=t), randn(g, N, K, dtype=t), randn(g, N), randn(g, M, N, dtype=t), randn(g, M, N, dtype=t),
            randn(g, M, N, dtype=t)]
    got = []
    for behind in (7.0, float("nan")):
        x, w, b, res, dy, z = (put(a, behind) for a in args)
        got.append((B.csa_linear_fwd(p, x, w, b, res), *B.csa_linear_bwd(p, dy, x, w, z)))
    for a, b in zip(*got):
        assert bool(a.isfinite().all()) and torch.equal(a, b)


def test_autograd_sees_what_the_calls_write():
    """A graph kept over an optimizer step, or over a call that writes to one of its tensors, refuses its backward pass."""
    g = gen(3)
    p = B.LinearParams(24, 16, 16, "f32")
    x, w = randn(g, 24, 16).requires_grad_(True), randn(g, 16, 16).requires_grad_(True)
    y = B.csa_linear(x, w, params=p)
    state = B.AdamWTensors.zero_state([w])
    B.csa_adamw(B.AdamWTensors([w.detach()], [torch.ones(16, 16, device="cuda")], **state), 1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    r = B.RopeParams(24, 1, 16, "f32")
    pos, f = torch.arange(24, device="cuda", dtype=torch.int32)[None], torch.ones(8, device="cuda", dtype=torch.float64)
    dy = randn(g, 24, 16)
    for write in (lambda t: B.csa_rope(r, t, pos, f, out=t), lambda t: B.csa_linear_fwd(p, dy, w.detach(), residual=t, out=t),
                  lambda t: B.csa_linear_fwd(p, dy, w.detach(), preact=t),
                  lambda t: B.csa_linear_bwd(p, dy, dy.clone(), w.detach(), out=(t, None, None))):
        x = randn(g, 24, 16)
        y = B.csa_linear(x, w, params=p)
        write(x)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    with torch.inference_mode():                 # tensors without a counter
        out = torch.empty(24, 16, device="cuda")
        assert B.csa_linear_fwd(p, dy, w.detach(), out=out) is out and B.csa_rope(r, out, pos, f, out=out) is out
    # an unchanged graph goes through
    B.csa_linear(randn(g, 24, 16), w, params=p).sum().backward()
