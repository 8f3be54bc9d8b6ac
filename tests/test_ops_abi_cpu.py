"""The entry points around the step (projections, rotary positions, AdamW) on a machine without a GPU: sizes,
refusals and fault injection; no compute call gets past the host checks."""
import ctypes

import pytest

BIG = 1 << 40


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


# ------------------------------------------------------------------ projections

def linear(B, **kw):
    base = dict(rows=100, in_features=64, out_features=48, activation="silu")
    base.update(kw)
    return B.LinearParams(**base)


def linear_fwd(B, p, x=addr(1), w=addr(2), bias=addr(3), res=addr(4), y=addr(5), z=addr(6), ws=addr(7), n=BIG):
    return B._lib.csa_linear_fwd(p.ref, x, w, bias, res, y, z, ws, n, None)


def linear_bwd(B, p, dy=addr(1), x=addr(2), w=addr(3), z=addr(4), dx=addr(5), dw=addr(6), db=addr(7), ws=addr(8), n=BIG):
    return B._lib.csa_linear_bwd(p.ref, dy, x, w, z, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("field,value,status", [
    ("dtype", 5, 1), ("out_dtype", -1, 1), ("activation", 4, 1), ("in_features", 0, 1), ("out_features", 0, 1),
    ("rows", -1, 1), ("alpha", float("nan"), 1), ("x_stride", 63, 1), ("residual_stride", 47, 1), ("dy_stride", 47, 1),
    ("rows", 1 << 31, 2), ("x_stride", 1 << 37, 2), ("rows", 0x7fff0001, 2), ("in_features", 0x7fff0001, 2),
    ("out_features", 0x7fff0001, 2)])
def test_linear_params_refused(B, field, value, status):
    p = linear(B)
    setattr(p.c, field, value)
    assert p.fwd_workspace_bytes == 0 and p.bwd_workspace_bytes == 0
    assert linear_fwd(B, p) == status and linear_bwd(B, p) == status


def test_linear_bf16_output_of_f32_values_refused(B):
    p = linear(B, dtype="f32", out_dtype="bf16")
    assert linear_fwd(B, p) == 2 and linear_bwd(B, p) == 2


def test_linear_pointers_refused(B):
    p = linear(B)
    assert linear_fwd(B, p, x=None) == 1 and linear_fwd(B, p, w=None) == 1 and linear_fwd(B, p, y=None) == 1
    for name in ("x", "w", "bias", "res", "y", "z"):
        assert linear_fwd(B, p, **{name: addr(9) + 8}) == 3, name
    assert linear_bwd(B, p, z=None) == 1                      # an activation's gradient needs its argument
    assert linear_bwd(B, p, dy=None) == 1 and linear_bwd(B, p, x=None) == 1 and linear_bwd(B, p, w=None) == 1
    for name in ("dy", "x", "w", "z", "dx", "dw", "db"):
        assert linear_bwd(B, p, **{name: addr(9) + 4}) == 3, name
    # the residual as the output: only with the output's own row stride
    assert linear_fwd(B, linear(B, residual_stride=56), res=addr(5)) == 1


def test_linear_an_output_over_another_argument_refused(B):
    p = linear(B)
    for name in ("x", "w", "bias", "z"):
        assert linear_fwd(B, p, **{name: addr(5)}) == 1, name       # y
    for name in ("x", "w", "bias", "res"):
        assert linear_fwd(B, p, **{name: addr(6)}) == 1, name       # preact
    assert linear_fwd(B, p, res=addr(5), z=None) == 5               # the residual in place: past the checks, no GPU
    for out in (5, 6, 7):
        for name in ("dy", "x", "w", "z"):
            assert linear_bwd(B, p, **{name: addr(out)}) == 1, (out, name)
    assert linear_bwd(B, p, dw=addr(5)) == linear_bwd(B, p, db=addr(5)) == linear_bwd(B, p, db=addr(6)) == 1
    # what is not read may hold a gradient
    assert linear_bwd(B, p, dx=addr(2), dw=None) == linear_bwd(B, p, dx=None, dw=addr(3)) == 5
    assert linear_bwd(B, linear(B, activation="none"), dx=addr(4)) == 5


def test_linear_workspace_refused(B):
    p = linear(B)
    assert p.bwd_workspace_bytes > 0
    assert linear_bwd(B, p, n=p.bwd_workspace_bytes - 1) == 4
    assert linear_bwd(B, p, ws=None) == 4
    assert linear_bwd(B, p, n=p.bwd_workspace_bytes) == 5     # past the checks: no GPU


def test_linear_without_rows_enqueues_nothing_forward(B):
    assert linear_fwd(B, linear(B, rows=0), x=None, y=None, z=None, res=None) == 0


def test_linear_names_refused(B):
    with pytest.raises(ValueError):
        linear(B, activation="tanh")
    with pytest.raises(ValueError):
        linear(B, dtype="fp16")


# ------------------------------------------------------------------ rotary positions

def rope(B, **kw):
    base = dict(rows=10, heads=4, head_dim=64, rot_dim=32, sections=[8, 4, 4])
    base.update(kw)
    return B.RopeParams(**base)


def call_rope(B, p, x=addr(1), pos=addr(2), f=addr(3), out=addr(4)):
    return B._lib.csa_rope(p.ref, x, pos, f, out, None)


@pytest.mark.parametrize("field,value,status", [
    ("dtype", 2, 1), ("heads", 0, 1), ("head_dim", 0, 1), ("rot_offset", -2, 1), ("rot_offset", 33, 1), ("rot_dim", 31, 1),
    ("rot_dim", 30, 1), ("interleaved", 2, 1), ("inverse", -1, 1), ("positions_64", 3, 1), ("axes", 0, 1), ("axes", 5, 1),
    ("axes", 2, 1), ("rows", -1, 1), ("x_head_stride", 63, 1), ("out_head_stride", 63, 1), ("x_row_stride", 63, 1),
    ("out_row_stride", 200, 1), ("rows", 1 << 41, 2), ("x_row_stride", 1 << 41, 2)])
def test_rope_params_refused(B, field, value, status):
    p = rope(B)
    setattr(p.c, field, value)
    assert call_rope(B, p) == status


def test_rope_sections_refused(B):
    p = rope(B)
    p.c.sections[1], p.c.sections[2] = -4, 12                # the right sum, one negative
    assert call_rope(B, p) == 1
    with pytest.raises(ValueError):
        rope(B, sections=[2] * 5)
    assert call_rope(B, rope(B, head_dim=2048, rot_dim=1026, sections=[513])) == 2


def test_rope_pointers_refused(B):
    p = rope(B)
    for name in ("x", "pos", "f", "out"):
        assert call_rope(B, p, **{name: None}) == 1, name
    assert call_rope(B, p, x=addr(9) + 8) == 3 and call_rope(B, p, out=addr(9) + 8) == 3
    assert call_rope(B, p, pos=addr(9) + 2) == 3 and call_rope(B, p, f=addr(9) + 4) == 3
    assert call_rope(B, rope(B, positions_64=True), pos=addr(9) + 4) == 3
    assert call_rope(B, rope(B, x_row_stride=512), out=addr(1)) == 1    # in place, but other strides
    assert call_rope(B, rope(B, rows=0), x=None, pos=None, f=None, out=None) == 0


def test_rope_heads_outermost_accepted(B):
    """[heads, rows, head_dim]: rows lie within a head's stride."""
    assert call_rope(B, rope(B, out_row_stride=64, out_head_stride=640)) == 5
    assert call_rope(B, rope(B, out_row_stride=64, out_head_stride=639)) == 1


# ------------------------------------------------------------------ AdamW

def adamw(B, tensors, **kw):
    base = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1)
    base.update(kw)
    p = B.csa_adamw_params(**base)
    table = (B.csa_adamw_tensor * len(tensors))(*tensors)
    return B._lib.csa_adamw(ctypes.byref(p), table, len(tensors), None)


def tensor(B, k=1, **kw):
    base = dict(param=addr(10 * k), grad=addr(10 * k + 1), master=None, m=addr(10 * k + 2), v=addr(10 * k + 3),
                m_scale=addr(10 * k + 4), v_scale=addr(10 * k + 5), numel=1000, param_dtype=1, grad_dtype=1, state_dtype=1)
    base.update(kw)
    return B.csa_adamw_tensor(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(lr=float("inf")), 1), (dict(beta1=1.0), 1), (dict(beta2=-0.1), 1), (dict(beta1=float("nan")), 1),
    (dict(eps=-1.0), 1), (dict(weight_decay=float("nan")), 1), (dict(step=0), 1), (dict(lr_dev=addr(90) + 2), 3),
    (dict(step_dev=addr(90) + 4), 3), (dict(grad_scale=addr(90) + 1), 3), (dict(found_inf=addr(90) + 2), 3)])
def test_adamw_params_refused(B, kw, status):
    assert adamw(B, [tensor(B)], **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(param=None), 1), (dict(grad=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(m_scale=None), 1),
    (dict(v_scale=None), 1), (dict(numel=-1), 1), (dict(numel=1 << 41), 2), (dict(param_dtype=2), 1),
    (dict(grad_dtype=-1), 1), (dict(state_dtype=2), 1), (dict(param=addr(90) + 2), 3), (dict(grad=addr(90) + 8), 3),
    (dict(master=addr(90) + 4), 3), (dict(m=addr(90) + 1), 3), (dict(v_scale=addr(90) + 2), 3)])
def test_adamw_tensors_refused(B, kw, status):
    assert adamw(B, [tensor(B, 2), tensor(B, **kw)]) == status


@pytest.mark.parametrize("field", ["param", "m", "v", "m_scale", "v_scale", "master"])
def test_adamw_the_same_buffer_twice_refused(B, field):
    a, b = tensor(B, 1, master=addr(16)), tensor(B, 2, master=addr(26))
    assert adamw(B, [a, b]) == 5                               # past the checks: no GPU
    setattr(b, field, getattr(a, field))
    assert adamw(B, [a, b]) == 1


def test_adamw_of_nothing(B):
    assert adamw(B, []) == 0
    p = B.csa_adamw_params(step=1)
    assert B._lib.csa_adamw(ctypes.byref(p), None, 0, None) == 0
    assert B._lib.csa_adamw(ctypes.byref(p), None, 1, None) == 1
    assert B._lib.csa_adamw(None, None, 0, None) == 1
    assert adamw(B, [tensor(B, numel=0, param=None, grad=None, m=None, v=None)]) == 0


def test_fault_injection_reaches_every_entry(B, monkeypatch):
    monkeypatch.setenv("CSA_FAULT", "timeout")
    assert linear_fwd(B, linear(B)) == linear_bwd(B, linear(B)) == call_rope(B, rope(B)) == adamw(B, [tensor(B)]) == 6
