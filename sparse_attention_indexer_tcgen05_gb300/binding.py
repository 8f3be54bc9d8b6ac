"""Thin PyTorch binding of libcsa_indexer.so (ctypes).

Argument marshalling only: every step of the path runs in the library's CUDA kernels.  PyTorch supplies
device memory (outputs and workspace) and the current stream.  The functions keep the C ABI's names:

    csa_indexer_fwd(params, q_idx, w, k_idx)                        -> (ids, selscore)
    csa_teacher(params, q, kv, kv_c, sink, ids)                     -> teacher
    csa_teacher_from_lse(params, q, kv_c, lse_nc, ids)              -> teacher
    csa_indexer_bwd(params, q_idx, w, k_idx, q, kv, kv_c, sink, ids, selscore[, teacher])
                                                                    -> (loss, dq_idx, dw, dk_idx)
    csa_scores_debug(params, q_idx, w, k_idx, row_begin, row_count) -> scores

Around the step (what makes q_idx, w and k_idx out of hidden states, and updates the weights that do):

    csa_linear_fwd(params, x, weight[, bias, residual])             -> y            (projection with its epilogue)
    csa_linear_bwd(params, dy, x, weight[, preact])                 -> (dx, dw, db)
    csa_rope(params, x, positions, inv_freq)                        -> out          (rotary positions; also their gradient)
    csa_adamw(tensors, step, ...)                                                   (AdamW over many tensors, in place)
    csa_layernorm_fwd(params, x[, weight, bias])                    -> y            (the norm of rows)
    csa_layernorm_bwd(params, dy, x, weight, stats)                 -> (dx, dweight, dbias)

The model's own loss (labels, a teacher's top logits, or both).  The scores of a vocabulary go by without being kept; for gradients the
exponentials of as many rows as 4 GiB hold are (VocabLossParams' piece_rows: of so many):

    csa_vocab_loss_fwd(params, x, weight[, labels, teacher_ids, teacher_logits, teacher_lse])   -> loss
    csa_vocab_loss_bwd(params, x, weight[, ...])                                                -> (loss, dx, dw)

with ``CSALinear`` / ``csa_linear``, ``CSARope`` / ``csa_rotary``, ``CSALayerNorm`` / ``csa_layernorm`` and ``CSAVocabLoss`` /
``csa_vocab_loss`` as their autograd forms.  ``CSAIndexerLoss`` wraps the step as an autograd function (forward returns ids and
the loss; backward returns the stored indexer gradients scaled by the incoming gradient).

Importing this module loads the library and raises ImportError if it has not been built: there is no
fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import warnings

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa_indexer.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python -m sparse_attention_indexer_tcgen05_gb300.build` (or __graft_entry__.build())")

_lib = ctypes.CDLL(LIB_PATH)

SBHD, BSHD, THD = 0, 1, 2
F32, BF16 = 0, 1
LAYOUTS = {"sbhd": SBHD, "bshd": BSHD, "thd": THD}
DTYPES = {"f32": F32, "bf16": BF16, torch.float32: F32, torch.bfloat16: BF16}
TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16}

STATUS = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_ALIGNMENT",
          4: "CSA_ERR_WORKSPACE", 5: "CSA_ERR_CUDA", 6: "CSA_ERR_TIMEOUT"}


# csa_teacher_mode: the full-CSA teacher, or the compressed-only one the issue reports (A/B control)
TEACHER_MODES = {"full": 0, "compressed_only": 1}


class csa_params(ctypes.Structure):
    _fields_ = [
        ("layout", ctypes.c_int32), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32),
        ("seqlen", ctypes.c_int32), ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_q_unpadded", ctypes.c_void_p),
        ("max_seqlen_q", ctypes.c_int32), ("key_rows", ctypes.c_int32), ("compress_ratio", ctypes.c_int32),
        ("window", ctypes.c_int32), ("topk", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float), ("sparse_loss", ctypes.c_int32), ("reduction", ctypes.c_int32),
        ("loss_coeff", ctypes.c_float), ("teacher_mode", ctypes.c_int32),
        ("require_tensor_cores", ctypes.c_int32),
    ]


# csa_activation and csa_state_dtype
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu_tanh": 3}
STATE_F32, STATE_E4M3 = 0, 1
ADAMW_BLOCK = 256      # elements that share one scale of an 8-bit state
NEAREST_BETA2 = 0.89   # up to here a step without gradient moves every e4m3 root by more than half a code
ROPE_MAX_AXES = 4


class csa_linear_params(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("activation", ctypes.c_int32),
        ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("alpha", ctypes.c_float),
        ("rows", ctypes.c_int64), ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
        ("dy_stride", ctypes.c_int64),
    ]


class csa_rope_params(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rot_offset", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
        ("inverse", ctypes.c_int32), ("positions_64", ctypes.c_int32), ("axes", ctypes.c_int32),
        ("sections", ctypes.c_int32 * ROPE_MAX_AXES), ("rows", ctypes.c_int64),
        ("x_row_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
    ]


class csa_layernorm_params(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("cols", ctypes.c_int32), ("eps", ctypes.c_float),
        ("rows", ctypes.c_int64), ("x_stride", ctypes.c_int64), ("dy_stride", ctypes.c_int64),
    ]


class csa_vocab_loss_params(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("features", ctypes.c_int32), ("vocab", ctypes.c_int32), ("slots", ctypes.c_int32),
        ("labels_64", ctypes.c_int32), ("ids_64", ctypes.c_int32), ("reduction", ctypes.c_int32), ("alpha", ctypes.c_float),
        ("label_weight", ctypes.c_float), ("teacher_weight", ctypes.c_float), ("rows", ctypes.c_int64),
        ("x_stride", ctypes.c_int64), ("piece_rows", ctypes.c_int64),
    ]


class csa_vocab_targets(ctypes.Structure):
    _fields_ = [
        ("labels", ctypes.c_void_p), ("teacher_ids", ctypes.c_void_p), ("teacher_logits", ctypes.c_void_p),
        ("teacher_lse", ctypes.c_void_p),
    ]


class csa_adamw_tensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("numel", ctypes.c_int64),
        ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32),
    ]


class csa_adamw_params(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
        ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64), ("lr_dev", ctypes.c_void_p),
        ("step_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p), ("found_inf", ctypes.c_void_p),
        ("seed", ctypes.c_uint64), ("stochastic", ctypes.c_int32),
    ]


_P = ctypes.POINTER(csa_params)
_PL, _PR, _PA = (ctypes.POINTER(t) for t in (csa_linear_params, csa_rope_params, csa_adamw_params))
_PN, _PV, _PT = (ctypes.POINTER(t) for t in (csa_layernorm_params, csa_vocab_loss_params, csa_vocab_targets))
_vp, _sz, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
for _name, _args, _res in [
    ("csa_topk_width", [_P], ctypes.c_int32),
    ("csa_key_width", [_P], ctypes.c_int32),
    ("csa_teacher_width", [_P], ctypes.c_int32),
    ("csa_rows", [_P], ctypes.c_int64),
    ("csa_compressed_rows", [_P], ctypes.c_int64),
    ("csa_workspace_size", [_P], ctypes.c_size_t),
    ("csa_indexer_fwd", [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_teacher", [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_teacher_from_lse", [_P, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_indexer_bwd", [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                         _vp],
     ctypes.c_int),
    ("csa_scores_debug", [_P, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_indexer_bwd_noalloc", [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
     ctypes.c_int),
    ("csa_linear_fwd_workspace_size", [_PL], ctypes.c_size_t),
    ("csa_linear_bwd_workspace_size", [_PL], ctypes.c_size_t),
    ("csa_linear_fwd", [_PL, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_linear_bwd", [_PL, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_rope", [_PR, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    ("csa_adamw", [_PA, _vp, ctypes.c_int32, _vp], ctypes.c_int),
    ("csa_layernorm_bwd_workspace_size", [_PN], ctypes.c_size_t),
    ("csa_layernorm_fwd", [_PN, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    ("csa_layernorm_bwd", [_PN, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_vocab_loss_fwd_workspace_size", [_PV], ctypes.c_size_t),
    ("csa_vocab_loss_bwd_workspace_size", [_PV], ctypes.c_size_t),
    ("csa_vocab_loss_fwd", [_PV, _vp, _vp, _PT, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_vocab_loss_bwd", [_PV, _vp, _vp, _PT, _vp, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
    ("csa_check_device_status", [_vp], ctypes.c_int),
    ("csa_selftest_bounded_wait", [_vp], ctypes.c_int),
    ("csa_last_timeout_site", [], ctypes.c_int32),
    ("csa_last_path", [], ctypes.c_char_p),
    ("csa_last_cuda_error", [], ctypes.c_char_p),
    ("csa_kernel_launches", [], ctypes.c_uint64),
    ("csa_status_string", [ctypes.c_int], ctypes.c_char_p),
]:
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res

EXPORTED = ("csa_topk_width", "csa_key_width", "csa_teacher_width", "csa_rows", "csa_compressed_rows",
            "csa_workspace_size", "csa_indexer_fwd", "csa_teacher", "csa_teacher_from_lse", "csa_indexer_bwd",
            "csa_scores_debug",
            "csa_indexer_bwd_noalloc",
            "csa_linear_fwd_workspace_size", "csa_linear_bwd_workspace_size", "csa_linear_fwd", "csa_linear_bwd",
            "csa_rope", "csa_adamw",
            "csa_layernorm_bwd_workspace_size", "csa_layernorm_fwd", "csa_layernorm_bwd",
            "csa_vocab_loss_fwd_workspace_size", "csa_vocab_loss_bwd_workspace_size", "csa_vocab_loss_fwd",
            "csa_vocab_loss_bwd",
            "csa_check_device_status", "csa_selftest_bounded_wait", "csa_last_timeout_site", "csa_last_path",
            "csa_last_cuda_error",
            "csa_kernel_launches",
            "csa_status_string")


class CSAError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        msg = _lib.csa_status_string(status).decode()
        if status == 5:  # CSA_ERR_CUDA
            msg += " (" + _lib.csa_last_cuda_error().decode() + ")"
        if status == 6:  # CSA_ERR_TIMEOUT
            msg += f" (kernel {_lib.csa_last_timeout_site() // 100}, wait site {_lib.csa_last_timeout_site() % 100})"
        super().__init__(f"{call}: {msg}")


def _check(status: int, call: str):
    if status != 0:
        raise CSAError(status, call)


class Params:
    """Geometry and flags of one step (the C struct csa_params plus references to its cu_seqlens tensors).

    For THD, ``cu_seqlens_q`` / ``cu_seqlens_q_unpadded`` are int32 CUDA tensors, ``batch`` is the number of
    segments, ``seqlen`` the physical rows, ``max_seqlen_q`` the longest unpadded segment (host int) and
    ``key_rows`` the rows of k_idx / kv_c.
    """

    def __init__(self, layout, dtype, batch, seqlen, compress_ratio, window, topk, heads, head_dim, idx_heads,
                 idx_dim, softmax_scale, sparse_loss=True, reduction="mean", loss_coeff=1.0, cu_seqlens_q=None,
                 cu_seqlens_q_unpadded=None, max_seqlen_q=0, key_rows=0, teacher_mode="full",
                 require_tensor_cores=False):
        self.cu = cu_seqlens_q
        self.cur = cu_seqlens_q_unpadded
        for t in (self.cu, self.cur):
            if t is not None and (t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous()):
                raise ValueError("cu_seqlens tensors must be contiguous int32 CUDA tensors")
        lay = LAYOUTS[layout] if isinstance(layout, str) else int(layout)
        if lay == THD and self.cu is not None:
            batch = self.cu.numel() - 1
        self.c = csa_params(lay, DTYPES[dtype] if not isinstance(dtype, int) else dtype, int(batch), int(seqlen),
                            self.cu.data_ptr() if self.cu is not None else None,
                            self.cur.data_ptr() if self.cur is not None else None, int(max_seqlen_q), int(key_rows),
                            int(compress_ratio), int(window), int(topk), int(heads), int(head_dim), int(idx_heads),
                            int(idx_dim), float(softmax_scale), 1 if sparse_loss else 0,
                            0 if reduction in ("mean", 0) else 1, float(loss_coeff),
                            TEACHER_MODES[teacher_mode] if isinstance(teacher_mode, str) else int(teacher_mode),
                            1 if require_tensor_cores else 0)

    @property
    def ref(self):
        return ctypes.byref(self.c)

    @property
    def K(self) -> int:
        return _lib.csa_topk_width(self.ref)

    @property
    def key_width(self) -> int:
        return _lib.csa_key_width(self.ref)

    @property
    def teacher_width(self) -> int:
        return _lib.csa_teacher_width(self.ref)

    @property
    def rows(self) -> int:
        return _lib.csa_rows(self.ref)

    @property
    def compressed_rows(self) -> int:
        return _lib.csa_compressed_rows(self.ref)

    @property
    def workspace_bytes(self) -> int:
        return _lib.csa_workspace_size(self.ref)

    @property
    def value_dtype(self) -> torch.dtype:
        return TORCH_DTYPE[self.c.dtype]


def csa_topk_width(p: Params) -> int:
    return p.K


def csa_workspace_size(p: Params) -> int:
    return p.workspace_bytes


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _check_tensor(t, name, dtype, device, numel=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def _workspace(p: Params, device, workspace):
    n = p.workspace_bytes
    if workspace is None:
        workspace = torch.empty(max(n, 1), dtype=torch.uint8, device=device)
    return workspace, workspace.numel()


@contextlib.contextmanager
def _nvtx(name):
    torch.cuda.nvtx.range_push(name)
    try:
        yield
    finally:
        torch.cuda.nvtx.range_pop()


def csa_indexer_fwd(p: Params, q_idx, w, k_idx, workspace=None, ids=None, selscore=None):
    """Steps 1-2: scores + top-k.  Returns (ids [rows, K] int32, selscore [rows, K] fp32)."""
    dev = q_idx.device
    rows, K, HI, DI = p.rows, p.K, p.c.idx_heads, p.c.idx_dim
    _check_tensor(q_idx, "q_idx", p.value_dtype, dev, rows * HI * DI)
    _check_tensor(w, "w", torch.float32, dev, rows * HI)
    _check_tensor(k_idx, "k_idx", p.value_dtype, dev, p.compressed_rows * DI)
    if ids is None:
        ids = torch.empty((rows, K), dtype=torch.int32, device=dev)
    if selscore is None:
        selscore = torch.empty((rows, K), dtype=torch.float32, device=dev)
    ws, nws = _workspace(p, dev, workspace)
    with _nvtx("csa_indexer_fwd"):
        st = _lib.csa_indexer_fwd(p.ref, _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(ids), _ptr(selscore), _ptr(ws), nws,
                                  _stream(dev))
    _check(st, "csa_indexer_fwd")
    return ids, selscore


def csa_teacher(p: Params, q, kv, kv_c, sink, ids, workspace=None, out=None):
    """Step 3: full-CSA teacher for the given ids.  Returns teacher [rows, teacher_width] fp32."""
    dev = q.device
    rows, H, D = p.rows, p.c.heads, p.c.head_dim
    _check_tensor(q, "q", p.value_dtype, dev, rows * H * D)
    _check_tensor(kv, "kv", p.value_dtype, dev, rows * D)
    _check_tensor(kv_c, "kv_c", p.value_dtype, dev, p.compressed_rows * D)
    _check_tensor(sink, "sink", torch.float32, dev, H)
    _check_tensor(ids, "ids", torch.int32, dev, rows * p.K)
    if out is None:
        out = torch.empty((rows, p.teacher_width), dtype=torch.float32, device=dev)
    ws, nws = _workspace(p, dev, workspace)
    with _nvtx("csa_teacher"):
        st = _lib.csa_teacher(p.ref, _ptr(q), _ptr(kv), _ptr(kv_c), _ptr(sink), _ptr(ids), _ptr(out), _ptr(ws), nws,
                              _stream(dev))
    _check(st, "csa_teacher")
    return out


def csa_teacher_from_lse(p: Params, q, kv_c, lse_nc, ids, workspace=None, out=None):
    """Step 3 from a given non-compressed log-sum-exp lse_nc [rows, heads] fp32 (natural log of exp(sink) plus
    the window's exponentials, per row and head).  Returns teacher [rows, teacher_width] fp32."""
    dev = q.device
    rows, H, D = p.rows, p.c.heads, p.c.head_dim
    _check_tensor(q, "q", p.value_dtype, dev, rows * H * D)
    _check_tensor(kv_c, "kv_c", p.value_dtype, dev, p.compressed_rows * D)
    _check_tensor(lse_nc, "lse_nc", torch.float32, dev, rows * H)
    _check_tensor(ids, "ids", torch.int32, dev, rows * p.K)
    if out is None:
        out = torch.empty((rows, p.teacher_width), dtype=torch.float32, device=dev)
    ws, nws = _workspace(p, dev, workspace)
    with _nvtx("csa_teacher_from_lse"):
        st = _lib.csa_teacher_from_lse(p.ref, _ptr(q), _ptr(kv_c), _ptr(lse_nc), _ptr(ids), _ptr(out), _ptr(ws), nws,
                                       _stream(dev))
    _check(st, "csa_teacher_from_lse")
    return out


def csa_indexer_bwd(p: Params, q_idx, w, k_idx, q, kv, kv_c, sink, ids, selscore, teacher=None, workspace=None,
                    out=None, row_loss=None):
    """Steps 3-5: teacher (unless given), KL and indexer gradients.
    Returns (loss [] fp32, dq_idx like q_idx, dw like w, dk_idx like k_idx).  If row_loss (a [rows] fp32 tensor)
    is given, it receives the unscaled per-row KL."""
    dev = q_idx.device
    rows, K, HI, DI = p.rows, p.K, p.c.idx_heads, p.c.idx_dim
    _check_tensor(q_idx, "q_idx", p.value_dtype, dev, rows * HI * DI)
    _check_tensor(w, "w", torch.float32, dev, rows * HI)
    _check_tensor(k_idx, "k_idx", p.value_dtype, dev, p.compressed_rows * DI)
    _check_tensor(ids, "ids", torch.int32, dev, rows * K)
    _check_tensor(selscore, "selscore", torch.float32, dev, rows * K)
    if teacher is None:
        H, D = p.c.heads, p.c.head_dim
        _check_tensor(q, "q", p.value_dtype, dev, rows * H * D)
        _check_tensor(kv, "kv", p.value_dtype, dev, rows * D)
        _check_tensor(kv_c, "kv_c", p.value_dtype, dev, p.compressed_rows * D)
        _check_tensor(sink, "sink", torch.float32, dev, H)
    else:
        _check_tensor(teacher, "teacher", torch.float32, dev, rows * p.teacher_width)
    if out is None:
        out = (torch.empty((), dtype=torch.float32, device=dev), torch.empty_like(q_idx), torch.empty_like(w),
               torch.empty_like(k_idx))
    loss, dq, dw, dk = out
    if row_loss is not None:
        _check_tensor(row_loss, "row_loss", torch.float32, dev, rows)
    ws, nws = _workspace(p, dev, workspace)
    with _nvtx("csa_indexer_bwd"):
        st = _lib.csa_indexer_bwd(p.ref, _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q), _ptr(kv), _ptr(kv_c), _ptr(sink),
                                  _ptr(ids), _ptr(selscore), _ptr(teacher), _ptr(loss), _ptr(row_loss), _ptr(dq),
                                  _ptr(dw), _ptr(dk), _ptr(ws), nws, _stream(dev))
    _check(st, "csa_indexer_bwd")
    return loss, dq, dw, dk


NOALLOC_SCRATCH_BYTES = 64 << 20


def csa_indexer_bwd_noalloc(p: Params, q_idx, w, k_idx, q, kv, kv_c, sink, ids, selscore, teacher=None, out=None,
                            row_loss=None):
    """csa_indexer_bwd without a workspace, for callers that cannot allocate device memory: the library uses
    its own fixed 64 MiB device scratch (shared by every call on a device; serialise overlapping calls).
    Returns (loss, dq_idx, dw, dk_idx); raises CSAError (CSA_ERR_WORKSPACE) if the problem needs more scratch."""
    dev = q_idx.device
    rows = p.rows
    if out is None:
        out = (torch.empty((), dtype=torch.float32, device=dev), torch.empty_like(q_idx), torch.empty_like(w),
               torch.empty_like(k_idx))
    loss, dq, dw, dk = out
    with _nvtx("csa_indexer_bwd_noalloc"):
        st = _lib.csa_indexer_bwd_noalloc(p.ref, _ptr(q_idx), _ptr(w), _ptr(k_idx), _ptr(q), _ptr(kv), _ptr(kv_c),
                                          _ptr(sink), _ptr(ids), _ptr(selscore), _ptr(teacher), _ptr(loss),
                                          _ptr(row_loss), _ptr(dq), _ptr(dw), _ptr(dk), _stream(dev))
    _check(st, "csa_indexer_bwd_noalloc")
    return loss, dq, dw, dk


def csa_scores_debug(p: Params, q_idx, w, k_idx, row_begin=0, row_count=None, workspace=None):
    """Test aid: the fp32 scores the forward selects from, [row_count, key_width] (-inf where not visible)."""
    dev = q_idx.device
    if row_count is None:
        row_count = p.rows - row_begin
    out = torch.empty((row_count, p.key_width), dtype=torch.float32, device=dev)
    ws, nws = _workspace(p, dev, workspace)
    st = _lib.csa_scores_debug(p.ref, _ptr(q_idx), _ptr(w), _ptr(k_idx), int(row_begin), int(row_count), _ptr(out),
                               _ptr(ws), nws, _stream(dev))
    _check(st, "csa_scores_debug")
    return out


def csa_check_device_status(device=None):
    st = _lib.csa_check_device_status(_stream(device) if torch.cuda.is_available() else None)
    _check(st, "csa_check_device_status")


def csa_last_path() -> str:
    return _lib.csa_last_path().decode()


def csa_last_timeout_site() -> int:
    """100 x kernel + wait site of the last timeout csa_check_device_status reported (0 before any)."""
    return int(_lib.csa_last_timeout_site())


def csa_last_cuda_error() -> str:
    return _lib.csa_last_cuda_error().decode()


def csa_kernel_launches() -> int:
    return int(_lib.csa_kernel_launches())


class CSAIndexerLoss(torch.autograd.Function):
    """ids, loss = CSAIndexerLoss.apply(q_idx, w, k_idx, q, kv, kv_c, sink, params).

    The forward runs the whole step (scores + top-k, teacher, KL, gradients) and keeps only the three
    indexer gradients for the backward, so no score graph is ever retained.  Gradients flow to q_idx,
    w and k_idx only; q, kv, kv_c and sink receive none (they are the detached teacher side)."""

    @staticmethod
    def forward(ctx, q_idx, w, k_idx, q, kv, kv_c, sink, params):
        ids, sel = csa_indexer_fwd(params, q_idx.contiguous(), w.contiguous(), k_idx.contiguous())
        loss, dq, dw, dk = csa_indexer_bwd(params, q_idx.contiguous(), w.contiguous(), k_idx.contiguous(),
                                           q.contiguous(), kv.contiguous(), kv_c.contiguous(), sink.contiguous(),
                                           ids, sel)
        ctx.save_for_backward(dq, dw, dk)
        ctx.mark_non_differentiable(ids)
        return ids, loss

    @staticmethod
    def backward(ctx, _gid, gloss):
        dq, dw, dk = ctx.saved_tensors
        return (dq * gloss.to(dq.dtype), dw * gloss, dk * gloss.to(dk.dtype), None, None, None, None, None)


def csa_indexer_loss(q_idx, w, k_idx, q, kv, kv_c, sink, params: Params):
    return CSAIndexerLoss.apply(q_idx, w, k_idx, q, kv, kv_c, sink, params)


# ------------------------------------------------------------------ around the step

# These calls are short enough that the host side shows: one expression checks a tensor, the error is found afterwards.

_raw_stream = torch._C._cuda_getCurrentRawStream
_push, _pop = torch.cuda.nvtx.range_push, torch.cuda.nvtx.range_pop
_current_device = torch._C._cuda_getDevice
# torch's allocation without its dispatcher (on the current device), 4 us less in a call; not every build has it
_quick_empty = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


# Kernels write through addresses.  Autograd learns from its version counter that a tensor of the caller's has changed, and
# refuses a backward pass that would read what a forward pass saved of it.
_changed = torch.autograd.graph.increment_version


def _empty(shape, strides, dtype, index):
    if _quick_empty is not None and _current_device() == index:
        return _quick_empty(shape, strides, dtype)
    return torch.empty_strided(shape, strides, dtype=dtype, device=torch.device("cuda", index))


def _invoke(name, fn, device_index, *args):
    """fn(*args, stream) with the tensors' device as the current one (launches go there), inside an NVTX range."""
    _push(name)
    try:
        if _current_device() == device_index:
            st = fn(*args, _raw_stream(device_index))
        else:
            with torch.cuda.device(device_index):
                st = fn(*args, _raw_stream(device_index))
    finally:
        _pop()
    if st != 0:
        raise CSAError(st, name)


def _on_cuda(t, name):
    """The index of t's device."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _check_flat(t, name, dtype, index, numel):
    """A contiguous tensor of `numel` values on device `index`."""
    if t is not None and t.dtype is dtype and t.get_device() == index and t.numel() == numel and t.is_contiguous():
        return
    _check_tensor(t, name, dtype, torch.device("cuda", index), numel)


def _check_weight(t, dtype, index, out_features, in_features):
    """[out_features, in_features]; one of as many values that lies the other way round is refused."""
    if (t is not None and t.dtype is dtype and t.get_device() == index and t.shape == (out_features, in_features) and
            t.is_contiguous()):
        return
    _check_flat(t, "weight", dtype, index, out_features * in_features)
    if t.dim() > 1 and t.shape[-1] != in_features:
        raise ValueError(f"weight has shape {tuple(t.shape)}, expected [{out_features}, {in_features}]")


def _dtype(d):
    if isinstance(d, int) and d in TORCH_DTYPE:
        return d
    if d not in DTYPES:
        raise ValueError(f"dtype must be f32 or bf16, got {d}")
    return DTYPES[d]


def _check_rows(t, name, dtype, index, rows, cols, stride):
    """A [rows, cols] tensor whose rows lie `stride` elements apart (0: cols; leading dimensions may be folded into
    rows)."""
    if (t is not None and t.dtype is dtype and t.get_device() == index and t.shape == (rows, cols) and
            t.is_contiguous() and (not stride or stride == cols)):
        return
    device = torch.device("cuda", index)
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() < 1 or t.shape[-1] != cols or t.numel() != rows * cols:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{rows}, {cols}]")
    if t.numel() == 0:
        return
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    expect = stride or cols
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n > 1 and st != expect:
            raise ValueError(f"{name} has row stride {st}, expected {expect}")
        expect = expect * n


class LinearParams:
    """One projection y = act(alpha x W^T + bias) + residual (the C struct csa_linear_params): x [rows, in_features],
    W [out_features, in_features].  dtype is that of x, W and their gradients; out_dtype that of y, residual and dy
    (dtype, or f32).  Strides are elements from row to row, 0 for contiguous rows."""

    def __init__(self, rows, in_features, out_features, dtype="bf16", out_dtype=None, activation="none", alpha=1.0,
                 x_stride=0, residual_stride=0, dy_stride=0):
        if isinstance(activation, str):
            if activation not in ACTIVATIONS:
                raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation}")
            activation = ACTIVATIONS[activation]
        dt = _dtype(dtype)
        self.c = csa_linear_params(dt, dt if out_dtype is None else _dtype(out_dtype), int(activation),
                                   int(in_features), int(out_features), float(alpha), int(rows), int(x_stride),
                                   int(residual_stride), int(dy_stride))
        self.ref = ctypes.byref(self.c)
        self.value_dtype, self.out_value_dtype = TORCH_DTYPE[self.c.dtype], TORCH_DTYPE[self.c.out_dtype]

    @property
    def fwd_workspace_bytes(self) -> int:
        return _lib.csa_linear_fwd_workspace_size(self.ref)

    @property
    def bwd_workspace_bytes(self) -> int:
        return _lib.csa_linear_bwd_workspace_size(self.ref)

    @property
    def workspace_bytes(self) -> int:
        """Enough for either direction."""
        return max(self.fwd_workspace_bytes, self.bwd_workspace_bytes)


def _check_workspace(workspace, index):
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{index}")
    return workspace.data_ptr(), workspace.nbytes


def csa_linear_fwd(p: LinearParams, x, weight, bias=None, residual=None, workspace=None, out=None, preact=None):
    """y = act(alpha x weight^T + bias) + residual, in one pass with fp32 sums.  Returns y [rows, out_features].
    preact (a [rows, out_features] tensor of p's dtype) receives the activation's argument, which csa_linear_bwd reads.
    out may be the residual itself (contiguous)."""
    c, dev = p.c, _on_cuda(x, "x")
    M, K, N = c.rows, c.in_features, c.out_features
    _check_rows(x, "x", p.value_dtype, dev, M, K, c.x_stride)
    _check_weight(weight, p.value_dtype, dev, N, K)
    if bias is not None:
        _check_flat(bias, "bias", torch.float32, dev, N)
    if residual is not None:
        _check_rows(residual, "residual", p.out_value_dtype, dev, M, N, c.residual_stride)
    given = out is not None
    if not given:
        out = _empty((M, N), (N, 1), p.out_value_dtype, dev)
    else:
        _check_flat(out, "out", p.out_value_dtype, dev, M * N)
    if preact is not None:
        _check_flat(preact, "preact", p.value_dtype, dev, M * N)
    if workspace is None:
        workspace = _empty((p.fwd_workspace_bytes,), (1,), torch.uint8, dev)
    ws, nws = _check_workspace(workspace, dev)
    _invoke("csa_linear_fwd", _lib.csa_linear_fwd, dev, p.ref, x.data_ptr(), weight.data_ptr(), _ptr(bias),
            _ptr(residual), out.data_ptr(), _ptr(preact), ws, nws)
    if given:
        _changed(out)
    if preact is not None:
        _changed(preact)
    return out


def csa_linear_bwd(p: LinearParams, dy, x, weight, preact=None, need_dx=True, need_dw=True, need_db=True, workspace=None,
                   out=None):
    """The gradients of csa_linear_fwd for dy: (dx [rows, in_features], dw like weight, db [out_features] fp32), None
    in the place of one that is not asked for.  preact is what the forward wrote there (not read without an
    activation).  out: a tuple of the three to write to."""
    c, dev = p.c, _on_cuda(dy, "dy")
    M, K, N = c.rows, c.in_features, c.out_features
    _check_rows(dy, "dy", p.out_value_dtype, dev, M, N, c.dy_stride)
    if need_dw:
        _check_rows(x, "x", p.value_dtype, dev, M, K, c.x_stride)
    if need_dx:
        _check_weight(weight, p.value_dtype, dev, N, K)
    if c.activation != 0:
        _check_flat(preact, "preact", p.value_dtype, dev, M * N)
    else:
        preact = None

    def output(i, name, shape, strides, dtype, numel):
        if out is None or out[i] is None:
            return _empty(shape, strides, dtype, dev)
        _check_flat(out[i], name, dtype, dev, numel)
        return out[i]

    dx = output(0, "dx", (M, K), (K, 1), p.value_dtype, M * K) if need_dx else None
    dw = output(1, "dw", (N, K), (K, 1), p.value_dtype, N * K) if need_dw else None
    db = output(2, "db", (N,), (1,), torch.float32, N) if need_db else None
    if workspace is None:
        workspace = _empty((p.bwd_workspace_bytes,), (1,), torch.uint8, dev)
    ws, nws = _check_workspace(workspace, dev)
    _invoke("csa_linear_bwd", _lib.csa_linear_bwd, dev, p.ref, dy.data_ptr(), _ptr(x), _ptr(weight), _ptr(preact),
            _ptr(dx), _ptr(dw), _ptr(db), ws, nws)
    if out is not None:
        _changed([t for t in (dx, dw, db) if t is not None])
    return dx, dw, db


class RopeParams:
    """Rotary positions on [rows, heads, head_dim] values (the C struct csa_rope_params).  rot_dim values from
    rot_offset on rotate (default: all); sections gives the frequency pairs of each position axis (default: one axis);
    interleaved pairs are (2 i, 2 i + 1), others (i, i + rot_dim / 2); inverse turns back (the gradient)."""

    def __init__(self, rows, heads, head_dim, dtype="bf16", rot_dim=None, rot_offset=0, sections=None,
                 interleaved=False, inverse=False, positions_64=False, x_row_stride=0, x_head_stride=0,
                 out_row_stride=0, out_head_stride=0):
        rot_dim = int(head_dim - rot_offset if rot_dim is None else rot_dim)
        sections = [rot_dim // 2] if sections is None else [int(n) for n in sections]
        if not 1 <= len(sections) <= ROPE_MAX_AXES:
            raise ValueError(f"sections must name 1 to {ROPE_MAX_AXES} axes, got {len(sections)}")
        self.c = csa_rope_params(_dtype(dtype), int(heads), int(head_dim), int(rot_offset), rot_dim,
                                 1 if interleaved else 0, 1 if inverse else 0, 1 if positions_64 else 0, len(sections),
                                 (ctypes.c_int32 * ROPE_MAX_AXES)(*sections), int(rows), int(x_row_stride),
                                 int(x_head_stride), int(out_row_stride), int(out_head_stride))
        self.ref = ctypes.byref(self.c)
        self.value_dtype = TORCH_DTYPE[self.c.dtype]

    def inverted(self) -> "RopeParams":
        """The same rotation backwards, on contiguous values: what a gradient of out takes."""
        c = self.c
        return RopeParams(c.rows, c.heads, c.head_dim, c.dtype, c.rot_dim, c.rot_offset, list(c.sections[:c.axes]),
                          c.interleaved, not c.inverse, c.positions_64)


def _check_heads(t, name, p, index, row_stride, head_stride):
    c = p.c
    if (not row_stride and not head_stride and t.dtype is p.value_dtype and t.get_device() == index and
            t.is_contiguous() and t.numel() == c.rows * c.heads * c.head_dim):
        return
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    if t.dtype != p.value_dtype:
        raise ValueError(f"{name} must be {p.value_dtype}, got {t.dtype}")
    head_stride = head_stride or c.head_dim
    row_stride = row_stride or c.heads * head_stride
    if head_stride == c.head_dim and row_stride == c.heads * head_stride:  # contiguous: any shape of that many values
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (or its strides given to RopeParams)")
        if t.numel() != c.rows * c.heads * c.head_dim:
            raise ValueError(f"{name} has {t.numel()} elements, expected {c.rows * c.heads * c.head_dim}")
        return
    if tuple(t.shape) != (c.rows, c.heads, c.head_dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(c.rows, c.heads, c.head_dim)}")
    want = (row_stride, head_stride, 1)
    if t.numel() and any(n > 1 and a != b for n, a, b in zip(t.shape, t.stride(), want)):
        raise ValueError(f"{name} has strides {t.stride()}, expected {want}")


def csa_rope(p: RopeParams, x, positions, inv_freq, out=None):
    """x [rows, heads, head_dim] with its pairs turned by positions [axes, rows] (int32, or int64 with positions_64)
    times inv_freq [rot_dim / 2] (fp64).  Returns out; out=x works in place."""
    c, dev = p.c, _on_cuda(x, "x")
    _check_heads(x, "x", p, dev, c.x_row_stride, c.x_head_stride)
    _check_flat(positions, "positions", torch.int64 if c.positions_64 else torch.int32, dev, c.axes * c.rows)
    if c.axes > 1 and positions.dim() > 1 and positions.shape[0] != c.axes:
        raise ValueError(f"positions has shape {tuple(positions.shape)}, expected [{c.axes}, {c.rows}]")
    _check_flat(inv_freq, "inv_freq", torch.float64, dev, c.rot_dim // 2)
    given = out is not None
    if not given:
        if c.out_row_stride or c.out_head_stride:
            raise ValueError("out is required where RopeParams gives its strides")
        out = _empty(tuple(x.shape), x.stride(), x.dtype, dev) if x.is_contiguous() else \
            _empty((c.rows, c.heads, c.head_dim), (c.heads * c.head_dim, c.head_dim, 1), x.dtype, dev)
    else:
        _check_heads(out, "out", p, dev, c.out_row_stride, c.out_head_stride)
    _invoke("csa_rope", _lib.csa_rope, dev, p.ref, x.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), out.data_ptr())
    if given:
        _changed(out)
    return out


class LayerNormParams:
    """The norm of rows of `cols` values (the C struct csa_layernorm_params).  param_dtype is that of weight, bias and their
    gradients.  Strides are elements from row to row, 0 for contiguous rows."""

    def __init__(self, rows, cols, dtype="bf16", param_dtype="f32", eps=1e-5, x_stride=0, dy_stride=0):
        self.c = csa_layernorm_params(_dtype(dtype), _dtype(param_dtype), int(cols), float(eps), int(rows), int(x_stride),
                                      int(dy_stride))
        self.ref = ctypes.byref(self.c)
        self.value_dtype, self.param_value_dtype = TORCH_DTYPE[self.c.dtype], TORCH_DTYPE[self.c.param_dtype]

    @property
    def bwd_workspace_bytes(self) -> int:
        return _lib.csa_layernorm_bwd_workspace_size(self.ref)


def csa_layernorm_fwd(p: LayerNormParams, x, weight=None, bias=None, out=None, stats=None):
    """y = (x - mean) rstd weight + bias of each row of x [rows, cols] (weight None: ones, bias None: zeros).  Returns y.
    stats (a [2, rows] fp32 tensor) receives the rows' means and rstd, which csa_layernorm_bwd reads.  out may be x itself
    (contiguous)."""
    c, dev = p.c, _on_cuda(x, "x")
    M, N = c.rows, c.cols
    _check_rows(x, "x", p.value_dtype, dev, M, N, c.x_stride)
    if weight is not None:
        _check_flat(weight, "weight", p.param_value_dtype, dev, N)
    if bias is not None:
        _check_flat(bias, "bias", p.param_value_dtype, dev, N)
    given = out is not None
    if not given:
        out = _empty((M, N), (N, 1), p.value_dtype, dev)
    else:
        _check_flat(out, "out", p.value_dtype, dev, M * N)
    if stats is not None:
        _check_flat(stats, "stats", torch.float32, dev, 2 * M)
    _invoke("csa_layernorm_fwd", _lib.csa_layernorm_fwd, dev, p.ref, x.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(),
            _ptr(stats))
    if given:
        _changed(out)
    if stats is not None:
        _changed(stats)
    return out


def csa_layernorm_bwd(p: LayerNormParams, dy, x, weight=None, stats=None, need_dx=True, need_dweight=True, need_dbias=True,
                      workspace=None, out=None):
    """The gradients of csa_layernorm_fwd for dy: (dx [rows, cols], dweight [cols], dbias [cols]), None in the place of one
    that is not asked for.  stats is what the forward wrote there.  out: a tuple of the three to write to; dx may be dy or x
    (contiguous)."""
    c, dev = p.c, _on_cuda(dy, "dy")
    M, N = c.rows, c.cols
    _check_rows(dy, "dy", p.value_dtype, dev, M, N, c.dy_stride)
    if need_dx or need_dweight or need_dbias:
        _check_rows(x, "x", p.value_dtype, dev, M, N, c.x_stride)
        _check_flat(stats, "stats", torch.float32, dev, 2 * M)
    if weight is not None:
        _check_flat(weight, "weight", p.param_value_dtype, dev, N)

    def output(i, name, need, shape, strides, dtype):
        if not need:
            return None
        if out is None or out[i] is None:
            return _empty(shape, strides, dtype, dev)
        _check_flat(out[i], name, dtype, dev, M * N if i == 0 else N)
        return out[i]

    dx = output(0, "dx", need_dx, (M, N), (N, 1), p.value_dtype)
    dw = output(1, "dweight", need_dweight, (N,), (1,), p.param_value_dtype)
    db = output(2, "dbias", need_dbias, (N,), (1,), p.param_value_dtype)
    if workspace is None:
        workspace = _empty((p.bwd_workspace_bytes,), (1,), torch.uint8, dev)
    ws, nws = _check_workspace(workspace, dev)
    _invoke("csa_layernorm_bwd", _lib.csa_layernorm_bwd, dev, p.ref, dy.data_ptr(), _ptr(x), _ptr(weight), _ptr(stats), _ptr(dx),
            _ptr(dw), _ptr(db), ws, nws)
    if out is not None:
        _changed([t for t in (dx, dw, db) if t is not None])
    return dx, dw, db


class VocabLossParams:
    """Losses of the scores z = alpha x W^T (the C struct csa_vocab_loss_params): x [rows, features], W [vocab, features].
    alpha scales the scores of both losses; a teacher's logits are taken as they are given (at a temperature: divided by the caller).
    slots: a teacher's candidates a row (0: labels alone; a call may leave the teacher, or the labels, out).  reduction "mean": each loss over the rows that have it; "sum".
    piece_rows: rows whose scores' exponentials are held at a time for gradients (0: as many as 4 GiB hold)."""

    def __init__(self, rows, features, vocab, dtype="bf16", slots=0, alpha=1.0, label_weight=1.0, teacher_weight=1.0,
                 reduction="mean", labels_64=False, ids_64=False, x_stride=0, piece_rows=0):
        if reduction not in ("mean", "sum"):
            raise ValueError(f"reduction must be mean or sum, got {reduction}")
        self.c = csa_vocab_loss_params(_dtype(dtype), int(features), int(vocab), int(slots), 1 if labels_64 else 0,
                                       1 if ids_64 else 0, 0 if reduction == "mean" else 1, float(alpha), float(label_weight),
                                       float(teacher_weight), int(rows), int(x_stride), int(piece_rows))
        self.ref = ctypes.byref(self.c)
        self.value_dtype = TORCH_DTYPE[self.c.dtype]

    @property
    def fwd_workspace_bytes(self) -> int:
        return _lib.csa_vocab_loss_fwd_workspace_size(self.ref)

    @property
    def bwd_workspace_bytes(self) -> int:
        return _lib.csa_vocab_loss_bwd_workspace_size(self.ref)


def _vocab_targets(p, dev, labels, teacher_ids, teacher_logits, teacher_lse):
    """The targets' addresses.  Without slots the teacher's tensors are refused; with them either target may be left out."""
    c = p.c
    if labels is not None:
        _check_flat(labels, "labels", torch.int64 if c.labels_64 else torch.int32, dev, c.rows)
    taught = teacher_ids is not None or teacher_logits is not None or teacher_lse is not None
    if taught and not c.slots:
        raise ValueError("a teacher needs VocabLossParams(slots=...)")
    if taught:
        for name, t, dtype in (("teacher_ids", teacher_ids, torch.int64 if c.ids_64 else torch.int32),
                               ("teacher_logits", teacher_logits, torch.float32)):
            _check_flat(t, name, dtype, dev, c.rows * c.slots)
            if t.dim() > 1 and t.shape[-1] != c.slots:
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{c.rows}, {c.slots}]")
        if teacher_lse is not None:
            _check_flat(teacher_lse, "teacher_lse", torch.float32, dev, c.rows)
    elif labels is None:
        raise ValueError("labels or a teacher are required")
    return csa_vocab_targets(_ptr(labels), _ptr(teacher_ids), _ptr(teacher_logits), _ptr(teacher_lse))


def csa_vocab_loss_fwd(p: VocabLossParams, x, weight, labels=None, teacher_ids=None, teacher_logits=None, teacher_lse=None,
                       row_loss=None, workspace=None, out=None):
    """The loss (a device scalar) of labels [rows] (negative: none), of a teacher's candidates teacher_ids [rows, slots]
    (negative: none) with their teacher_logits (f32), or of both.  teacher_lse [rows]: the teacher's own log-sum-exp; without
    it the candidates' shares sum to 1.  row_loss (a [2, rows] f32 tensor) receives the rows' label and teacher losses."""
    c, dev = p.c, _on_cuda(x, "x")
    _check_rows(x, "x", p.value_dtype, dev, c.rows, c.features, c.x_stride)
    _check_weight(weight, p.value_dtype, dev, c.vocab, c.features)
    targets = _vocab_targets(p, dev, labels, teacher_ids, teacher_logits, teacher_lse)
    given = out is not None
    if not given:
        out = _empty((), (), torch.float32, dev)
    else:
        _check_flat(out, "out", torch.float32, dev, 1)
    if row_loss is not None:
        _check_flat(row_loss, "row_loss", torch.float32, dev, 2 * c.rows)
    if workspace is None:
        workspace = _empty((p.fwd_workspace_bytes,), (1,), torch.uint8, dev)
    ws, nws = _check_workspace(workspace, dev)
    _invoke("csa_vocab_loss_fwd", _lib.csa_vocab_loss_fwd, dev, p.ref, x.data_ptr(), weight.data_ptr(), ctypes.byref(targets),
            out.data_ptr(), _ptr(row_loss), ws, nws)
    if given:
        _changed(out)
    if row_loss is not None:
        _changed(row_loss)
    return out


def csa_vocab_loss_bwd(p: VocabLossParams, x, weight, labels=None, teacher_ids=None, teacher_logits=None, teacher_lse=None,
                       row_loss=None, need_dx=True, need_dw=True, workspace=None, out=None):
    """The loss of csa_vocab_loss_fwd and its gradients: (loss, dx [rows, features], dw [vocab, features]), None in the place
    of one that is not asked for.  out: a tuple of the three to write to."""
    c, dev = p.c, _on_cuda(x, "x")
    M, K, V = c.rows, c.features, c.vocab
    _check_rows(x, "x", p.value_dtype, dev, M, K, c.x_stride)
    _check_weight(weight, p.value_dtype, dev, V, K)
    targets = _vocab_targets(p, dev, labels, teacher_ids, teacher_logits, teacher_lse)

    def output(i, name, need, shape, strides, dtype, numel):
        if not need:
            return None
        if out is None or out[i] is None:
            return _empty(shape, strides, dtype, dev)
        _check_flat(out[i], name, dtype, dev, numel)
        return out[i]

    loss = output(0, "loss", True, (), (), torch.float32, 1)
    dx = output(1, "dx", need_dx, (M, K), (K, 1), p.value_dtype, M * K)
    dw = output(2, "dw", need_dw, (V, K), (K, 1), p.value_dtype, V * K)
    if row_loss is not None:
        _check_flat(row_loss, "row_loss", torch.float32, dev, 2 * M)
    if workspace is None:
        workspace = _empty((p.bwd_workspace_bytes,), (1,), torch.uint8, dev)
    ws, nws = _check_workspace(workspace, dev)
    _invoke("csa_vocab_loss_bwd", _lib.csa_vocab_loss_bwd, dev, p.ref, x.data_ptr(), weight.data_ptr(), ctypes.byref(targets),
            loss.data_ptr(), _ptr(row_loss), _ptr(dx), _ptr(dw), ws, nws)
    if out is not None:
        _changed([t for t in (loss, dx, dw) if t is not None])
    if row_loss is not None:
        _changed(row_loss)
    return loss, dx, dw


class AdamWTensors:
    """The tensors of csa_adamw, checked and laid out once.  Lists of equal length: param (f32 or bf16), grad (f32 or
    bf16), the moments m and v (both f32, or both float8_e4m3fn with their f32 scales m_scale and v_scale, one per
    ADAMW_BLOCK elements, last block short), and master: an f32 copy that the step updates, param being its rounding
    (a list, with None for a tensor that has none).  ``AdamWTensors.zero_state`` makes m, v and scales.

    seed (an integer; zero_state gives one with 8-bit moments) rounds 8-bit moments stochastically, by a hash of seed,
    tensor, element and step: they then follow their recurrences.  None rounds to nearest, which over many steps follows
    changes of more than half a code (5.6 %) a step only: beta2 up to NEAREST_BETA2."""

    def __init__(self, param, grad, m, v, m_scale=None, v_scale=None, master=None, seed=None):
        n = len(param)
        none = [None] * n
        columns = dict(param=list(param), grad=list(grad), m=list(m), v=list(v), m_scale=list(m_scale or none),
                       v_scale=list(v_scale or none), master=list(master or none))
        for name, c in columns.items():
            if len(c) != n:
                raise ValueError(f"{name} has {len(c)} tensors, param has {n}")
        self.tensors = columns                       # keeps the buffers alive
        self.device = param[0].device if n else None
        self.count = n
        self.seed = None if seed is None else int(seed) % 2 ** 64
        self.nearest = False                         # whether 8-bit moments are rounded to nearest
        self.table = (csa_adamw_tensor * n)()
        for i, e in enumerate(self.table):
            t = {name: c[i] for name, c in columns.items()}
            numel = t["param"].numel()
            for name in ("param", "grad"):
                if t[name].dtype not in DTYPES:
                    raise ValueError(f"{name}[{i}] must be f32 or bf16, got {t[name].dtype}")
                _check_tensor(t[name], f"{name}[{i}]", t[name].dtype, self.device, numel)
            eight = t["m"].dtype == torch.float8_e4m3fn
            self.nearest = self.nearest or (eight and seed is None)
            for name in ("m", "v"):
                _check_tensor(t[name], f"{name}[{i}]", torch.float8_e4m3fn if eight else torch.float32, self.device, numel)
            for name in ("m_scale", "v_scale") if eight else ():
                _check_tensor(t[name], f"{name}[{i}]", torch.float32, self.device, -(-numel // ADAMW_BLOCK))
            if t["master"] is not None:
                _check_tensor(t["master"], f"master[{i}]", torch.float32, self.device, numel)
            e.param, e.grad, e.master = _ptr(t["param"]), _ptr(t["grad"]), _ptr(t["master"])
            e.m, e.v, e.m_scale, e.v_scale = _ptr(t["m"]), _ptr(t["v"]), _ptr(t["m_scale"]), _ptr(t["v_scale"])
            e.numel, e.param_dtype, e.grad_dtype = numel, DTYPES[t["param"].dtype], DTYPES[t["grad"].dtype]
            e.state_dtype = STATE_E4M3 if eight else STATE_F32
        # what a graph may have saved; views of one buffer share its version counter
        saved = (t if t._base is None else t._base for name in ("param", "master") for t in columns[name] if t is not None)
        self.written = list({id(t): t for t in saved}.values())
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name, i)
                       for name, c in columns.items() if name != "grad" for i, t in enumerate(c)
                       if t is not None and t.numel())
        for (_, end, a, i), (begin, _, b, j) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError(f"{a}[{i}] and {b}[{j}] overlap")

    @staticmethod
    def zero_state(param, eight_bit=False, seed=0):
        """m, v (for 8 bits also their scales and the seed of their rounding) before the first step, as keyword arguments
        of AdamWTensors."""
        dt = torch.float8_e4m3fn if eight_bit else torch.float32
        state = {k: [torch.zeros(t.shape, dtype=torch.uint8, device=t.device).view(dt) if eight_bit
                     else torch.zeros(t.shape, dtype=dt, device=t.device) for t in param] for k in ("m", "v")}
        if eight_bit:
            state.update({k: [torch.zeros(-(-t.numel() // ADAMW_BLOCK), dtype=torch.float32, device=t.device)
                              for t in param] for k in ("m_scale", "v_scale")}, seed=seed)
        return state

    def set_grads(self, grad):
        """Other gradient tensors of the same sizes (types may differ) for the next steps."""
        if len(grad) != self.count:
            raise ValueError(f"grad has {len(grad)} tensors, param has {self.count}")
        for i, (g, e) in enumerate(zip(grad, self.table)):
            if g.dtype not in DTYPES:
                raise ValueError(f"grad[{i}] must be f32 or bf16, got {g.dtype}")
            _check_tensor(g, f"grad[{i}]", g.dtype, self.device, e.numel)
        for g, e in zip(grad, self.table):
            e.grad, e.grad_dtype = g.data_ptr(), DTYPES[g.dtype]
        self.tensors["grad"] = list(grad)


def csa_adamw(tensors: AdamWTensors, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
              grad_scale=None, found_inf=None):
    """One AdamW step over all tensors, in place.  step (1 for the first) and lr are numbers, or device scalars (int64,
    f32) that are read when the step runs, for a captured graph; grad_scale (f32 device scalar) multiplies every
    gradient; found_inf (f32 device scalar), when not 0, leaves everything as it is."""
    p = csa_adamw_params(0.0, float(beta1), float(beta2), float(eps), float(weight_decay), 1, None, None, None, None,
                         tensors.seed or 0, tensors.seed is not None)
    if tensors.nearest and p.beta2 > NEAREST_BETA2:
        tensors.nearest = False  # said once
        warnings.warn(f"8-bit moments rounded to nearest do not follow beta2 = {p.beta2} over many steps: give AdamWTensors "
                      "a seed", stacklevel=2)
    dev = tensors.device
    if dev is None:
        return
    index = dev.index
    if isinstance(lr, torch.Tensor):
        _check_flat(lr, "lr", torch.float32, index, 1)
        p.lr_dev = lr.data_ptr()
    else:
        p.lr = lr
    if isinstance(step, torch.Tensor):
        _check_flat(step, "step", torch.int64, index, 1)
        p.step_dev = step.data_ptr()
    else:
        p.step = step
    if grad_scale is not None:
        _check_flat(grad_scale, "grad_scale", torch.float32, index, 1)
        p.grad_scale = grad_scale.data_ptr()
    if found_inf is not None:
        _check_flat(found_inf, "found_inf", torch.float32, index, 1)
        p.found_inf = found_inf.data_ptr()
    _invoke("csa_adamw", _lib.csa_adamw, index, ctypes.byref(p), tensors.table, tensors.count)
    _changed(tensors.written)  # after the launch: 50 ns a tensor


def _own(grad):
    """A gradient as the kernels read it: contiguous, and on 16 bytes (autograd may hand over a slice of a larger one)."""
    grad = grad.contiguous()
    return grad.clone() if grad.data_ptr() % 16 else grad


class _GradModeFunction(torch.autograd.Function):
    """A function whose forward is told, by its last argument, whether autograd is on.  ctx.needs_input_grad is what the inputs ask
    for, also under no_grad and inference_mode, and says nothing of whether there will be a backward pass."""

    @classmethod
    def apply(cls, *args):
        return super().apply(*args, torch.is_grad_enabled())


class CSALinear(_GradModeFunction):
    """y = CSALinear.apply(x, weight, bias, residual, params): gradients flow to all four tensors (bias and residual
    may be None)."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, params, grad):
        c = params.c
        preact = None
        if grad and c.activation != 0 and any(ctx.needs_input_grad[:3]):
            preact = torch.empty((c.rows, c.out_features), dtype=params.value_dtype, device=x.device)
        y = csa_linear_fwd(params, x, weight.contiguous(), bias, residual, preact=preact)
        ctx.params, ctx.x_shape = params, x.shape
        ctx.bias_shape = bias.shape if bias is not None else None
        ctx.residual_shape = residual.shape if residual is not None else None
        ctx.save_for_backward(x, weight, preact)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, preact = ctx.saved_tensors
        c = ctx.params.c
        need = ctx.needs_input_grad
        dx = dw = db = dres = None
        given, dy = dy, _own(dy)
        if need[3]:
            # Autograd may keep what it is handed as a .grad and add to it, unless it is the incoming tensor itself: a view
            # of that one would share its memory with the caller's gradient and with other leaves' .grad.
            dres = dy if dy.shape == ctx.residual_shape else dy.reshape(ctx.residual_shape)
            if dres is not given and dres.data_ptr() == given.data_ptr():
                dres = dres.clone()
        if any(need[:3]):
            p = ctx.params
            if c.dy_stride:  # autograd hands contiguous gradients over
                p = LinearParams(c.rows, c.in_features, c.out_features, c.dtype, c.out_dtype, c.activation, c.alpha,
                                 c.x_stride)
            dx, dw, db = csa_linear_bwd(p, dy, x, weight.contiguous(), preact, need[0], need[1], need[2])
        return (dx.view(ctx.x_shape) if dx is not None else None, dw.view(weight.shape) if dw is not None else None,
                db.view(ctx.bias_shape) if db is not None else None,
                dres, None, None)


def csa_linear(x, weight, bias=None, residual=None, *, params: LinearParams):
    return CSALinear.apply(x, weight, bias, residual, params)


class CSARope(torch.autograd.Function):
    """out = CSARope.apply(x, positions, inv_freq, params): the gradient of x is the inverse rotation of out's."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, params):
        ctx.params = params
        ctx.save_for_backward(positions, inv_freq)
        return csa_rope(params, x, positions, inv_freq)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        positions, inv_freq = ctx.saved_tensors
        if ctx.needs_input_grad[2]:
            raise ValueError("inv_freq has no gradient here: detach it")
        return csa_rope(ctx.params.inverted(), _own(dout), positions, inv_freq), None, None, None


def csa_rotary(x, positions, inv_freq, params: RopeParams):
    return CSARope.apply(x, positions, inv_freq, params)


class CSALayerNorm(_GradModeFunction):
    """y = CSALayerNorm.apply(x, weight, bias, params): gradients flow to all three tensors (weight and bias may be None)."""

    @staticmethod
    def forward(ctx, x, weight, bias, params, grad):
        keep = grad and any(ctx.needs_input_grad[:3])
        stats = torch.empty((2, params.c.rows), dtype=torch.float32, device=x.device) if keep else None
        y = csa_layernorm_fwd(params, x, weight, bias, stats=stats)
        ctx.params, ctx.x_shape = params, x.shape
        ctx.shapes = [t.shape if t is not None else None for t in (weight, bias)]
        ctx.save_for_backward(x, weight, stats)
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, stats = ctx.saved_tensors
        p, need = ctx.params, ctx.needs_input_grad
        c = p.c
        if c.dy_stride:  # autograd hands contiguous gradients over
            p = LayerNormParams(c.rows, c.cols, c.dtype, c.param_dtype, c.eps, c.x_stride)
        grads = csa_layernorm_bwd(p, _own(dy), x, weight, stats, need[0], need[1], need[2])
        return (*(g.view(shape) if g is not None else None for g, shape in zip(grads, (ctx.x_shape, *ctx.shapes))), None, None)


def csa_layernorm(x, weight=None, bias=None, *, params: LayerNormParams):
    return CSALayerNorm.apply(x, weight, bias, params)


class CSAVocabLoss(_GradModeFunction):
    """loss = CSAVocabLoss.apply(x, weight, labels, teacher_ids, teacher_logits, teacher_lse, params): gradients flow to x and
    weight.  As with CSAIndexerLoss the forward makes them with the loss (the loss alone where autograd is off) and keeps nothing
    else for the backward; the teacher's side receives none."""

    @staticmethod
    def forward(ctx, x, weight, labels, teacher_ids, teacher_logits, teacher_lse, params, grad):
        need_dx, need_dw = (grad and need for need in ctx.needs_input_grad[:2])
        targets = [t.contiguous() if t is not None else None for t in (labels, teacher_ids, teacher_logits, teacher_lse)]
        weight = weight.contiguous()
        if not (need_dx or need_dw):
            return csa_vocab_loss_fwd(params, x, weight, *targets)
        loss, dx, dw = csa_vocab_loss_bwd(params, x, weight, *targets, need_dx=need_dx, need_dw=need_dw)
        ctx.save_for_backward(dx.view(x.shape) if need_dx else None, dw.view(weight.shape) if need_dw else None)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, gloss):
        dx, dw = ctx.saved_tensors
        # scaled in fp32: gloss in bf16 would be off by one factor for all of a gradient's values
        return (*((g.float() * gloss).to(g.dtype) if g is not None else None for g in (dx, dw)), *[None] * 6)


def csa_vocab_loss(x, weight, labels=None, teacher_ids=None, teacher_logits=None, teacher_lse=None, *, params: VocabLossParams):
    return CSAVocabLoss.apply(x, weight, labels, teacher_ids, teacher_logits, teacher_lse, params)
