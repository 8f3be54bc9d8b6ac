"""One training step of the indexer's own weights, from hidden states to updated weights.

    q_idx = rope(x Wq^T)         [rows, idx_heads, idx_dim]       k_idx = rope(x_c Wk^T)   [compressed rows, idx_dim]
                                                                  (key_norm: k_idx = rope(norm(x_c Wk^T)))
    w     = scale x Ww^T         [rows, idx_heads] fp32            ids, scores = csa_indexer_fwd(q_idx, w, k_idx)
    loss, dq_idx, dw, dk_idx = csa_indexer_bwd(...)                the gradients go back through the rotation and the
                                                                   projections into the weights, which AdamW updates.

x are the hidden states of the queries, x_c those of the compressed keys; both are inputs here (no gradient flows to
them, as none flows to the teacher's side).  Every buffer is made once, so that ``step`` allocates nothing and can be
captured into a CUDA graph; the step count lives on the device.  Nothing here goes through autograd: a captured step
shares no gradient node with an eager one.
"""
from __future__ import annotations

import torch

from . import binding as B


class IndexerTrainer:
    """The weights wq [idx_heads * idx_dim, hidden], wk [idx_dim, hidden] and ww [idx_heads, hidden] (params' dtype,
    updated in place), their gradients and their AdamW state.

    rot_dim values of each indexer head rotate (0: none), by `sections` of the position axes.  weight_scale is the
    indexer's scale, folded into w.  key_norm: (weight, bias) [idx_dim] of a layer norm of the keys between their projection
    and their rotation, trained with the others (f32 or bf16; bias may be None).  eight_bit holds the moments in e4m3; bf16
    weights get fp32 master copies."""

    def __init__(self, params: B.Params, wq, wk, ww, rot_dim=0, sections=None, interleaved=False, weight_scale=1.0,
                 lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, eight_bit=False, positions_64=False,
                 key_norm=None, key_norm_eps=1e-6):
        c = params.c
        self.params, self.wq, self.wk, self.ww = params, wq, wk, ww
        dev, dt = wq.device, params.value_dtype
        rows, keys, heads, dim, hidden = params.rows, params.compressed_rows, c.idx_heads, c.idx_dim, wq.shape[-1]
        for name, t, n in (("wq", wq, heads * dim), ("wk", wk, dim), ("ww", ww, heads)):
            if tuple(t.shape) != (n, hidden) or t.dtype != dt:
                raise ValueError(f"{name} must be {dt} [{n}, {hidden}], got {t.dtype} {tuple(t.shape)}")
        self.hyper = dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay)
        self.step_count = torch.zeros((), dtype=torch.int64, device=dev)
        self.taken = torch.empty((), dtype=torch.bool, device=dev)  # whether a step with found_inf counted

        self.p_q = B.LinearParams(rows, hidden, heads * dim, c.dtype)
        self.p_k = B.LinearParams(keys, hidden, dim, c.dtype)
        self.p_w = B.LinearParams(rows, hidden, heads, c.dtype, "f32", alpha=weight_scale)
        if rot_dim:
            kw = dict(dtype=c.dtype, rot_dim=rot_dim, sections=sections, interleaved=interleaved, positions_64=positions_64)
            self.r_q, self.r_k = B.RopeParams(rows, heads, dim, **kw), B.RopeParams(keys, 1, dim, **kw)
            self.r_dq, self.r_dk = self.r_q.inverted(), self.r_k.inverted()
        else:
            self.r_q = None

        new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        f32 = torch.float32
        self.q_idx, self.k_idx, self.w = new(rows, heads, dim), new(keys, dim), new(rows, heads, dtype=f32)
        self.ids, self.selscore = new(rows, params.K, dtype=torch.int32), new(rows, params.K, dtype=f32)
        self.loss = new(dtype=f32)
        self.dq_idx, self.dk_idx, self.dw = new(rows, heads, dim), new(keys, dim), new(rows, heads, dtype=f32)
        weights = [wq, wk, ww]
        need = [params.workspace_bytes] + [p.workspace_bytes for p in (self.p_q, self.p_k, self.p_w)]
        self.norm = None
        if key_norm is not None:
            self.key_norm = tuple(key_norm)
            for name, t in zip(("weight", "bias"), self.key_norm, strict=True):
                if t is None and name == "bias":
                    continue
                if tuple(t.shape) != (dim,) or t.dtype != self.key_norm[0].dtype:
                    raise ValueError(f"key_norm's {name} must be {self.key_norm[0].dtype} [{dim}], got {t.dtype} {tuple(t.shape)}")
            self.norm = B.LayerNormParams(keys, dim, c.dtype, self.key_norm[0].dtype, key_norm_eps)
            self.k_proj, self.k_stats = new(keys, dim), new(2, keys, dtype=f32)
            weights += [t for t in self.key_norm if t is not None]
            need.append(self.norm.bwd_workspace_bytes)
        self.grads = [torch.empty_like(t) for t in weights]
        self.workspace = new(max(1, *need), dtype=torch.uint8)  # one call after the other uses it
        master = [t.float() if t.dtype != f32 else None for t in weights] if dt != f32 or self.norm is not None else None
        self.tensors = B.AdamWTensors(weights, self.grads, master=master, **B.AdamWTensors.zero_state(weights, eight_bit))

    def project(self, x, x_c, positions=None, key_positions=None, inv_freq=None):
        """q_idx, w and k_idx of the hidden states, into the trainer's buffers."""
        B.csa_linear_fwd(self.p_q, x, self.wq, workspace=self.workspace, out=self.q_idx)
        B.csa_linear_fwd(self.p_k, x_c, self.wk, workspace=self.workspace, out=self.k_idx if self.norm is None else self.k_proj)
        if self.norm is not None:
            B.csa_layernorm_fwd(self.norm, self.k_proj, *self.key_norm, out=self.k_idx, stats=self.k_stats)
        B.csa_linear_fwd(self.p_w, x, self.ww, workspace=self.workspace, out=self.w)
        if self.r_q is not None:
            B.csa_rope(self.r_q, self.q_idx, positions, inv_freq, out=self.q_idx)
            B.csa_rope(self.r_k, self.k_idx, key_positions, inv_freq, out=self.k_idx)
        return self.q_idx, self.w, self.k_idx

    def gradients(self, x, x_c, q, kv, kv_c, sink, positions=None, key_positions=None, inv_freq=None):
        """Forward and backward: the loss (a device scalar) and the gradients of wq, wk and ww (and of the keys' norm), in the
        trainer's buffers."""
        p = self.params
        q_idx, w, k_idx = self.project(x, x_c, positions, key_positions, inv_freq)
        B.csa_indexer_fwd(p, q_idx, w, k_idx, workspace=self.workspace, ids=self.ids, selscore=self.selscore)
        B.csa_indexer_bwd(p, q_idx, w, k_idx, q, kv, kv_c, sink, self.ids, self.selscore, workspace=self.workspace,
                          out=(self.loss, self.dq_idx, self.dw, self.dk_idx))
        if self.r_q is not None:
            B.csa_rope(self.r_dq, self.dq_idx, positions, inv_freq, out=self.dq_idx)
            B.csa_rope(self.r_dk, self.dk_idx, key_positions, inv_freq, out=self.dk_idx)
        if self.norm is not None:
            weight, bias = self.key_norm
            B.csa_layernorm_bwd(self.norm, self.dk_idx, self.k_proj, weight, self.k_stats, need_dbias=bias is not None,
                                workspace=self.workspace, out=(self.dk_idx, self.grads[3], self.grads[4] if bias is not None else None))
        for lp, dy, rows, weight, dw in ((self.p_q, self.dq_idx.view(-1, self.wq.shape[0]), x, self.wq, self.grads[0]),
                                         (self.p_k, self.dk_idx, x_c, self.wk, self.grads[1]),
                                         (self.p_w, self.dw, x, self.ww, self.grads[2])):
            B.csa_linear_bwd(lp, dy, rows, weight, need_dx=False, need_db=False, workspace=self.workspace, out=(None, dw, None))
        return self.loss, self.grads

    def step(self, x, x_c, q, kv, kv_c, sink, positions=None, key_positions=None, inv_freq=None, grad_scale=None,
             found_inf=None):
        """gradients() and the weights' AdamW step.  Returns the loss, a device scalar.  found_inf (f32 device scalar),
        when not 0, leaves weights, state and step count as they are."""
        self.gradients(x, x_c, q, kv, kv_c, sink, positions, key_positions, inv_freq)
        if found_inf is None:
            self.step_count.add_(1)
        else:
            self.step_count.add_(torch.eq(found_inf.view(()), 0, out=self.taken))
        B.csa_adamw(self.tensors, self.step_count, grad_scale=grad_scale, found_inf=found_inf, **self.hyper)
        return self.loss
