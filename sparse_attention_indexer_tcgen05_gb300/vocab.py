"""One training step of a model's last layer norm and vocabulary weight, beside the indexer's: from hidden states to the
loss, the gradient that goes back into the model, and updated weights.

    y = norm(x) [rows, features]            loss, dy, dW = csa_vocab_loss_bwd(y, W, labels and/or a teacher's top logits)
    dx, dnorm = csa_layernorm_bwd(dy)       AdamW updates W and the norm's weight and bias

dx [rows, features] is the gradient of the hidden states: what the model, whose attention reads the indexer's keys, trains
on, with labels or with the dense model's top logits.  Every buffer is made once, so that ``step`` allocates nothing and
can be captured into a CUDA graph; the step count lives on the device.  Nothing here goes through autograd.
"""
from __future__ import annotations

import torch

from . import binding as B


class VocabTrainer:
    """weight [vocab, features] (params' dtype) and the norm's norm_weight and norm_bias [features] (f32 or bf16; bias may
    be None), updated in place, their gradients and their AdamW state.

    eight_bit holds the moments in e4m3; bf16 weights get fp32 master copies."""

    def __init__(self, params: B.VocabLossParams, weight, norm_weight, norm_bias=None, eps=1e-5, lr=1e-4, beta1=0.9,
                 beta2=0.95, adam_eps=1e-8, weight_decay=0.0, eight_bit=False):
        c = params.c
        self.params, self.weight, self.norm_weight, self.norm_bias = params, weight, norm_weight, norm_bias
        dev, dt = weight.device, params.value_dtype
        if tuple(weight.shape) != (c.vocab, c.features) or weight.dtype != dt:
            raise ValueError(f"weight must be {dt} [{c.vocab}, {c.features}], got {weight.dtype} {tuple(weight.shape)}")
        if c.x_stride not in (0, c.features):
            raise ValueError("the loss reads the norm's rows, which are contiguous")
        for name, t in (("norm_weight", norm_weight), ("norm_bias", norm_bias)):
            if t is not None and (tuple(t.shape) != (c.features,) or t.dtype != norm_weight.dtype):
                raise ValueError(f"{name} must be {norm_weight.dtype} [{c.features}], got {t.dtype} {tuple(t.shape)}")
        self.norm = B.LayerNormParams(c.rows, c.features, c.dtype, norm_weight.dtype, eps)
        self.hyper = dict(lr=lr, beta1=beta1, beta2=beta2, eps=adam_eps, weight_decay=weight_decay)
        self.step_count = torch.zeros((), dtype=torch.int64, device=dev)
        self.taken = torch.empty((), dtype=torch.bool, device=dev)  # whether a step with found_inf counted

        new = lambda *shape, dtype=dt: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        self.y, self.dx = new(c.rows, c.features), new(c.rows, c.features)
        self.stats, self.loss = new(2, c.rows, dtype=torch.float32), new(dtype=torch.float32)
        self.row_loss = new(2, c.rows, dtype=torch.float32)
        weights = [t for t in (weight, norm_weight, norm_bias) if t is not None]
        self.grads = [torch.empty_like(t) for t in weights]
        need = max(1, params.bwd_workspace_bytes, params.fwd_workspace_bytes, self.norm.bwd_workspace_bytes)
        self.workspace = new(need, dtype=torch.uint8)  # one call after the other uses it
        master = [t.float() if t.dtype != torch.float32 else None for t in weights]
        self.tensors = B.AdamWTensors(weights, self.grads, master=master, **B.AdamWTensors.zero_state(weights, eight_bit))

    def evaluate(self, x, **targets):
        """The loss alone (a device scalar), with the targets of csa_vocab_loss_fwd; the rows' losses are in row_loss."""
        B.csa_layernorm_fwd(self.norm, x, self.norm_weight, self.norm_bias, out=self.y)
        return B.csa_vocab_loss_fwd(self.params, self.y, self.weight, **targets, row_loss=self.row_loss,
                                    workspace=self.workspace, out=self.loss)

    def gradients(self, x, **targets):
        """Forward and backward: the loss, dx and the gradients of weight, norm_weight and norm_bias, in the trainer's
        buffers."""
        B.csa_layernorm_fwd(self.norm, x, self.norm_weight, self.norm_bias, out=self.y, stats=self.stats)
        # the gradient of y takes dx's place, and dx then its own
        B.csa_vocab_loss_bwd(self.params, self.y, self.weight, **targets, row_loss=self.row_loss, workspace=self.workspace,
                             out=(self.loss, self.dx, self.grads[0]))
        B.csa_layernorm_bwd(self.norm, self.dx, x, self.norm_weight, self.stats, need_dbias=self.norm_bias is not None,
                            workspace=self.workspace, out=(self.dx, self.grads[1], self.grads[2] if self.norm_bias is not None else None))
        return self.loss, self.dx, self.grads

    def step(self, x, grad_scale=None, found_inf=None, **targets):
        """gradients() and the weights' AdamW step.  Returns the loss (a device scalar) and dx.  found_inf (f32 device
        scalar), when not 0, leaves weights, state and step count as they are."""
        self.gradients(x, **targets)
        if found_inf is None:
            self.step_count.add_(1)
        else:
            self.step_count.add_(torch.eq(found_inf.view(()), 0, out=self.taken))
        B.csa_adamw(self.tensors, self.step_count, grad_scale=grad_scale, found_inf=found_inf, **self.hyper)
        return self.loss, self.dx
