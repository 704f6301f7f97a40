"""The token operators as torch modules with gradients, for a model whose parameters `Muon` updates: its embedding
table, its norms and its loss. All arithmetic runs in libdmuon's kernels (token_ops.py).

    self.embed = dm.Embedding(vocab, dim, scale=dim ** 0.5, dtype=torch.bfloat16)
    self.norm = dm.AddRMSNorm(dim)
    y, h = self.norm(x, h)                     # h + x, and its norm
    loss, logp = dm.PolicyLoss(kl_coef=0.05)(logits, targets, old_logp, advantages, weights, ref_logp)

Parameters are fp32, as Muon asks; activations fp32 or bf16. Muon gives all of these parameters to AdamW. Gradients are of
first order: differentiating them again raises an error.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import token_ops


class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale, dtype, padding_idx):
        ids = ids.contiguous()
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale, ctx.padding_idx = table.shape[0], scale, padding_idx
        return token_ops.embedding(table, ids, scale, dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        (ids,) = ctx.saved_tensors
        return (token_ops.embedding_grad(grad.contiguous(), ids, ctx.rows, ctx.scale, ctx.padding_idx), None, None, None,
                None)


class Embedding(torch.nn.Embedding):
    """torch.nn.Embedding whose output is scale * table[ids], of `dtype` (the table stays fp32), with a dense gradient."""

    def __init__(self, num_embeddings, embedding_dim, padding_idx=None, scale=1.0, dtype=None, device="cuda"):
        super().__init__(num_embeddings, embedding_dim, padding_idx=padding_idx, device=device, dtype=torch.float32)
        self.scale, self.out_dtype = float(scale), dtype or torch.float32

    @classmethod
    def from_pretrained(cls, embeddings, freeze=True, padding_idx=None, scale=1.0, dtype=None):
        """The module over an fp32 table of its own, which is not copied; without a gradient if `freeze`."""
        if embeddings.dim() != 2 or embeddings.dtype != torch.float32:
            raise ValueError("embeddings must be a 2-D float32 tensor")
        rows, dim = embeddings.shape
        embed = cls(rows, dim, padding_idx=padding_idx, scale=scale, dtype=dtype, device="meta")
        embed.weight = torch.nn.Parameter(embeddings, requires_grad=not freeze)
        return embed

    def forward(self, ids):
        return _Lookup.apply(self.weight, ids, self.scale, self.out_dtype, self.padding_idx)


class _AddNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gain, eps):
        ctx.set_materialize_grads(False)
        x = x.contiguous()
        y, h = token_ops.add_rmsnorm(x, None if residual is None else residual.contiguous(), gain, eps)
        ctx.save_for_backward(h, gain)
        ctx.eps, ctx.alone = eps, residual is None
        return (y, h.view_as(h)) if ctx.alone else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, gain = ctx.saved_tensors
        if dy is None:
            return dh, None if ctx.alone else dh, None, None
        dx, dgain = token_ops.add_rmsnorm_grad(dy.contiguous(), h, gain, None if dh is None else dh.contiguous(), ctx.eps)
        return dx, None if ctx.alone else dx, dgain, None


class AddRMSNorm(torch.nn.Module):
    """(y, h) = (RMS norm of h with a gain, h = x + residual); h is x without a residual."""

    def __init__(self, dim, eps=1e-6, device="cuda"):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(dim, dtype=torch.float32, device=device))
        self.eps = float(eps)

    def forward(self, x, residual=None):
        return _AddNorm.apply(x, residual, self.weight, self.eps)


class _Policy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, old_logp, advantages, weights, ref_logp, options):
        loss, logp, _ = token_ops.policy_loss(logits, targets, old_logp, advantages, weights, ref_logp, dlogits=False,
                                              **options)
        ctx.save_for_backward(logits, targets, old_logp, advantages, weights, ref_logp)
        ctx.options = options
        ctx.mark_non_differentiable(logp)
        return loss, logp

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        logits, targets, old_logp, advantages, weights, ref_logp = ctx.saved_tensors
        # The gradient is linear in the weights, so what arrives from behind the loss goes into them.
        dlogits = token_ops.policy_loss(logits, targets, old_logp, advantages, weights * dloss, ref_logp, **ctx.options)[2]
        return dlogits, None, None, None, None, None, None


class PolicyLoss(torch.nn.Module):
    """(loss, logp) of token_ops.policy_loss, differentiable in the logits: one pass over them forward and one backward.
    A step that needs nothing between the two gets both in one pass from policy_loss itself:
    `loss, logp, dlogits = dm.policy_loss(...); logits.backward(dlogits)`."""

    def __init__(self, clip_low=0.2, clip_high=0.2, kl_coef=0.0, temperature=1.0):
        super().__init__()
        self.options = dict(clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef, temperature=temperature)

    def forward(self, logits, targets, old_logp, advantages, weights, ref_logp=None):
        return _Policy.apply(logits, targets, old_logp, advantages, weights, ref_logp, self.options)
