"""The token operators as torch modules with gradients, for a model whose parameters `Muon` updates: its embedding
table, its norms, its attention and its loss. All arithmetic runs in libdmuon's kernels (token_ops.py).

    self.embed = dm.Embedding(vocab, dim, scale=dim ** 0.5, dtype=torch.bfloat16)
    self.norm = dm.AddRMSNorm(dim)
    y, h = self.norm(x, h)                     # h + x, and its norm
    self.rotary = dm.QKNormRotary(head_dim)
    q, k = self.rotary(q, k, positions)        # (..., heads, head_dim)
    out = dm.Attention()(q, k, v, offsets)     # causal, sequences packed one behind the other
    loss, logp = dm.PolicyLoss(kl_coef=0.05)(logits, targets, old_logp, advantages, weights, ref_logp)
    stats = dm.TokenStats(top=5)(logits, targets)      # logp and entropy with gradients, alternatives

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


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_gain, k_gain, positions, options):
        positions = positions.contiguous()
        out = token_ops.qk_norm_rotary(q, k, positions, q_gain, k_gain, **options)
        ctx.save_for_backward(q, k, q_gain, k_gain, positions)
        ctx.options = options
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_gain, k_gain, positions = ctx.saved_tensors
        grads = token_ops.qk_norm_rotary_grad(dq_out.contiguous(), None if k is None else dk_out.contiguous(), q, k,
                                              positions, q_gain, k_gain, **ctx.options)
        return grads + (None, None)


class QKNormRotary(torch.nn.Module):
    """(q, k) with each head's RMS norm (fp32 gains that the heads share) and the position rotation:
    token_ops.qk_norm_rotary, whose options it takes. norm=False rotates alone and has no parameters."""

    def __init__(self, dim, norm=True, rotary_dim=None, base=10000.0, freqs=None, sections=None, interleaved=False, eps=1e-6,
                 device="cuda"):
        super().__init__()
        for name in ("q_weight", "k_weight"):
            gain = torch.nn.Parameter(torch.ones(dim, dtype=torch.float32, device=device)) if norm else None
            self.register_parameter(name, gain)
        self.options = dict(norm=norm, rotary_dim=rotary_dim, base=base, freqs=freqs, sections=sections,
                            interleaved=interleaved, eps=eps)

    def forward(self, q, k, positions):
        return _Rotary.apply(q, k, self.q_weight, self.k_weight, positions, self.options)


def _reachable(t):
    """t, or a copy of it where attention's 16-byte accesses would not reach its heads."""
    try:
        strides = token_ops._heads(t, "heads")[3:]
    except ValueError:
        return t.contiguous()
    if t.data_ptr() % 16 or any(s % 8 or s == 0 for s in strides):
        return t.clone(memory_format=torch.contiguous_format)
    return t


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, offsets, causal, scale):
        q, k, v = _reachable(q), _reachable(k), _reachable(v)
        offsets = None if offsets is None else offsets.contiguous()
        out, lse = token_ops.attention(q, k, v, offsets, causal, scale)
        ctx.save_for_backward(q, k, v, out, lse, offsets)
        ctx.causal, ctx.scale = causal, scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, offsets = ctx.saved_tensors
        return token_ops.attention_grad(_reachable(dout), q, k, v, out, lse, offsets, ctx.causal, ctx.scale) + (
            None, None, None)


class Attention(torch.nn.Module):
    """token_ops.attention over whole prompts, with its gradient: (tokens, heads, dim), a batch (batch, length, heads, dim),
    or sequences packed by `offsets`."""

    def __init__(self, causal=True, scale=None):
        super().__init__()
        self.causal, self.scale = causal, scale

    def forward(self, q, k, v, offsets=None):
        return _Attention.apply(q, k, v, offsets, self.causal, self.scale)


class _Stats(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, top, temperature):
        ctx.set_materialize_grads(False)
        logits = logits.contiguous() if logits.dim() != 2 else logits
        stats = token_ops.token_stats(logits, targets, top, temperature)
        ctx.save_for_backward(logits, targets, stats.norm, stats.entropy)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(stats.top_logp, stats.top_ids, stats.norm)
        return tuple(stats)

    @staticmethod
    @once_differentiable
    def backward(ctx, dlogp, dentropy, *_):
        logits, targets, norm, entropy = ctx.saved_tensors
        if dlogp is None and dentropy is None:
            return None, None, None, None
        dlogits = token_ops.token_stats_grad(logits, targets, norm, entropy, None if dlogp is None else dlogp.contiguous(),
                                             None if dentropy is None else dentropy.contiguous(), ctx.temperature)
        return dlogits, None, None, None


class TokenStats(torch.nn.Module):
    """token_ops.token_stats, with gradients of logp and entropy in the logits; the alternatives have none."""

    def __init__(self, top=0, temperature=1.0):
        super().__init__()
        self.top, self.temperature = top, temperature

    def forward(self, logits, targets=None):
        return token_ops.TokenStats(*_Stats.apply(logits, targets, self.top, self.temperature))
