"""Policy-gradient steps of a small language model: embedding, residual RMS norms, rotated positions, causal attention, a
clipped policy loss with a KL term, and the Muon optimizer, all on libdmuon's kernels; matrix products are torch's.

    python examples/policy_step.py [--steps 20] [--vocab 32000] [--dim 512] [--layers 4]

Each step draws tokens from the model itself, rewards the even ones, and takes two optimizer steps on them. The
reward (0.5 for a model that knows nothing) rises.
"""

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_momentum_gb300 as dm  # noqa: E402


class Linear(torch.nn.Module):
    """fp32 weights, as Muon asks, in bf16 products."""

    def __init__(self, inputs, outputs):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.randn(outputs, inputs, device="cuda") * inputs ** -0.5)

    def forward(self, x):
        return F.linear(x, self.weight.to(torch.bfloat16))


class Block(torch.nn.Module):
    def __init__(self, dim, heads):
        super().__init__()
        self.heads = heads
        self.norm_attn, self.norm_mlp = dm.AddRMSNorm(dim), dm.AddRMSNorm(dim)
        self.rotary, self.attention = dm.QKNormRotary(dim // heads, norm=False), dm.Attention()
        self.qkv, self.out = Linear(dim, 3 * dim), Linear(dim, dim)
        self.up, self.down = Linear(dim, 4 * dim), Linear(4 * dim, dim)

    def forward(self, x, h):
        y, h = self.norm_attn(x, h)
        b, t, d = y.shape
        q, k, v = self.qkv(y).view(b, t, 3, self.heads, d // self.heads).unbind(2)
        q, k = self.rotary(q, k, torch.arange(t, device="cuda").expand(b, t))
        x = self.out(self.attention(q, k, v).view(b, t, d))
        y, h = self.norm_mlp(x, h)
        return self.down(F.gelu(self.up(y))), h


class Model(torch.nn.Module):
    def __init__(self, vocab, dim, layers, heads):
        super().__init__()
        self.embed = dm.Embedding(vocab, dim, scale=1.0, dtype=torch.bfloat16)
        self.blocks = torch.nn.ModuleList(Block(dim, heads) for _ in range(layers))
        self.norm = dm.AddRMSNorm(dim)
        self.lm_head = Linear(dim, vocab)

    def forward(self, ids):
        x, h = self.embed(ids), None
        for block in self.blocks:
            x, h = block(x, h)
        return self.lm_head(self.norm(x, h)[0])


def train(steps=20, vocab=32000, dim=512, layers=4, batch=8, length=128, seed=0, report=print):
    torch.manual_seed(seed)
    model = Model(vocab, dim, layers, heads=dim // 64)
    # The gradients of the first steps are nearly of rank one; the YOU table takes a singular value of 1, which
    # POLAR_EXPRESS's first step maps to 2.45 and the later ones out of fp16's range.
    opt = dm.Muon(model, lr=0.005, adamw_lr=2e-3, coefficients=dm.YOU)
    rewards = []
    for step in range(steps):
        prompt = torch.randint(0, vocab, (batch, length), device="cuda")
        with torch.no_grad():
            logits = model(prompt).view(-1, vocab)
            targets = torch.distributions.Categorical(logits=logits.float()).sample()
            drawn = dm.token_stats(logits, targets)
            old_logp = drawn.logp
        reward = (targets % 2 == 0).float()
        advantages = (reward - reward.mean()) / (reward.std() + 1e-6)
        weights = torch.full_like(reward, 1.0 / reward.numel())
        for _ in range(2):
            opt.zero_grad()
            logits = model(prompt).view(-1, vocab)
            # Loss and gradient in one pass over the logits; old_logp serves as the reference too.
            loss, logp, dlogits = dm.policy_loss(logits.detach(), targets, old_logp, advantages, weights,
                                                 ref_logp=old_logp, kl_coef=0.01)
            logits.backward(dlogits)
            opt.step()
        rewards.append(reward.mean())
        report(f"step {step}: reward {float(reward.mean()):.3f}  loss {float(loss):+.4f}  "
               f"log-ratio {float((logp - old_logp).mean()):+.4f}  entropy {float(drawn.entropy.mean()):.3f}")
    dm.check_status()
    return [float(r) for r in rewards]


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 20), ("vocab", 32000), ("dim", 512), ("layers", 4)):
        parser.add_argument(f"--{name}", type=int, default=value)
    train(**vars(parser.parse_args()))
