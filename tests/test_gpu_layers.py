"""GPU: the token operators' modules. Gradients against torch's autograd over the same formulas in float64, and the
example's training loop.

Tolerances: fp32 activations; relative Frobenius 1e-5 (sums of up to 300 products, 300 x 2^-24 = 2e-5 at the worst and
its square root in practice), and 2^-7 where activations are bf16 (two roundings of 2^-8 each)."""

import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 2.0 ** -7)], ids=["f32", "bf16"])
def test_modules_against_autograd(dm, dtype, tol):
    """Embedding, two norms in a row along the residual stream, a product, the loss scaled by 3 behind it."""
    torch.manual_seed(0)
    vocab, dim, n = 300, 96, 40
    embed = dm.Embedding(vocab, dim, padding_idx=7, scale=2.0, dtype=dtype)
    norms = [dm.AddRMSNorm(dim), dm.AddRMSNorm(dim)]
    head = torch.nn.Parameter(torch.randn(vocab, dim, device="cuda") * 0.2)
    for norm in norms:
        with torch.no_grad():
            norm.weight.normal_(1.0, 0.2)
    ids = torch.randint(0, vocab, (4, n // 4), device="cuda")
    ids[0, :3] = 7
    targets = torch.randint(0, vocab, (n,), device="cuda")
    adv, ref_shift = torch.randn(n, device="cuda"), torch.randn(n, device="cuda") * 0.2
    weights = torch.rand(n, device="cuda") / n
    weights[5] = 0

    x = embed(ids)
    y, h = norms[0](x)
    z, h = norms[1](y, h)
    logits = (z + 0.5 * h).view(n, dim) @ head.to(dtype).T
    with torch.no_grad():
        lp = dm.token_logprobs(logits.detach(), targets)
    old, ref = lp + 0.05, lp + ref_shift
    loss, logp = dm.PolicyLoss(kl_coef=0.1, temperature=0.8)(logits, targets, old, adv, weights, ref)
    (3.0 * loss).backward()

    E, W, G = embed.weight.detach().double().requires_grad_(), head.detach().double().requires_grad_(), [
        norm.weight.detach().double().requires_grad_() for norm in norms]

    def norm64(v, g):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * g

    x64 = 2.0 * E[ids]
    y64 = norm64(x64, G[0])
    h64 = y64 + x64
    z64 = norm64(h64, G[1])
    ls = torch.log_softmax((z64 + 0.5 * h64).view(n, dim) @ W.T / 0.8, 1)
    lp64 = ls[torch.arange(n), targets]
    r = torch.exp(lp64 - old.double())
    d = ref.double() - lp64
    each = -torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv) + 0.1 * (torch.exp(d) - d - 1)
    # the log-probabilities at other temperatures than the module's are not compared
    want = 3.0 * (each * weights.double()).sum()
    want.backward()
    E.grad[7] = 0
    if dtype == torch.float32:
        lp_at = torch.where(weights != 0, lp64.detach(), torch.zeros_like(lp64))
        assert rel(logp, lp_at) < tol
    assert rel(head.grad, W.grad) < 8 * tol
    for norm, g in zip(norms, G):
        assert rel(norm.weight.grad, g.grad) < 8 * tol
    assert rel(embed.weight.grad, E.grad) < 8 * tol
    assert embed.weight.grad[7].abs().max() == 0
    assert not logp.requires_grad
    dm.check_status()


def test_norm_module_without_a_use_of_its_norm(dm):
    """Only h is used: its gradient passes through."""
    norm = dm.AddRMSNorm(32)
    x = torch.randn(5, 32, device="cuda", requires_grad=True)
    r = torch.randn(5, 32, device="cuda", requires_grad=True)
    norm(x, r)[1].sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(r.grad, torch.ones_like(r)) and norm.weight.grad is None


def test_muon_gives_these_parameters_to_adamw(dm):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import policy_step
    model = policy_step.Model(64, 64, 1, 1)
    opt = dm.Muon(model)
    rest = {id(p) for g in opt.param_groups if not g["use_muon"] for p in g["params"]}
    assert rest == {id(model.embed.weight), id(model.lm_head.weight), id(model.norm.weight),
                    id(model.blocks[0].norm_attn.weight), id(model.blocks[0].norm_mlp.weight)}


def test_example_learns(dm):
    """The rewarded half of the vocabulary is drawn more often after a few steps: 0.5 at first, give or take
    0.5 / sqrt(1024) = 0.016."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import policy_step
    rewards = policy_step.train(steps=15, vocab=1000, dim=128, layers=2, report=lambda line: None)
    assert rewards[0] < 0.58 and rewards[-1] > 0.65, rewards
