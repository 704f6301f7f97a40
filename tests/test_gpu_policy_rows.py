"""GPU: rows of the policy loss where the ways through its kernels differ: in place, and at the borders of the shares into
which a row is cut."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_token_ops import TYPE_IDS, TYPES, check_policy, place, policy_inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


# A warp's rows, clusters of each size of CTA, more rows than there are clusters.
SIZES = [(700, 2003), (40, 9001), (300, 25003), (200, 50257), (300, 128256), (40, 262147)]


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,vocab", SIZES)
def test_in_place_over_several_turns(dm, n, vocab, dt, layout):
    """The gradient over the logits is the gradient beside them, though each row's target is read while other warps
    finish the row: its value has to be on its way before the sum that lets them. Targets lie all over the row."""
    g = torch.Generator(device="cuda").manual_seed(n)
    logits = place(torch.empty(n, vocab, device="cuda").normal_(0, 2, generator=g).to(dt), layout)
    # the first row's every share in turn, its ends among them
    targets = torch.linspace(0, vocab - 1, n, device="cuda").round().long()
    targets[1::2] = targets[1::2].flip(0)
    old = dm.token_logprobs(logits, targets) + 0.05
    adv = torch.empty(n, device="cuda").normal_(generator=g)
    w = torch.full((n,), 1.0 / n, device="cuda")
    w[5::7] = 0
    want = dm.policy_loss(logits, targets, old, adv, w, old, kl_coef=0.1)
    for _ in range(3):
        over = place(logits.clone(), layout)
        got = dm.policy_loss(over, targets, old, adv, w, old, kl_coef=0.1, dlogits=over)
        assert got[2] is over and all(torch.equal(a, b) for a, b in zip(got, want))
    live = w != 0
    p = torch.log_softmax(logits[live].float(), 1).gather(1, targets[live][:, None])[:, 0]
    assert torch.allclose(want[1][live], p, rtol=0, atol=2e-5)
    dm.check_status()


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("vocab", [515, 9001, 50257, 128256])
def test_targets_at_the_borders_of_the_shares(dm, vocab, dt):
    """Targets at a row's ends, and around multiples of its length's 8th to 128th part, against the 64-bit oracle."""
    at = {0, 1, vocab - 2, vocab - 1} | {min(vocab - 1, vocab * k // 16 + d) for k in range(1, 16, 3) for d in (-1, 0, 1)}
    n = len(at)
    for layout in ("plain", "offset"):
        s = policy_inputs(n, vocab, dt, 1.0, vocab, layout, masked=0.0)
        s["targets"] = torch.tensor(sorted(at), device="cuda")
        s["old_logp"] = torch.log_softmax(s["logits"].double(), 1).gather(1, s["targets"][:, None])[:, 0].float() + 0.03
        s["ref_logp"] = s["old_logp"] - 0.1
        check_policy(dm, s, 1.0, 0.1)
    dm.check_status()


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("dt,vocab", [(torch.float32, 292869), (torch.float32, 400001), (torch.bfloat16, 585733),
                                      (torch.bfloat16, 700000)])
def test_rows_beyond_the_memory_of_a_cluster(dm, dt, vocab, layout):
    """Read twice, by a CTA each: with and without a gradient, in place, masked rows and masked logits among them."""
    n = 7
    s = policy_inputs(n, vocab, dt, 1.0, vocab, layout, masked=0.0)
    s["weights"][2] = 0
    s["targets"][4] = -1
    s["logits"][5, vocab // 2:] = float("-inf")
    s["targets"][5] = 3
    s["old_logp"] = torch.log_softmax(s["logits"].double(), 1).gather(1, s["targets"].clamp(min=0)[:, None])[:, 0].float()
    s["ref_logp"] = s["old_logp"] - 0.1
    loss, logp, d = check_policy(dm, s, 1.0, 0.1)
    args = dict(clip_low=0.2, clip_high=0.25, kl_coef=0.1)
    alone = dm.policy_loss(**s, **args, dlogits=False)
    assert torch.equal(alone[0], loss) and torch.equal(alone[1], logp)
    got = dm.policy_loss(**s, **args, dlogits=s["logits"])
    assert all(torch.equal(a, b) for a, b in zip(got, (loss, logp, d)))
    dm.check_status()


@pytest.mark.parametrize("temperature", [1.0, 1.3, 0.7])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("vocab", [700, 50257])
def test_log_probabilities_lean_to_no_side(dm, vocab, dt, temperature):
    """The mean of the signed errors over 4000 rows, which a loss adds up. The exponentials are off by 2^-24 to one side in
    the mean, in the sum and again in the logarithm's step: 2^-23. Roundings of values up to 16 (4.8e-7 at most) average
    out to 4.8e-7 / sqrt(4000) = 8e-9, of which three are allowed. The temperature is the fp32 one of the call."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    n, t32 = 4000, float(torch.tensor(temperature, dtype=torch.float32))
    logits = torch.empty(n, vocab, device="cuda").normal_(0, 2, generator=g).to(dt)
    targets = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    got = dm.token_logprobs(logits, targets, temperature).double()
    want = torch.cat([torch.log_softmax(part.double() / t32, 1).gather(1, at[:, None])[:, 0]
                      for part, at in zip(logits.split(500), targets.split(500))])
    assert abs(float((got - want).mean())) < 2.0 ** -23 + 2.4e-8, float((got - want).mean())
