"""GPU: token statistics and their gradient against the float64 oracle.

Tolerances with u = 2^-24: those of a log-probability in test_gpu_token_ops (2^x within 4 u, a term's exponent within 4 u of
itself, a row's sums within (vocab / 32 + 40) u for a thread of the smallest CTA): off(x) = 8 u (max |z - max z| + log vocab
+ |value|) + (vocab / 32 + 40) u. The entropy's sum of |z - max| p has the same relative errors: off + those of itself, so
twice its value more. The gradient's p is off by off relative to itself and its factors by as much and by 8 u."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import token_ops as ref  # noqa: E402
from tests.test_gpu_token_ops import ROUND, TYPE_IDS, TYPES, U, f64, place, randn, within  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def reach(logits, temperature):
    """Largest finite |z - max z| of each row."""
    z = logits / temperature
    gap = z.max(axis=1, keepdims=True) - z
    return np.where(np.isfinite(gap), gap, 0.0).max(axis=1)


def sum_off(vocab):
    return (vocab / 32 + 40) * U


def logits_for(n, vocab, dt, layout, banned, seed):
    x = randn((n, vocab), seed, 3.0, dt)
    if banned:
        ban = torch.rand(n, vocab, generator=torch.Generator().manual_seed(seed)) < 0.3
        ban[:, vocab // 2] = False
        x[ban.cuda()] = float("-inf")
    return place(x, layout)


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,vocab,top,temp", [(1, 1, 1, 1.0), (3, 5, 5, 0.7), (40, 31, 3, 1.0), (7, 257, 32, 1.3),
                                              (70, 1000, 20, 1.0), (3, 2049, 1, 1.0), (4, 4100, 0, 0.5),
                                              (9, 8200, 32, 1.0), (400, 5003, 7, 1.0), (2, 50257, 20, 1.3), (5, 70001, 5, 1.0)])
def test_token_stats(dm, n, vocab, top, temp, dt, layout):
    banned = vocab > 300 and n % 2 == 1
    x = logits_for(n, vocab, dt, layout, banned, n + vocab)
    targets = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(3))
    targets[0] = vocab // 2
    if n > 3:
        targets[2] = -1
    on_gpu = targets.to(torch.int32 if n % 2 else torch.int64).cuda()
    got = dm.token_stats(x, on_gpu, top=top, temperature=temp)
    x64 = f64(x)
    logp, entropy, top_logp, top_ids, norm = ref.token_stats(x64, targets.tolist(), top, temp)
    assert got.top_ids.shape == (n, top) and got.top_ids.tolist() == top_ids.tolist()
    off = 8 * U * (reach(x64, temp) + np.log(vocab)) + sum_off(vocab)
    finite = np.isfinite(logp)
    assert np.array_equal(f64(got.logp)[~finite], logp[~finite])
    within(got.logp[torch.from_numpy(finite).cuda()], logp[finite], (off + 8 * U * np.abs(logp))[finite])
    within(got.entropy, entropy, 2 * off + 2 * (sum_off(vocab) + 8 * U * reach(x64, temp)) * entropy)
    some = np.isfinite(top_logp)
    assert np.array_equal(f64(got.top_logp)[~some], top_logp[~some])
    bound = off[:, None] + 8 * U * np.where(some, np.abs(top_logp), 0)
    assert (np.abs(f64(got.top_logp) - top_logp)[some] <= bound[some]).all()
    assert np.array_equal(f64(got.norm)[:, 0], norm[:, 0])
    within(got.norm[:, 1], norm[:, 1], (sum_off(vocab) + 8 * U * reach(x64, temp)) * norm[:, 1])
    again = dm.token_stats(x, on_gpu, top=top, temperature=temp)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "bits differ"
    # The gradient at what the forward pass stored
    g, h = randn((n,), 5), randn((n,), 6, 0.3)
    for dlogp, dentropy in ((g, h), (g, None), (None, h)):
        want, size = ref.token_stats_grad(x64, targets.tolist(), None if dlogp is None else f64(g),
                                          None if dentropy is None else f64(h), temp)
        out = place(torch.empty(n, vocab, dtype=dt, device="cuda"), "rows" if n % 2 else layout)
        d = dm.token_stats_grad(x, on_gpu, got.norm, got.entropy, dlogp, dentropy, temperature=temp, dlogits=out)
        assert d is out
        # p, log p and the entropy are off by `off` and a few u; so are their products
        rel = 3 * off[:, None] + 3 * sum_off(vocab) + 8 * U * reach(x64, temp)[:, None] + 16 * U
        more = np.exp(np.where(np.isfinite(x64), ref.log_softmax(x64, temp), -np.inf)) * np.abs(f64(h))[:, None] / temp
        within(d, want, rel * size + 3 * off[:, None] * (more if dentropy is not None else 0) + ROUND[dt] * np.abs(want))
    dm.check_status()


@pytest.mark.parametrize("layout", ["plain", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n, vocab, top", [(640, 200, 5), (700, 2600, 3), (1300, 999, 32), (1300, 5003, 5), (2500, 1, 1),
                                           (2500, 3001, 20), (2500, 9001, 1), (1250, 17000, 2)])
def test_many_rows(dm, n, vocab, top, dt, layout):
    """More rows than the widest CTAs hold at once, so that a row has fewer warps: values by the formula for some of them,
    ids for all, rows that do not count or hold no number, and the gradient."""
    x = logits_for(n, vocab, dt, layout, vocab > 300, n + vocab)
    x[5] = float("-inf")
    x[6, vocab // 2] = float("nan")
    x[7] = 1.5  # equal logits
    targets = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(3))
    targets[8:n:9] = -1
    on_gpu = targets.cuda()
    got = dm.token_stats(x, on_gpu, top=top, temperature=1.3)
    parts = [dm.token_stats(x[i:i + 500], on_gpu[i:i + 500], top=top, temperature=1.3) for i in range(0, n, 500)]
    assert torch.equal(got.top_ids, torch.cat([part.top_ids for part in parts]))
    assert got.logp[5:7].isnan().all() and got.entropy[5:7].isnan().all()
    picks = [0, 1, 2, 3, 4, 7, 8, 9, 17, n // 2, n - 2, n - 1]
    some, few = torch.tensor(picks).cuda(), [targets[i].item() for i in picks]
    x64 = f64(x[some])
    logp, entropy, top_logp, top_ids, norm = ref.token_stats(x64, few, top, 1.3)
    off = 8 * U * (reach(x64, 1.3) + np.log(vocab)) + sum_off(vocab)
    assert got.top_ids[some].tolist() == top_ids.tolist()
    finite = np.isfinite(logp)
    within(got.logp[some][torch.from_numpy(finite).cuda()], logp[finite], (off + 8 * U * np.abs(logp))[finite])
    within(got.entropy[some], entropy, 2 * off + 2 * (sum_off(vocab) + 8 * U * reach(x64, 1.3)) * entropy)
    within(got.norm[some][:, 1], norm[:, 1], (sum_off(vocab) + 8 * U * reach(x64, 1.3)) * norm[:, 1])
    g, h = randn((n,), 5), randn((n,), 6, 0.3)
    d = dm.token_stats_grad(x, on_gpu, got.norm, got.entropy, g, h, temperature=1.3)
    want, size = ref.token_stats_grad(x64, few, f64(g[some]), f64(h[some]), 1.3)
    rel = 3 * off[:, None] + 3 * sum_off(vocab) + 8 * U * reach(x64, 1.3)[:, None] + 16 * U
    more = np.exp(np.where(np.isfinite(x64), ref.log_softmax(x64, 1.3), -np.inf)) * np.abs(f64(h[some]))[:, None] / 1.3
    within(d[some], want, rel * size + 3 * off[:, None] * more + ROUND[dt] * np.abs(want))
    assert not d[targets.cuda() < 0].any()
    dm.check_status()


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("vocab", [40, 1111, 5000, 40000])
def test_equal_logits(dm, vocab, dt):
    """Rows of equal logits, of few different ones, of a few allowed tokens, zeros of both signs: ids by column."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.zeros(7, vocab)
    x[1] = torch.randint(0, 3, (vocab,), generator=g).float()
    x[2] = float("-inf")
    x[2, vocab // 3], x[2, vocab - 1] = 1.0, 1.0
    x[3, ::2] = -0.0
    x[4] = torch.arange(vocab).float().clamp(max=256) * -1
    x[5] = torch.arange(vocab).float() % 251
    x[6] = torch.arange(vocab).float().div(64).floor()
    x = x.to(dt).cuda()
    for top in (1, 5, 32):
        got = dm.token_stats(x, top=top)
        _, entropy, _, ids, _ = ref.token_stats(f64(x) + 0.0, None, top)
        assert got.logp is None and got.top_ids.tolist() == ids.tolist()
        within(got.entropy, entropy, 3 * (sum_off(vocab) + 8 * U * (reach(f64(x), 1.0) + np.log(vocab))) * (1 + entropy))
    dm.check_status()


def test_not_numbers_and_infinities(dm):
    """A row that holds NaN or +infinity, or nothing but -infinity, gives NaN; other rows do not notice."""
    for vocab in (100, 3000, 20000):
        x = randn((6, vocab), 1)
        clean = dm.token_stats(x, top=4)
        x[1, 7] = float("nan")
        x[2, vocab - 3] = float("inf")
        x[3] = float("-inf")
        x[4] = float("nan")
        got = dm.token_stats(x, torch.zeros(6, dtype=torch.int64, device="cuda"), top=4)
        assert got.entropy[1:5].isnan().all() and got.logp[1:5].isnan().all() and got.top_logp[1:5].isnan().all()
        assert torch.equal(got.entropy[[0, 5]], clean.entropy[[0, 5]])
        assert torch.equal(got.top_ids[[0, 1, 5]], clean.top_ids[[0, 1, 5]]) or 7 in clean.top_ids[1]
        assert got.top_ids[2, 0] == vocab - 3 and got.top_ids[3].tolist() == [0, 1, 2, 3]
        assert got.top_ids[4].tolist() == [-1] * 4
        d = dm.token_stats_grad(x, None, got.norm, got.entropy, dentropy=torch.ones(6, device="cuda"))
        assert d[1:5].isnan().any(1).all() and d[[0, 5]].isfinite().all()
    dm.check_status()


def test_targets_outside(dm):
    x = randn((4, 600), 1)
    got = dm.token_stats(x, torch.tensor([5, 600, 1 << 40, -7], device="cuda"), top=2)
    with pytest.raises(dm.DmuonError) as e:
        dm.check_status()
    assert e.value.status == dm.ERR_INDEX
    assert got.top_ids[1:].tolist() == [[-1, -1]] * 3 and not got.logp[1:].any() and not got.norm[1:].any()
    d = dm.token_stats_grad(x, torch.tensor([5, 600, 1 << 40, -7], device="cuda"), got.norm, got.entropy,
                            dlogp=torch.ones(4, device="cuda"))
    with pytest.raises(dm.DmuonError):
        dm.check_status()
    assert not d[1:].any() and d[0].any()
    dm.check_status()


def test_shapes_in_place_and_agreement(dm):
    """Batches; the gradient over the logits; the log-probabilities of token_logprobs; no rows."""
    x = randn((3, 4, 700), 1, 2.0, torch.bfloat16)
    targets = torch.randint(0, 700, (3, 4), device="cuda")
    got = dm.token_stats(x, targets, top=3)
    assert got.logp.shape == (3, 4) and got.top_ids.shape == (3, 4, 3) and got.norm.shape == (3, 4, 2)
    assert (got.logp - dm.token_logprobs(x, targets)).abs().max() < 1e-5
    assert dm.token_stats(x).entropy.shape == (3, 4)
    g = torch.ones(3, 4, device="cuda")
    want = dm.token_stats_grad(x, targets, got.norm, got.entropy, g, g)
    y = x.clone()
    assert dm.token_stats_grad(y, targets, got.norm, got.entropy, g, g, dlogits=y) is y and torch.equal(y, want)
    assert dm.token_stats(x[:0], targets[:0], top=2).top_logp.shape == (0, 4, 2)
    for word, call in (("top", lambda: dm.token_stats(x, targets, top=33)),
                       ("top", lambda: dm.token_stats(x[..., :8].contiguous(), top=9)),
                       ("temperature", lambda: dm.token_stats(x, targets, temperature=0.0)),
                       ("targets", lambda: dm.token_stats_grad(x, None, got.norm, got.entropy, g)),
                       ("entropy", lambda: dm.token_stats_grad(x, targets, got.norm, None, g, g))):
        with pytest.raises(dm.DmuonError, match=word):
            call()
    dm.check_status()
