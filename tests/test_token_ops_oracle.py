"""CPU: the float64 token operators against differences of their own forward forms, and the C entry points'
and binding's refusals (arguments are checked before a device is touched).

Central differences with step s of a function with third derivative f3 are off by s^2 f3 / 6 + 2^-52 |f| / s:
at s = 1e-5 and values around 1, under 1e-8; 1e-6 is asked for."""

import ctypes

import numpy as np
import pytest

import newton_schulz_momentum_gb300 as dm
from newton_schulz_momentum_gb300 import build as dmbuild
from oracle import token_ops as ref

STEP, TOL = 1e-5, 1e-6


def differences(f, x):
    got = np.zeros_like(x)
    for k in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[k] += STEP
        down[k] -= STEP
        got[k] = (f(up) - f(down)) / (2 * STEP)
    return got


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(0)
    table, ids, dout = rng.normal(size=(5, 3)), np.array([4, 0, 4, 2, 4]), rng.normal(size=(5, 3))
    want = differences(lambda t: (ref.embedding(t, ids, 1.5) * dout).sum(), table)
    got, _, count = ref.embedding_grad(dout, ids, 5, 1.5)
    assert np.abs(got - want).max() < TOL and count.tolist() == [1, 0, 1, 0, 3]
    assert np.abs(ref.embedding_grad(dout, ids, 5, 1.5, padding_idx=4)[0][4]).max() == 0


@pytest.mark.parametrize("eps", [1e-6, 0.5])
def test_norm_gradient_against_differences(eps):
    rng = np.random.default_rng(1)
    x, r, gain = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7)
    dy, dh = rng.normal(size=(3, 7)), rng.normal(size=(3, 7))

    def out(x, gain):
        y, h = ref.add_rmsnorm(x, r, gain, eps)
        return (y * dy).sum() + (h * dh).sum()

    dx, dgain, _, _ = ref.add_rmsnorm_grad(dy, x + r, gain, dh, eps)
    assert np.abs(dx - differences(lambda v: out(v, gain), x)).max() < TOL
    assert np.abs(dgain - differences(lambda v: out(x, v), gain)).max() < TOL


@pytest.mark.parametrize("temperature", [1.0, 0.7])
@pytest.mark.parametrize("kl", [0.0, 0.3])
def test_policy_gradient_against_differences(temperature, kl):
    rng = np.random.default_rng(2)
    n, vocab = 8, 6
    logits, targets = rng.normal(size=(n, vocab)), rng.integers(0, vocab, size=n)
    adv, w = rng.normal(size=n), rng.uniform(0.1, 1.0, size=n)
    w[3] = 0.0
    targets[5] = -1
    lp = np.array([ref.log_softmax(logits, temperature)[t, max(0, a)] for t, a in enumerate(targets)])
    old, rlp = lp + rng.choice([-0.5, -0.05, 0.07, 0.6], size=n), lp + rng.normal(size=n) * 0.3

    def loss(x):
        return ref.policy_loss(x, targets, old, adv, w, rlp, 0.2, 0.3, kl, temperature)[0]

    got = ref.policy_loss(logits, targets, old, adv, w, rlp, 0.2, 0.3, kl, temperature)[2]
    assert np.abs(got - differences(loss, logits)).max() < TOL
    assert np.abs(got[[3, 5]]).max() == 0


# ---------------------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def L():
    dmbuild.build()
    return dm.lib()


A, B, C = 4096, 8192, 16384  # stand-in addresses, never read
NAN, INF = float("nan"), float("inf")


def replaced(args, changes):
    args = list(args)
    for k, v in changes.items():
        args[k] = v
    return args


def refused(L, f, args, changes, status, word):
    rc = f(*replaced(args, changes), None)
    message = L.dmuon_last_error().decode()
    assert rc == status and word in message, (changes, rc, message)


# table, dtype, rows, dim, ld, ids, id_bytes, n, scale, out, out_dtype, ld_out
EMBED = (A, 0, 10, 8, 8, B, 8, 4, 1.0, C, 1, 8)


@pytest.mark.parametrize("changes,word", [
    ({0: None}, "table"), ({1: 2}, "dtype of table"), ({2: 0}, "rows"), ({2: 1 << 31}, "rows"), ({3: 0}, "dim"),
    ({4: 7}, "leading dimension of table"), ({5: None}, "ids"), ({5: B + 4}, "aligned"), ({6: 2}, "id_bytes"),
    ({7: -1}, "n must"), ({7: 1 << 31}, "n must"), ({8: NAN}, "scale"), ({8: INF}, "scale"), ({9: None}, "out"),
    ({9: C + 1}, "aligned"), ({10: 3}, "dtype of out"), ({11: 7}, "leading dimension of out"), ({0: A + 2}, "aligned")])
def test_embedding_refuses(L, changes, word):
    refused(L, L.dmuon_embedding, EMBED, changes, dm.ERR_INVALID_ARG, word)


# grad_out, dtype, ld, ids, id_bytes, n, rows, dim, scale, padding_idx, grad, ld_grad, accumulate
EMBED_GRAD = (A, 1, 8, B, 4, 4, 10, 8, 1.0, -1, C, 8, 0)


@pytest.mark.parametrize("changes,word", [
    ({0: None}, "grad_out"), ({1: 7}, "dtype of grad_out"), ({2: 4}, "leading dimension of grad_out"), ({3: None}, "ids"),
    ({4: 0}, "id_bytes"), ({5: -5}, "n must"), ({6: 0}, "rows"), ({7: 0}, "dim"), ({8: NAN}, "scale"),
    ({9: 10}, "padding_idx"), ({10: None}, "grad"), ({10: C + 2}, "aligned"), ({11: 7}, "leading dimension of grad")])
def test_embedding_grad_refuses(L, changes, word):
    refused(L, L.dmuon_embedding_grad, EMBED_GRAD, changes, dm.ERR_INVALID_ARG, word)


# x, ldx, residual, ldr, dtype, gain, n, dim, eps, h, ldh, y, y_dtype, ldy, scales, group
NORM = (A, 8, B, 8, 1, C, 4, 8, 1e-6, A, 8, B, 1, 8, None, 0)


@pytest.mark.parametrize("changes,word", [
    ({0: None}, "x must"), ({1: 7}, "leading dimension of x"), ({3: 7}, "leading dimension of residual"), ({4: 2}, "dtype"),
    ({5: C + 2}, "gain"), ({6: -1}, "n must"), ({7: 0}, "dim"), ({8: -1e-6}, "eps"), ({8: NAN}, "eps"),
    ({10: 7}, "leading dimension of h"), ({11: None}, "y must"), ({12: 0}, "y_dtype"), ({13: 7}, "leading dimension of y"),
    ({14: A}, "scales"), ({12: 2}, "scales"), ({12: 2, 14: A, 15: 48}, "group"), ({12: 2, 14: A, 15: -1}, "group"),
    ({12: 2, 14: A + 2}, "aligned"), ({12: 2, 14: A, 13: 7}, "leading dimension of y")])
def test_norm_refuses(L, changes, word):
    refused(L, L.dmuon_add_rmsnorm, NORM, changes, dm.ERR_INVALID_ARG, word)


# dy, lddy, h, ldh, dh, lddh, dtype, gain, n, dim, eps, dx, lddx, dgain, accumulate
NORM_GRAD = (A, 8, B, 8, C, 8, 0, A, 4, 8, 1e-6, B, 8, C, 0)


@pytest.mark.parametrize("changes,word", [
    ({0: None}, "dy"), ({1: 7}, "leading dimension of dy"), ({2: None}, "h must"), ({3: 7}, "leading dimension of h"),
    ({5: 7}, "leading dimension of dh"), ({6: 2}, "dtype"), ({7: A + 1}, "gain"), ({8: -1}, "n must"), ({9: 0}, "dim"),
    ({10: INF}, "eps"), ({11: None}, "dx"), ({12: 7}, "leading dimension of dx"), ({13: C + 2}, "dgain")])
def test_norm_grad_refuses(L, changes, word):
    refused(L, L.dmuon_add_rmsnorm_grad, NORM_GRAD, changes, dm.ERR_INVALID_ARG, word)


# logits, dtype, ld, n, vocab, targets, id_bytes, old, ref, adv, weights, lo, hi, kl, temp, loss, logp, dlogits, ldd
POLICY = (A, 1, 16, 4, 16, B, 8, C, C, C, C, 0.2, 0.2, 0.1, 1.0, A, B, C, 16)


@pytest.mark.parametrize("changes,word", [
    ({0: None}, "logits"), ({1: 3}, "dtype of logits"), ({2: 15}, "leading dimension of logits"), ({3: -1}, "n must"),
    ({4: 0}, "vocab"), ({5: None}, "ids"), ({6: 16}, "id_bytes"), ({7: None}, "old_logp"), ({8: None}, "ref_logp"),
    ({9: None}, "advantages"), ({10: None}, "weights"), ({11: -0.1}, "clip_low"), ({12: NAN}, "clip"), ({13: INF}, "kl_coef"),
    ({14: 0.0}, "temperature"), ({14: -1.0}, "temperature"), ({14: NAN}, "temperature"), ({15: None}, "loss"),
    ({16: B + 2}, "aligned"), ({18: 15}, "leading dimension of dlogits")])
def test_policy_refuses(L, changes, word):
    refused(L, L.dmuon_policy_loss, POLICY, changes, dm.ERR_INVALID_ARG, word)


# logits, dtype, ld, n, vocab, targets, id_bytes, temperature, logp
LOGP = (A, 1, 16, 4, 16, B, 8, 1.0, C)


@pytest.mark.parametrize("changes,word", [
    ({0: None}, "logits"), ({1: 2}, "dtype of logits"), ({2: 15}, "leading dimension"), ({4: 0}, "vocab"), ({5: None}, "ids"),
    ({6: 1}, "id_bytes"), ({7: 0.0}, "temperature"), ({8: None}, "logp"), ({8: C + 1}, "aligned")])
def test_logprobs_refuses(L, changes, word):
    refused(L, L.dmuon_token_logprobs, LOGP, changes, dm.ERR_INVALID_ARG, word)


def test_row_lengths_beyond_the_limit_are_unsupported(L):
    big = (1 << 24) + 1
    refused(L, L.dmuon_embedding, EMBED, {3: big, 4: big, 11: big}, dm.ERR_UNSUPPORTED, "dim")
    refused(L, L.dmuon_token_logprobs, LOGP, {2: big, 4: big}, dm.ERR_UNSUPPORTED, "vocab")


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dm.embedding(x, ids), lambda: dm.embedding_grad(x, ids, 4), lambda: dm.add_rmsnorm(x),
                 lambda: dm.add_rmsnorm_fp8(x), lambda: dm.add_rmsnorm_grad(x, x),
                 lambda: dm.policy_loss(x, ids, x[0], x[0], x[0]), lambda: dm.token_logprobs(x, ids)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert ctypes.sizeof(ctypes.c_void_p) == 8
