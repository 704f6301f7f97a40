"""CPU: the float64 oracle of per-head norm with rotation, attention and token statistics, against closed forms,
differences and planted mistakes."""

import numpy as np
import pytest

from oracle import token_ops as ref


def difference(f, x, step=1e-6):
    """Gradient of the scalar f by central differences."""
    g = np.zeros_like(x)
    flat, out = x.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + step
        up = f()
        flat[i] = keep - step
        out[i] = (up - f()) / (2 * step)
        flat[i] = keep
    return g


def test_turns_and_closed_forms():
    """A quarter of a revolution swaps a pair; opposite turns cancel; lengths stay; sections pick their axis."""
    rng = np.random.default_rng(0)
    z = rng.standard_normal((3, 2, 8))
    quarter = np.full((3, 3), np.pi / 2)
    got = ref.turn(z, quarter, 6, False)
    assert np.allclose(got[..., :3], -z[..., 3:6]) and np.allclose(got[..., 3:6], z[..., :3])
    assert np.array_equal(got[..., 6:], z[..., 6:])
    got = ref.turn(z, quarter, 6, True)
    assert np.allclose(got[..., 0:6:2], -z[..., 1:6:2]) and np.allclose(got[..., 1:6:2], z[..., 0:6:2])
    angles = rng.standard_normal((3, 4))
    assert np.allclose(ref.turn(ref.turn(z, angles, 8, True), -angles, 8, True), z)
    assert np.allclose((ref.turn(z, angles, 8, False) ** 2).sum(-1), (z ** 2).sum(-1))
    pos = np.array([[1, 2, 3], [10, 20, 30]])
    got = ref.turns(pos, 6, base=100.0, sections=(1, 2))
    assert np.allclose(got[:, 0], pos[0]) and np.allclose(got[:, 1], pos[1] * 100.0 ** (-1 / 3))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_gradient_by_differences(interleaved, norm):
    rng = np.random.default_rng(1)
    x, dy, gain = rng.standard_normal((3, 2, 6)), rng.standard_normal((3, 2, 6)), rng.standard_normal(6) + 2
    angles = ref.turns(np.array([0, 5, 1000]), 4)
    f = lambda: (dy * ref.qk_norm_rotary(x, gain if norm else None, angles, 4, interleaved, norm, 1e-3)).sum()
    dx, dgain, dx_size, dgain_size = ref.qk_norm_rotary_grad(dy, x, gain if norm else None, angles, 4, interleaved, norm, 1e-3)
    assert np.allclose(dx, difference(f, x), atol=1e-7)
    assert (np.abs(dx) <= dx_size * (1 + 1e-12)).all()
    if norm:
        assert np.allclose(dgain, difference(f, gain), atol=1e-7) and (np.abs(dgain) <= dgain_size).all()


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradient_by_differences(causal):
    rng = np.random.default_rng(2)
    n, heads, kv, dim = 7, 4, 2, 3
    q, k, v = (rng.standard_normal((n, h, dim)) for h in (heads, kv, kv))
    ends, dout = [1, 4, 4, 6], rng.standard_normal((n, heads, dim))  # an empty sequence, tokens of none at both ends
    out, lse, size, _ = ref.attention(q, k, v, ends, causal)
    assert (np.abs(out) <= size + 1e-15).all() and not out[0].any() and not out[6].any() and not lse[:, [0, 6]].any()
    f = lambda: (dout * ref.attention(q, k, v, ends, causal)[0]).sum()
    got, off = ref.attention_grad(dout, q, k, v, out, lse, ends, causal, p_off=0.1, dot_off=0.1)
    for g, x, o in zip(got, (q, k, v), off):
        assert np.allclose(g, difference(f, x), atol=1e-7)
        assert (o >= 0).all() and o[1:6].min() > 0 and not o[0].any() and not g[6].any()


def test_attention_closed_forms():
    """The first token of a causal sequence sees itself; equal keys give the mean; sequences do not mix."""
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((6, 1, 4)) for _ in range(3))
    out, lse, _, _ = ref.attention(q, k, v, [0, 4, 6], True, 0.5)
    assert np.allclose(out[[0, 4]], v[[0, 4]]) and np.isclose(lse[0, 4], 0.5 * (q[4, 0] @ k[4, 0]))
    same = np.broadcast_to(k[:1], k.shape)
    assert np.allclose(ref.attention(q, same, v, [0, 4, 6], False)[0][5, 0], v[4:, 0].mean(0))
    k2 = k.copy()
    k2[4:] += 1
    assert np.array_equal(ref.attention(q, k2, v, [0, 4, 6])[0][:4], out[:4] * 0 + ref.attention(q, k, v, [0, 4, 6])[0][:4])


def test_token_stats_closed_forms_and_differences():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [1.0, 3.0, 3.0, -np.inf], [5.0, 1.0, 2.0, 0.0]])
    logp, entropy, top_logp, top_ids, norm = ref.token_stats(x, np.array([2, 1, -1]), 3, 2.0)
    assert np.isclose(logp[0], -np.log(4)) and np.isclose(entropy[0], np.log(4)) and top_ids[0].tolist() == [0, 1, 2]
    assert top_ids[1].tolist() == [1, 2, 0] and np.isclose(norm[1, 1], 2 + np.exp(-1.0)) and norm[1, 0] == 3.0
    assert logp[2] == entropy[2] == 0 and top_ids[2].tolist() == [-1] * 3
    rng = np.random.default_rng(4)
    x, targets = rng.standard_normal((3, 5)) * 2, np.array([4, 0, -1])
    g, h = rng.standard_normal(3), rng.standard_normal(3)
    f = lambda: (g * ref.token_stats(x, targets, 0, 0.7)[0]).sum() + (h * ref.token_stats(x, targets, 0, 0.7)[1]).sum()
    got, size = ref.token_stats_grad(x, targets, g, h, 0.7)
    assert np.allclose(got, difference(f, x), atol=1e-7) and (np.abs(got) <= size + 1e-15).all()


def test_planted_mistakes_are_seen():
    """A wrong sign of a turn, a key in place of another: each is far outside the tolerances."""
    rng = np.random.default_rng(5)
    q, k, v = (rng.standard_normal((40, 2, 8)) for _ in range(3))
    out = ref.attention(q, k, v, [0, 40])[0]
    k2 = k.copy()
    k2[3] = k[4]
    assert np.abs(ref.attention(q, k2, v, [0, 40])[0] - out).max() > 2.0 ** -6
    angles = ref.turns(np.arange(1, 41), 8)
    assert np.abs(ref.turn(q, angles, 8, False) - ref.turn(q, -angles, 8, False)).max() > 0.1
