"""GPU: per-head norm with rotation and its gradient against the float64 oracle.

Tolerances, elementwise, with u = 2^-24 and the output's own rounding r (2^-8 bf16, u fp32). A sine or cosine: the angle in
halves of a revolution is rounded to 24 bits after a step of 2^-32, pi 2^-25 + 2^-31 <= 1.6 u off, and sincospif's two units
of the last place are 2 u: 4 u. The root of the mean: a lane adds at most 16 squares and up to 5 steps join them, each
product and sum u, half of it for the root, rsqrtf 2 ulp = 4 u: 16 u; the products with it and the gain 3 u. So an output is
within 32 u (|z1| + |z2|) + r |y|. Backward the sum over the row has 3 products a term and the terms are off by 4 u before,
and 1 / dim, rho^2 and the last product add a few: 64 u of the sum of the absolute terms, + r |dx|. A gain's gradient adds
n heads terms, each within 40 u of itself, in any order: (40 + n heads) u of the sum of their absolute values."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import token_ops as ref  # noqa: E402
from tests.test_gpu_token_ops import ROUND, TYPE_IDS, TYPES, U, f64, randn, within  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def heads_like(n, heads, dim, layout, dtype, seed, std=1.0):
    """Values (n, heads, dim) in one of several layouts."""
    t = randn((n, heads, dim), seed, std, dtype)
    if layout == "qkv":  # a part of wider rows
        wide = torch.full((n, heads + 3, dim), float("nan"), dtype=dtype, device="cuda")
        wide[:, 2:2 + heads] = t
        return wide[:, 2:2 + heads]
    if layout == "odd":  # off any alignment
        flat = torch.full((n * heads * (dim + 3) + 1,), float("nan"), dtype=dtype, device="cuda")
        view = flat[1:].view(n, heads, dim + 3)[..., :dim]
        view.copy_(t)
        return view
    if layout == "by_head":  # heads in front of tokens
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    return t


def positions_for(n, axes, far, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(-far // 4, far, (axes, n), generator=g)
    return (pos if axes > 1 else pos[0]).to(dtype).cuda()


CASES = [  # n, heads, kv_heads, dim, rotary_dim, axes, far
    (1, 1, 1, 2, 2, 1, 10), (1, 32, 8, 128, 128, 1, 1 << 30), (5, 3, 1, 64, 64, 3, 5000), (3, 7, 0, 128, 64, 1, 1000),
    (33, 9, 3, 78, 20, 1, 100000), (2, 2, 2, 256, 256, 4, 1 << 20), (17, 5, 5, 254, 250, 2, 1 << 24), (64, 4, 2, 96, 96, 1, 9),
    (700, 12, 4, 32, 32, 1, 4096), (130, 2, 1, 66, 0, 1, 7), (1025, 1, 1, 130, 66, 3, 100)]


@pytest.mark.parametrize("layout", ["plain", "qkv", "odd", "by_head"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_qk_norm_rotary(dm, case, dt, layout):
    n, hq, hk, dim, rd, axes, far = case
    inter, norm, gains = n % 2 == 1, dim != 96, dim != 64
    q, k = heads_like(n, hq, dim, layout, dt, 1), heads_like(n, hk, dim, layout, dt, 2, 3.0) if hk else None
    qg, kg = (randn((dim,), 3) + 1, randn((dim,), 4) + 1) if norm and gains else (None, None)
    kg = kg if hk else None
    sections = None
    if axes > 1:
        parts = [rd // 2 // axes] * axes
        parts[0] += rd // 2 - sum(parts)
        sections = tuple(parts)
    pos = positions_for(n, axes, far, 5, torch.int32 if n % 3 == 0 else torch.int64)
    options = dict(norm=norm, rotary_dim=rd, base=500.0, sections=sections, interleaved=inter, eps=1e-5)
    got = dm.qk_norm_rotary(q, k, pos, qg, kg, **options)
    angles = ref.turns(pos.cpu().numpy(), rd, 500.0, None, sections)
    for t, g, out in ((q, qg, got[0]), (k, kg, got[1])):
        if t is None:
            assert out is None
            continue
        want = ref.qk_norm_rotary(f64(t), None if g is None else f64(g), angles, rd, inter, norm, 1e-5)
        # |z1| + |z2| of every pair, through the gradient's bound of its terms
        z = ref.qk_norm_rotary(f64(t), None if g is None else f64(g), angles * 0, rd, inter, norm, 1e-5)
        size = ref.qk_norm_rotary_grad(z, z, None, angles, rd, inter, False)[2]
        within(out, want, 32 * U * size + ROUND[dt] * np.abs(want))
    dq_out, dk_out = heads_like(n, hq, dim, layout, dt, 6), heads_like(n, hk, dim, layout, dt, 7) if hk else None
    grads = dm.qk_norm_rotary_grad(dq_out, dk_out, q, k, pos, qg, kg, **options)
    for t, d, g, dx, dg in ((q, dq_out, qg, grads[0], grads[2]), (k, dk_out, kg, grads[1], grads[3])):
        if t is None:
            assert dx is None and dg is None
            continue
        want, wantg, size, sizeg = ref.qk_norm_rotary_grad(f64(d), f64(t), None if g is None else f64(g), angles, rd, inter,
                                                           norm, 1e-5)
        within(dx, want, 64 * U * size + ROUND[dt] * np.abs(want))
        if g is None:
            assert dg is None
        else:
            within(dg, wantg, (40 + n * t.shape[1]) * U * sizeg)
    again = dm.qk_norm_rotary_grad(dq_out, dk_out, q, k, pos, qg, kg, **options)
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b), "bits differ"
    dm.check_status()


def test_in_place_shapes_and_frequencies(dm):
    """Outputs over the inputs; batches; given frequencies; no tokens; expanded gradients."""
    q, k = randn((2, 5, 4, 64), 1, dtype=torch.bfloat16), randn((2, 5, 2, 64), 2, dtype=torch.bfloat16)
    pos = torch.arange(5, device="cuda").expand(2, 5).contiguous()
    qg, kg = randn((64,), 3) + 1, randn((64,), 4) + 1
    q1, k1 = dm.qk_norm_rotary(q, k, pos, qg, kg)
    freqs = [10000.0 ** (-2 * j / 64) for j in range(32)]
    q2, k2 = dm.qk_norm_rotary(q, k, pos, qg, kg, freqs=freqs)
    assert torch.equal(q1, q2) and torch.equal(k1, k2)
    flat = dm.qk_norm_rotary(q.view(10, 4, 64), k.view(10, 2, 64), pos.view(10), qg, kg)
    assert torch.equal(flat[0].view(q.shape), q1)
    sliced = dm.qk_norm_rotary(q[:, :, 1:3], k, pos, qg, kg)[0]
    assert torch.equal(sliced, q1[:, :, 1:3])
    d = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda").expand(2, 5, 4, 64)
    dk = torch.ones_like(k)
    a = dm.qk_norm_rotary_grad(d, dk, q, k, pos, qg, kg)
    b = dm.qk_norm_rotary_grad(d.contiguous(), dk, q, k, pos, qg, kg)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    over = d.contiguous()
    c = dm.qk_norm_rotary_grad(over, dk, q, k, pos, qg, kg, dq=over)
    assert c[0] is over and torch.equal(over, a[0])
    qq, kk = q.clone(), k.clone()
    got = dm.qk_norm_rotary(qq, kk, pos, qg, kg, q_out=qq, k_out=kk)
    assert got[0] is qq and torch.equal(qq, q1) and torch.equal(kk, k1)
    none = dm.qk_norm_rotary_grad(q[:0], k[:0], q[:0], k[:0], pos[:0], qg, kg)
    assert none[0].shape == (0, 5, 4, 64) and not none[2].any() and not none[3].any()
    dm.check_status()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layout", ["plain", "qkv", "odd"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("hq, hk, dim, rd", [(5, 1, 64, 64), (9, 3, 78, 20), (1, 2, 128, 64), (3, 0, 250, 250), (21, 4, 32, 16)])
def test_more_tokens_than_warps(dm, hq, hk, dim, rd, dt, layout, in_place):
    """Warps that go through several tokens, over heads that do not fill their batches: every token's rows are those of a
    call with few tokens, bit by bit, and the gains' sums those of the formula."""
    n, few = 9001, 37
    inter = dim == 78
    q, k = heads_like(n, hq, dim, layout, dt, 1), heads_like(n, hk, dim, layout, dt, 2) if hk else None
    qg, kg = randn((dim,), 3) + 1, randn((dim,), 4) + 1 if hk else None
    pos = positions_for(n, 1, 100000, 5, torch.int64)
    options = dict(rotary_dim=rd, interleaved=inter)
    dq_out, dk_out = heads_like(n, hq, dim, layout, dt, 6), heads_like(n, hk, dim, layout, dt, 7) if hk else None
    picks = [slice(0, few), slice(4000, 4000 + few), slice(n - few, n)]
    part = lambda t, at: None if t is None else t[at]
    small = [dm.qk_norm_rotary(q[at], part(k, at), pos[at], qg, kg, **options) for at in picks]
    small_grads = [dm.qk_norm_rotary_grad(dq_out[at], part(dk_out, at), q[at], part(k, at), pos[at], qg, kg, **options)
                   for at in picks]
    into = dict(dq=dq_out, dk=dk_out) if in_place else {}
    wants = []  # the gains' gradients, and what their terms add up to without their signs
    angles = ref.turns(pos.cpu().numpy(), rd, 10000.0, None, None)
    for t, d, g in ((q, dq_out, qg), (k, dk_out, kg)):
        if t is not None:
            wants.append(ref.qk_norm_rotary_grad(f64(d), f64(t), f64(g), angles, rd, inter, True, 1e-6)[1::2])
    grads = dm.qk_norm_rotary_grad(dq_out, dk_out, q, k, pos, qg, kg, **options, **into)
    into = dict(q_out=q, k_out=k) if in_place else {}
    out = dm.qk_norm_rotary(q, k, pos, qg, kg, **options, **into)
    for at, o, g in zip(picks, small, small_grads):
        for a, b in list(zip(out, o)) + list(zip(grads[:2], g[:2])):
            assert (a is None and b is None) or torch.equal(a[at], b)
    for got, heads, (want, size) in zip(grads[2:], (hq, hk), wants):
        within(got, want, (40 + n * heads) * U * size)
    dm.check_status()


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n", [3, 700, 9001])
def test_in_place_again_and_again(dm, n, dt):
    """Calls over their own inputs, each set up while the one before it still runs, read what that one wrote."""
    q, k = randn((n, 5, 64), 1, dtype=dt), randn((n, 2, 64), 2, dtype=dt)
    qg, kg = randn((64,), 3) + 1, randn((64,), 4) + 1
    pos = positions_for(n, 1, 1000, 5, torch.int64)
    a, b = q, k
    for _ in range(20):
        a, b = dm.qk_norm_rotary(a, b, pos, qg, kg)
        torch.cuda.synchronize()
    for _ in range(20):
        dm.qk_norm_rotary(q, k, pos, qg, kg, q_out=q, k_out=k)
    assert torch.equal(a, q) and torch.equal(b, k)
    dm.check_status()


def test_far_positions_are_as_exact_as_near_ones(dm):
    """A revolution of every frequency more or less, at positions up to 2^31: frequencies of k / 4096 revolutions, whose
    angles repeat every 4096 positions."""
    freqs = [2 * np.pi * j / 4096 for j in range(32)]
    q = randn((6, 2, 64), 1)
    near = torch.tensor([0, 1, 17, 4095, 2, 3], device="cuda")
    far = near + 4096 * torch.tensor([0, 1, 1 << 10, 1 << 18, -(1 << 18), (1 << 19) - 1], device="cuda")
    a, _ = dm.qk_norm_rotary(q, None, near, norm=False, freqs=freqs)
    b, _ = dm.qk_norm_rotary(q, None, far, norm=False, freqs=freqs)
    # a frequency is a double: off by 2^-53 of itself, times 2^31 positions and 2 pi
    assert (a - b).abs().max() < 2.0 ** -18


def test_a_row_of_one_token_does_not_reach_another(dm):
    q = randn((40, 3, 64), 1, dtype=torch.bfloat16)
    pos = torch.arange(40, device="cuda")
    clean, _ = dm.qk_norm_rotary(q, None, pos)
    q[7, 1] = float("nan")
    q[9, 0, 3] = float("inf")
    got, _ = dm.qk_norm_rotary(q, None, pos)
    same = torch.ones(40, 3, dtype=torch.bool)
    same[7, 1] = same[9, 0] = False
    assert torch.equal(got[same.cuda()], clean[same.cuda()]) and got[7, 1].isnan().all()


def test_refusals(dm):
    q, k, pos = randn((4, 2, 64), 1), randn((4, 1, 64), 2), torch.arange(4, device="cuda")
    for word, call in (
            ("shape", lambda: dm.qk_norm_rotary(q, k, pos[:3])),
            ("tokens", lambda: dm.qk_norm_rotary(q, k[:3], pos)),
            ("freqs", lambda: dm.qk_norm_rotary(q, k, pos, freqs=[1.0])),
            ("dimensions", lambda: dm.qk_norm_rotary(q[0], k, pos)),
            ("int32", lambda: dm.qk_norm_rotary(q, k, pos.float())),
            ("bfloat16", lambda: dm.qk_norm_rotary(q.half(), k.half(), pos)),
            ("float32", lambda: dm.qk_norm_rotary(q, k.bfloat16(), pos)),
            ("contiguous", lambda: dm.qk_norm_rotary(q.transpose(1, 2)[:, :64:2], k, pos))):
        with pytest.raises(ValueError, match=word):
            call()
    for word, call in (
            ("sections", lambda: dm.qk_norm_rotary(q, k, pos.expand(2, 4).contiguous(), sections=(1, 2))),
            ("rotary_dim", lambda: dm.qk_norm_rotary(q, k, pos, rotary_dim=66)),
            ("rotary_dim", lambda: dm.qk_norm_rotary(q, k, pos, rotary_dim=7)),
            ("even", lambda: dm.qk_norm_rotary(q[..., :63].contiguous(), k[..., :63].contiguous(), pos)),
            ("gains", lambda: dm.qk_norm_rotary(q, k, pos, torch.ones(64, device="cuda"), norm=False)),
            ("base", lambda: dm.qk_norm_rotary(q, k, pos, base=0.0)),
            ("strides must be equal", lambda: dm.qk_norm_rotary(
                q, k, pos, q_out=q.view(-1)[:8 * 64].as_strided((4, 2, 64), (64, 256, 1)))),
            ("overlap", lambda: dm.qk_norm_rotary(q, k, pos, q_out=torch.empty(4, 1, 64, device="cuda").expand(4, 2, 64)))):
        with pytest.raises(dm.DmuonError, match=word):
            call()
    dm.check_status()
