"""GPU: per-head norm with rotation, attention and token statistics as they are used together: modules and their gradients
against torch's autograd over the same formulas in float64, in captured graphs, on several streams.

Tolerances: relative Frobenius. fp32 operators (rotation, statistics) 1e-5: sums of up to 300 products, 300 x 2^-24 at the
worst. Everything through bf16 attention: q, k, v and dout are rounded to bf16 at its border (2^-8 each at the worst, a third
of it in the root mean square), its p, ds and outputs inside once more; a gradient passes four to six such roundings, so 6 x
2^-8 = 0.024 bounds the worst that errors in line would add up to."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def rel(a, b):
    return float((a.detach().double() - b).norm() / b.norm())


def normal(*shape, seed=0, std=1.0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g).to(dtype)


def norm_turn64(x, gain, pos, eps=1e-6):
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * gain
    half = x.shape[-1] // 2
    angle = pos.double()[:, None] * 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def attention64(q, k, v, ends):
    group = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    out = []
    for b, e in zip(ends, ends[1:]):
        x = torch.einsum("ihd,jhd->hij", q[b:e], k[b:e]) * q.shape[-1] ** -0.5
        x = x.masked_fill(torch.ones(e - b, e - b, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(x, -1), v[b:e]))
    return torch.cat(out)


def test_a_layer_and_a_loss(dm):
    """qkv in one product, norm and rotation, attention over packed sequences, a head, a loss of log-probabilities with an
    entropy bonus: gradients of the input, the gains and the head."""
    n, hq, hk, dim, vocab = 300, 6, 2, 64, 500
    ends = [0, 130, 131, 131, 300]
    offsets = torch.tensor(ends, device="cuda")
    pos = torch.cat([torch.arange(b - a) for a, b in zip(ends, ends[1:])]).cuda()
    x = normal(n, hq + 2 * hk, dim, seed=1).requires_grad_()
    head = (normal(vocab, hq * dim, seed=2) * (hq * dim) ** -0.5).requires_grad_()
    targets = torch.randint(0, vocab, (n,), device="cuda")
    targets[7] = -1
    w = torch.rand(n, device="cuda")
    rotary = dm.QKNormRotary(dim)
    with torch.no_grad():
        rotary.q_weight.copy_(1 + 0.2 * normal(dim, seed=3))
        rotary.k_weight.copy_(1 + 0.2 * normal(dim, seed=4))
    qkv = x.to(BF16)
    q, k = rotary(qkv[:, :hq], qkv[:, hq:hq + hk], pos)
    out = dm.Attention()(q, k, qkv[:, hq + hk:], offsets)
    logits = out.reshape(n, -1).float() @ head.T
    stats = dm.TokenStats(top=3)(logits, targets)
    loss = -(w * stats.logp).sum() - 0.1 * (w * stats.entropy).sum()
    (2.0 * loss).backward()

    x64, h64 = x.detach().double().requires_grad_(), head.detach().double().requires_grad_()
    gq, gk = (g.detach().double().requires_grad_() for g in (rotary.q_weight, rotary.k_weight))
    out64 = attention64(norm_turn64(x64[:, :hq], gq, pos), norm_turn64(x64[:, hq:hq + hk], gk, pos), x64[:, hq + hk:], ends)
    ls = torch.log_softmax(out64.reshape(n, -1) @ h64.T, -1)
    live = targets >= 0
    lp = ls[torch.arange(n), targets.clamp(min=0)]
    entropy = -(ls.exp() * ls).sum(-1)
    want = -(w * torch.where(live, lp + 0.1 * entropy, 0.0)).sum()
    (2.0 * want).backward()
    assert rel(out, out64.detach()) < 0.024 and abs(float(loss - want)) < 0.02 * abs(float(want))
    for got, ref in ((x.grad, x64.grad), (head.grad, h64.grad), (rotary.q_weight.grad, gq.grad), (rotary.k_weight.grad, gk.grad)):
        assert rel(got, ref) < 0.024
    # bf16 logits may order nearly equal tokens otherwise: the first alternative is within rounding of the largest
    assert (ls.max(-1).values - ls.gather(1, stats.top_ids.clamp(min=0))[:, 0])[live].max() < 0.05
    dm.check_status()


def test_fp32_modules_against_autograd(dm):
    n, h, dim, vocab = 40, 3, 24, 300
    x, g = normal(n, h, dim, seed=1).requires_grad_(), normal(n, h, dim, seed=2)
    pos = torch.randint(0, 5000, (n,), device="cuda")
    rotary = dm.QKNormRotary(dim)
    out, none = rotary(x, None, pos)
    assert none is None
    (out * g).sum().backward()
    x64, w64 = x.detach().double().requires_grad_(), rotary.q_weight.detach().double().requires_grad_()
    want = norm_turn64(x64, w64, pos)
    (want * g).sum().backward()
    assert rel(out, want.detach()) < 1e-5 and rel(x.grad, x64.grad) < 1e-5 and rel(rotary.q_weight.grad, w64.grad) < 1e-5
    assert rotary.k_weight.grad is None
    bare = dm.QKNormRotary(dim, norm=False)
    assert not list(bare.parameters())
    y = x.detach().clone().requires_grad_()
    bare(y, None, pos)[0].sum().backward()
    assert (y.grad.norm() - (n * h * dim) ** 0.5).abs() < 1e-2  # a turn keeps lengths
    z, a = normal(n, vocab, seed=3, std=2.0).requires_grad_(), torch.randint(0, vocab, (n,), device="cuda")
    stats = dm.TokenStats(top=2, temperature=0.7)(z, a)
    (stats.logp.sum() * 2 - stats.entropy.sum()).backward()
    z64 = z.detach().double().requires_grad_()
    ls = torch.log_softmax(z64 / 0.7, -1)
    (2 * ls[torch.arange(n), a].sum() + (ls.exp() * ls).sum()).backward()
    assert rel(z.grad, z64.grad) < 1e-5
    dm.check_status()


def test_gradients_against_differences(dm):
    """Along a random direction, in fp32: a step of 1e-2 is off by its square, and by 2^-24 of the value over the step."""
    n, h, dim, vocab = 20, 2, 32, 100
    x, v, g = normal(n, h, dim, seed=1), normal(n, h, dim, seed=2), normal(n, h, dim, seed=3)
    pos, gain = torch.randint(0, 100000, (n,), device="cuda"), 1 + 0.2 * normal(dim, seed=4)
    f = lambda x: float((dm.qk_norm_rotary(x, None, pos, gain)[0].double() * g).sum())
    dx = dm.qk_norm_rotary_grad(g, None, x, None, pos, gain)[0]
    want, got = (f(x + 1e-2 * v) - f(x - 1e-2 * v)) / 2e-2, float((dx.double() * v).sum())
    assert abs(want - got) < 1e-2 * (1 + abs(want))
    z, u, a = normal(n, vocab, seed=5), normal(n, vocab, seed=6), torch.randint(0, vocab, (n,), device="cuda")
    one = torch.ones(n, device="cuda")

    def l(z):
        s = dm.token_stats(z, a)
        return float(s.logp.double().sum() + s.entropy.double().sum())
    s = dm.token_stats(z, a)
    dz = dm.token_stats_grad(z, a, s.norm, s.entropy, one, one)
    want, got = (l(z + 1e-2 * u) - l(z - 1e-2 * u)) / 2e-2, float((dz.double() * u).sum())
    assert abs(want - got) < 1e-2 * (1 + abs(want))
    # attention in bf16: a difference is off by the outputs' roundings over the step, so a large step and a loose bound
    q, k, v = (normal(200, h, 64, seed=i, dtype=BF16) for i, h in enumerate((2, 1, 1)))
    d, u = normal(200, 2, 64, seed=8, dtype=BF16), normal(200, 2, 64, seed=9, dtype=BF16)
    o = lambda q: float((dm.attention(q, k, v)[0].double() * d.double()).sum())
    out, lse = dm.attention(q, k, v)
    dq = dm.attention_grad(d, q, k, v, out, lse)[0]
    up, down = (q + 0.25 * u), (q - 0.25 * u)
    want, got = o(up) - o(down), float((dq.double() * (up.double() - down.double())).sum())
    assert abs(want - got) < 0.1 * float(dq.double().norm() * (up.double() - down.double()).norm())
    dm.check_status()


def test_views_of_one_array(dm):
    """q, k and v of one product, and their gradients into one array."""
    n, hq, hk, dim = 200, 4, 2, 64
    qkv, dqkv = normal(n, hq + 2 * hk, dim, seed=1, dtype=BF16), torch.full((n, hq + 2 * hk, dim), 7.0, dtype=BF16, device="cuda")
    q, k, v = qkv.split([hq, hk, hk], 1)
    out, lse = dm.attention(q, k, v)
    plain, _ = dm.attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(out, plain)
    d = normal(n, hq, dim, seed=2, dtype=BF16)
    dq, dk, dv = dqkv.split([hq, hk, hk], 1)
    dm.attention_grad(d, q, k, v, out, lse, dq=dq, dk=dk, dv=dv)
    want = dm.attention_grad(d, q.contiguous(), k.contiguous(), v.contiguous(), out, lse)
    assert torch.equal(dqkv, torch.cat(want, 1))
    # gradients with strides of 0 and heads in front reach the module
    leaf = qkv.clone().requires_grad_()
    dm.Attention()(*leaf.split([hq, hk, hk], 1)).sum().backward()
    ones = dm.attention_grad(torch.ones_like(out), q, k, v, out, lse)
    assert torch.equal(leaf.grad, torch.cat(ones, 1))
    heads_first = qkv.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(dm.Attention()(*heads_first.split([hq, hk, hk], 1)), out)
    odd = torch.zeros(n, hq, dim + 1, dtype=BF16, device="cuda")
    odd[..., :dim] = q
    assert torch.equal(dm.Attention()(odd[..., :dim], k, v), out)  # copied: its rows are off 16 bytes
    dm.check_status()


def everything(dm, s):
    q, k = dm.qk_norm_rotary(s["q"], s["k"], s["pos"], s["g"], s["g"])
    out, lse = dm.attention(q, k, s["v"], s["offsets"])
    grads = dm.attention_grad(s["d"], q, k, s["v"], out, lse, s["offsets"])
    back = dm.qk_norm_rotary_grad(grads[0], grads[1], s["q"], s["k"], s["pos"], s["g"], s["g"])
    stats = dm.token_stats(s["z"], s["a"], top=5)
    dz = dm.token_stats_grad(s["z"], s["a"], stats.norm, stats.entropy, s["w"], s["w"])
    return [q, k, out, lse, *grads, *back, *stats, dz]


def inputs(seed, n=260, lengths=(100, 0, 160)):
    g = torch.Generator().manual_seed(seed)
    return {"q": normal(n, 4, 64, seed=seed, dtype=BF16), "k": normal(n, 2, 64, seed=seed + 1, dtype=BF16),
            "v": normal(n, 2, 64, seed=seed + 2, dtype=BF16), "d": normal(n, 4, 64, seed=seed + 3, dtype=BF16),
            "g": 1 + 0.1 * normal(64, seed=seed + 4), "pos": torch.randint(0, 9999, (n,), generator=g).cuda(),
            "offsets": torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda(),
            "z": normal(n, 3000, seed=seed + 5, std=2.0), "a": torch.randint(0, 3000, (n,), generator=g).cuda(),
            "w": torch.rand(n, generator=g).cuda()}


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_in_captured_graphs(dm):
    """Two graphs of different sizes captured, replayed in turn with new inputs and other calls between them."""
    sets = [inputs(1), inputs(50, 400, (400,))]
    for s in sets:
        everything(dm, s)
    graphs, outs = [], []
    for s in sets:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(everything(dm, s))
        graphs.append(g)
    for seed in (100, 200):
        fresh = [inputs(seed, 260, (1, 259, 0)), inputs(seed + 50, 400, (400,))]
        for s, f in zip(sets, fresh):
            for name in s:
                s[name].copy_(f[name])
        graphs[0].replay()
        dm.release_workspace()
        other = everything(dm, inputs(seed + 7, 900, (900,)))
        graphs[1].replay()
        for f, out in zip(fresh, outs):
            assert same(out, everything(dm, f))
        assert all(o.isfinite().all() for o in other if o.is_floating_point())
    dm.check_status()


def test_on_several_streams(dm):
    """Calls on two streams at once, many times, give each the bits that it has alone."""
    sets = [inputs(1, 700, (300, 400)), inputs(30, 500, (500,))]
    want = [everything(dm, s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(everything(dm, s))
        torch.cuda.synchronize()
        assert all(same(g, w) for g, w in zip(got, want))
    # the stream argument, with tensors made on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = dm.attention(sets[0]["q"], sets[0]["k"], sets[0]["v"], stream=side)
    side.synchronize()
    assert torch.equal(out, dm.attention(sets[0]["q"], sets[0]["k"], sets[0]["v"])[0])
    dm.check_status()


def test_offsets_out_of_order(dm):
    """Offsets that fall or leave the arrays are reported; sequences in order beside them are as they should be."""
    s = inputs(1, 300, (300,))
    q, k, v, d = s["q"], s["k"], s["v"], s["d"]
    good, good_lse = dm.attention(q, k, v, torch.tensor([0, 100, 200, 300], device="cuda"))
    for bad in ([0, 100, 50, 50], [0, 100, 301], [0, 100, 1 << 40], [-5, 0, 100], [0, 100, -1]):
        offsets = torch.tensor(bad, device="cuda")
        out, lse = dm.attention(q, k, v, offsets)
        with pytest.raises(dm.DmuonError) as e:
            dm.check_status()
        assert e.value.status == dm.ERR_INDEX
        if bad[1] == 100:
            assert torch.equal(out[:50], good[:50])
        dm.attention_grad(d, q, k, v, out, lse, offsets)
        with pytest.raises(dm.DmuonError):
            dm.check_status()
    dm.check_status()


def test_many_sequences(dm):
    """More sequences than a warp looks at at once, most of them short or empty; rows by hand."""
    lengths = [(i * 7) % 5 for i in range(400)] + [300] + [0] * 50 + [1] * 70
    ends = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    s = inputs(1, ends[-1], lengths)
    out, lse = dm.attention(s["q"], s["k"], s["v"], s["offsets"])
    grads = dm.attention_grad(s["d"], s["q"], s["k"], s["v"], out, lse, s["offsets"])
    for i in (0, 1, 2, 33, 399, 400, 451, 520):
        b, e = ends[i], ends[i + 1]
        if b == e:
            continue
        o, l = dm.attention(s["q"][b:e], s["k"][b:e], s["v"][b:e])
        assert torch.equal(o, out[b:e]) and torch.equal(l, lse[:, b:e])
        gr = dm.attention_grad(s["d"][b:e], s["q"][b:e], s["k"][b:e], s["v"][b:e], o, l)
        assert all(torch.equal(x, y[b:e]) for x, y in zip(gr, grads))
    dm.check_status()


def test_launch_records(dm):
    """The per-launch timing names these calls."""
    s = inputs(1)
    everything(dm, s)
    torch.cuda.synchronize()
    dm.timing_enable(True)
    try:
        everything(dm, s)
        names = [name for name, _ in dm.timing_read_launches()]
    finally:
        dm.timing_enable(False)
    assert names == ["qk_rotary", "attention", "attention", "qk_rotary", "token_stats", "token_stats"]


@pytest.mark.slow
def test_long_sequences(dm):
    """One sequence of 9011 tokens, and one of 3 behind it: rows near both ends against 64 bits, one head."""
    n = 9014
    q, k, v, d = (normal(n, 1, 64, seed=i, dtype=BF16) for i in range(4))
    offsets = torch.tensor([0, 9011, n], device="cuda")
    out, lse = dm.attention(q, k, v, offsets)
    dq, dk, dv = dm.attention_grad(d, q, k, v, out, lse, offsets)
    x = (q[:9011, 0].double() @ k[:9011, 0].double().T) * 0.125
    x.masked_fill_(torch.ones(9011, 9011, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
    p = torch.softmax(x, -1)
    want = p @ v[:9011, 0].double()
    assert rel(out[:9011, 0], want) < 0.01
    dp = d[:9011, 0].double() @ v[:9011, 0].double().T
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * 0.125
    assert rel(dq[:9011, 0], ds @ k[:9011, 0].double()) < 0.01
    assert rel(dk[:9011, 0], ds.T @ q[:9011, 0].double()) < 0.01
    assert rel(dv[:9011, 0], p.T @ d[:9011, 0].double()) < 0.01
    dm.check_status()
