"""GPU: the token operators against their float64 oracle, at the sizes, strides and masks where they can go wrong.

Tolerances, elementwise, with u = 2^-24 (fp32) and the output's own rounding r = 2^-8 (bf16, 8 significant bits) or u (fp32):
- a lookup is one product: (u + r) |out|;
- a sum of k terms in any order is within k u of the sum of their absolute values, twice that for the products;
- a row's sum of squares: a thread adds at most dim / 32 + 8 terms and the threads' sums join in at most 16 steps, so
  it is within (dim / 32 + 24) u of itself; half of that for its root, and 8 u for the root's and the products' own;
- a log-probability: logits scaled by log2(e) / temperature are each within 2 u of themselves, 2^x within 4 u, a
  row's sum within (vocab / 256 + 32) u, and the logarithm and the final differences within 8 u of the values they
  join: 8 u (max |z| + log vocab + |log-probability|) + (vocab / 256 + 40) u. A probability and the ratio are off by
  as much relative to themselves. Rows whose ratio is within 1e-3 of a clip bound are not drawn.
- e4m3 keeps three bits after the leading one: |q scale - y| <= 2^-4 |y|, or half its smallest step, 2^-10 scale;
  both grow by y's own error."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import token_ops as ref  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.bfloat16]
TYPE_IDS = ["f32", "bf16"]


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def randn(shape, seed, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def place(t, layout):
    """The same values in another layout: "rows" strides a 2-D tensor wider than its rows; "offset" starts it one element
    after an aligned address."""
    if layout == "plain":
        return t
    n, d = t.shape
    if layout == "rows":
        wide = torch.full((n, d + 5), float("nan"), dtype=t.dtype, device=t.device)
        wide[:, :d] = t
        return wide[:, :d]
    flat = torch.empty(n * d + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(n, d)


def within(got, want, bound):
    got, want = f64(got), np.asarray(want)
    assert got.shape == want.shape
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound
    assert over.max(initial=-1.0) <= 0, f"off by {np.abs(got - want).max():.3e}, {over.max():.3e} over its bound"


# ---------------------------------------------------------------------------- embedding


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("tt,to", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                   (torch.float32, torch.float32), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("n,rows,dim", [(1, 7, 1), (1, 100, 4096), (5, 3, 8), (33, 50, 257), (700, 1000, 64),
                                        (64, 9, 8200), (3, 2, 20000)])
def test_embedding(dm, n, rows, dim, tt, to, layout):
    table = place(randn((rows, dim), 1, dtype=tt), layout)
    ids = torch.randint(0, rows, (n,), generator=torch.Generator().manual_seed(n))
    ids[0], ids[-1] = rows - 1, 0
    for kind in (torch.int64, torch.int32):
        out = place(torch.empty(n, dim, dtype=to, device="cuda"), layout)
        got = dm.embedding(table, ids.to(kind).cuda(), scale=1.5, out=out)
        assert got is out
        want = ref.embedding(f64(table), ids.tolist(), 1.5)
        within(out, want, (U + ROUND[to]) * np.abs(want))
    dm.check_status()


def test_embedding_shapes_and_bad_ids(dm):
    table = randn((6, 16), 2)
    ids = torch.tensor([[0, 5, 2], [1, 1, 3]], device="cuda")
    assert torch.equal(dm.embedding(table, ids), table[ids])
    assert dm.embedding(table, ids[:0]).shape == (0, 3, 16)
    dm.check_status()
    bad = torch.tensor([0, 6, -1, 1 << 40, 5], device="cuda")
    got = dm.embedding(table, bad)
    with pytest.raises(dm.DmuonError) as e:
        dm.check_status()
    assert e.value.status == dm.ERR_INDEX
    assert torch.equal(got[[0, 4]], table[[0, 5]]) and got[1:4].abs().max() == 0
    grad = dm.embedding_grad(torch.ones(5, 16, device="cuda"), bad, 6)
    with pytest.raises(dm.DmuonError) as e:
        dm.check_status()
    assert e.value.status == dm.ERR_INDEX
    assert grad.sum(1).tolist() == [16, 0, 0, 0, 0, 16]
    dm.check_status()


def spread_ids(kind, n, rows):
    g = torch.Generator().manual_seed(n + rows)
    if kind == "one":  # every token the same
        return torch.full((n,), rows // 2)
    if kind == "distinct":
        return torch.randperm(max(n, rows), generator=g)[:n] % rows
    if kind == "falling":  # many of the small ids, few of the others
        return ((torch.rand(n, generator=g, dtype=torch.float64) * np.log(rows + 1)).exp() - 1).long().clamp(0, rows - 1)
    return torch.randint(0, rows, (n,), generator=g)


@pytest.mark.parametrize("kind", ["one", "distinct", "falling", "even"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,rows,dim", [(0, 5, 8), (1, 1, 1), (1, 300, 64), (31, 1000, 7), (257, 64, 129),
                                        (1000, 70000, 16), (4099, 257, 40), (20000, 30, 8), (70001, 66000, 4),
                                        (513, 20, 2056), (40, 11, 16400)])
def test_embedding_grad(dm, n, rows, dim, dt, kind):
    ids = spread_ids(kind, n, rows)
    dout = randn((n, dim), 3, dtype=dt)
    pad = int(ids[n // 2]) if n > 2 and kind == "even" else None
    want, size, count = ref.embedding_grad(f64(dout), ids.tolist(), rows, 0.75, -1 if pad is None else pad)
    bound = (2 + count[:, None]) * U * size
    on_gpu = ids.to(torch.int32 if n % 2 else torch.int64).cuda()
    grad = torch.full((rows, dim), float("nan"), device="cuda")
    got = dm.embedding_grad(dout, on_gpu, rows, scale=0.75, padding_idx=pad, grad=grad)
    assert got is grad
    within(got, want, bound)
    assert torch.equal(got, dm.embedding_grad(dout, on_gpu, rows, scale=0.75, padding_idx=pad)), "bits differ"
    start = randn((rows, dim), 4)
    want, size, count = ref.embedding_grad(f64(dout), ids.tolist(), rows, 0.75, -1 if pad is None else pad, f64(start))
    bare = torch.from_numpy(count == 0).cuda()
    got = dm.embedding_grad(dout, on_gpu, rows, scale=0.75, padding_idx=pad, grad=start.clone(), accumulate=True)
    within(got, want, (3 + count[:, None]) * U * size)
    assert torch.equal(got[bare], start[bare])
    dm.check_status()


@pytest.mark.parametrize("layout", ["rows", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
def test_embedding_grad_layouts(dm, dt, layout):
    n, rows, dim = 300, 40, 264
    ids = spread_ids("falling", n, rows)
    dout = place(randn((n, dim), 5, dtype=dt), layout)
    want, size, count = ref.embedding_grad(f64(dout), ids.tolist(), rows, 2.0)
    grad = place(torch.full((rows, dim), float("nan"), device="cuda"), layout)
    dm.embedding_grad(dout, ids.cuda(), rows, scale=2.0, grad=grad)
    within(grad, want, (2 + count[:, None]) * U * size)
    if layout == "rows":
        assert torch.isnan(grad.as_strided((rows, 5), (dim + 5, 1), dim)).all(), "written between the rows"


@pytest.mark.parametrize("kind", ["one", "distinct", "falling", "even"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,rows,dim", [(256, 5, 1030), (255, 300, 33), (2, 1, 5)])
def test_embedding_grad_of_few_tokens(dm, n, rows, dim, dt, kind):
    """Up to 256 tokens are added without a sort."""
    test_embedding_grad(dm, n, rows, dim, dt, kind)


def test_embedding_offsets_past_32_bits(dm):
    """A table of over 2^32 elements: the last rows are looked up and receive their gradients."""
    rows, dim = (1 << 20) + 5, 4100
    table = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    table[rows - 1], table[rows - 2] = 3.0, 5.0
    ids = torch.tensor([rows - 1, 0, rows - 2, rows - 1], device="cuda")
    got = dm.embedding(table, ids, scale=2.0)
    assert got[:, 0].tolist() == [6.0, 0.0, 10.0, 6.0] and got[:, -1].tolist() == [6.0, 0.0, 10.0, 6.0]
    del table
    grad = dm.embedding_grad(torch.ones(4, dim, device="cuda"), ids, rows)
    assert grad[rows - 3:].sum(1).tolist() == [0.0, dim, 2.0 * dim] and float(grad.double().sum()) == 4.0 * dim
    dm.check_status()
    del grad
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------- residual RMS norm


def norm_error(dim):
    return ((dim / 32 + 24) / 2 + 8) * U


NORM_SIZES = [(1, 1), (1, 4096), (3, 7), (37, 128), (5, 129), (2, 1000), (300, 64), (2, 8200), (3, 16384), (2, 16385),
              (1, 40000), (1025, 96)]


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", NORM_SIZES)
def test_add_rmsnorm(dm, n, dim, dt, layout):
    x, r = place(randn((n, dim), 6, dtype=dt), layout), place(randn((n, dim), 7, 3.0, dt), layout)
    gain = randn((dim,), 8)
    for residual, g in ((r, gain), (None, gain), (r, None)):
        wy, wh = ref.add_rmsnorm(f64(x), None if residual is None else f64(residual), None if g is None else f64(g), 1e-5)
        y = place(torch.empty(n, dim, dtype=dt, device="cuda"), layout)
        y, h = dm.add_rmsnorm(x, residual, g, eps=1e-5, y=y)
        # where x and residual nearly cancel, y's error is that of their fp32 sum
        lost = U * (np.abs(wy) + (0 if residual is None else np.abs(wy)))
        within(y, wy, (norm_error(dim) + ROUND[dt]) * np.abs(wy) + lost)
        if residual is None:
            assert h is x
        else:
            within(h, wh, (U + ROUND[dt]) * np.abs(wh))
    if layout != "rows":  # in place: h over the residual, y over x
        y0, h0 = dm.add_rmsnorm(x, r, gain)
        x1, r1 = x.clone(), r.clone()
        y1, h1 = dm.add_rmsnorm(x1, r1, gain, y=x1, h=r1)
        assert y1 is x1 and h1 is r1 and torch.equal(y1, y0) and torch.equal(h1, h0)


@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", [(1, 1), (1, 4096), (3, 31), (7, 257), (300, 96), (2, 8200), (2, 16385), (65, 320)])
def test_add_rmsnorm_fp8(dm, n, dim, dt, group):
    x, r, gain = randn((n, dim), 9, dtype=dt), randn((n, dim), 10, 3.0, dt), randn((dim,), 11)
    x[0, :min(dim, 64)] = 0  # a group of zeros in the first row
    r[0, :min(dim, 64)] = 0
    for residual, layout in ((r, "plain"), (None, "offset")):
        q, scales, h = dm.add_rmsnorm_fp8(place(x, layout), residual, gain, group=group)
        wy, wh = ref.add_rmsnorm(f64(x), None if residual is None else f64(residual), f64(gain), 1e-6)
        ws = ref.group_scales(wy, group)
        err = norm_error(dim) + 3 * U
        within(scales, ws, err * np.abs(ws))
        wide = np.repeat(f64(scales), group or dim, axis=1)[:, :dim]
        got = f64(q.float()) * wide
        assert np.abs(f64(q.float())).max() <= 448
        bound = np.maximum(2.0 ** -4 * np.abs(wy), 2.0 ** -10 * wide) + 4 * err * np.abs(wy) + 1e-300
        assert (np.abs(got - wy) <= bound * (1 + 1e-6)).all()
        if residual is not None:
            within(h, wh, (U + ROUND[dt]) * np.abs(wh))


def test_add_rmsnorm_extremes(dm):
    """A row of zeros, rows of the type's largest and smallest values, and a row with NaN or infinity beside sound ones."""
    x = randn((6, 256), 12)
    x[0] = 0
    x[1] *= 1e-30
    x[3, 5] = float("nan")
    x[4, 9] = float("inf")
    gain = torch.ones(256, device="cuda")
    y, _ = dm.add_rmsnorm(x, None, gain, eps=0.0)
    assert torch.isnan(y[0]).all() and torch.isnan(y[3]).all()
    y, _ = dm.add_rmsnorm(x, None, gain, eps=1e-6)
    assert y[0].abs().max() == 0 and torch.isnan(y[3]).all()
    assert torch.isnan(y[4, 9]) and y[4, :9].abs().max() == 0
    for k in (2, 5):
        within(y[k], ref.add_rmsnorm(f64(x[k:k + 1]), None, None, 1e-6)[0][0], 1e-5)
    q, scales, _ = dm.add_rmsnorm_fp8(x, None, gain, group=128)
    assert scales[0].tolist() == [1.0, 1.0] and q[0].float().abs().max() == 0
    assert torch.isnan(q[3].float()).all()
    assert torch.isfinite(q[[0, 1, 2, 5]].float()).all()
    assert dm.add_rmsnorm(x[:0], None, gain)[0].shape == (0, 256)


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", NORM_SIZES + [(70, 4096), (5000, 16), (700, 129)])
def test_add_rmsnorm_grad(dm, n, dim, dt, layout):
    dy, h = place(randn((n, dim), 13, dtype=dt), layout), place(randn((n, dim), 14, 2.0, dt), layout)
    dh, gain = place(randn((n, dim), 15, dtype=dt), layout), randn((dim,), 16)
    err = 3 * norm_error(dim) + (dim / 32 + 24) * U
    for through, g in ((dh, gain), (None, gain), (dh, None)):
        wx, wg, sx, sg = ref.add_rmsnorm_grad(f64(dy), f64(h), None if g is None else f64(g),
                                              None if through is None else f64(through), 1e-5)
        dx, dgain = dm.add_rmsnorm_grad(dy, h, g, dh=through, eps=1e-5)
        within(dx, wx, err * sx + ROUND[dt] * np.abs(wx))
        if g is None:
            assert dgain is None
            continue
        within(dgain, wg, (n * U + norm_error(dim) + 4 * U) * sg)
        again = dm.add_rmsnorm_grad(dy, h, g, dh=through, eps=1e-5)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dgain), "bits differ"
    dx, dgain = dm.add_rmsnorm_grad(dy, h, gain, dh=dh)
    more = dgain.clone()
    over = dy.clone()
    dx1, more1 = dm.add_rmsnorm_grad(over, h, gain, dh=dh, dx=over, dgain=more, accumulate=True)
    assert more1 is more and torch.equal(dx1, dx) and torch.equal(more, dgain + dgain)
    over = dh.clone()
    assert torch.equal(dm.add_rmsnorm_grad(dy, h, gain, dh=over, dx=over)[0], dx)


def test_add_rmsnorm_grad_without_rows(dm):
    x, gain = torch.zeros(0, 96, device="cuda"), torch.ones(96, device="cuda")
    dx, dgain = dm.add_rmsnorm_grad(x, x, gain)
    assert dx.shape == (0, 96) and dgain.abs().max() == 0
    keep = torch.full((96,), 2.0, device="cuda")
    assert dm.add_rmsnorm_grad(x, x, gain, dgain=keep, accumulate=True)[1].tolist() == [2.0] * 96


# Rows of every length that has its own split among threads, and more of them than the GPU holds at a time.
NORM_TURNS = [(4001, 300), (4001, 515), (2500, 700), (1500, 1500), (1500, 2051), (700, 5003), (700, 6005), (400, 9301),
              (400, 12289), (400, 16000)]


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", NORM_TURNS)
def test_add_rmsnorm_in_turns(dm, n, dim, dt):
    test_add_rmsnorm(dm, n, dim, dt, "plain")
    test_add_rmsnorm_fp8(dm, n, dim, dt, 128)


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", NORM_TURNS)
def test_add_rmsnorm_grad_in_turns(dm, n, dim, dt):
    test_add_rmsnorm_grad(dm, n, dim, dt, "plain")


def test_norm_gradient_against_differences(dm):
    """The kernels' own forward in differences: a step of 1e-2 in fp32 values of order 1 is off by about 1e-4 (its square)
    and the rounding of a sum of 40 values, 40 u / 1e-2 = 2.4e-4; 2e-3 is asked for."""
    x, r, gain, dy, dh = (randn((1, 40), 20 + k) for k in range(5))
    gain = gain[0]

    def f(x):
        y, h = dm.add_rmsnorm(x, r, gain)
        return float((y.double() * dy).sum() + (h.double() * dh).sum())

    _, h = dm.add_rmsnorm(x, r, gain)
    dx, _ = dm.add_rmsnorm_grad(dy, h, gain, dh=dh)
    for k in range(40):
        step = torch.zeros_like(x)
        step[0, k] = 1e-2
        assert abs((f(x + step) - f(x - step)) / 2e-2 - float(dx[0, k])) < 2e-3


# ---------------------------------------------------------------------------- policy loss


def policy_inputs(n, vocab, dt, temperature, seed, layout="plain", masked=0.2):
    g = torch.Generator().manual_seed(seed)
    logits = randn((n, vocab), seed, 2.0, dt)
    targets = torch.randint(0, vocab, (n,), generator=g)
    logits[torch.arange(n), targets.cuda()] += (torch.rand(n, generator=g) * 8).to(dt).cuda()
    logits = place(logits, layout)
    lp = ref.log_softmax(f64(logits), temperature)[np.arange(n), targets.numpy()] if n else np.zeros(0)
    rng = np.random.default_rng(seed)
    old, rlp = lp + rng.normal(size=n) * 0.2, lp + rng.normal(size=n) * 0.3
    for bound in (0.8, 1.25):  # clear of the clip bounds
        near = np.abs(np.exp(lp - old) - bound) < 1e-3
        old[near] = lp[near]
    w = np.where(rng.random(n) < masked, 0.0, rng.uniform(0.5, 1.5, size=n) / max(n, 1))
    make = lambda v: torch.from_numpy(np.asarray(v)).float().cuda()  # noqa: E731
    return dict(logits=logits, targets=targets.cuda(), old_logp=make(old), advantages=make(rng.normal(size=n)),
                weights=make(w), ref_logp=make(rlp))


def check_policy(dm, s, temperature, kl, dlogits=None):
    n, vocab = s["logits"].shape
    args = dict(clip_low=0.2, clip_high=0.25, kl_coef=kl, temperature=temperature)
    z = f64(s["logits"])
    dt = s["logits"].dtype
    # the fp32 constants as the kernels get them
    wl, wlp, wd, terms, coef = ref.policy_loss(z, s["targets"].tolist(), *(f64(s[k]) for k in
                                               ("old_logp", "advantages", "weights", "ref_logp")), **args)
    live = (f64(s["weights"]) != 0) & (s["targets"].cpu().numpy() >= 0)
    zs = np.where(live[:, None], np.where(np.isfinite(z), np.abs(z), 0), 0).max(axis=1, initial=0) / temperature
    lp_err = 8 * U * (zs + np.log(vocab) + np.abs(wlp)) + (vocab / 256 + 40) * U
    loss, logp, d = dm.policy_loss(**s, **args, dlogits=dlogits)
    assert loss.shape == () and logp.shape == s["targets"].shape
    within(logp, wlp, lp_err * live)
    # A term's slope in lp is its coefficient; its own products round to 8 u of their values.
    reach = np.abs(coef) + f64(s["weights"]) * (np.abs(f64(s["advantages"])) * 2 + kl * 4)
    within(loss, wl, (lp_err * reach).sum() + (n + 16) * U * np.abs(terms).sum() + 1e-30)
    p = np.abs(wd)
    c_err = (reach * (lp_err + 16 * U)) / temperature
    ls = np.exp(ref.log_softmax(np.where(live[:, None], z, 0), temperature)) if n else z
    hit = np.zeros_like(z)
    hit[np.arange(n)[live], s["targets"].cpu().numpy()[live]] = 1
    bound = c_err[:, None] * (ls + hit) + (np.abs(coef) / temperature * (lp_err + 8 * U))[:, None] * (ls + hit * 0)
    within(d, wd, bound + ROUND[dt] * p + 4 * U * (np.abs(coef) / temperature)[:, None] * hit + 1e-38)
    assert f64(d)[~live].any() == False  # noqa: E712
    assert torch.equal(dm.token_logprobs(s["logits"], s["targets"], temperature)[torch.from_numpy(live).cuda()],
                       logp[torch.from_numpy(live).cuda()])
    return loss, logp, d


POLICY_SIZES = [(1, 1), (1, 2), (3, 33), (2, 1000), (70, 513), (5, 4096), (2, 50257), (3, 128256), (400, 100), (1, 262147),
                (9, 8191)]


@pytest.mark.parametrize("layout", ["plain", "rows", "offset"])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,vocab", POLICY_SIZES)
def test_policy_loss(dm, n, vocab, dt, layout):
    for temperature, kl in ((1.0, 0.1), (0.7, 0.0)):
        s = policy_inputs(n, vocab, dt, temperature, n + vocab, layout)
        loss, logp, d = check_policy(dm, s, temperature, kl)
        again = dm.policy_loss(**s, clip_low=0.2, clip_high=0.25, kl_coef=kl, temperature=temperature)
        assert torch.equal(again[0], loss) and torch.equal(again[1], logp) and torch.equal(again[2], d), "bits differ"
        alone = dm.policy_loss(**s, clip_low=0.2, clip_high=0.25, kl_coef=kl, temperature=temperature, dlogits=False)
        assert alone[2] is None and torch.equal(alone[0], loss) and torch.equal(alone[1], logp)
        # into a buffer of another layout, then over the logits themselves
        for other in ("plain", "rows", "offset"):
            into = place(torch.full((n, vocab), float("nan"), dtype=dt, device="cuda"), other)
            got = dm.policy_loss(**s, clip_low=0.2, clip_high=0.25, kl_coef=kl, temperature=temperature, dlogits=into)[2]
            assert got is into and torch.equal(into, d)
        got = dm.policy_loss(**s, clip_low=0.2, clip_high=0.25, kl_coef=kl, temperature=temperature,
                             dlogits=s["logits"])[2]
        assert torch.equal(got, d)
    dm.check_status()


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,vocab", [(400, 5003), (250, 12000), (250, 25003), (90, 50257)])
def test_policy_in_turns(dm, n, vocab, dt):
    """Clusters of every size of CTA, each with several rows."""
    s = policy_inputs(n, vocab, dt, 1.0, 9)
    loss, logp, d = check_policy(dm, s, 1.0, 0.1)
    some = {k: v[n // 2:] for k, v in s.items()}
    got = dm.policy_loss(**some, clip_low=0.2, clip_high=0.25, kl_coef=0.1)
    assert torch.equal(got[1], logp[n // 2:]) and torch.equal(got[2], d[n // 2:]), "a row's bits depend on the others"
    dm.check_status()


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
def test_policy_many_rows(dm, dt):
    s = policy_inputs(3001, 700, dt, 1.0, 5)
    check_policy(dm, s, 1.0, 0.1)
    s["targets"] = s["targets"].to(torch.int32)
    check_policy(dm, s, 1.0, 0.1)


def test_policy_masks(dm):
    """Rows that no weight or target asks for are not read, whatever they hold; none left is a loss of 0."""
    s = policy_inputs(6, 1000, torch.bfloat16, 1.0, 6, masked=0.0)
    s["weights"][1] = 0
    s["targets"][2] = -100
    s["logits"][1] = float("nan")
    s["logits"][2] = float("inf")
    s["old_logp"][1] = float("nan")
    s["advantages"][2] = float("inf")
    clean = {k: v.clone() for k, v in s.items()}
    clean["logits"][1:3] = 0
    clean["old_logp"][1] = 0
    clean["advantages"][2] = 0
    want = check_policy(dm, clean, 1.0, 0.1)
    got = dm.policy_loss(**s, clip_high=0.25, kl_coef=0.1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s["weights"].zero_()
    loss, logp, d = dm.policy_loss(**s, kl_coef=0.1)
    assert float(loss) == 0 and logp.abs().max() == 0 and d.abs().max() == 0
    empty = {k: v[:0] for k, v in s.items()}
    loss, logp, d = dm.policy_loss(**empty, kl_coef=0.1)
    assert float(loss) == 0 and logp.shape == (0,) and d.shape == (0, 1000)
    dm.check_status()


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("vocab", [40, 1000, 70001])
def test_policy_masked_logits(dm, vocab, dt):
    """Logits of -infinity and of the type's lowest value are tokens of probability 0, in stretches of any length."""
    s = policy_inputs(4, vocab, dt, 1.0, 7, masked=0.0)
    low = torch.finfo(dt).min
    t = s["targets"]
    for k, value in ((0, float("-inf")), (1, low), (2, float("-inf"))):
        keep = s["logits"][k, t[k]].clone()
        s["logits"][k, vocab // 3:] = value
        if k == 2:
            s["logits"][k] = value  # all but the target
        s["logits"][k, t[k]] = keep
    z = f64(s["logits"])
    lp = ref.log_softmax(z, 1.0)[np.arange(4), t.cpu().numpy()]
    s["old_logp"] = torch.from_numpy(lp + 0.05).float().cuda()
    s["ref_logp"] = torch.from_numpy(lp - 0.1).float().cuda()
    check_low = {k: v.clone() for k, v in s.items()}
    check_low["logits"][1][check_low["logits"][1] == low] = float("-inf")  # the bounds go by the sizes of live logits
    _, logp, d = check_policy(dm, check_low, 1.0, 0.1)
    got = dm.policy_loss(**s, clip_high=0.25, kl_coef=0.1)
    assert torch.equal(got[1], logp) and torch.equal(got[2], d)
    assert float(logp[2]) == 0


@pytest.mark.parametrize("vocab", [40, 1000, 70001])
def test_policy_unsound_rows(dm, vocab):
    """NaN, +infinity and a row of nothing but -infinity give NaN in their own rows alone."""
    s = policy_inputs(5, vocab, torch.float32, 1.0, 8, masked=0.0)
    s["logits"][1, vocab // 2] = float("nan")
    s["logits"][2, vocab - 1] = float("inf")
    s["logits"][3] = float("-inf")
    loss, logp, d = dm.policy_loss(**s, kl_coef=0.1)
    assert torch.isnan(loss) and torch.isnan(logp[1:4]).all() and torch.isnan(d[1:4]).all()
    one = {k: v[[0, 4]] for k, v in s.items()}
    _, lp, dd = dm.policy_loss(**one, kl_coef=0.1)
    assert torch.equal(logp[[0, 4]], lp) and torch.equal(d[[0, 4]], dd) and torch.isfinite(dd).all()


def test_policy_bad_targets(dm):
    s = policy_inputs(4, 64, torch.float32, 1.0, 9, masked=0.0)
    s["targets"][1], s["targets"][3] = 64, 1 << 40
    _, logp, d = dm.policy_loss(**s)
    with pytest.raises(dm.DmuonError) as e:
        dm.check_status()
    assert e.value.status == dm.ERR_INDEX
    assert logp[[1, 3]].abs().max() == 0 and d[[1, 3]].abs().max() == 0 and d[[0, 2]].abs().max() > 0
    s["weights"][[1, 3]] = 0  # a masked row's target is not looked at
    dm.policy_loss(**s)
    dm.check_status()


def test_policy_offsets_past_32_bits(dm):
    """Logits of over 2^32 elements in all: the last rows are read and written."""
    n, vocab = 20000, 215000
    logits = torch.zeros(n, vocab, dtype=torch.bfloat16, device="cuda")
    targets = torch.zeros(n, dtype=torch.int64, device="cuda")
    logits[n - 1, 7], targets[n - 1] = 20.0, 7
    z = torch.zeros(n, device="cuda")
    loss, logp, d = dm.policy_loss(logits, targets, z - 1.0, z + 1.0, z + 1.0, clip_high=1e9, dlogits=logits)
    want = ref.log_softmax(np.eye(1, vocab, 7) * 20.0, 1.0)[0, 7]
    assert abs(float(logp[-1]) - want) < 1e-4 and abs(float(logp[0]) + np.log(vocab)) < 1e-4
    r = np.exp(want + 1.0)
    assert abs(float(d[-1, 7]) + r * (1 - np.exp(want))) < 0.01 * r * (1 - np.exp(want)) + 1e-4
    dm.check_status()
    del logits, d
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------- streams and capture


def test_on_another_stream_and_in_a_graph(dm):
    s = policy_inputs(33, 3000, torch.bfloat16, 1.0, 10)
    x, r, gain = randn((33, 512), 1, dtype=torch.bfloat16), randn((33, 512), 2, dtype=torch.bfloat16), randn((512,), 3)
    ids = spread_ids("falling", 33, 100).cuda()
    table = randn((100, 512), 4)

    def all_of_them():
        y, h = dm.add_rmsnorm(dm.embedding(table, ids, 2.0, torch.bfloat16), r, gain)
        q, scales, _ = dm.add_rmsnorm_fp8(x, r, gain)
        dx, dgain = dm.add_rmsnorm_grad(x, h, gain, dh=r)
        return (y, h, q.float(), scales, dx, dgain, dm.embedding_grad(dx, ids, 100), *dm.policy_loss(**s, kl_coef=0.1))

    want = all_of_them()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(1000000)
        got = all_of_them()
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of_them()
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    dm.check_status()


def test_timing_records(dm):
    x = randn((8, 64), 1)
    dm.add_rmsnorm(x)
    dm.timing_enable(True)
    try:
        dm.add_rmsnorm(x)
        dm.token_logprobs(x, torch.zeros(8, dtype=torch.int64, device="cuda"))
        dm.embedding(x, torch.zeros(3, dtype=torch.int64, device="cuda"))
        names = [name for name, ms in dm.timing_read_launches() if ms > 0]
    finally:
        dm.timing_enable(False)
    assert names == ["rmsnorm", "policy_loss", "embedding"]
