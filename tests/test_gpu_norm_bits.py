"""GPU: the forward norm's 8-bit output, bit for bit: the same wherever rows lie, and its scales rounded once."""

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_token_ops import TYPE_IDS, TYPES, place, randn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", [(700, 96), (600, 129), (900, 1027), (300, 4096), (200, 8200), (100, 16383)])
def test_fp8_rows_do_not_depend_on_where_they_lie(dm, n, dim, dt, group):
    """Arrays on 16 bytes, off them alike, off them each in another way, and every row by itself."""
    x, r, gain = randn((n, dim), 40, dtype=dt), randn((n, dim), 41, 3.0, dt), randn((dim,), 42)
    want = dm.add_rmsnorm_fp8(x, r, gain, group=group)
    for lx, lr, lh in (("rows", "rows", "rows"), ("offset", "offset", "offset"), ("plain", "rows", "offset"),
                       ("offset", "plain", "rows")):
        h = place(torch.empty(n, dim, dtype=dt, device="cuda"), lh)
        got = dm.add_rmsnorm_fp8(place(x, lx), place(r, lr), gain, group=group, h=h)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a,
                               b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b), (lx, lr, lh)
    for k in (0, n // 2, n - 1):
        got = dm.add_rmsnorm_fp8(x[k:k + 1], r[k:k + 1], gain, group=group)
        assert torch.equal(got[0].view(torch.uint8), want[0][k:k + 1].view(torch.uint8))
        assert torch.equal(got[1], want[1][k:k + 1])


@pytest.mark.parametrize("dim", [64, 256, 4096])
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
def test_fp8_scales_are_rounded_once(dm, dim, dt):
    """Rows of +-1 with eps 0 have a norm of exactly 1, so y is the gain, and a group's scale the quotient of its largest
    gain and 448, rounded to fp32. q is y over that scale, but for quotients within 2^-22 of a border between two
    e4m3 values, which the two roundings to fp32 can move across it."""
    g = torch.Generator().manual_seed(dim)
    x = torch.where(torch.rand(30, dim, generator=g) < 0.5, -1.0, 1.0).to(dt).cuda()
    for seed in range(20):
        gain = randn((dim,), 100 + seed)
        q, scales, _ = dm.add_rmsnorm_fp8(x, None, gain, eps=0.0, group=32)
        top = gain.abs().view(-1, 32).amax(1).double()
        want = (top / 448.0).float()
        assert torch.equal(scales, want.expand(30, -1))
        y = x.double() * gain.double()
        exact = y / want.double().repeat_interleave(32)
        safe = (exact * (1 + 2.0 ** -22)).float().to(torch.float8_e4m3fn).float() == (
            exact * (1 - 2.0 ** -22)).float().to(torch.float8_e4m3fn).float()
        assert safe.double().mean() > 0.999
        assert torch.equal(q.float()[safe], exact.float().to(torch.float8_e4m3fn).float()[safe])


@pytest.mark.parametrize("dim", [129, 4096])
def test_gain_sums_are_added_pairwise(dm, dim):
    """152 rows, one per CTA, whose terms are all positive, so that the sums over the CTAs are what rounds. A rounding's
    error has a deviation of about 0.41 u of the value (u = 2^-24). Pairwise over 2^L equal terms the last sum counts
    in full, the two before it by half and so on: 0.41 u sqrt(2) = 0.6 u in all, and the terms' own errors average out
    to a tenth of theirs. One after the other over 32 warps' sums it would be 0.41 u sqrt(32 / 3) = 1.35 u. The root mean
    square over the columns has to be below 1 u."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    h = torch.randn(152, dim, generator=g, device="cuda")
    dy = h.sign() * (0.5 + torch.rand(152, dim, generator=g, device="cuda"))
    _, dgain = dm.add_rmsnorm_grad(dy, h, torch.ones(dim, device="cuda"), eps=1e-6)
    h64 = h.double()
    want = (dy.double() * h64 * torch.rsqrt((h64 * h64).mean(1, keepdim=True) + 1e-6)).sum(0)
    error = ((dgain.double() - want) / want).pow(2).mean().sqrt()
    assert float(error) < 2.0 ** -24, float(error) * 2 ** 24
