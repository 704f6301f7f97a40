"""GPU: the norms with every array in the same strided or shifted layout, so that rows stay in registers as they do in
contiguous tensors, with more rows than the GPU holds at a time. Tolerances as in test_gpu_token_ops.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import token_ops as ref  # noqa: E402
from tests.test_gpu_token_ops import (NORM_TURNS, ROUND, TYPE_IDS, TYPES, U, f64, norm_error, place, randn,  # noqa: E402
                                      within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


# Gaps of 5 elements (rows at every offset from 16 bytes), of 16 (rows on 16 bytes where their length is), a start one
# element behind an aligned address, and both of these.
LAYOUTS = {"rows": 5, "wide": 16, "offset": None, "shifted": 16}


def lay(t, layout):
    if layout not in ("wide", "shifted"):
        return place(t, layout)
    n, d = t.shape
    flat = torch.full((n * (d + 16) + 1,), float("nan"), dtype=t.dtype, device=t.device)
    view = flat[1 if layout == "shifted" else 0:][:n * (d + 16)].view(n, d + 16)
    view[:, :d] = t
    return view[:, :d]


def blank(n, dim, dt, layout):
    return lay(torch.full((n, dim), float("nan"), dtype=dt, device="cuda"), layout)


def gaps_untouched(t, layout):
    gap = LAYOUTS[layout]
    if gap is None:
        return True
    n, d = t.shape
    return bool(torch.isnan(t.as_strided((n, gap), (d + gap, 1), t.storage_offset() + d)).all())


# Lengths of which rows end on 16 bytes, so that `wide` stays clear of the kernels for rows with edges.
SIZES = NORM_TURNS + [(5000, 128), (3000, 512), (2000, 2048), (900, 4096), (400, 8192), (300, 16384)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", SIZES)
def test_forward(dm, n, dim, dt, layout):
    """Bit for bit what contiguous tensors give (which are held against the oracle elsewhere), gaps left alone."""
    x, r, gain = randn((n, dim), 50, dtype=dt), randn((n, dim), 51, 3.0, dt), randn((dim,), 52)
    want_y, want_h = dm.add_rmsnorm(x, r, gain)
    want_q, want_s, _ = dm.add_rmsnorm_fp8(x, r, gain)
    alone, _ = dm.add_rmsnorm(x, None, gain)
    xs, rs, y, h = lay(x, layout), lay(r, layout), blank(n, dim, dt, layout), blank(n, dim, dt, layout)
    dm.add_rmsnorm(xs, rs, gain, y=y, h=h)
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    assert gaps_untouched(y, layout) and gaps_untouched(h, layout)
    h = blank(n, dim, dt, layout)
    q, s, _ = dm.add_rmsnorm_fp8(xs, rs, gain, h=h)
    assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
    assert torch.equal(h, want_h) and gaps_untouched(h, layout)
    y = blank(n, dim, dt, layout)
    assert torch.equal(dm.add_rmsnorm(xs, None, gain, y=y)[0], alone)
    dm.add_rmsnorm(xs, rs, gain, y=xs, h=rs)  # in place
    assert torch.equal(xs, want_y) and torch.equal(rs, want_h) and gaps_untouched(xs, layout) and gaps_untouched(rs, layout)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", SIZES)
def test_gradient(dm, n, dim, dt, layout):
    dy, h = lay(randn((n, dim), 53, dtype=dt), layout), lay(randn((n, dim), 54, 2.0, dt), layout)
    dh, gain = lay(randn((n, dim), 55, dtype=dt), layout), randn((dim,), 56)
    wx, wg, sx, sg = ref.add_rmsnorm_grad(f64(dy), f64(h), f64(gain), f64(dh), 1e-5)
    dx = blank(n, dim, dt, layout)
    _, dgain = dm.add_rmsnorm_grad(dy, h, gain, dh=dh, eps=1e-5, dx=dx)
    err = 3 * norm_error(dim) + (dim / 32 + 24) * U
    within(dx, wx, err * sx + ROUND[dt] * np.abs(wx))
    within(dgain, wg, (n * U + norm_error(dim) + 4 * U) * sg)
    assert gaps_untouched(dx, layout)
    for over in (dy, dh):
        keep = over.clone()
        again = dm.add_rmsnorm_grad(dy, h, gain, dh=dh, eps=1e-5, dx=over)
        assert torch.equal(over, dx) and torch.equal(again[1], dgain) and gaps_untouched(over, layout)
        over.copy_(keep)


@pytest.mark.parametrize("dt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("n,dim", [(2500, 700), (700, 6005), (500, 4096)])
def test_arrays_in_different_layouts(dm, n, dim, dt):
    x, r, gain = randn((n, dim), 57, dtype=dt), randn((n, dim), 58, dtype=dt), randn((dim,), 59)
    want = dm.add_rmsnorm(x, r, gain)
    y, h = blank(n, dim, dt, "rows"), blank(n, dim, dt, "shifted")
    dm.add_rmsnorm(lay(x, "offset"), lay(r, "wide"), gain, y=y, h=h)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    assert gaps_untouched(y, "rows") and gaps_untouched(h, "shifted")
    wx, wg, sx, sg = ref.add_rmsnorm_grad(f64(x), f64(r), f64(gain), None, 1e-5)
    dx = blank(n, dim, dt, "rows")
    _, dgain = dm.add_rmsnorm_grad(lay(x, "offset"), lay(r, "wide"), gain, eps=1e-5, dx=dx)
    within(dx, wx, (3 * norm_error(dim) + (dim / 32 + 24) * U) * sx + ROUND[dt] * np.abs(wx))
    within(dgain, wg, (n * U + norm_error(dim) + 4 * U) * sg)
    assert gaps_untouched(dx, "rows")
