"""GPU: attention over packed prompts and its gradient against the float64 oracle.

Tolerances, elementwise, with u = 2^-24 and bf16's rounding b = 2^-8. A score's product adds dim terms in fp32, which the
tensor cores may cut rather than round: 2 dim u of the sum of its absolute terms, and as much again for the maximum it is
taken from; the exponent's products 4 u |x| and 2^x 4 u. So p is off by x_off = 4 dim u reach + 16 u (1 + reach) of
itself, with reach the row's largest scale sum |q k|. Forward: p is rounded to bf16 beside a sum that is not, and the sums
over len keys are fp32: (b + x_off + 2 len u) sum p |v| + b |out|; lse: x_off + 2 len u + 4 u (1 + |lse|). Backward, at the
stored out and lse: p and ds are rounded to bf16, dout . v and D add dim terms: p_off = 2 b + x_off, dot_off = 4 dim u, sums
of len (times the group's heads) terms 4 len group u, and the result's own rounding b. D = dout . out has what out lost in
its rounding; the kernel adds the sum of ds to it, which is exactly that, in some of its sums: with D + t rest, t in [0, 1],
ds is p |rest| off at most, which the oracle adds to its bounds."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import token_ops as ref  # noqa: E402
from tests.test_gpu_token_ops import U, f64, randn, within  # noqa: E402

pytestmark = pytest.mark.gpu

B = 2.0 ** -8


@pytest.fixture(scope="module")
def dm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import newton_schulz_momentum_gb300 as dm
    return dm


def heads_like(n, heads, dim, layout, seed, std=1.0):
    t = randn((n, heads, dim), seed, std, torch.bfloat16)
    if layout == "part":  # a part of wider rows, with rows of NaN around it
        wide = torch.full((n, heads + 2, dim + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 1:1 + heads, :dim] = t
        return wide[:, 1:1 + heads, :dim]
    if layout == "by_head":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    return t


def check(dm, n, ends, heads, kv, dim, causal, layout="plain", scale=None, packed=True, seed=1, std=1.0):
    q, k, v = (heads_like(n, h, dim, layout, seed + i, std) for i, h in enumerate((heads, kv, kv)))
    offsets = torch.tensor(ends, dtype=torch.int32 if n % 2 else torch.int64).cuda() if packed else None
    kw = dict(offsets=offsets, causal=causal, scale=scale)
    if ends[0] > 0 or ends[-1] < n:  # tokens of no sequence hold NaN
        for t in (q, k, v):
            t[:ends[0]] = float("nan")
            t[ends[-1]:] = float("nan")
    got, lse = dm.attention(q, k, v, **kw)
    zero = np.zeros((n, 1, 1))
    zero[ends[0]:ends[-1]] = 1.0
    q64, k64, v64 = (np.where(zero > 0, f64(t), 0.0) for t in (q, k, v))
    want, want_lse, size, reach = ref.attention(q64, k64, v64, ends, causal, scale)
    length = max(b - a for a, b in zip(ends, ends[1:])) if len(ends) > 1 else 0
    x_off = 4 * dim * U * reach + 16 * U * (1 + reach)
    within(got, want, (B + x_off.T[..., None] + 2 * length * U) * size + B * np.abs(want))
    within(lse, want_lse, x_off + 2 * length * U + 4 * U * (1 + np.abs(want_lse)))
    again, lse2 = dm.attention(q, k, v, **kw)
    assert torch.equal(got, again) and torch.equal(lse, lse2), "bits differ"
    dout = heads_like(n, heads, dim, layout, seed + 7)
    if ends[0] > 0 or ends[-1] < n:
        dout[:ends[0]] = float("nan")
        dout[ends[-1]:] = float("nan")
    do64 = np.where(zero > 0, f64(dout), 0.0)
    grads = dm.attention_grad(dout, q, k, v, got, lse, **kw)
    wants, offs = ref.attention_grad(do64, q64, k64, v64, f64(got), f64(lse), ends, causal, scale,
                                     p_off=2 * B + x_off.max(initial=0) + 4 * length * heads // kv * U, dot_off=4 * dim * U)
    for g, w, o in zip(grads, wants, offs):
        within(g, w, o + B * np.abs(w) + 1e-30)
    again = dm.attention_grad(dout, q, k, v, got, lse, **kw)
    assert all(torch.equal(a, b) for a, b in zip(grads, again)), "bits differ"
    dm.check_status()


LENGTHS = [[1], [2], [127], [128], [129], [255], [256], [257], [61], [640, 1, 0, 0, 129, 3], [1, 1, 1, 1], [0, 0, 300, 0],
           [63, 64, 65, 66], [385, 511]]


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("heads,kv,dim", [(1, 1, 64), (2, 2, 128), (4, 1, 64), (3, 1, 128), (6, 2, 128)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_attention(dm, lengths, heads, kv, dim, causal):
    ends = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    check(dm, ends[-1], ends, heads, kv, dim, causal, packed=len(lengths) > 1)


@pytest.mark.parametrize("layout", ["plain", "part", "by_head"])
@pytest.mark.parametrize("heads,kv,dim", [(2, 1, 8), (1, 1, 16), (5, 5, 40), (2, 1, 72), (7, 1, 80), (4, 2, 96), (2, 2, 120)])
def test_dims_and_layouts(dm, heads, kv, dim, layout):
    """Tokens of no sequence in front and behind, whose NaN must reach nothing."""
    check(dm, 470, [5, 135, 136, 400, 461], heads, kv, dim, True, layout, scale=0.3)
    check(dm, 200, [0, 200], heads, kv, dim, False, layout, packed=False)


def test_sharp_and_growing_scores(dm):
    """Scores of up to several hundred, negative scales, and keys that grow along the sequence, so that the running maximum
    moves at every step."""
    check(dm, 700, [0, 700], 2, 1, 64, True, std=4.0)
    check(dm, 300, [0, 300], 2, 1, 128, False, scale=-0.2)
    n = 900
    q = torch.ones(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    k = (torch.arange(n, device="cuda").float() / 16).to(torch.bfloat16)[:, None, None].expand(n, 1, 64).contiguous()
    v = randn((n, 1, 64), 3, dtype=torch.bfloat16)
    for sign in (1.0, -1.0):
        got, lse = dm.attention(q, k, v, causal=False, scale=sign)
        x = f64(q)[:, 0] @ f64(k)[:, 0].T * sign
        p = np.exp(x - x.max(1, keepdims=True))
        want = p @ f64(v)[:, 0] / p.sum(1, keepdims=True)
        assert np.abs(f64(got)[:, 0] - want).max() < 2.0 ** -6
        assert np.abs(f64(lse)[0] - (x.max(1) + np.log(p.sum(1)))).max() < 1e-2
    dm.check_status()


def test_batches_equal_sequences(dm):
    """(batch, length, heads, dim) is a sequence each, as with offsets; and a sequence gives the same bits alone."""
    q, k, v = (randn((3, 150, h, 64), i, dtype=torch.bfloat16) for i, h in enumerate((4, 2, 2)))
    got, lse = dm.attention(q, k, v)
    offsets = torch.tensor([0, 150, 300, 450], device="cuda")
    flat, lse2 = dm.attention(q.view(450, 4, 64), k.view(450, 2, 64), v.view(450, 2, 64), offsets)
    assert torch.equal(got.view(450, 4, 64), flat) and torch.equal(lse, lse2) and lse.shape == (4, 450)
    one, lse1 = dm.attention(q[1], k[1], v[1])
    assert torch.equal(one, got[1]) and torch.equal(lse1, lse[:, 150:300])
    d = randn((3, 150, 4, 64), 9, dtype=torch.bfloat16)
    a = dm.attention_grad(d, q, k, v, got, lse)
    b = dm.attention_grad(d[1], q[1], k[1], v[1], one, lse1)
    assert all(torch.equal(x[1], y) for x, y in zip(a, b))
    dm.check_status()


def test_not_finite_values_stay_in_their_sequence(dm):
    """NaN and infinities in every tensor of one sequence; its neighbours in the same tiles do not notice."""
    ends = [0, 70, 75, 140, 300]
    offsets = torch.tensor(ends, device="cuda")
    for dim in (64, 128):
        q, k, v, d = (randn((300, h, dim), i, dtype=torch.bfloat16) for i, h in enumerate((4, 2, 2, 4)))
        for causal in (True, False):
            out, lse = dm.attention(q, k, v, offsets, causal)
            grads = dm.attention_grad(d, q, k, v, out, lse, offsets, causal)
            bad = [t.clone() for t in (q, k, v, d)]
            for t in bad:
                t[70:75] = float("nan")
                t[72] = float("inf")
                t[73] = float("-inf")
            out2, lse2 = dm.attention(*bad[:3], offsets, causal)
            grads2 = dm.attention_grad(bad[3], *bad[:3], out2, lse2, offsets, causal)
            rest = [i for i in range(300) if not 70 <= i < 75]
            assert torch.equal(out[rest], out2[rest]) and torch.equal(lse[:, rest], lse2[:, rest])
            assert all(torch.equal(a[rest], b[rest]) for a, b in zip(grads, grads2))
            assert out2[70:75].isnan().all()
    dm.check_status()


def test_given_outputs_keep_other_tokens(dm):
    """Rows of no sequence stay as they were in given outputs, and are zeros in new ones."""
    n, offsets = 200, torch.tensor([10, 60, 150], device="cuda", dtype=torch.int32)
    q, k, v, d = (randn((n, h, 64), i, dtype=torch.bfloat16) for i, h in enumerate((2, 1, 1, 2)))
    new = [torch.full_like(t, 7.0) for t in (q, q, k, v)]
    lse = torch.full((2, n), 7.0, device="cuda")
    out, got_lse = dm.attention(q, k, v, offsets, out=new[0], lse=lse)
    assert out is new[0] and got_lse is lse
    plain, plain_lse = dm.attention(q, k, v, offsets)
    grads = dm.attention_grad(d, q, k, v, out, lse, offsets, dq=new[1], dk=new[2], dv=new[3])
    zeros = dm.attention_grad(d, q, k, v, plain, plain_lse, offsets)
    for a, b in zip((out, *grads), (plain, *zeros)):
        assert torch.equal(a[10:150], b[10:150])
        assert (a[:10] == 7).all() and (a[150:] == 7).all() and not b[:10].any() and not b[150:].any()
    assert (lse[:, :10] == 7).all() and (lse[:, 150:] == 7).all() and not plain_lse[:, 150:].any()
    none, _ = dm.attention(q, k, v, offsets[:1])  # no sequence at all
    assert not none.any()
    empty, _ = dm.attention(q[:0], k[:0], v[:0])
    assert empty.shape == (0, 2, 64)
    dm.check_status()


def test_refusals(dm):
    q, k, v = (randn((8, h, 64), i, dtype=torch.bfloat16) for i, h in enumerate((4, 2, 2)))
    for word, call in (("bfloat16", lambda: dm.attention(q.float(), k.float(), v.float())),
                       ("shape", lambda: dm.attention(q, k, v[:7])),
                       ("tokens", lambda: dm.attention(q, k[:7], v)),
                       ("offsets", lambda: dm.attention(q, k, v, torch.zeros(2, 2, dtype=torch.int32, device="cuda"))),
                       ("lse", lambda: dm.attention_grad(q, q, k, v, q, torch.zeros(3, device="cuda")))):
        with pytest.raises(ValueError, match=word):
            call()
    wide = torch.zeros(8, 4, 66, dtype=torch.bfloat16, device="cuda")
    for word, call in (("multiple of kv_heads", lambda: dm.attention(q[:, :3], k, v)),
                       ("multiple of 8", lambda: dm.attention(q[..., :60], k[..., :60], v[..., :60])),
                       ("strides", lambda: dm.attention(wide[..., :64], k, v)),
                       ("16-byte", lambda: dm.attention(wide.view(-1)[1:8 * 256 + 1].view(8, 4, 64), k, v)),
                       ("out cannot", lambda: dm.attention(q, k, v, out=q)),
                       ("finite", lambda: dm.attention(q, k, v, scale=float("inf"))),
                       ("cannot go over", lambda: dm.attention_grad(q, q, k, v, q, torch.zeros(4, 8, device="cuda"), dq=q)),
                       ("at most 128", lambda: dm.attention(*(torch.zeros(4, 1, 136, dtype=torch.bfloat16, device="cuda"),) * 3))):
        with pytest.raises(dm.DmuonError, match=word):
            call()
    dm.check_status()
