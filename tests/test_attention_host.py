"""CPU checks of the host side of per-head norm with rotation, attention and token statistics: devices, refusals."""

import ctypes

import pytest

from tests.test_token_ops_host import Stub, entry_body

ENTRIES = ("dmuon_qk_norm_rotary", "dmuon_qk_norm_rotary_grad", "dmuon_attention", "dmuon_attention_grad",
           "dmuon_token_stats", "dmuon_token_stats_grad")
A, B, C, D = 0x10000, 0x20000, 0x30000, 0x40000  # aligned addresses, never read


@pytest.mark.parametrize("name", ENTRIES)
def test_entries_let_no_exception_out(name):
    body = entry_body(name).strip()
    assert body.startswith("try {") and "catch (const std::exception" in body


class Heads(Stub):
    def stride(self, k=None):
        out, step = [], 1
        for size in reversed(self.shape):
            out.insert(0, step)
            step *= size
        return tuple(out) if k is None else out[k]

    def zero_(self):
        return self


@pytest.fixture
def calls(monkeypatch):
    """The entry points' calls, as (name, device that was current, stream), with device 0 current at first."""
    import contextlib
    import types
    torch = pytest.importorskip("torch")
    from newton_schulz_momentum_gb300 import token_ops
    current, made = [0], []

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    def entry(name):
        def call(*args):
            made.append((name, current[0], args[-1]))
            return 0
        return call

    def empty(*shape, dtype=None, device=None):
        return Heads(*(shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape), dtype=dtype,
                     device=int(device.split(":")[1]))

    monkeypatch.setattr(token_ops, "lib", lambda: types.SimpleNamespace(**{n: entry(n) for n in ENTRIES}))
    monkeypatch.setattr(token_ops, "_current_device", lambda: current[0])
    monkeypatch.setattr(token_ops, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", empty)
    return made


def all_calls(at, odd=None):
    """One call of each function with every tensor on device `at`, but for argument `odd` of (function, argument, device)."""
    import torch
    from newton_schulz_momentum_gb300 import token_ops as ops
    i64, i32, b16, n, d = torch.int64, torch.int32, torch.bfloat16, 4, 8
    q, k, lse = (n, 2, d, b16), (n, 1, d, b16), (2, n)
    kinds = {
        "qk_norm_rotary": dict(q=q, k=k, positions=(n, i64), q_gain=(d,), k_gain=(d,), q_out=q, k_out=k),
        "qk_norm_rotary_grad": dict(dq_out=q, dk_out=k, q=q, k=k, positions=(n, i64), q_gain=(d,), k_gain=(d,), dq=q, dk=k),
        "attention": dict(q=q, k=k, v=k, offsets=(3, i32), out=q, lse=lse),
        "attention_grad": dict(dout=q, q=q, k=k, v=k, out=q, lse=lse, offsets=(3, i32), dq=q, dk=k, dv=k),
        "token_stats": dict(logits=(n, d), targets=(n, i64)),
        "token_stats_grad": dict(logits=(n, d), targets=(n, i64), norm=(n, 2), entropy=(n,), dlogp=(n,), dentropy=(n,),
                                 dlogits=(n, d)),
    }
    for name, shapes in kinds.items():
        if odd is not None and odd[0] != name:
            continue
        args = {}
        for arg, shape in shapes.items():
            dtype = shape[-1] if isinstance(shape[-1], torch.dtype) else torch.float32
            sizes = [v for v in shape if isinstance(v, int)]
            args[arg] = Heads(*sizes, dtype=dtype, device=odd[2] if odd is not None and odd[1] == arg else at)
        yield name, args, lambda fn=getattr(ops, name), a=args: fn(**a)


def test_calls_run_on_their_tensors_device(calls):
    for at in (0, 1):
        for name, args, call in all_calls(at):
            del calls[:]
            call()
            assert [c[1:] for c in calls] == [(at, 100 + at)], name


def test_tensors_of_two_devices_are_refused(calls):
    seen = 0
    for name, args, _ in list(all_calls(1)):
        for arg in args:
            for where, word in ((0, "cuda"), (-1, "CUDA")):
                ((_, _, call),) = all_calls(1, odd=(name, arg, where))
                with pytest.raises(ValueError, match=word):
                    call()
                assert not calls
                seen += 1
    assert seen == 2 * 41


def heads(ptr, token=16, head=8):
    return [ptr, token, head]


def rotary(q=None, k=None, q_out=None, k_out=None, heads_=2, kv=1, dtype=1, gains=(None, None), norm=1, eps=1e-6, n=4, dim=8,
           rd=8, base=1e4, freqs=None, pos=D, id_bytes=8, axes=1, stride=4, sections=None):
    parts = None if sections is None else (ctypes.c_int64 * len(sections))(*sections)
    f = None if freqs is None else (ctypes.c_double * len(freqs))(*freqs)
    return [*(q or heads(A)), heads_, *(k or heads(B, 8)), kv, dtype, *gains, norm, eps, n, dim, rd, 0, base, f, pos,
            id_bytes, axes, stride, parts, *(q_out or heads(C)), *(k_out or heads(0x50000, 8)), None]


def attention(q=None, k=None, v=None, out=None, dtype=1, n=4, heads_=2, kv=1, dim=8, offsets=None, id_bytes=4, sequences=1,
              scale=0.3, lse=D):
    return [*(q or heads(A)), *(k or heads(B, 8)), *(v or heads(0x28000, 8)), dtype, n, heads_, kv, dim, offsets, id_bytes,
            sequences, 1, scale, 0, *(out or heads(C)), lse, None]


def stats(dtype=1, ld=16, n=4, vocab=16, targets=B, id_bytes=8, top=2, temp=1.0, logp=C, entropy=C, top_logp=C, top_ids=C,
          norm=C):
    return [A, dtype, ld, n, vocab, targets, id_bytes, top, temp, logp, entropy, top_logp, top_ids, norm, None]


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("entry,args,word", [
    ("dmuon_qk_norm_rotary", rotary(dtype=2), "dtype"),
    ("dmuon_qk_norm_rotary", rotary(heads_=0), "heads"),
    ("dmuon_qk_norm_rotary", rotary(dim=7), "even"),
    ("dmuon_qk_norm_rotary", rotary(rd=10), "rotary_dim"),
    ("dmuon_qk_norm_rotary", rotary(axes=5), "axes"),
    ("dmuon_qk_norm_rotary", rotary(axes=2), "sections"),
    ("dmuon_qk_norm_rotary", rotary(axes=2, sections=(1, 2)), "add up"),
    ("dmuon_qk_norm_rotary", rotary(axes=2, sections=(5, -1)), "sections"),
    ("dmuon_qk_norm_rotary", rotary(id_bytes=2), "id_bytes"),
    ("dmuon_qk_norm_rotary", rotary(pos=None), "NULL"),
    ("dmuon_qk_norm_rotary", rotary(eps=NAN), "eps"),
    ("dmuon_qk_norm_rotary", rotary(base=0.0), "base"),
    ("dmuon_qk_norm_rotary", rotary(freqs=(1.0, NAN, 0.0, 0.0)), "frequency 1"),
    ("dmuon_qk_norm_rotary", rotary(gains=(A, None), norm=0), "norm"),
    ("dmuon_qk_norm_rotary", rotary(gains=(A + 2, None)), "aligned"),
    ("dmuon_qk_norm_rotary", rotary(q=heads(None)), "q must not be NULL"),
    ("dmuon_qk_norm_rotary", rotary(q=heads(A + 1)), "aligned"),
    ("dmuon_qk_norm_rotary", rotary(q_out=heads(C, 8, 8)), "overlap"),
    ("dmuon_qk_norm_rotary", rotary(q_out=heads(C, 16, 4)), "overlap"),
    ("dmuon_qk_norm_rotary", rotary(q=heads(A, -16, 8)), "negative"),
    ("dmuon_qk_norm_rotary", rotary(q=heads(A), q_out=heads(A, 24, 8)), "strides must be equal"),
    ("dmuon_qk_norm_rotary", rotary(n=-1), "n must be"),
    ("dmuon_attention", attention(dtype=0), "BF16"),
    ("dmuon_attention", attention(heads_=3, kv=2), "multiple of kv_heads"),
    ("dmuon_attention", attention(dim=12), "multiple of 8"),
    ("dmuon_attention", attention(n=-1), "n must be"),
    ("dmuon_attention", attention(sequences=3), "equal length"),
    ("dmuon_attention", attention(sequences=0), "sequences"),
    ("dmuon_attention", attention(offsets=D + 2), "aligned"),
    ("dmuon_attention", attention(offsets=D, id_bytes=3), "id_bytes"),
    ("dmuon_attention", attention(scale=INF), "finite"),
    ("dmuon_attention", attention(scale=0.0), "not 0"),
    ("dmuon_attention", attention(q=heads(A + 8)), "16-byte"),
    ("dmuon_attention", attention(k=heads(B, 12)), "multiples of 8"),
    ("dmuon_attention", attention(q=heads(A, 0, 8)), "must not be 0"),
    ("dmuon_attention", attention(out=heads(C, 8, 8)), "overlap"),
    ("dmuon_attention", attention(out=heads(A)), "out cannot go over"),
    ("dmuon_attention", attention(lse=None), "lse"),
    ("dmuon_token_stats", stats(dtype=3), "dtype"),
    ("dmuon_token_stats", stats(ld=15), "leading dimension"),
    ("dmuon_token_stats", stats(top=33), "top"),
    ("dmuon_token_stats", stats(top=-1), "top"),
    ("dmuon_token_stats", stats(vocab=1, top=2), "top"),
    ("dmuon_token_stats", stats(temp=0.0), "temperature"),
    ("dmuon_token_stats", stats(logp=None), "logp"),
    ("dmuon_token_stats", stats(entropy=None), "entropy"),
    ("dmuon_token_stats", stats(top_ids=None), "top_ids"),
    ("dmuon_token_stats", stats(top_ids=C + 4), "top_ids"),
    ("dmuon_token_stats", stats(norm=C + 2), "norm"),
    ("dmuon_token_stats_grad", [A, 1, 16, 4, 16, None, 8, C, C, C, None, 1.0, D, 16, None], "targets"),
    ("dmuon_token_stats_grad", [A, 1, 16, 4, 16, B, 8, C, None, C, C, 1.0, D, 16, None], "entropy"),
    ("dmuon_token_stats_grad", [A, 1, 16, 4, 16, B, 8, C, C, C, C, 1.0, A, 24, None], "dlogits is written over logits"),
], ids=lambda v: v if isinstance(v, str) else "")
def test_invalid_arguments_are_refused(entry, args, word):
    """Before a device is asked for anything."""
    import newton_schulz_momentum_gb300 as dm
    from newton_schulz_momentum_gb300 import build
    build.build()
    rc = getattr(dm.lib(), entry)(*args)
    message = dm.lib().dmuon_last_error().decode()
    assert rc == dm.ERR_INVALID_ARG and word in message, (rc, message)


def test_beyond_the_limits():
    import newton_schulz_momentum_gb300 as dm
    for entry, args in (("dmuon_qk_norm_rotary", rotary(dim=258, rd=8)), ("dmuon_attention", attention(dim=136)),
                        ("dmuon_attention", attention(n=(1 << 30) + 1)), ("dmuon_attention", attention(n=1 << 30, heads_=60000, q=heads(A, 480000, 8), out=heads(C, 480000, 8)))):
        assert getattr(dm.lib(), entry)(*args) == dm.ERR_UNSUPPORTED, (entry, dm.lib().dmuon_last_error())


def test_attention_gradient_outputs_must_be_apart():
    import newton_schulz_momentum_gb300 as dm

    def call(dq, dk, dv):
        args = [*heads(A), *heads(B), *heads(C, 8), *heads(0x38000, 8), *heads(D), D, 1, 4, 2, 1, 8, None, 4, 1, 1, 0.3, 0,
                *heads(dq), *heads(dk, 8), *heads(dv, 8), None]
        rc = dm.lib().dmuon_attention_grad(*args)
        return rc, dm.lib().dmuon_last_error().decode()

    for bad in ((A, 0x60000, 0x70000), (0x60000, C, 0x70000), (0x60000, 0x60000, 0x70000), (0x50000, 0x60000, 0x60000)):
        rc, message = call(*bad)
        assert rc == dm.ERR_INVALID_ARG and ("cannot go over" in message or "different" in message), message


def test_heads_of_views():
    """One stride from token to token and one from head to head, whatever the dimensions in front."""
    torch = pytest.importorskip("torch")
    from newton_schulz_momentum_gb300.token_ops import _heads
    qkv = torch.empty(2, 5, 7, 8)
    assert _heads(qkv, "q") == (10, 7, 8, 56, 8)
    assert _heads(qkv[:, :, 2:4], "q") == (10, 2, 8, 56, 8)
    assert _heads(qkv[:, :, 2:4, :4], "q") == (10, 2, 4, 56, 8)
    assert _heads(qkv[1:, :, :1], "q") == (5, 1, 8, 56, 8)
    assert _heads(qkv[:, 0], "q") == (2, 7, 8, 280, 8)
    assert _heads(qkv[0].transpose(0, 1), "q") == (7, 5, 8, 8, 56)
    assert _heads(torch.empty(0, 7, 8), "q") == (0, 7, 8, 56, 8)
    for bad in (qkv[:, :4, 2:4], qkv[..., ::2], torch.empty(7, 8)):
        with pytest.raises(ValueError):
            _heads(bad, "q")


def test_second_derivatives_raise(monkeypatch):
    torch = pytest.importorskip("torch")
    from newton_schulz_momentum_gb300 import layers, token_ops
    plain = dict(
        qk_norm_rotary=lambda q, k, pos, qg, kg, **o: (q * qg, k * kg),
        qk_norm_rotary_grad=lambda dq, dk, q, k, pos, qg, kg, **o: (dq * qg, dk * kg, (dq * q).sum((0, 1)), (dk * k).sum((0, 1))),
        attention=lambda q, k, v, offsets, causal, scale: (q * v, q.sum((1, 2))),
        attention_grad=lambda do, q, k, v, out, lse, offsets, causal, scale: (do * v, torch.zeros_like(k), do * q),
        token_stats=lambda x, a, top, t: token_ops.TokenStats(x[:, 0] * 2, x[:, 1] * 3, x[:, :top] + 0, x[:, :top].long(), x + 0),
        token_stats_grad=lambda x, a, norm, h, g, ge, t: torch.stack([
            g * 2 if g is not None else x[:, 0] * 0, ge * 3 if ge is not None else x[:, 0] * 0], 1))
    for name, fn in plain.items():
        monkeypatch.setattr(token_ops, name, fn)
    q, k = torch.rand(3, 2, 8, requires_grad=True), torch.rand(3, 2, 8, requires_grad=True)
    x, ids = torch.rand(3, 2, requires_grad=True), torch.zeros(3, dtype=torch.int64)
    rotary_ = layers.QKNormRotary(8, device="cpu")
    outs = [(rotary_(q, k, ids)[0], q), (rotary_(q, k, ids)[1], rotary_.k_weight), (layers.Attention()(q, k, k), q),
            (layers.TokenStats(top=1)(x, ids).logp, x), (layers.TokenStats()(x).entropy, x)]
    for out, by in outs:
        total = (out.double() ** 3).sum()
        (want,) = torch.autograd.grad(total, by, retain_graph=True)
        (got,) = torch.autograd.grad(total, by, create_graph=True)
        assert torch.equal(want, got.detach()) and got.abs().sum() > 0
        with pytest.raises(RuntimeError, match="once_differentiable"):
            got.pow(2).sum().backward()
    got = layers.TokenStats(top=2)(x, ids)
    assert not got.top_logp.requires_grad and not got.norm.requires_grad and got.top_ids.dtype == torch.int64
