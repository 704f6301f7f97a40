"""CPU checks of the token operators' host side: what needs no GPU to be seen."""

import contextlib
import os
import re
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ENTRIES = ("dmuon_embedding", "dmuon_embedding_grad", "dmuon_add_rmsnorm", "dmuon_add_rmsnorm_grad", "dmuon_policy_loss",
           "dmuon_token_logprobs")


def entry_body(name):
    with open(os.path.join(ROOT, "newton_schulz_momentum_gb300", "csrc", "api.cu")) as f:
        src = f.read()
    found = re.search(r"^int %s\([^{]*\{\n(.*?)^\}" % name, src, re.S | re.M)
    assert found, name
    return found.group(1)


@pytest.mark.parametrize("name", ENTRIES)
def test_entries_let_no_exception_out(name):
    """A host allocation that fails (the list of timed launches, of workspace blocks) becomes a status: an exception that
    leaves a C function ends the process."""
    body = entry_body(name).strip()
    assert body.startswith("try {") and "catch (const std::exception" in body


class Stub:
    """What the wrappers ask of a tensor, on a device that need not exist."""

    def __init__(self, *shape, dtype=None, device=0):
        import torch
        self.shape, self.dtype, self.index = torch.Size(shape), dtype or torch.float32, device
        self.device, self.is_cuda = (f"cuda:{device}", True) if device >= 0 else ("cpu", False)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """The entry points' calls, as (name, device that was current, stream), with device 0 current at first."""
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

    monkeypatch.setattr(token_ops, "lib", lambda: types.SimpleNamespace(**{n: entry(n) for n in ENTRIES}))
    if hasattr(token_ops, "_current_device"):
        monkeypatch.setattr(token_ops, "_current_device", lambda: current[0])
    monkeypatch.setattr(token_ops, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch, "empty", lambda *shape, dtype=None, device=None: Stub(
        *(shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape), dtype=dtype,
        device=int(device.split(":")[1])))
    return made


def all_calls(at, odd=None):
    """One call of each function with every tensor on device `at`, but for argument `odd` of (function, argument)."""
    import torch
    from newton_schulz_momentum_gb300 import token_ops as ops
    i64, n, d = torch.int64, 4, 8
    kinds = {
        "embedding": dict(table=(9, d), ids=(n, i64), out=(n, d)),
        "embedding_grad": dict(grad_out=(n, d), ids=(n, i64), grad=(9, d)),
        "add_rmsnorm": dict(x=(n, d), residual=(n, d), gain=(d,), y=(n, d), h=(n, d)),
        "add_rmsnorm_fp8": dict(x=(n, d), residual=(n, d), gain=(d,), h=(n, d)),
        "add_rmsnorm_grad": dict(dy=(n, d), h=(n, d), gain=(d,), dh=(n, d), dx=(n, d), dgain=(d,)),
        "policy_loss": dict(logits=(n, d), targets=(n, i64), old_logp=(n,), advantages=(n,), weights=(n,), ref_logp=(n,),
                            dlogits=(n, d)),
        "token_logprobs": dict(logits=(n, d), targets=(n, i64)),
    }
    for name, shapes in kinds.items():
        if odd is not None and odd[0] != name:
            continue
        args = {}
        for arg, shape in shapes.items():
            dtype = shape[-1] if isinstance(shape[-1], torch.dtype) else torch.float32
            sizes = [v for v in shape if isinstance(v, int)]
            args[arg] = Stub(*sizes, dtype=dtype, device=odd[2] if odd is not None and odd[1] == arg else at)
        if name == "embedding_grad":
            args["rows"] = 9
        yield name, args, lambda fn=getattr(ops, name), a=args: fn(**a)


def test_calls_run_on_their_tensors_device(calls):
    """The library launches on the current device: the tensors' device is made current around the call."""
    for at in (0, 1):
        for name, _, call in all_calls(at):
            del calls[:]
            call()
            assert [c[1:] for c in calls] == [(at, 100 + at)], name


def test_tensors_of_two_devices_are_refused(calls):
    """Every tensor argument of every function is looked at; a refused call reaches no entry point."""
    seen = 0
    for name, args, _ in list(all_calls(1)):
        for arg in [a for a in args if isinstance(args[a], Stub)]:
            for where, word in ((0, "cuda"), (-1, "CUDA")):
                ((_, _, call),) = all_calls(1, odd=(name, arg, where))
                with pytest.raises(ValueError, match=word):
                    call()
                assert not calls
                seen += 1
    assert seen == 2 * 30


@pytest.fixture
def plain_kernels(monkeypatch):
    """The functions behind the modules, in torch on the CPU."""
    torch = pytest.importorskip("torch")
    from newton_schulz_momentum_gb300 import token_ops

    def norm(x, residual, gain, eps):
        h = x if residual is None else x + residual
        return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * gain, h

    def norm_grad(dy, h, gain, dh, eps):
        rho = torch.rsqrt((h * h).mean(-1, keepdim=True) + eps)
        d = dy * gain
        dx = rho * d - h * rho ** 3 * (d * h).mean(-1, keepdim=True) + (0 if dh is None else dh)
        return dx, (dy * h * rho).sum(0)

    def loss(logits, targets, old, adv, weights, ref, dlogits=None, **options):
        p = torch.softmax(logits, 1)
        return (p[:, 0] * weights).sum(), p[:, 0], None if dlogits is False else p * weights[:, None]

    def grad(dy, ids, rows, scale, pad):
        return torch.zeros(rows, dy.shape[-1]).index_add(0, ids, dy * scale)

    for name, fn in (("embedding", lambda table, ids, scale, dtype: (scale * table[ids]).to(dtype)),
                     ("embedding_grad", grad), ("add_rmsnorm", norm), ("add_rmsnorm_grad", norm_grad),
                     ("policy_loss", loss)):
        monkeypatch.setattr(token_ops, name, fn)
    return torch


def test_second_derivatives_raise(plain_kernels):
    """The backward passes are not differentiable themselves: a gradient penalty gets an error, not a gradient without
    its terms. First derivatives are as before, with create_graph too."""
    torch = plain_kernels
    from newton_schulz_momentum_gb300 import layers
    torch.manual_seed(0)
    n, d = 5, 8
    ids = torch.tensor([0, 2, 2, 1, 0])
    embed, norm = layers.Embedding(3, d, scale=2.0, device="cpu"), layers.AddRMSNorm(d, device="cpu")
    x = torch.randn(n, d, requires_grad=True)
    v = torch.rand(n) + 0.5
    for out, by in ((embed(ids), embed.weight), (norm(x)[0], x), (norm(x, x.detach())[0], norm.weight),
                    (layers.PolicyLoss()(x, ids, v, v, v)[0], x)):
        total = (out.double() ** 3).sum()
        (want,) = torch.autograd.grad(total, by, retain_graph=True)
        (got,) = torch.autograd.grad(total, by, create_graph=True)
        assert torch.equal(want, got.detach())
        with pytest.raises(RuntimeError, match="once_differentiable"):
            got.pow(2).sum().backward()


def test_embedding_from_pretrained(plain_kernels):
    """torch.nn.Embedding's constructor from a table, with this module's own options."""
    torch = plain_kernels
    from newton_schulz_momentum_gb300 import layers
    table = torch.arange(12.0).view(4, 3)
    embed = layers.Embedding.from_pretrained(table, padding_idx=-1, scale=3.0, dtype=torch.bfloat16)
    assert embed.weight.data_ptr() == table.data_ptr() and not embed.weight.requires_grad and embed.padding_idx == 3
    assert torch.equal(embed(torch.tensor([2, 0])), (3.0 * table[[2, 0]]).bfloat16())
    embed = layers.Embedding.from_pretrained(table, freeze=False)
    assert embed.weight.requires_grad and embed.padding_idx is None and embed(torch.tensor([1])).dtype == torch.float32
    assert (embed.num_embeddings, embed.embedding_dim) == (4, 3)
    with pytest.raises(ValueError, match="2-D"):
        layers.Embedding.from_pretrained(table[0])
    with pytest.raises(ValueError, match="float32"):
        layers.Embedding.from_pretrained(table.bfloat16())


A, B, C = 0x10000, 0x20000, 0x30000  # 16-byte aligned addresses, never read


@pytest.mark.parametrize("entry,args,word", [
    # logits, dtype, ld, n, vocab, targets, id_bytes, old, ref, adv, weights, lo, hi, kl, temp, loss, logp, dlogits, ldd
    ("dmuon_policy_loss", (A, 1, 16, 4, 16, B, 8, C, C, C, C, 0.2, 0.2, 0.1, 1.0, C, B, A, 24), "logits"),
    # x, ldx, residual, ldr, dtype, gain, n, dim, eps, h, ldh, y, y_dtype, ldy, scales, group
    ("dmuon_add_rmsnorm", (A, 8, B, 8, 1, None, 4, 8, 1e-6, A, 9, C, 1, 8, None, 0), "h is written over x"),
    ("dmuon_add_rmsnorm", (A, 8, B, 8, 1, None, 4, 8, 1e-6, B, 16, C, 1, 8, None, 0), "h is written over residual"),
    ("dmuon_add_rmsnorm", (A, 8, B, 8, 1, None, 4, 8, 1e-6, None, 0, A, 1, 9, None, 0), "y is written over x"),
    ("dmuon_add_rmsnorm", (A, 8, B, 16, 1, None, 4, 8, 1e-6, None, 0, B, 1, 8, None, 0), "y is written over residual"),
    ("dmuon_add_rmsnorm", (A, 8, B, 8, 1, None, 1, 8, 1e-6, None, 0, A, 2, 8, C, 0), "another type"),
    # dy, lddy, h, ldh, dh, lddh, dtype, gain, n, dim, eps, dx, lddx, dgain, accumulate
    ("dmuon_add_rmsnorm_grad", (A, 8, B, 8, C, 8, 0, None, 4, 8, 1e-6, A, 12, None, 0), "dx is written over dy"),
    ("dmuon_add_rmsnorm_grad", (A, 8, B, 8, C, 8, 0, None, 4, 8, 1e-6, C, 12, None, 0), "dx is written over dh")])
def test_rows_in_place_with_another_stride_are_refused(entry, args, word):
    """Rows of the output would fall on input rows that are still to be read."""
    import newton_schulz_momentum_gb300 as dm
    from newton_schulz_momentum_gb300 import build
    build.build()
    rc = getattr(dm.lib(), entry)(*args, None)
    message = dm.lib().dmuon_last_error().decode()
    assert rc == dm.ERR_INVALID_ARG and word in message, (rc, message)


def test_rows_of_one_element_have_no_stride_within():
    """A column of a matrix: whatever lies between the elements of a row that has one does not matter."""
    torch = pytest.importorskip("torch")
    from newton_schulz_momentum_gb300.token_ops import _layout
    column = torch.empty(6, 9)[:, ::4][:, 1:2]
    assert column.stride() == (9, 4) and _layout(column, "x") == (6, 1, 9)
    assert _layout(torch.empty(6, 9)[:, :4], "x") == (6, 4, 9) and _layout(torch.empty(2, 3, 5), "x") == (6, 5, 5)
    assert _layout(torch.empty(0, 5), "x") == (0, 5, 5) and _layout(torch.empty(1, 9)[:, :4], "x") == (1, 4, 4)
    for bad in (torch.empty(6, 9)[:, ::4], torch.empty(1, 9).expand(6, 9), torch.empty(4, 6, 9)[:, :, :5], torch.empty(9, 6).T):
        with pytest.raises(ValueError, match="contiguous"):
            _layout(bad, "x")
