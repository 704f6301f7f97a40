"""The token operators of libdmuon: what a language model's training step runs beside its matrix products, on
the parameters that AdamW updates, and between them. Argument marshalling only: each function is one C call, enqueued
on the current CUDA stream of its tensors' device, which is the same for all of them; all are reachable as attributes of
the package.

    y = dm.embedding(table, ids, scale=64.0)                       # lookup
    grad = dm.embedding_grad(dy, ids, rows=table.shape[0])         # its dense fp32 gradient
    y, h = dm.add_rmsnorm(x, residual, gain)                       # h = x + residual, y = rms norm of h
    q, scales, h = dm.add_rmsnorm_fp8(x, residual, gain)           # the same with e4m3 outputs
    dx, dgain = dm.add_rmsnorm_grad(dy, h, gain, dh=dh)
    loss, logp, dlogits = dm.policy_loss(logits, targets, old_logp, advantages, weights)
    logp = dm.token_logprobs(logits, targets)
    q, k = dm.qk_norm_rotary(q, k, positions, q_gain, k_gain)      # norm of each head, and the position rotation
    out, lse = dm.attention(q, k, v, offsets)                      # causal, over packed sequences
    dq, dk, dv = dm.attention_grad(dout, q, k, v, out, lse, offsets)
    dq, dk, dq_gain, dk_gain = dm.qk_norm_rotary_grad(dq, dk, q0, k0, positions, q_gain, k_gain)
    stats = dm.token_stats(logits, targets, top=5)                 # logp, entropy, top_logp, top_ids, norm
    dlogits = dm.token_stats_grad(logits, targets, stats.norm, stats.entropy, dlogp, dentropy)

Activations are fp32 or bf16 CUDA tensors whose last dimension is the row; a 2-D tensor may have any row
stride, others must be contiguous. Heads are (..., heads, dim) with any stride from head to head and from token to
token. Ids and positions are int32 or int64. layers.py holds the autograd forms.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import BF16, E4M3, F32, _check, lib

_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
# The current stream's address without a Stream object around it (a third of a small call's time), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream, dev):
    """Address of `stream`, by default the current one of device `dev`."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _elsewhere(call, dev, *args):
    """call(*args) with device `dev` current: the library works on the current one."""
    with torch.cuda.device(dev):
        return call(*args)


def _device(t, name):
    """Index of a CUDA tensor's device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _same_device(t, name, dev):
    at = _device(t, name)
    if at != dev:
        raise ValueError(f"{name} is on cuda:{at}, but the call's other tensors are on cuda:{dev}")


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return code


def _layout(t, name):
    """(rows, row length, row stride) of a tensor."""
    size = t.shape
    if not size:
        raise ValueError(f"{name} must have at least one dimension")
    dim = size[-1]
    if t.is_contiguous():
        return (size[0] if len(size) == 2 else t.numel() // dim if dim else 0), dim, dim
    if len(size) != 2 or (dim > 1 and t.stride(1) != 1) or t.stride(0) < dim:
        raise ValueError(f"{name} must be contiguous, or 2-D with contiguous rows that do not overlap")
    return size[0], dim, t.stride(0)


def _rows(t, name, dev, shape, dtype):
    """Row stride of a tensor of the given shape and dtype (None: any) on device `dev`."""
    if t.get_device() != dev:
        _same_device(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    return t.shape[-1] if t.is_contiguous() else _layout(t, name)[2]


def _vector(t, name, dev, n, dtype=torch.float32):
    """Device address of a contiguous tensor of n elements on device `dev` (None stays None)."""
    if t is None:
        return None
    if t.get_device() != dev:
        _same_device(t, name, dev)
    if t.numel() != n or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _ids(t, name, dev, n=None):
    """(address, bytes per id) of a list of token ids on device `dev`."""
    size = _ID_BYTES.get(t.dtype)
    if t.get_device() != dev:
        _same_device(t, name, dev)
    if size is None or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 or int64 CUDA tensor")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, not {t.numel()}")
    return t.data_ptr(), size


def embedding(table, ids, scale=1.0, dtype=None, out=None, stream=None):
    """scale * table[ids], shaped ids.shape + (dim,), of `dtype` (the table's by default) or into `out`. An id outside
    the table gives zeros, and check_status() raises ERR_INDEX."""
    if table.dim() != 2:
        raise ValueError("table must be a 2-D tensor")
    dev = table.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(embedding, _device(table, "table"), table, ids, scale, dtype, out, stream)
    rows, dim, ld = _layout(table, "table")
    ptr, size = _ids(ids, "ids", dev)
    if out is None:
        out = torch.empty(ids.shape + (dim,), dtype=dtype or table.dtype, device=table.device)
        n, ldo = ids.numel(), dim
    else:
        n, ldo = ids.numel(), _rows(out, "out", dev, ids.shape + (dim,), dtype)
    status = lib().dmuon_embedding(table.data_ptr(), _code(table, "table"), rows, dim, ld, ptr, size, n, scale,
                                   out.data_ptr(), _code(out, "out"), ldo, _stream(stream, dev))
    if status:
        _check(status)
    return out


def embedding_grad(grad_out, ids, rows, scale=1.0, padding_idx=None, grad=None, accumulate=False, stream=None):
    """The dense fp32 gradient, rows x dim, of embedding()'s table: row v is scale times the sum of grad_out over the
    tokens of id v (none for padding_idx). Into `grad` where given: written over, or added to with accumulate."""
    dev = grad_out.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(embedding_grad, _device(grad_out, "grad_out"), grad_out, ids, rows, scale, padding_idx,
                          grad, accumulate, stream)
    n, dim, ld = _layout(grad_out, "grad_out")
    ptr, size = _ids(ids, "ids", dev, n)
    if grad is None:
        if accumulate:
            raise ValueError("accumulate needs a grad to add to")
        grad = torch.empty((rows, dim), dtype=torch.float32, device=grad_out.device)
        ldg = dim
    else:
        ldg = _rows(grad, "grad", dev, (rows, dim), torch.float32)
    status = lib().dmuon_embedding_grad(grad_out.data_ptr(), _code(grad_out, "grad_out"), ld, ptr, size, n, rows, dim,
                                        scale, -1 if padding_idx is None else padding_idx, grad.data_ptr(), ldg,
                                        1 if accumulate else 0, _stream(stream, dev))
    if status:
        _check(status)
    return grad


def _norm_args(dev, x, residual, gain, h):
    n, dim, ldx = _layout(x, "x")
    ldr, ldh, hp = 0, 0, None
    if residual is not None:
        ldr = _rows(residual, "residual", dev, x.shape, x.dtype)
        if h is None:
            h, ldh = torch.empty(x.shape, dtype=x.dtype, device=x.device), dim
            hp = h.data_ptr()
    if hp is None and h is not None:
        ldh = _rows(h, "h", dev, x.shape, x.dtype)
        hp = h.data_ptr()
    return (dim, h, (x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, _code(x, "x"),
                     _vector(gain, "gain", dev, dim), n, dim), (hp, ldh))


def add_rmsnorm(x, residual=None, gain=None, eps=1e-6, y=None, h=None, stream=None):
    """(y, h) with h = x + residual and y = gain * h / sqrt(mean(h^2) + eps) over the last dimension, both of x's
    dtype. Without a residual h is x itself. `h` may be x or residual, to update the residual stream in place."""
    dev = x.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(add_rmsnorm, _device(x, "x"), x, residual, gain, eps, y, h, stream)
    dim, h, head, tail = _norm_args(dev, x, residual, gain, h)
    if y is None:
        y, ldy = torch.empty(x.shape, dtype=x.dtype, device=x.device), dim
    else:
        ldy = _rows(y, "y", dev, x.shape, x.dtype)
    status = lib().dmuon_add_rmsnorm(*head, eps, *tail, y.data_ptr(), head[4], ldy, None, 0, _stream(stream, dev))
    if status:
        _check(status)
    return y, (x if h is None else h)


def add_rmsnorm_fp8(x, residual=None, gain=None, eps=1e-6, group=128, h=None, stream=None):
    """(q, scales, h): add_rmsnorm with y in 8 bits. Each `group` of columns (32, 64, 128 or 256; 0 for the whole row) is
    held as q = float8_e4m3fn(y / scale) with scale = max |y| / 448, fp32, shaped x.shape[:-1] + (groups,)."""
    dev = x.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(add_rmsnorm_fp8, _device(x, "x"), x, residual, gain, eps, group, h, stream)
    dim, h, head, tail = _norm_args(dev, x, residual, gain, h)
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(x.shape[:-1] + (-(-dim // group) if group else 1,), dtype=torch.float32, device=x.device)
    status = lib().dmuon_add_rmsnorm(*head, eps, *tail, q.data_ptr(), E4M3, dim, scales.data_ptr(), group,
                                     _stream(stream, dev))
    if status:
        _check(status)
    return q, scales, (x if h is None else h)


def add_rmsnorm_grad(dy, h, gain=None, dh=None, eps=1e-6, dx=None, dgain=None, accumulate=False, stream=None):
    """(dx, dgain) of add_rmsnorm at its h: dx is the gradient of x and of residual alike, `dh` (the gradient that
    reaches h itself) included; dgain is fp32, or None without a gain. dx may be dy or dh. With accumulate the gain's
    gradient is added to `dgain`."""
    dev = dy.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(add_rmsnorm_grad, _device(dy, "dy"), dy, h, gain, dh, eps, dx, dgain, accumulate, stream)
    n, dim, ldy = _layout(dy, "dy")
    ldh = _rows(h, "h", dev, dy.shape, dy.dtype)
    lddh = 0 if dh is None else _rows(dh, "dh", dev, dy.shape, dy.dtype)
    if dx is None:
        dx, lddx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device), dim
    else:
        lddx = _rows(dx, "dx", dev, dy.shape, dy.dtype)
    if dgain is None and gain is not None:
        if accumulate:
            raise ValueError("accumulate needs a dgain to add to")
        dgain = torch.empty(dim, dtype=torch.float32, device=dy.device)
    status = lib().dmuon_add_rmsnorm_grad(dy.data_ptr(), ldy, h.data_ptr(), ldh, None if dh is None else dh.data_ptr(),
                                          lddh, _code(dy, "dy"), _vector(gain, "gain", dev, dim), n, dim, eps,
                                          dx.data_ptr(), lddx, _vector(dgain, "dgain", dev, dim),
                                          1 if accumulate else 0, _stream(stream, dev))
    if status:
        _check(status)
    return dx, dgain


def policy_loss(logits, targets, old_logp, advantages, weights, ref_logp=None, clip_low=0.2, clip_high=0.2,
                kl_coef=0.0, temperature=1.0, dlogits=None, stream=None):
    """(loss, logp, dlogits) of the clipped policy loss with a KL term (dmuon_policy_loss): loss is an fp32 scalar
    tensor, logp the targets' log-probabilities, dlogits the loss's gradient, of the logits' dtype.

    weights holds mask and mean (1 / number of tokens, and 0 for a prompt's or padding's); a row of weight 0 or with a
    negative target is not read. dlogits may be a tensor to write into (the logits themselves among them), or False
    for the loss alone."""
    dev = logits.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(policy_loss, _device(logits, "logits"), logits, targets, old_logp, advantages, weights,
                          ref_logp, clip_low, clip_high, kl_coef, temperature, dlogits, stream)
    n, vocab, ld = _layout(logits, "logits")
    ptr, size = _ids(targets, "targets", dev, n)
    ldd, dptr = 0, None
    if dlogits is None:
        dlogits, ldd = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device), vocab
        dptr = dlogits.data_ptr()
    elif dlogits is False:
        dlogits = None
    else:
        ldd = _rows(dlogits, "dlogits", dev, logits.shape, logits.dtype)
        dptr = dlogits.data_ptr()
    loss = torch.empty((), dtype=torch.float32, device=logits.device)
    logp = torch.empty(targets.shape, dtype=torch.float32, device=logits.device)
    status = lib().dmuon_policy_loss(logits.data_ptr(), _code(logits, "logits"), ld, n, vocab, ptr, size,
                                     _vector(old_logp, "old_logp", dev, n), _vector(ref_logp, "ref_logp", dev, n),
                                     _vector(advantages, "advantages", dev, n), _vector(weights, "weights", dev, n),
                                     clip_low, clip_high, kl_coef, temperature, loss.data_ptr(), logp.data_ptr(), dptr,
                                     ldd, _stream(stream, dev))
    if status:
        _check(status)
    return loss, logp, dlogits


def token_logprobs(logits, targets, temperature=1.0, stream=None):
    """log softmax(logits / temperature)[targets], fp32, shaped like targets; 0 where a target is negative."""
    dev = logits.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(token_logprobs, _device(logits, "logits"), logits, targets, temperature, stream)
    n, vocab, ld = _layout(logits, "logits")
    ptr, size = _ids(targets, "targets", dev, n)
    logp = torch.empty(targets.shape, dtype=torch.float32, device=logits.device)
    status = lib().dmuon_token_logprobs(logits.data_ptr(), _code(logits, "logits"), ld, n, vocab, ptr, size,
                                        temperature, logp.data_ptr(), _stream(stream, dev))
    if status:
        _check(status)
    return logp


def _heads(t, name):
    """(tokens, heads, head length, token stride, head stride) of a tensor (..., heads, dim)."""
    size = t.shape
    if len(size) < 3:
        raise ValueError(f"{name} must have the dimensions (..., heads, dim)")
    heads, dim = size[-2:]
    if t.is_contiguous():
        return (size[0] if len(size) == 3 else size[:-2].numel()), heads, dim, heads * dim, dim
    strides = t.stride()
    if dim > 1 and strides[-1] != 1:
        raise ValueError(f"{name} must have contiguous heads")
    token, n = heads * dim, 1
    for count, stride in zip(reversed(size[:-2]), reversed(strides[:-2])):
        if count != 1:
            if n == 1:
                token = stride
            elif stride != token * n:
                raise ValueError(f"{name} must have one stride from token to token")
            n *= count
    return n, heads, dim, token, strides[-2] if heads > 1 else dim


def _head_array(t, name, dev, shape, dtype):
    """(address, token stride, head stride) of heads of the given shape and dtype on device `dev`."""
    if t.get_device() != dev:
        _same_device(t, name, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.is_contiguous():
        dim = shape[-1]
        return t.data_ptr(), shape[-2] * dim, dim
    return (t.data_ptr(),) + _heads(t, name)[3:]


def _new(t):
    return torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _new_heads(t):
    """A new tensor like t, and its (address, token stride, head stride)."""
    new = _new(t)
    dim = t.shape[-1]
    return new, (new.data_ptr(), t.shape[-2] * dim, dim)


def _like_q(k, q):
    if k.dim() < 3 or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError("k must have q's tokens and head length")


def _rotary_args(dev, q, n, dim, positions, q_gain, k_gain, norm, rotary_dim, base, freqs, sections, interleaved, eps):
    """The C calls' arguments from dtype to sections."""
    rotary_dim = dim if rotary_dim is None else rotary_dim
    axes, axis_list = 1, None
    tokens = q.shape[:-2]
    if sections is not None:
        axes = len(sections)
        axis_list = (ctypes.c_int64 * axes)(*sections)
        tokens = (axes,) + tuple(tokens)
    pos, id_bytes = _ids(positions, "positions", dev)
    if positions.shape != tokens:
        raise ValueError(f"positions must have shape {tuple(tokens)}, not {tuple(positions.shape)}")
    if freqs is not None:
        freqs = [float(f) for f in freqs]
        if len(freqs) != rotary_dim // 2:
            raise ValueError(f"freqs must have rotary_dim / 2 = {rotary_dim // 2} elements, not {len(freqs)}")
        freqs = (ctypes.c_double * max(len(freqs), 1))(*freqs)
    return (_code(q, "q"), _vector(q_gain, "q_gain", dev, dim), _vector(k_gain, "k_gain", dev, dim), 1 if norm else 0, eps,
            n, dim, rotary_dim, 1 if interleaved else 0, base, freqs, pos, id_bytes, axes, n, axis_list)


_NO_HEADS = (None, 0, 0)


def qk_norm_rotary(q, k, positions, q_gain=None, k_gain=None, norm=True, rotary_dim=None, base=10000.0, freqs=None,
                   sections=None, interleaved=False, eps=1e-6, q_out=None, k_out=None, stream=None):
    """(q_out, k_out): the RMS norm of each head of q (..., heads, dim) and k (..., kv_heads, dim; or None) over its
    columns, times a gain that all heads share, and the position rotation of the first rotary_dim columns (all by
    default), in pairs (j, j + rotary_dim / 2) or, interleaved, (2j, 2j + 1). norm=False rotates alone.

    positions are integers, shaped like q without its last two dimensions; with sections = (s0, s1, ...), which add up to
    rotary_dim / 2, one more dimension in front: s0 frequencies follow positions[0], the next s1 positions[1], ... The
    angles per position are base^(-2j / rotary_dim), or `freqs` (rotary_dim / 2 numbers). q_out may be q, and k_out k."""
    dev = q.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(qk_norm_rotary, _device(q, "q"), q, k, positions, q_gain, k_gain, norm, rotary_dim, base, freqs,
                          sections, interleaved, eps, q_out, k_out, stream)
    n, heads, dim, token, head = _heads(q, "q")
    turns = _rotary_args(dev, q, n, dim, positions, q_gain, k_gain, norm, rotary_dim, base, freqs, sections, interleaved, eps)
    if q_out is None:
        q_out, q_out_at = _new_heads(q)
    else:
        q_out_at = _head_array(q_out, "q_out", dev, q.shape, q.dtype)
    kv_heads, k_at, k_out_at = 0, _NO_HEADS, _NO_HEADS
    if k is None:
        k_out = None
    else:
        _like_q(k, q)
        kv_heads, k_at = k.shape[-2], _head_array(k, "k", dev, k.shape, q.dtype)
        if k_out is None:
            k_out, k_out_at = _new_heads(k)
        else:
            k_out_at = _head_array(k_out, "k_out", dev, k.shape, q.dtype)
    status = lib().dmuon_qk_norm_rotary(q.data_ptr(), token, head, heads, *k_at, kv_heads, *turns, *q_out_at, *k_out_at,
                                        _stream(stream, dev))
    if status:
        _check(status)
    return q_out, k_out


def qk_norm_rotary_grad(dq_out, dk_out, q, k, positions, q_gain=None, k_gain=None, norm=True, rotary_dim=None,
                        base=10000.0, freqs=None, sections=None, interleaved=False, eps=1e-6, dq=None, dk=None,
                        stream=None):
    """(dq, dk, dq_gain, dk_gain) of qk_norm_rotary at its q and k: the gains' gradients are fp32, None without a gain. dq
    may be dq_out or q, and dk dk_out or k."""
    dev = q.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(qk_norm_rotary_grad, _device(q, "q"), dq_out, dk_out, q, k, positions, q_gain, k_gain, norm,
                          rotary_dim, base, freqs, sections, interleaved, eps, dq, dk, stream)
    n, heads, dim, token, head = _heads(q, "q")
    turns = _rotary_args(dev, q, n, dim, positions, q_gain, k_gain, norm, rotary_dim, base, freqs, sections, interleaved, eps)
    if dq is None:
        dq, dq_at = _new_heads(q)
    else:
        dq_at = _head_array(dq, "dq", dev, q.shape, q.dtype)
    kv_heads, k_at, dk_out_at, dk_at = 0, _NO_HEADS, _NO_HEADS, _NO_HEADS
    if k is None:
        dk = None
    else:
        _like_q(k, q)
        kv_heads, k_at = k.shape[-2], _head_array(k, "k", dev, k.shape, q.dtype)
        dk_out_at = _head_array(dk_out, "dk_out", dev, k.shape, q.dtype)
        if dk is None:
            dk, dk_at = _new_heads(k)
        else:
            dk_at = _head_array(dk, "dk", dev, k.shape, q.dtype)
    dq_gain = None if q_gain is None else torch.empty(dim, dtype=torch.float32, device=q.device)
    dk_gain = None if k_gain is None or k is None else torch.empty(dim, dtype=torch.float32, device=q.device)
    status = lib().dmuon_qk_norm_rotary_grad(
        *_head_array(dq_out, "dq_out", dev, q.shape, q.dtype), q.data_ptr(), token, head, heads, *dk_out_at, *k_at,
        kv_heads, *turns, *dq_at, *dk_at, None if dq_gain is None else dq_gain.data_ptr(),
        None if dk_gain is None else dk_gain.data_ptr(), _stream(stream, dev))
    if status:
        _check(status)
    return dq, dk, dq_gain, dk_gain


def _prompts(dev, q, k, offsets, causal, scale, zero_outside):
    """(number of tokens, heads, the C calls' q, their arguments from dtype to zero_outside) of an attention call."""
    n, heads, dim, token, head = _heads(q, "q")
    _like_q(k, q)
    if q.dtype is not torch.bfloat16:
        raise ValueError(f"q must be {torch.bfloat16}, not {q.dtype}")
    if offsets is None:
        at, id_bytes, sequences = None, 4, q.shape[:-3].numel() or 1
    else:
        at, id_bytes = _ids(offsets, "offsets", dev)
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be a list of one more elements than sequences")
        sequences = offsets.numel() - 1
    return n, heads, (q.data_ptr(), token, head), (
        BF16, n, heads, k.shape[-2], dim, at, id_bytes, sequences, 1 if causal else 0,
        dim ** -0.5 if scale is None else scale, 1 if zero_outside else 0)


def attention(q, k, v, offsets=None, causal=True, scale=None, out=None, lse=None, stream=None):
    """(out, lse): softmax attention over whole prompts. q (..., heads, dim), k and v (..., kv_heads, dim), bf16; query
    head h reads key head h // (heads // kv_heads). `scale` is dim^-1/2 by default. out is like q; lse, (heads, tokens)
    fp32, holds each row's log of the sum of exponentials, which attention_grad reads.

    Without `offsets` the dimension in front of the heads is a sequence: (tokens, heads, dim) is one, (batch, length,
    heads, dim) is a batch of them. `offsets`, sequences + 1 integers, packs sequences of different lengths (0 among
    them): sequence s is tokens offsets[s] to offsets[s + 1]. Tokens of no sequence get zeros, or, where `out` is
    given, stay as they were. dim is a multiple of 8, at most 128; addresses and strides are multiples of 16 bytes."""
    dev = q.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(attention, _device(q, "q"), q, k, v, offsets, causal, scale, out, lse, stream)
    n, heads, q_at, prompts = _prompts(dev, q, k, offsets, causal, scale, out is None and lse is None)
    given = out is not None
    if given:
        out_at = _head_array(out, "out", dev, q.shape, q.dtype)
    else:
        out, out_at = _new_heads(q)
        if lse is not None:
            out.zero_()
    if lse is None:
        lse = (torch.zeros if given else torch.empty)((heads, n), dtype=torch.float32, device=q.device)
    status = lib().dmuon_attention(*q_at, *_head_array(k, "k", dev, k.shape, q.dtype),
                                   *_head_array(v, "v", dev, k.shape, q.dtype), *prompts, *out_at,
                                   _vector(lse, "lse", dev, heads * n), _stream(stream, dev))
    if status:
        _check(status)
    return out, lse


def attention_grad(dout, q, k, v, out, lse, offsets=None, causal=True, scale=None, dq=None, dk=None, dv=None,
                   stream=None):
    """(dq, dk, dv) of attention at its out and lse, like q, k and v. Tokens of no sequence get zeros, or, where any of
    the three is given, stay as they were in it."""
    dev = q.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(attention_grad, _device(q, "q"), dout, q, k, v, out, lse, offsets, causal, scale, dq, dk, dv,
                          stream)
    all_new = dq is None and dk is None and dv is None
    n, heads, q_at, prompts = _prompts(dev, q, k, offsets, causal, scale, all_new)
    grads, places = [], []
    for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", k)):
        if t is None:
            t, at = _new_heads(like)
            if not all_new:
                t.zero_()
        else:
            at = _head_array(t, name, dev, like.shape, q.dtype)
        grads.append(t)
        places += at
    status = lib().dmuon_attention_grad(*_head_array(dout, "dout", dev, q.shape, q.dtype), *q_at,
                                        *_head_array(k, "k", dev, k.shape, q.dtype),
                                        *_head_array(v, "v", dev, k.shape, q.dtype),
                                        *_head_array(out, "out", dev, q.shape, q.dtype),
                                        _vector(lse, "lse", dev, heads * n), *prompts, *places, _stream(stream, dev))
    if status:
        _check(status)
    return tuple(grads)


class TokenStats(NamedTuple):
    """Of each row of logits: its target's log-probability (None without targets), the entropy of its distribution, the
    log-probabilities and ids of its most likely tokens, and (largest logit, sum of exp((x - largest) / temperature))."""
    logp: Optional[torch.Tensor]
    entropy: torch.Tensor
    top_logp: torch.Tensor
    top_ids: torch.Tensor
    norm: torch.Tensor


def token_stats(logits, targets=None, top=0, temperature=1.0, stream=None):
    """TokenStats(logp, entropy, top_logp, top_ids, norm) of softmax(logits / temperature), fp32 and, the ids, int64,
    in one pass over the logits. The first three are shaped like targets (logits without their last dimension), the
    next two with `top` (at most 32) alternatives behind, best first, the lower id among equals. A row whose target is
    negative is not read: zeros, and ids of -1."""
    dev = logits.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(token_stats, _device(logits, "logits"), logits, targets, top, temperature, stream)
    n, vocab, ld = _layout(logits, "logits")
    ptr, size = (None, 8) if targets is None else _ids(targets, "targets", dev, n)
    shape, at = logits.shape[:-1] if targets is None else targets.shape, logits.device
    logp = None if targets is None else torch.empty(shape, dtype=torch.float32, device=at)
    entropy = torch.empty(shape, dtype=torch.float32, device=at)
    top_logp = torch.empty(shape + (max(top, 0),), dtype=torch.float32, device=at)
    top_ids = torch.empty(shape + (max(top, 0),), dtype=torch.int64, device=at)
    norm = torch.empty(shape + (2,), dtype=torch.float32, device=at)
    status = lib().dmuon_token_stats(logits.data_ptr(), _code(logits, "logits"), ld, n, vocab, ptr, size, top, temperature,
                                     None if logp is None else logp.data_ptr(), entropy.data_ptr(), top_logp.data_ptr(),
                                     top_ids.data_ptr(), norm.data_ptr(), _stream(stream, dev))
    if status:
        _check(status)
    return TokenStats(logp, entropy, top_logp, top_ids, norm)


def token_stats_grad(logits, targets, norm, entropy, dlogp=None, dentropy=None, temperature=1.0, dlogits=None,
                     stream=None):
    """The gradient of token_stats' logp and entropy in the logits, of their dtype, at its norm and entropy. Without dlogp
    targets may be None; without dentropy entropy may be. dlogits may be a tensor to write into, the logits among them."""
    dev = logits.get_device()
    if dev < 0 or dev != _current_device():
        return _elsewhere(token_stats_grad, _device(logits, "logits"), logits, targets, norm, entropy, dlogp, dentropy,
                          temperature, dlogits, stream)
    n, vocab, ld = _layout(logits, "logits")
    ptr, size = (None, 8) if targets is None else _ids(targets, "targets", dev, n)
    if dlogits is None:
        dlogits, ldd = _new(logits), vocab
    else:
        ldd = _rows(dlogits, "dlogits", dev, logits.shape, logits.dtype)
    status = lib().dmuon_token_stats_grad(logits.data_ptr(), _code(logits, "logits"), ld, n, vocab, ptr, size,
                                          _vector(norm, "norm", dev, 2 * n), _vector(entropy, "entropy", dev, n),
                                          _vector(dlogp, "dlogp", dev, n), _vector(dentropy, "dentropy", dev, n),
                                          temperature, dlogits.data_ptr(), ldd, _stream(stream, dev))
    if status:
        _check(status)
    return dlogits
