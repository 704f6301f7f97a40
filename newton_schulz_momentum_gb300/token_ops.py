"""The token operators of libdmuon: what a language model's training step runs beside its matrix products, on
the parameters that AdamW updates. Argument marshalling only: each function is one C call, enqueued on the current
CUDA stream of its tensors' device, which is the same for all of them; all are reachable as attributes of the package.

    y = dm.embedding(table, ids, scale=64.0)                       # lookup
    grad = dm.embedding_grad(dy, ids, rows=table.shape[0])         # its dense fp32 gradient
    y, h = dm.add_rmsnorm(x, residual, gain)                       # h = x + residual, y = rms norm of h
    q, scales, h = dm.add_rmsnorm_fp8(x, residual, gain)           # the same with e4m3 outputs
    dx, dgain = dm.add_rmsnorm_grad(dy, h, gain, dh=dh)
    loss, logp, dlogits = dm.policy_loss(logits, targets, old_logp, advantages, weights)
    logp = dm.token_logprobs(logits, targets)

Activations are fp32 or bf16 CUDA tensors whose last dimension is the row; a 2-D tensor may have any row
stride, others must be contiguous. Ids are int32 or int64. layers.py holds the autograd forms.
"""

from __future__ import annotations

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
