"""Operators for training a small recurrent student of a large teacher: what makes the
gradients that ``OneBitAdam`` and ``LocoAdam`` step with.

``gated_scan``         the student's sequence mixing: a gated linear recurrence over time
``gated_scan_step``    one token of it, for generation
``distill_loss``       the loss against a teacher's top logits, one value per row
``distill_loss_grad``  the same with the gradient by the logits, in one pass over them
``read_status``        whether a kernel's bounded wait has run out since it was last asked

Each is a call of the CUDA library (the contracts are in include/ob.h); ``gated_scan`` and
``distill_loss`` are differentiable by autograd. Work is enqueued on the current torch
stream of the tensors' device. A wrong shape raises ValueError, a wrong type TypeError,
before anything is enqueued; a refusal or failure of the library raises ``ob.ObError``.
"""
import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import ob

SCAN_CHUNK = 64
DISTILL_MAX_K = 1024


def _need(t, name, shape, dtype, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise TypeError("%s must be a %s tensor" % (name, str(dtype).replace("torch.", "")))
    if t.shape != shape:
        raise ValueError("%s must have the shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s is on %s, not %s" % (name, t.device, device))
    return t if t.is_contiguous() else t.contiguous()


def _need_data(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in ob.DTYPES:
        raise TypeError("%s must be a float32, float16 or bfloat16 tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s is on %s: the operators run on a CUDA device" % (name, t.device))


def _need_flags(t, name, shape, device):
    if isinstance(t, torch.Tensor) and t.dtype == torch.uint8:
        return _need(t, name, shape, torch.uint8, device)
    return _need(t, name, shape, torch.bool, device)


def _rows_apart(t):
    """The tensor itself where its last axis is adjacent, else a copy."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


@functools.lru_cache(maxsize=None)
def _function(name):
    return getattr(ob.load(), name)


def _call(device, name, *args):
    """Enqueue on the current stream of ``device``, whichever device is current."""
    index = device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        rc = _function(name)(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = _function(name)(*args, stream)
    if rc != ob.OB_OK:
        raise ob.ObError(name, rc)


def read_status(device=None):
    """Waits for the current stream of ``device`` (None: the current device), then reports and
    clears its status: 0 when all the operators' kernels there have finished normally, 1 when one
    has given up a wait (each is bounded, some seconds; what it wrote from there on is NaN)."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if device.index is None:
        device = torch.device(device.type, torch.cuda.current_device())
    status = ctypes.c_uint()
    _call(device, "ob_operators_read_status", ctypes.byref(status))
    return status.value


def _view(t):
    stride = t.stride()
    return ctypes.byref(ob.View(t.data_ptr(), stride[0], stride[1]))


# ---- gated scan ----------------------------------------------------------------------------------


def _scan_inputs(x, r, i, decay, reset, dims):
    _need_data(x, "x")
    shape, dtype, device = x.shape, x.dtype, x.device
    if len(shape) != dims:
        raise ValueError("x must be %s, not of shape %s" % ("[B, T, D]" if dims == 3 else "[B, D]", tuple(shape)))
    for t, name in ((r, "r"), (i, "i")):
        if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
            _need_data(t, name)
            raise TypeError("%s must have the type of x" % name)
        if t.shape != shape or t.device != device:
            raise ValueError("%s must have the shape and device of x" % name)
    if decay is None:
        raise TypeError("decay must be a float32 tensor")
    decay = _need(decay, "decay", shape[-1:], torch.float32, device)
    if reset is not None:
        reset = _need_flags(reset, "reset", shape[:-1], device)
    if x.stride(-1) != 1 or r.stride(-1) != 1 or i.stride(-1) != 1:
        x, r, i = _rows_apart(x), _rows_apart(r), _rows_apart(i)
    return x, r, i, decay, reset


def _differentiates(*tensors):
    if not torch.is_grad_enabled():
        return False
    for t in tensors:
        if t is not None and t.requires_grad:
            return True
    return False


@functools.lru_cache(maxsize=256)
def _scan_workspace_bytes(B, T, D, dtype, backward):
    return ob.load().ob_gated_scan_workspace_bytes(B, T, D, dtype, backward)


def _scan_workspace(x, backward):
    size = _scan_workspace_bytes(*x.shape, ob.DTYPES[x.dtype], backward)
    return torch.empty(size, dtype=torch.uint8, device=x.device)


def _scan_forward(x, r, i, decay, h0, reset, keep_states):
    B, T, D = x.shape
    y = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    h_last = torch.empty((B, D), dtype=torch.float32, device=x.device)
    states = None
    if keep_states:
        states = torch.empty((B, -(-T // SCAN_CHUNK), D), dtype=torch.float32, device=x.device)
    ws = _scan_workspace(x, 0)
    _call(x.device, "ob_gated_scan_fwd", B, T, D, ob.DTYPES[x.dtype], _view(x), _view(r), _view(i), decay.data_ptr(),
          ob._ptr(h0), ob._ptr(reset), y.data_ptr(), h_last.data_ptr(), ob._ptr(states), ws.data_ptr())
    return y, h_last, states


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, decay, h0, reset):
        ctx.set_materialize_grads(False)
        y, h_last, states = _scan_forward(x, r, i, decay, h0, reset, True)
        ctx.save_for_backward(x, r, i, decay, reset, states)
        ctx.has_h0 = h0 is not None
        return y, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        x, r, i, decay, reset, states = ctx.saved_tensors
        if dy is None and dh is None:
            return None, None, None, None, None, None
        B, T, D = x.shape
        dy = None if dy is None else _rows_apart(dy)
        dh = None if dh is None else dh.contiguous()
        grads = [torch.empty((B, T, D), dtype=x.dtype, device=x.device) for _ in range(3)]
        ddecay = torch.empty(D, dtype=torch.float32, device=x.device)
        dh0 = torch.empty((B, D), dtype=torch.float32, device=x.device) if ctx.has_h0 else None
        ws = _scan_workspace(x, 1)
        _call(x.device, "ob_gated_scan_bwd", B, T, D, ob.DTYPES[x.dtype], _view(x), _view(r), _view(i),
              decay.data_ptr(), ob._ptr(reset), states.data_ptr(), None if dy is None else _view(dy), ob._ptr(dh),
              *[g.data_ptr() for g in grads], ddecay.data_ptr(), ob._ptr(dh0), ws.data_ptr())
        return (*grads, ddecay, dh0, None)


def gated_scan(x, r, i, decay, h0=None, reset=None):
    """The gated scan over x, r, i [B, T, D] (one type, float32, float16 or bfloat16), s the
    logistic function::

        a_t = exp(-decay * s(r_t))
        h_t = a_t * h_{t-1} + sqrt(1 - a_t^2) * s(i_t) * x_t

    ``decay`` [D] float32, from 0 to 1e28 (not checked; a negative one gives NaN), is the rate
    at an open gate; ``h0`` [B, D] float32 the state before the first token (None: zero);
    ``reset`` [B, T] bool marks tokens that start a sequence, before which the state is
    dropped, whatever it is. Returns y [B, T, D] in the type of x and the last state [B, D]
    in float32. Differentiable by x, r, i, decay and h0; the state is float32 throughout, in
    the backward pass too. Batch and time strides are free (slices of a joint projection need
    no copy); channels that are not adjacent are copied first.
    """
    x, r, i, decay, reset = _scan_inputs(x, r, i, decay, reset, 3)
    h0 = _need(h0, "h0", (x.shape[0], x.shape[2]), torch.float32, x.device)
    if _differentiates(x, r, i, decay, h0):
        return _GatedScan.apply(x, r, i, decay, h0, reset)
    return _scan_forward(x, r, i, decay, h0, reset, False)[:2]


def gated_scan_step(x, r, i, decay, h, reset=None):
    """One token of the scan for B sequences: x, r, i [B, D]; ``h`` [B, D] float32 is updated
    in place; ``reset`` [B] bool marks sequences that begin. Returns y [B, D] in the type of
    x. It has no backward pass: call it under ``torch.no_grad()``."""
    x, r, i, decay, reset = _scan_inputs(x, r, i, decay, reset, 2)
    if h is None or (isinstance(h, torch.Tensor) and not h.is_contiguous()):
        raise ValueError("h must be a contiguous float32 tensor: it is updated in place")
    h = _need(h, "h", x.shape, torch.float32, x.device)
    if _differentiates(x, r, i, decay, h):
        raise ValueError("gated_scan_step has no backward pass: call it under torch.no_grad()")
    B, D = x.shape
    y = torch.empty((B, D), dtype=x.dtype, device=x.device)
    _call(x.device, "ob_gated_scan_step", B, D, ob.DTYPES[x.dtype], x.data_ptr(), x.stride(0), r.data_ptr(),
          r.stride(0), i.data_ptr(), i.stride(0), decay.data_ptr(), ob._ptr(reset), h.data_ptr(), y.data_ptr())
    increment_version(h)
    return y


# ---- distillation loss -----------------------------------------------------------------------------


def _distill_inputs(logits, index, top, top_lse, temperature, weight):
    _need_data(logits, "logits")
    _need_data(top, "top")
    if logits.dim() < 2 or logits.shape[-1] < 1:
        raise ValueError("logits must be [..., V] with V >= 1, not %s" % (tuple(logits.shape),))
    if not isinstance(index, torch.Tensor) or index.dtype not in (torch.int32, torch.int64):
        raise TypeError("index must be an int32 or int64 tensor")
    rows = logits.shape[:-1]
    if index.dim() != logits.dim() or index.shape[:-1] != rows or top.shape != index.shape:
        raise ValueError("index and top must be %s, not %s and %s"
                         % (tuple(rows) + ("K",), tuple(index.shape), tuple(top.shape)))
    if index.shape[-1] > DISTILL_MAX_K:
        raise ValueError("at most %d entries per row, not %d" % (DISTILL_MAX_K, index.shape[-1]))
    if index.device != logits.device or top.device != logits.device:
        raise ValueError("index and top must be on the device of logits")
    temperature = float(temperature)
    if not 0.0 < temperature < float("inf"):
        raise ValueError("temperature must be positive and finite")
    top_lse = _need(top_lse, "top_lse", rows, torch.float32, logits.device)
    weight = _need(weight, "weight", rows, torch.float32, logits.device)
    flat = _rows_apart(logits if logits.dim() == 2 else logits.flatten(0, -2))
    return flat, index.contiguous(), top.contiguous(), top_lse, temperature, weight


def _distill_args(flat, index, top, top_lse, temperature, weight):
    N, V = flat.shape
    return [N, V, index.shape[-1], ob.DTYPES[flat.dtype], flat.data_ptr(), flat.stride(0), index.data_ptr(),
            8 * index.element_size(), top.data_ptr(), ob.DTYPES[top.dtype], ob._ptr(top_lse), ob._ptr(weight),
            temperature]


@functools.lru_cache(maxsize=256)
def _distill_workspace_bytes(N, V, dtype):
    return ob.load().ob_distill_workspace_bytes(N, V, dtype)


def _distill_forward(args, flat, dlogits, stats):
    N, V = flat.shape
    loss = torch.empty(N, dtype=torch.float32, device=flat.device)
    ws = None
    if dlogits is not None:
        size = _distill_workspace_bytes(N, V, ob.DTYPES[flat.dtype])
        ws = torch.empty(size, dtype=torch.uint8, device=flat.device) if size else None
    _call(flat.device, "ob_distill", *args, loss.data_ptr(), ob._ptr(dlogits),
          V if dlogits is None else dlogits.stride(0), ob._ptr(stats), ob._ptr(ws))
    return loss


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, flat, index, top, top_lse, temperature, weight):
        stats = torch.empty((flat.shape[0], 4), dtype=torch.float32, device=flat.device)
        loss = _distill_forward(_distill_args(flat, index, top, top_lse, temperature, weight), flat, None, stats)
        ctx.save_for_backward(flat, index, top, top_lse, weight, stats)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        flat, index, top, top_lse, weight, stats = ctx.saved_tensors
        dloss = dloss.contiguous()
        d = torch.empty(flat.shape, dtype=flat.dtype, device=flat.device)
        _call(flat.device, "ob_distill_bwd", *_distill_args(flat, index, top, top_lse, ctx.temperature, weight),
              stats.data_ptr(), dloss.data_ptr(), d.data_ptr(), flat.shape[1])
        return d, None, None, None, None, None


def distill_loss(logits, index, top, top_lse=None, temperature=1.0, weight=None):
    """Distillation loss of logits [..., V] against a teacher's top logits, one float32 value
    per row: weight * KL(teacher || student), q = softmax(logits / temperature).

    ``index`` [..., K] int32 or int64 and ``top`` [..., K] are the tokens and values the
    teacher sent; entries with an index outside [0, V) are padding. Without ``top_lse`` the
    teacher is the softmax of those values / temperature. With it ([...] float32, the
    log-sum-exp of all the teacher's logits / temperature) the tokens outside the list are
    one more entry, with the mass that both sides have left there (a student without any has an
    infinite loss, unless the teacher's is within rounding of 0). ``weight`` [...] float32
    multiplies the loss; rows of weight 0 (padding) and, without ``top_lse``, rows without an
    entry give 0. Differentiable by logits alone: the others must not require a gradient.
    Reduce it as the training loop wants; where the gradient's row factors are known
    beforehand, ``distill_loss_grad`` reads the logits once instead of twice.
    """
    flat, index, top, top_lse, temperature, weight = _distill_inputs(logits, index, top, top_lse, temperature, weight)
    if _differentiates(top, top_lse, weight):
        raise ValueError("distill_loss is differentiable by logits alone: detach top, top_lse and weight")
    if torch.is_grad_enabled() and flat.requires_grad:
        loss = _Distill.apply(flat, index, top, top_lse, temperature, weight)
    else:
        loss = _distill_forward(_distill_args(flat, index, top, top_lse, temperature, weight), flat, None, None)
    return loss if logits.dim() == 2 else loss.view(logits.shape[:-1])


def distill_loss_grad(logits, index, top, top_lse=None, temperature=1.0, weight=None, out=None):
    """The loss of ``distill_loss`` and the gradient of its sum by the logits, in one pass:
    put what the loss is scaled by (1 / tokens, a loss scale, 0 for padding) into ``weight``
    and call ``logits.backward(dlogits)``. Returns (loss [...], dlogits [..., V] in the type
    of logits). ``out`` receives dlogits; it may be ``logits`` itself where nothing reads
    those again (autograd raises where an operation has saved them for its backward pass), and
    must not overlap them otherwise."""
    _need_data(logits, "logits")
    flat, index, top, top_lse, temperature, weight = _distill_inputs(logits.detach(), index, top, top_lse, temperature,
                                                                     weight)
    given = out
    if given is None:
        d = torch.empty(flat.shape, dtype=flat.dtype, device=flat.device)
        out = d if logits.dim() == 2 else d.view(logits.shape)
    else:
        if not isinstance(out, torch.Tensor) or out.dtype != logits.dtype:
            raise TypeError("out must have the type of logits")
        if out.shape != logits.shape or out.device != logits.device:
            raise ValueError("out must have the shape and device of logits")
        if out.stride(-1) != 1 and out.shape[-1] > 1:
            raise ValueError("out must have adjacent tokens")
        try:
            d = out.detach().view(flat.shape)
        except RuntimeError:
            raise ValueError("out must have rows at one stride") from None
    loss = _distill_forward(_distill_args(flat, index, top, top_lse, temperature, weight), flat, d, None)
    if given is not None:
        increment_version(given)
    return loss if logits.dim() == 2 else loss.view(logits.shape[:-1]), out
