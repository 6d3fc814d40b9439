"""The operators around the cross-entropy on [T, V] logits: top K, distillation from a teacher's
top K, and the processing of logits (``include/vce_logits.h``).

Argument checks and marshalling only, as in the package's other wrappers.  A tensor argument must
lie on the logits' device; outputs that the caller does not pass are allocated on the stream that
the call runs on (``stream``, default the device's current stream), which becomes their stream.
Shape, type and device errors raise ValueError or TypeError before anything is enqueued; the
library's own refusals raise VceError.

The calls may be captured into CUDA graphs.  Of the two autograd functions, forward and backward
are captured together, and no graph of the same leaves built outside the capture may still be alive
then (PyTorch ties a leaf's gradient to the stream that first used it).
"""
from __future__ import annotations

import torch

from . import _DT, IGNORE_INDEX, RED, ROW_STATS, VceError, _get

MAX_TOPK = 256

_F32, _I64, _I32 = torch.float32, torch.int64, torch.int32

# the current stream's handle on a device (2 us less a call than through a Stream object)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _matrix(t, name, dev=None, shape=None):
    """Dtype code, rows, columns and leading dimension of a 2-D tensor with unit column stride."""
    code = _DT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}; use float32 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    T, V = t.shape
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {[T, V]}")
    if V > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: expected unit column stride")
    d = t.device
    if d.type != "cuda" or (dev is not None and d != dev):
        raise ValueError(f"{name}: on {d}, expected {'a CUDA device' if dev is None else dev}")
    return code, T, V, (t.stride(0) if T > 1 else max(t.stride(0), V))


def _flat(t, name, dtype, shape, dev):
    """The address of a contiguous tensor of this dtype and shape (None: 0)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {list(shape)}, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    return t.data_ptr()


def _new(shape, dtype, dev, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _out(t, name, dtype, shape, dev, stream):
    """An output, the caller's or a new one, and its address."""
    if t is None:
        t = _new(shape, dtype, dev, stream)
        return t, t.data_ptr()
    return t, _flat(t, name, dtype, shape, dev)


def _matrix_out(t, name, T, V, dtype, dev, stream):
    """A [T, V] output, the caller's or a new one, its address, dtype code and leading dimension."""
    if t is None:
        t = _new((T, V), dtype, dev, stream)
    code, _, _, ld = _matrix(t, name, dev, (T, V))
    return t, t.data_ptr(), code, ld


def _run(fn, dev, stream, *args):
    """Calls the library on the tensors' device and stream."""
    if stream is None:
        handle = _raw_stream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"stream: on {stream.device}, expected {dev}")
    else:
        handle = stream.cuda_stream
    f = getattr(_get(), fn)
    if torch.cuda.current_device() == dev.index:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, handle)
    if rc:
        raise VceError(fn, rc)


def _entries(k):
    """A number of entries a row that the library's 32-bit argument holds (it refuses those above its limit)."""
    if k >= 2 ** 31:
        raise ValueError(f"{k} entries a row, expected 1 to {MAX_TOPK}")
    return k


def ce_topk(logits, k, temperature=1.0, *, values=None, ids=None, lse=None, tail_lse=None, stream=None):
    """The k largest logits of each row in order (ties to the lowest column), their columns, and the
    log-sum-exp of logits / temperature over the row and over the columns left out.

    Returns (values [T, k] float32, ids [T, k] int64, lse [T], tail_lse [T]); where a row has fewer
    than k logits above -inf, the entries behind them are (-inf, -1).  No gradient.
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    k = _entries(int(k))
    if k < 1:
        raise ValueError(f"k: {k}, expected at least 1")
    values, p_values = _out(values, "values", _F32, (T, k), dev, stream)
    ids, p_ids = _out(ids, "ids", _I64, (T, k), dev, stream)
    lse, p_lse = _out(lse, "lse", _F32, (T,), dev, stream)
    tail_lse, p_tail = _out(tail_lse, "tail_lse", _F32, (T,), dev, stream)
    _run("ce_topk", dev, stream, logits.data_ptr(), dt, T, V, ld, k, temperature, p_values, p_ids, p_lse, p_tail)
    return values, ids, lse, tail_lse


def _teacher(ids, values, tail, T, dev):
    if ids.dim() != 2:
        raise ValueError("teacher_ids: expected a [T, K] tensor")
    K = _entries(ids.shape[1])
    tdt = _DT.get(values.dtype)
    if tdt is None:
        raise TypeError(f"teacher_values: unsupported dtype {values.dtype}; use float32 or bfloat16")
    return (K, _flat(ids, "teacher_ids", _I64, (T, K), dev),
            _flat(values, "teacher_values", values.dtype, (T, K), dev), tdt,
            _flat(tail, "teacher_tail", _F32, (T,), dev))


def ce_distill_forward(logits, teacher_ids, teacher_values, teacher_tail=None, temperature=1.0, labels=None,
                       ignore_index=IGNORE_INDEX, reduction="mean", *, loss_rows=None, loss_out=None,
                       row_stats=None, top_grads=None, status=None, stream=None):
    """Distillation loss of the student's logits against a teacher's top K (``ce_topk``'s ids, values
    and tail_lse at the same temperature; teacher_tail None: the teacher renormalised over its K).

    Returns (loss_out, loss_rows, row_stats, top_grads, status), the middle two for
    ce_distill_backward.
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    K, p_ids, p_values, tdt, p_tail = _teacher(teacher_ids, teacher_values, teacher_tail, T, dev)
    red = RED[reduction]
    loss_rows, p_rows = _out(loss_rows, "loss_rows", _F32, (T,), dev, stream)
    row_stats, p_stats = _out(row_stats, "row_stats", _F32, (T, ROW_STATS), dev, stream)
    top_grads, p_tops = _out(top_grads, "top_grads", _F32, (T, K), dev, stream)
    status, p_status = _out(status, "status", _I32, (1,), dev, stream)
    p_loss = None
    if red or loss_out is not None:
        loss_out, p_loss = _out(loss_out, "loss_out", _F32, (1,), dev, stream)
    _run("ce_distill_forward", dev, stream, logits.data_ptr(), dt, T, V, ld, p_ids, p_values, tdt, p_tail, K,
         temperature, _flat(labels, "labels", _I64, (T,), dev), ignore_index, red, p_rows, p_loss, p_stats, p_tops,
         p_status)
    return loss_out, loss_rows, row_stats, top_grads, status


def ce_distill_backward(logits, teacher_ids, row_stats, top_grads, grad_output, temperature=1.0, reduction="mean", *,
                        grad_logits=None, grad_dtype=None, stream=None):
    """Gradient of the distillation loss w.r.t. the student's logits.  Returns grad_logits."""
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids: expected a [T, K] tensor")
    K = _entries(teacher_ids.shape[1])
    red = RED[reduction]
    grad_logits, p_grad, gdt, gld = _matrix_out(grad_logits, "grad_logits", T, V, grad_dtype or logits.dtype, dev, stream)
    _run("ce_distill_backward", dev, stream, logits.data_ptr(), dt, T, V, ld,
         _flat(teacher_ids, "teacher_ids", _I64, (T, K), dev), K, temperature, red,
         _flat(row_stats, "row_stats", _F32, (T, ROW_STATS), dev), _flat(top_grads, "top_grads", _F32, (T, K), dev),
         _flat(grad_output, "grad_output", _F32, (1,) if red else (T,), dev), p_grad, gdt, gld)
    return grad_logits


def ce_distill_forward_backward(logits, teacher_ids, teacher_values, teacher_tail=None, temperature=1.0, labels=None,
                                ignore_index=IGNORE_INDEX, reduction="mean", *, grad_output=None, grad_logits=None,
                                grad_dtype=None, loss_rows=None, loss_out=None, row_stats=None, status=None,
                                stream=None):
    """Distillation loss and gradient in one pass over the logits (grad_output known; None: ones).

    Returns (loss_out, loss_rows, grad_logits, status).
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    K, p_ids, p_values, tdt, p_tail = _teacher(teacher_ids, teacher_values, teacher_tail, T, dev)
    red = RED[reduction]
    if grad_output is None:
        grad_output = _new((1,) if red else (T,), _F32, dev, stream)
        with torch.cuda.stream(stream):   # None: the current stream
            grad_output.fill_(1.0)
    grad_logits, p_grad, gdt, gld = _matrix_out(grad_logits, "grad_logits", T, V, grad_dtype or logits.dtype, dev, stream)
    loss_rows, p_rows = _out(loss_rows, "loss_rows", _F32, (T,), dev, stream)
    row_stats, p_stats = _out(row_stats, "row_stats", _F32, (T, ROW_STATS), dev, stream)
    status, p_status = _out(status, "status", _I32, (1,), dev, stream)
    p_loss = None
    if red or loss_out is not None:
        loss_out, p_loss = _out(loss_out, "loss_out", _F32, (1,), dev, stream)
    _run("ce_distill_forward_backward", dev, stream, logits.data_ptr(), dt, T, V, ld, p_ids, p_values, tdt, p_tail, K,
         temperature, _flat(labels, "labels", _I64, (T,), dev), ignore_index, red,
         _flat(grad_output, "grad_output", _F32, (1,) if red else (T,), dev), p_rows, p_loss, p_stats, p_grad, gdt, gld,
         p_status)
    return loss_out, loss_rows, grad_logits, status


class _Distill(torch.autograd.Function):
    """ce_distill_forward and _backward.  What the backward needs lies in one float32 buffer: row_stats
    [T, 4], top_grads [T, K], loss_rows [T], the status word."""

    @staticmethod
    def forward(ctx, logits, ids, values, tail, temperature, labels, ignore_index, reduction):
        dt, T, V, ld = _matrix(logits, "logits")
        dev = logits.device
        K, p_ids, p_values, tdt, p_tail = _teacher(ids, values, tail, T, dev)
        red = RED[reduction]
        kept = torch.empty(T * (ROW_STATS + K + 1) + 1, dtype=_F32, device=dev)
        loss = torch.empty((), dtype=_F32, device=dev) if red else torch.empty(T, dtype=_F32, device=dev)
        stats, p_loss = kept.data_ptr(), loss.data_ptr()
        tops = stats + 4 * ROW_STATS * T
        rows = tops + 4 * K * T
        _run("ce_distill_forward", dev, None, logits.data_ptr(), dt, T, V, ld, p_ids, p_values, tdt, p_tail, K,
             temperature, _flat(labels, "labels", _I64, (T,), dev), ignore_index, red, rows if red else p_loss,
             p_loss if red else None, stats, tops, rows + 4 * T)
        ctx.save_for_backward(logits, ids, kept)
        ctx.temperature, ctx.red = temperature, red
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        logits, ids, kept = ctx.saved_tensors
        dt, T, V, ld = _matrix(logits, "logits")
        if grad.dtype is not _F32 or not grad.is_contiguous():
            grad = grad.to(_F32).contiguous()
        g = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
        K, stats = ids.shape[1], kept.data_ptr()
        _run("ce_distill_backward", logits.device, None, logits.data_ptr(), dt, T, V, ld, ids.data_ptr(), K,
             ctx.temperature, ctx.red, stats, stats + 4 * ROW_STATS * T, grad.data_ptr(), g.data_ptr(), dt, V)
        return g, None, None, None, None, None, None, None


def distill_cross_entropy(logits, teacher_ids, teacher_values, teacher_tail=None, temperature=1.0, labels=None,
                          ignore_index=IGNORE_INDEX, reduction="mean"):
    """The distillation loss of [T, V] student logits with autograd: temperature^2 KL(teacher || student)
    over the teacher's K columns and, with teacher_tail, the rest as one outcome.  Rows whose first
    teacher id is -1 or whose label is ignore_index are ignored.  Gradient w.r.t. the logits only."""
    return _Distill.apply(logits, teacher_ids, teacher_values, teacher_tail, float(temperature), labels, ignore_index,
                          reduction)


def _list(ids, offsets, name, T, dev):
    """Addresses and length of a row-offset list."""
    if ids is None:
        if offsets is not None:
            raise ValueError(f"{name}_offsets without {name}_ids")
        return None, 0, None
    if offsets is None:
        raise ValueError(f"{name}_ids without {name}_offsets")
    if ids.dim() != 1:
        raise ValueError(f"{name}_ids: expected a 1-D tensor")
    n = ids.shape[0]
    # an empty tensor has no address; the offsets' is never read through it
    return (_flat(ids, f"{name}_ids", _I64, (n,), dev) or offsets.data_ptr(), n,
            _flat(offsets, f"{name}_offsets", _I64, (T + 1,), dev))


def _mask(mask, T, V, dev):
    if mask is None:
        return None, 0
    if mask.dtype is not _I32:
        raise TypeError(f"mask: expected int32 words, got {mask.dtype}")
    if mask.dim() != 2 or mask.shape[0] != T or mask.shape[1] * 32 < V or (mask.shape[1] > 1 and mask.stride(1) != 1):
        raise ValueError(f"mask: expected [{T}, at least {(V + 31) // 32}] words with unit column stride")
    if mask.device != dev:
        raise ValueError(f"mask: on {mask.device}, expected {dev}")
    return mask.data_ptr(), mask.stride(0) if T > 1 else mask.shape[1]


def logits_process(logits, *, temperature=None, repetition_penalty=None, frequency_penalty=None, presence_penalty=None,
                   history_ids=None, history_offsets=None, prompt_lens=None, bias_ids=None, bias_values=None,
                   bias_offsets=None, mask=None, out=None, out_dtype=None, row_status=None, stream=None):
    """Penalties for the tokens of each row's history, biases, temperature and a mask on the logits.

    Per-row parameters are float32 [T]; the history (and the biases) int64 ids of all rows one after
    another with int64 offsets [T + 1]; prompt_lens int64 [T], how many of a row's first tokens are its
    prompt; mask int32 words, bit j % 32 of word j // 32 allowing column j.

    Returns (out, row_status), row_status int32 [T]: 0, or an error of the row, which is NaN then.
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    out, p_out, odt, old = _matrix_out(out, "out", T, V, out_dtype or logits.dtype, dev, stream)
    row_status, p_status = _out(row_status, "row_status", _I32, (T,), dev, stream)
    h, n_h, h_off = _list(history_ids, history_offsets, "history", T, dev)
    b, n_b, b_off = _list(bias_ids, bias_offsets, "bias", T, dev)
    if b is not None and bias_values is None:
        raise ValueError("bias_ids without bias_values")
    bv = (_flat(bias_values, "bias_values", _F32, (n_b,), dev) or b) if b is not None else None
    m, mld = _mask(mask, T, V, dev)
    _run("logits_process", dev, stream, logits.data_ptr(), dt, T, V, ld,
         _flat(temperature, "temperature", _F32, (T,), dev),
         _flat(repetition_penalty, "repetition_penalty", _F32, (T,), dev),
         _flat(frequency_penalty, "frequency_penalty", _F32, (T,), dev),
         _flat(presence_penalty, "presence_penalty", _F32, (T,), dev), h, n_h, h_off,
         _flat(prompt_lens, "prompt_lens", _I64, (T,), dev), b, bv, n_b, b_off, m, mld, p_out, odt, old,
         p_status)
    return out, row_status


def logits_process_backward(grad_out, logits=None, *, temperature=None, repetition_penalty=None, history_ids=None,
                            history_offsets=None, mask=None, grad_logits=None, grad_dtype=None, row_status=None,
                            stream=None):
    """The gradient through logits_process w.r.t. its logits (the unprocessed ones, needed with a
    history only).  Returns (grad_logits, row_status); a row with an error has no gradient (+0.0)."""
    gdt, T, V, gld = _matrix(grad_out, "grad_out")
    dev = grad_out.device
    zdt, zld, z = gdt, V, None
    if logits is not None:
        zdt, _, _, zld = _matrix(logits, "logits", dev, (T, V))
        z = logits.data_ptr()
    grad_logits, p_grad, odt, old = _matrix_out(grad_logits, "grad_logits", T, V,
                                           grad_dtype or (grad_out if logits is None else logits).dtype, dev, stream)
    row_status, p_status = _out(row_status, "row_status", _I32, (T,), dev, stream)
    h, n_h, h_off = _list(history_ids, history_offsets, "history", T, dev)
    m, mld = _mask(mask, T, V, dev)
    _run("logits_process_backward", dev, stream, grad_out.data_ptr(), gdt, T, V, gld, z, zdt, zld,
         _flat(temperature, "temperature", _F32, (T,), dev),
         _flat(repetition_penalty, "repetition_penalty", _F32, (T,), dev), h, n_h, h_off, m, mld,
         p_grad, odt, old, p_status)
    return grad_logits, row_status


class _Process(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, out_dtype, kw):
        out, _ = logits_process(logits, out_dtype=out_dtype, **kw)
        keep = [kw.get(n) for n in ("temperature", "repetition_penalty", "history_ids", "history_offsets", "mask")]
        ctx.save_for_backward(logits, *keep)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        logits, temperature, repetition, ids, offsets, mask = ctx.saved_tensors
        if grad.dim() == 2 and (grad.stride(1) != 1 or grad.stride(0) < grad.shape[1]):
            grad = grad.contiguous()
        if ids is None or repetition is None:   # without a repetition penalty the history does not enter
            repetition = ids = offsets = None
        g, _ = logits_process_backward(grad, logits, temperature=temperature, repetition_penalty=repetition,
                                       history_ids=ids, history_offsets=offsets, mask=mask)
        return g, None, None


def process_logits(logits, *, out_dtype=None, **parameters):
    """logits_process with autograd (its keyword arguments but out, row_status and stream): the gradient
    w.r.t. the logits, the parameters as constants.  Rows with an error are NaN, and have no gradient."""
    for name in ("out", "row_status", "stream"):
        if name in parameters:
            raise TypeError(f"process_logits takes no {name}")
    return _Process.apply(logits, out_dtype, parameters)


# ---- test hooks: waits that give up -------------------------------------------------------------


def vce_test_topk_stall(logits, k, wait_ns=50_000_000, *, stream=None):
    """ce_topk of contiguous bfloat16 logits whose slices' last stages are never copied; its outputs."""
    T, V = logits.shape
    dev = logits.device
    out = (torch.zeros(T, k, device=dev), torch.zeros(T, k, dtype=_I64, device=dev), torch.zeros(T, device=dev),
           torch.zeros(T, device=dev))
    _run("vce_test_topk_stall", dev, stream, logits.data_ptr(), T, V, k, *(t.data_ptr() for t in out), int(wait_ns))
    return out


def vce_test_distill_stall(logits, teacher_ids, teacher_values, wait_ns=50_000_000, *, stream=None):
    """The one pass on contiguous bfloat16 logits, the gradient of each cluster's last block waiting in
    vain.  Returns (loss_out, loss_rows, grad_logits, status)."""
    T, V = logits.shape
    dev = logits.device
    go, loss, rows = torch.ones(1, device=dev), torch.zeros(1, device=dev), torch.zeros(T, device=dev)
    stats, grad = torch.zeros(T, ROW_STATS, device=dev), torch.zeros_like(logits)
    status = torch.full((1,), 0x7FFF1234, dtype=_I32, device=dev)
    _run("vce_test_distill_stall", dev, stream, logits.data_ptr(), T, V, teacher_ids.data_ptr(),
         teacher_values.data_ptr(), teacher_ids.shape[1], go.data_ptr(), rows.data_ptr(), loss.data_ptr(),
         stats.data_ptr(), grad.data_ptr(), int(wait_ns), status.data_ptr())
    return loss, rows, grad, status


def vce_test_distill_bwd_stall(logits, teacher_ids, row_stats, top_grads, wait_ns=50_000_000, *, stream=None):
    """The backward on contiguous bfloat16 logits, each row's last block waiting for its last stage in
    vain.  Returns grad_logits."""
    T, V = logits.shape
    dev = logits.device
    go, grad = torch.ones(1, device=dev), torch.zeros_like(logits)
    _run("vce_test_distill_bwd_stall", dev, stream, logits.data_ptr(), T, V, teacher_ids.data_ptr(),
         teacher_ids.shape[1], row_stats.data_ptr(), top_grads.data_ptr(), go.data_ptr(), grad.data_ptr(),
         int(wait_ns))
    return grad
