"""The post-training losses on [T, V] logits: log-probabilities of chosen tokens with the rows' entropies,
the clipped policy loss, and the preference loss over pairs of packed sequences (``include/vce_policy.h``).

Argument checks and marshalling only, as in the package's other wrappers (``logits_ops``): a tensor
argument must lie on the logits' device; outputs that the caller does not pass are allocated on the
stream that the call runs on; shape, type and device errors raise ValueError or TypeError before
anything is enqueued, the library's own refusals VceError.

The calls may be captured into CUDA graphs.  Of the autograd functions, forward and backward are
captured together, and no graph of the same leaves built outside the capture may still be alive then
(PyTorch ties a leaf's gradient to the stream that first used it).
"""
from __future__ import annotations

import ctypes

import torch

from . import IGNORE_INDEX, RED, ROW_STATS
from .logits_ops import _F32, _I32, _I64, _flat, _matrix, _matrix_out, _new, _out, _run

PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}


class _PolicyParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_float) for n in ("clip_low", "clip_high", "dual_clip", "kl_coef", "entropy_coef")]


class _PreferenceParams(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("beta", ctypes.c_float), ("label_smoothing", ctypes.c_float),
                ("margin", ctypes.c_float), ("average", ctypes.c_int)]


def _given(t, name, dtype, shape, dev):
    """The address of an argument that has to be there."""
    if t is None:
        raise TypeError(f"{name}: expected a tensor")
    return _flat(t, name, dtype, shape, dev)


# ---- log-probabilities --------------------------------------------------------------------------


def ce_logprobs_forward(logits, ids, temperature=1.0, ignore_index=IGNORE_INDEX, *, want_entropy=True, logprobs=None,
                        entropy=None, row_stats=None, status=None, stream=None):
    """log softmax(logits / temperature) at each row's id, and the rows' entropies.

    Returns (logprobs [T], entropy [T] or None, row_stats, status), float32; rows whose id is
    ignore_index are 0 and not read.
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    p_ids = _given(ids, "ids", _I64, (T,), dev)
    logprobs, p_lp = _out(logprobs, "logprobs", _F32, (T,), dev, stream)
    p_ent = None
    if want_entropy:
        entropy, p_ent = _out(entropy, "entropy", _F32, (T,), dev, stream)
    elif entropy is not None:
        raise ValueError("entropy given, but want_entropy is False")
    row_stats, p_stats = _out(row_stats, "row_stats", _F32, (T, ROW_STATS), dev, stream)
    status, p_status = _out(status, "status", _I32, (1,), dev, stream)
    _run("ce_logprobs_forward", dev, stream, logits.data_ptr(), dt, T, V, ld, p_ids, ignore_index, temperature, p_lp,
         p_ent, p_stats, p_status)
    return logprobs, entropy, row_stats, status


def ce_logprobs_backward(logits, ids, row_stats, grad_logprobs=None, grad_entropy=None, temperature=1.0, *,
                         grad_logits=None, grad_dtype=None, stream=None):
    """Gradient w.r.t. the logits from those of ce_logprobs_forward's outputs (None: 0; an entropy's only if
    the forward worked it out).  Returns grad_logits."""
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    grad_logits, p_grad, gdt, gld = _matrix_out(grad_logits, "grad_logits", T, V, grad_dtype or logits.dtype, dev, stream)
    _run("ce_logprobs_backward", dev, stream, logits.data_ptr(), dt, T, V, ld, _given(ids, "ids", _I64, (T,), dev),
         temperature, _given(row_stats, "row_stats", _F32, (T, ROW_STATS), dev),
         _flat(grad_logprobs, "grad_logprobs", _F32, (T,), dev), _flat(grad_entropy, "grad_entropy", _F32, (T,), dev),
         p_grad, gdt, gld)
    return grad_logits


def _as_f32(grad):
    return grad if grad is None or (grad.dtype is _F32 and grad.is_contiguous()) else grad.to(_F32).contiguous()


class _LogProbs(torch.autograd.Function):
    """What the backward needs, and the status word, lie in one float32 buffer (of the functions below too: an
    allocation costs a call more than its marshalling)."""

    @staticmethod
    def forward(ctx, logits, ids, temperature, ignore_index, want_entropy):
        dt, T, V, ld = _matrix(logits, "logits")
        dev = logits.device
        p_ids = _given(ids, "ids", _I64, (T,), dev)
        lp = torch.empty(T, dtype=_F32, device=dev)
        ent = torch.empty(T, dtype=_F32, device=dev) if want_entropy else None
        kept = torch.empty(ROW_STATS * T + 1, dtype=_F32, device=dev)
        stats = kept.data_ptr()
        _run("ce_logprobs_forward", dev, None, logits.data_ptr(), dt, T, V, ld, p_ids, ignore_index, temperature,
             lp.data_ptr(), ent.data_ptr() if want_entropy else None, stats, stats + 4 * ROW_STATS * T)
        ctx.save_for_backward(logits, ids, kept)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        return (lp, ent) if want_entropy else lp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_lp, grad_ent=None):
        logits, ids, kept = ctx.saved_tensors
        dt, T, V, ld = _matrix(logits, "logits")
        grad_lp, grad_ent = _as_f32(grad_lp), _as_f32(grad_ent)
        g = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
        _run("ce_logprobs_backward", logits.device, None, logits.data_ptr(), dt, T, V, ld, ids.data_ptr(),
             ctx.temperature, kept.data_ptr(), None if grad_lp is None else grad_lp.data_ptr(),
             None if grad_ent is None else grad_ent.data_ptr(), g.data_ptr(), dt, V)
        return g, None, None, None, None


def token_logprobs(logits, ids, temperature=1.0, ignore_index=IGNORE_INDEX, want_entropy=True):
    """ce_logprobs_forward with autograd: (logprobs [T], entropy [T] or None), gradients w.r.t. the logits."""
    out = _LogProbs.apply(logits, ids, float(temperature), ignore_index, bool(want_entropy))
    return out if want_entropy else (out, None)


# ---- policy loss --------------------------------------------------------------------------------


def _policy_args(actions, advantages, old_logprobs, ref_logprobs, weights, T, dev):
    return (_given(actions, "actions", _I64, (T,), dev), _flat(old_logprobs, "old_logprobs", _F32, (T,), dev),
            _given(advantages, "advantages", _F32, (T,), dev), _flat(ref_logprobs, "ref_logprobs", _F32, (T,), dev),
            _flat(weights, "weights", _F32, (T,), dev))


def policy_loss_forward(logits, actions, advantages, old_logprobs=None, ref_logprobs=None, weights=None, *,
                        clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0, temperature=1.0,
                        ignore_index=IGNORE_INDEX, reduction="mean", want_entropy=False, loss_rows=None, loss_out=None,
                        logprobs=None, entropy=None, row_stats=None, status=None, stream=None):
    """Clipped policy loss of [T, V] logits: per row, with the ratio r of the action's probability to its old
    one (old_logprobs None: the same), weights * (-min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
    + kl_coef (exp(d) - d - 1) - entropy_coef H), d = ref_logprobs - logprobs; dual_clip >= 1 bounds the
    first term by dual_clip A where A < 0.

    Returns (loss_out, loss_rows, logprobs, entropy or None, row_stats, status), row_stats for
    policy_loss_backward.
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    p_act, p_old, p_adv, p_ref, p_w = _policy_args(actions, advantages, old_logprobs, ref_logprobs, weights, T, dev)
    params = _PolicyParams(clip_low, clip_high, dual_clip, kl_coef, entropy_coef)
    red = RED[reduction]
    loss_rows, p_rows = _out(loss_rows, "loss_rows", _F32, (T,), dev, stream)
    logprobs, p_lp = _out(logprobs, "logprobs", _F32, (T,), dev, stream)
    p_ent = None
    if want_entropy or entropy is not None:
        entropy, p_ent = _out(entropy, "entropy", _F32, (T,), dev, stream)
    row_stats, p_stats = _out(row_stats, "row_stats", _F32, (T, ROW_STATS), dev, stream)
    status, p_status = _out(status, "status", _I32, (1,), dev, stream)
    p_loss = None
    if red or loss_out is not None:
        loss_out, p_loss = _out(loss_out, "loss_out", _F32, (1,), dev, stream)
    _run("policy_loss_forward", dev, stream, logits.data_ptr(), dt, T, V, ld, p_act, ignore_index, temperature, p_old,
         p_adv, p_ref, p_w, ctypes.byref(params), red, p_rows, p_loss, p_lp, p_ent, p_stats, p_status)
    return loss_out, loss_rows, logprobs, entropy, row_stats, status


def policy_loss_backward(logits, actions, row_stats, grad_output, temperature=1.0, reduction="mean", *,
                         grad_logits=None, grad_dtype=None, stream=None):
    """Gradient of the policy loss w.r.t. the logits.  Returns grad_logits."""
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    red = RED[reduction]
    grad_logits, p_grad, gdt, gld = _matrix_out(grad_logits, "grad_logits", T, V, grad_dtype or logits.dtype, dev, stream)
    _run("policy_loss_backward", dev, stream, logits.data_ptr(), dt, T, V, ld,
         _given(actions, "actions", _I64, (T,), dev), temperature, red,
         _given(row_stats, "row_stats", _F32, (T, ROW_STATS), dev),
         _given(grad_output, "grad_output", _F32, (1,) if red else (T,), dev), p_grad, gdt, gld)
    return grad_logits


def policy_loss_forward_backward(logits, actions, advantages, old_logprobs=None, ref_logprobs=None, weights=None, *,
                                 clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0,
                                 temperature=1.0, ignore_index=IGNORE_INDEX, reduction="mean", grad_output=None,
                                 want_entropy=False, grad_logits=None, grad_dtype=None, loss_rows=None, loss_out=None,
                                 logprobs=None, entropy=None, row_stats=None, status=None, stream=None):
    """policy_loss_forward and its gradient in one pass over the logits (grad_output known; None: ones).

    Returns (loss_out, loss_rows, logprobs, entropy or None, grad_logits, status).
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    p_act, p_old, p_adv, p_ref, p_w = _policy_args(actions, advantages, old_logprobs, ref_logprobs, weights, T, dev)
    params = _PolicyParams(clip_low, clip_high, dual_clip, kl_coef, entropy_coef)
    red = RED[reduction]
    if grad_output is None:
        grad_output = _new((1,) if red else (T,), _F32, dev, stream)
        with torch.cuda.stream(stream):   # None: the current stream
            grad_output.fill_(1.0)
    p_go = _flat(grad_output, "grad_output", _F32, (1,) if red else (T,), dev)
    grad_logits, p_grad, gdt, gld = _matrix_out(grad_logits, "grad_logits", T, V, grad_dtype or logits.dtype, dev, stream)
    loss_rows, p_rows = _out(loss_rows, "loss_rows", _F32, (T,), dev, stream)
    logprobs, p_lp = _out(logprobs, "logprobs", _F32, (T,), dev, stream)
    p_ent = None
    if want_entropy or entropy is not None:
        entropy, p_ent = _out(entropy, "entropy", _F32, (T,), dev, stream)
    row_stats, p_stats = _out(row_stats, "row_stats", _F32, (T, ROW_STATS), dev, stream)
    status, p_status = _out(status, "status", _I32, (1,), dev, stream)
    p_loss = None
    if red or loss_out is not None:
        loss_out, p_loss = _out(loss_out, "loss_out", _F32, (1,), dev, stream)
    _run("policy_loss_forward_backward", dev, stream, logits.data_ptr(), dt, T, V, ld, p_act, ignore_index, temperature,
         p_old, p_adv, p_ref, p_w, ctypes.byref(params), red, p_go, p_rows, p_loss, p_lp, p_ent, p_stats, p_grad, gdt,
         gld, p_status)
    return loss_out, loss_rows, logprobs, entropy, grad_logits, status


class _Policy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, actions, advantages, old, ref, weights, params, temperature, ignore_index, reduction):
        dt, T, V, ld = _matrix(logits, "logits")
        dev = logits.device
        p_act, p_old, p_adv, p_ref, p_w = _policy_args(actions, advantages, old, ref, weights, T, dev)
        red = RED[reduction]
        loss = torch.empty(() if red else T, dtype=_F32, device=dev)
        kept = torch.empty((ROW_STATS + 2) * T + 1, dtype=_F32, device=dev)   # row_stats, loss_rows, logprobs, status
        stats = kept.data_ptr()
        rows = stats + 4 * ROW_STATS * T
        _run("policy_loss_forward", dev, None, logits.data_ptr(), dt, T, V, ld, p_act, ignore_index, temperature, p_old,
             p_adv, p_ref, p_w, ctypes.byref(params), red, rows if red else loss.data_ptr(),
             loss.data_ptr() if red else None, rows + 4 * T, None, stats, rows + 8 * T)
        ctx.save_for_backward(logits, actions, kept)
        ctx.temperature, ctx.red = temperature, red
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        logits, actions, kept = ctx.saved_tensors
        dt, T, V, ld = _matrix(logits, "logits")
        grad = _as_f32(grad)
        g = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
        _run("policy_loss_backward", logits.device, None, logits.data_ptr(), dt, T, V, ld, actions.data_ptr(),
             ctx.temperature, ctx.red, kept.data_ptr(), grad.data_ptr(), g.data_ptr(), dt, V)
        return (g,) + (None,) * 9


def policy_loss(logits, actions, advantages, old_logprobs=None, ref_logprobs=None, weights=None, *, clip_low=0.2,
                clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0, temperature=1.0,
                ignore_index=IGNORE_INDEX, reduction="mean"):
    """policy_loss_forward with autograd: the loss (the rows' with reduction "none"), its gradient w.r.t. the
    logits; everything else is a constant."""
    return _Policy.apply(logits, actions, advantages, old_logprobs, ref_logprobs, weights,
                         _PolicyParams(clip_low, clip_high, dual_clip, kl_coef, entropy_coef), float(temperature),
                         ignore_index, reduction)


# ---- preference loss ----------------------------------------------------------------------------


def _pairs(offsets, dev):
    if offsets is None or offsets.dim() != 1 or offsets.shape[0] % 2 == 0:
        raise ValueError("offsets: expected a 1-D tensor of 2 P + 1 row offsets, P pairs of sequences")
    return offsets.shape[0] // 2, _flat(offsets, "offsets", _I64, tuple(offsets.shape), dev)


def preference_loss_forward(logits, labels, offsets, ref_logprobs=None, *, beta=0.1, kind="sigmoid",
                            label_smoothing=0.0, margin=0.0, average=False, temperature=1.0,
                            ignore_index=IGNORE_INDEX, reduction="mean", pair_losses=None, loss_out=None, rewards=None,
                            logprobs=None, row_stats=None, status=None, stream=None):
    """Preference loss over P pairs of sequences packed along the rows (sequence q is rows offsets[q] to
    offsets[q + 1]; 2 p is pair p's preferred one, 2 p + 1 the other): with a sequence's reward beta times
    the sum (average: mean) of logprobs - ref_logprobs and x the difference of a pair's rewards less
    margin, -log sigma(x) ("sigmoid", with label_smoothing), max(0, 1 - x) ("hinge") or
    ((x - 1/2) / beta)^2 ("ipo").

    Returns (loss_out, pair_losses [P], rewards [2 P], logprobs [T], row_stats, status), row_stats for
    preference_loss_backward.
    """
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    P, p_off = _pairs(offsets, dev)
    p_lab = _given(labels, "labels", _I64, (T,), dev)
    params = _PreferenceParams(PREFERENCE_KINDS[kind], beta, label_smoothing, margin, bool(average))
    red = RED[reduction]
    pair_losses, p_pair = _out(pair_losses, "pair_losses", _F32, (P,), dev, stream)
    rewards, p_rew = _out(rewards, "rewards", _F32, (2 * P,), dev, stream)
    logprobs, p_lp = _out(logprobs, "logprobs", _F32, (T,), dev, stream)
    row_stats, p_stats = _out(row_stats, "row_stats", _F32, (T, ROW_STATS), dev, stream)
    status, p_status = _out(status, "status", _I32, (1,), dev, stream)
    p_loss = None
    if red or loss_out is not None:
        loss_out, p_loss = _out(loss_out, "loss_out", _F32, (1,), dev, stream)
    _run("preference_loss_forward", dev, stream, logits.data_ptr(), dt, T, V, ld, p_lab, ignore_index, temperature,
         p_off, P, _flat(ref_logprobs, "ref_logprobs", _F32, (T,), dev), ctypes.byref(params), red, p_pair, p_loss,
         p_rew, p_lp, p_stats, p_status)
    return loss_out, pair_losses, rewards, logprobs, row_stats, status


def preference_loss_backward(logits, labels, row_stats, grad_output, pairs, temperature=1.0, reduction="mean", *,
                             grad_logits=None, grad_dtype=None, stream=None):
    """Gradient of the preference loss over `pairs` pairs w.r.t. the logits.  Returns grad_logits."""
    dt, T, V, ld = _matrix(logits, "logits")
    dev = logits.device
    red = RED[reduction]
    grad_logits, p_grad, gdt, gld = _matrix_out(grad_logits, "grad_logits", T, V, grad_dtype or logits.dtype, dev, stream)
    _run("preference_loss_backward", dev, stream, logits.data_ptr(), dt, T, V, ld,
         _given(labels, "labels", _I64, (T,), dev), temperature, pairs, red,
         _given(row_stats, "row_stats", _F32, (T, ROW_STATS), dev),
         _given(grad_output, "grad_output", _F32, (1,) if red else (pairs,), dev), p_grad, gdt, gld)
    return grad_logits


class _Preference(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, offsets, ref, params, temperature, ignore_index, reduction):
        dt, T, V, ld = _matrix(logits, "logits")
        dev = logits.device
        P, p_off = _pairs(offsets, dev)
        p_lab = _given(labels, "labels", _I64, (T,), dev)
        red = RED[reduction]
        loss = torch.empty(() if red else P, dtype=_F32, device=dev)
        # row_stats, logprobs, rewards, pair_losses, status
        kept = torch.empty((ROW_STATS + 1) * T + 3 * P + 1, dtype=_F32, device=dev)
        stats = kept.data_ptr()
        lp = stats + 4 * ROW_STATS * T
        rewards = lp + 4 * T
        pairs = rewards + 8 * P
        _run("preference_loss_forward", dev, None, logits.data_ptr(), dt, T, V, ld, p_lab, ignore_index, temperature,
             p_off, P, _flat(ref, "ref_logprobs", _F32, (T,), dev), ctypes.byref(params), red,
             pairs if red else loss.data_ptr(), loss.data_ptr() if red else None, rewards, lp, stats, pairs + 4 * P)
        ctx.save_for_backward(logits, labels, kept)
        ctx.pairs, ctx.temperature, ctx.red = P, temperature, red
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        logits, labels, kept = ctx.saved_tensors
        dt, T, V, ld = _matrix(logits, "logits")
        grad = _as_f32(grad)
        g = torch.empty((T, V), dtype=logits.dtype, device=logits.device)
        _run("preference_loss_backward", logits.device, None, logits.data_ptr(), dt, T, V, ld, labels.data_ptr(),
             ctx.temperature, ctx.pairs, ctx.red, kept.data_ptr(), grad.data_ptr(), g.data_ptr(), dt, V)
        return (g,) + (None,) * 7


def preference_loss(logits, labels, offsets, ref_logprobs=None, *, beta=0.1, kind="sigmoid", label_smoothing=0.0,
                    margin=0.0, average=False, temperature=1.0, ignore_index=IGNORE_INDEX, reduction="mean"):
    """preference_loss_forward with autograd: the loss (the pairs' with reduction "none"), its gradient w.r.t.
    the logits; ref_logprobs are constants."""
    return _Preference.apply(logits, labels, offsets, ref_logprobs,
                             _PreferenceParams(PREFERENCE_KINDS[kind], beta, label_smoothing, margin, bool(average)),
                             float(temperature), ignore_index, reduction)


# ---- test hooks: waits that give up -------------------------------------------------------------


def vce_test_policy_stall(logits, actions, advantages, wait_ns=50_000_000, *, stream=None):
    """The one pass on contiguous bfloat16 logits, the gradient of each cluster's last block waiting in vain.
    Returns (loss_out, loss_rows, logprobs, grad_logits, status)."""
    T, V = logits.shape
    dev = logits.device
    go, loss, rows, lp = (torch.ones(1, device=dev), torch.zeros(1, device=dev), torch.zeros(T, device=dev),
                          torch.zeros(T, device=dev))
    stats, grad = torch.zeros(T, ROW_STATS, device=dev), torch.zeros_like(logits)
    status = torch.full((1,), 0x7FFF1234, dtype=_I32, device=dev)
    _run("vce_test_policy_stall", dev, stream, logits.data_ptr(), T, V, actions.data_ptr(), advantages.data_ptr(),
         go.data_ptr(), rows.data_ptr(), loss.data_ptr(), lp.data_ptr(), stats.data_ptr(), grad.data_ptr(), int(wait_ns),
         status.data_ptr())
    return loss, rows, lp, grad, status


def vce_test_policy_bwd_stall(logits, actions, row_stats, wait_ns=50_000_000, *, stream=None):
    """The backward on contiguous bfloat16 logits, each row's last block waiting for its last stage in vain.
    Returns grad_logits."""
    T, V = logits.shape
    dev = logits.device
    go, grad = torch.ones(1, device=dev), torch.zeros_like(logits)
    _run("vce_test_policy_bwd_stall", dev, stream, logits.data_ptr(), T, V, actions.data_ptr(), row_stats.data_ptr(),
         go.data_ptr(), grad.data_ptr(), int(wait_ns))
    return grad
