"""Plain fp64 restatement (numpy, row by row) of the operators around the cross-entropy: top K with
log-sum-exps, the distillation loss against a teacher's top K with its gradient, and the processing of
logits with its gradient.  Shares no code with the CUDA path; test infrastructure only."""
import numpy as np

IGNORE_INDEX = -100


def lse(x):
    """log sum exp of a 1-D array; -inf of nothing."""
    x = np.asarray(x, np.float64)
    m = x.max() if x.size else -np.inf
    if m == -np.inf:
        return -np.inf
    return m + np.log(np.sum(np.exp(x - m)))


def topk(z, k, temperature=1.0):
    """(values, ids, lse, tail_lse) of fp64 logits [T, V]: descending, ties to the lowest column, -inf
    entries as (-inf, -1)."""
    T, V = z.shape
    values, ids = np.full((T, k), -np.inf), np.full((T, k), -1, np.int64)
    full, tail = np.empty(T), np.empty(T)
    for i in range(T):
        order = np.lexsort((np.arange(V), -z[i]))[:k]
        order = order[z[i][order] > -np.inf]
        values[i, :len(order)], ids[i, :len(order)] = z[i][order], order
        full[i] = lse(z[i] / temperature)
        rest = np.ones(V, bool)
        rest[order] = False
        tail[i] = lse(z[i][rest] / temperature)
    return values, ids, full, tail


def distill(z, ids, t, tail=None, temperature=1.0, labels=None, reduction="mean", grad_output=1.0,
            ignore_index=IGNORE_INDEX):
    """Losses and gradient of the K + 1 outcome KL divergence times temperature^2, from the definition.

    Returns a dict: loss_rows, loss_out, grad [T, V], p and q [T, V] (q's tail mass spread over the tail's
    columns as p is), kl, valid, n."""
    T, V = z.shape
    tau = float(temperature)
    valid = ids[:, 0] != -1
    if labels is not None:
        valid &= labels != ignore_index
    n = int(valid.sum())
    out = dict(loss_rows=np.zeros(T), kl=np.zeros(T), p=np.zeros((T, V)), q=np.zeros((T, V)), valid=valid, n=n)
    for i in np.nonzero(valid)[0]:
        s = z[i] / tau
        there = ids[i] >= 0
        cols, tv = ids[i][there], t[i][there] / tau
        r = -np.inf if tail is None else tail[i]
        total = lse(np.append(tv, r))
        q = np.exp(tv - total)
        q_tail = np.exp(r - total)
        rest = np.ones(V, bool)
        rest[cols] = False
        # log p from the entries' and the others' log-sum-exps, so that a mass near 1 keeps 1 - p
        top, other = lse(s[cols]), lse(s[rest])
        logp = s - top - np.logaddexp(0.0, other - top) if top > -np.inf else s - other
        log_p_tail = -np.logaddexp(0.0, top - other) if other > -np.inf else -np.inf
        with np.errstate(divide="ignore", invalid="ignore"):
            kl = np.sum(np.where(q > 0, q * (np.log(q) - logp[cols]), 0.0))
            if q_tail > 0:
                kl += q_tail * (np.log(q_tail) - log_p_tail)
            spread = np.exp(logp - log_p_tail) if log_p_tail > -np.inf else np.zeros(V)
        out["kl"][i], out["loss_rows"][i] = kl, tau * tau * kl
        out["p"][i] = np.exp(logp)
        full = np.where(rest, q_tail * spread, 0.0)
        full[cols] = q
        out["q"][i] = full
    rows = out["loss_rows"]
    out["loss_out"] = rows.sum() if reduction == "sum" else (rows.sum() / n if n else np.nan)
    c = np.broadcast_to(np.asarray(grad_output, np.float64), (T,)) * valid
    if reduction == "mean" and n:
        c = c / n
    out["c"] = c * tau
    out["grad"] = out["c"][:, None] * (out["p"] - out["q"])
    return out


def process(z, *, temperature=None, repetition=None, frequency=None, presence=None, history=None, prompt_lens=None,
            bias=None, allowed=None, upstream=None):
    """Processed fp64 logits, or with upstream the gradient w.r.t. z.  history: a list of id arrays, one
    a row; bias: a list of {column: value}; allowed: bool [T, V].  Also returns the sum of the terms'
    magnitudes per entry, for tolerances."""
    T, V = z.shape
    y, size = np.empty((T, V)), np.empty((T, V))
    for i in range(T):
        tau = 1.0 if temperature is None else float(temperature[i])
        r = 1.0 if repetition is None else float(repetition[i])
        f = 0.0 if frequency is None else float(frequency[i])
        p = 0.0 if presence is None else float(presence[i])
        factor, shift = np.ones(V), np.zeros(V)
        if history is not None:
            h = np.asarray(history[i], np.int64)
            start = 0 if prompt_lens is None else int(prompt_lens[i])
            for token in set(h.tolist()):
                factor[token] = 1.0 / r if z[i, token] > 0 else r
                count = int(np.sum(h[start:] == token))
                if count:
                    shift[token] = -f * count - p
        added = np.zeros(V)
        if bias is not None:
            for col, v in bias[i].items():
                added[col] = v
        if upstream is not None:
            y[i] = upstream[i] * factor / tau
            size[i] = np.abs(y[i])
        else:
            y[i] = (z[i] * factor + shift + added) / tau
            size[i] = (np.abs(z[i] * factor) + np.abs(shift) + np.abs(added)) / tau
        if allowed is not None:
            y[i][~allowed[i]] = 0.0 if upstream is not None else -np.inf
            size[i][~allowed[i]] = 0.0
    return y, size


def pack_mask(allowed):
    """bool [T, V] -> int32 words [T, ceil(V / 32)], bit j % 32 of word j // 32."""
    T, V = allowed.shape
    bits = np.zeros((T, (V + 31) // 32 * 32), np.uint64)
    bits[:, :V] = allowed
    words = (bits.reshape(T, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)
