"""Plain fp64 restatement (numpy, row by row) of the post-training losses on logits and of the fp8 head: token
log-probabilities with entropies, the clipped policy loss, the preference loss over pairs of packed sequences,
their gradients, block quantisation to e4m3 and the product of such matrices.  Shares no code with the CUDA
path; test infrastructure only."""
import numpy as np

IGNORE_INDEX = -100


def rows(z, ids, temperature=1.0, keep=None):
    """Of each row: log p, p [T, V], the token's log-probability and the entropy; rows left out (ids
    IGNORE_INDEX, or keep False) are 0.  log p of the token is taken through the other columns, so that a
    confident row keeps its digits."""
    T, V = z.shape
    logp, lp, ent = np.full((T, V), -np.inf), np.zeros(T), np.zeros(T)
    valid = ids != IGNORE_INDEX
    if keep is not None:
        valid = valid & keep
    for i in np.nonzero(valid)[0]:
        x = z[i] / temperature
        if np.isfinite(x.max()):
            x = x - x.max()   # beside logits of 1e20 the logarithm of a sum is lost in 64 bits too
        t = ids[i]
        rest = np.delete(x, t)
        m = rest.max() if rest.size else -np.inf
        other = m + np.log(np.exp(rest - m).sum()) if m > -np.inf else -np.inf
        lse = np.logaddexp(other, x[t])
        logp[i] = x - lse
        if x[t] == -np.inf:
            lp[i] = -np.inf
        elif other == -np.inf:
            lp[i] = 0.0
        else:
            lp[i] = -np.logaddexp(0.0, other - x[t])
        logp[i, t] = lp[i]
        p = np.exp(logp[i])
        ent[i] = -np.sum(p[p > 0] * logp[i][p > 0])
    return dict(logp=logp, p=np.exp(logp), lp=lp, ent=ent, valid=valid)


def gradient(r, ids, a, b, temperature=1.0):
    """dl/dz from a = dl/dlp and b = dl/dH per row."""
    T, V = r["p"].shape
    g = np.zeros((T, V))
    for i in np.nonzero(r["valid"])[0]:
        p, logp = r["p"][i], r["logp"][i]
        onehot = np.zeros(V)
        onehot[ids[i]] = 1.0
        inner = np.where(p > 0, logp + r["ent"][i], 0.0)
        diff = -p
        diff[ids[i]] = -np.expm1(r["lp"][i])   # 1 - p_t without cancellation
        g[i] = (a[i] * diff - b[i] * p * inner) / temperature
    return g


def policy(z, ids, adv, old=None, ref=None, weights=None, clip_low=0.2, clip_high=0.2, dual=0.0, kl=0.0, ent=0.0,
           temperature=1.0, reduction="mean", grad_output=1.0):
    r = rows(z, ids, temperature)
    lp, H, valid = r["lp"], r["ent"], r["valid"]
    w = np.ones(len(ids)) if weights is None else weights
    loss, a = np.zeros(len(ids)), np.zeros(len(ids))
    for i in np.nonzero(valid)[0]:
        ratio = 1.0 if old is None else np.exp(lp[i] - old[i])
        A = adv[i]
        one, two = ratio * A, min(max(ratio, 1 - clip_low), 1 + clip_high) * A
        s, slope = (one, one) if one <= two else (two, 0.0)
        if dual and A < 0 and s < dual * A:
            s, slope = dual * A, 0.0
        loss[i], a[i] = -s, -slope
        if kl:
            d = ref[i] - lp[i]
            loss[i] += kl * (np.expm1(d) - d)
            a[i] -= kl * np.expm1(d)
        loss[i] = w[i] * (loss[i] - ent * H[i])
        a[i] *= w[i]
    b = np.where(valid, -ent * w, 0.0)
    n = int(valid.sum())
    c = np.broadcast_to(np.asarray(grad_output, np.float64), (len(ids),)) * (1.0 / n if reduction == "mean" and n else 1.0)
    total = loss.sum() / n if reduction == "mean" and n else (np.nan if reduction == "mean" else loss.sum())
    return dict(r, loss_rows=loss, loss=total, a=a * c, b=b * c, grad=gradient(r, ids, a * c, b * c, temperature), n=n)


def preference(z, labels, offsets, ref=None, beta=0.1, kind="sigmoid", eps=0.0, margin=0.0, average=False,
               temperature=1.0, reduction="mean", grad_output=1.0):
    T = len(labels)
    P = (len(offsets) - 1) // 2
    inside = (np.arange(T) >= offsets[0]) & (np.arange(T) < offsets[-1])
    r = rows(z, labels, temperature, inside)
    rewards, share, pair = np.zeros(2 * P), np.ones(2 * P), np.zeros(P)
    for q in range(2 * P):
        n = 0
        for i in range(offsets[q], offsets[q + 1]):
            if r["valid"][i]:
                rewards[q] += r["lp"][i] - (0.0 if ref is None else ref[i])
                n += 1
        if average and n:
            share[q] = 1.0 / n
        rewards[q] *= beta * share[q]
    slope = np.zeros(P)
    for p in range(P):
        x = rewards[2 * p] - rewards[2 * p + 1] - margin
        if kind == "sigmoid":
            pair[p] = (1 - eps) * np.logaddexp(0, -x) + eps * np.logaddexp(0, x)
            slope[p] = -(1 - eps) / (1 + np.exp(x)) + eps / (1 + np.exp(-x))
        elif kind == "hinge":
            pair[p], slope[p] = max(0.0, 1 - x), -float(x < 1)
        else:
            pair[p], slope[p] = ((x - 0.5) / beta) ** 2, 2 * (x - 0.5) / beta ** 2
    c = np.broadcast_to(np.asarray(grad_output, np.float64), (P,)) * (1.0 / P if reduction == "mean" and P else 1.0)
    a = np.zeros(T)
    for q in range(2 * P):
        a[offsets[q]:offsets[q + 1]] = beta * slope[q // 2] * c[q // 2] * share[q] * (1 if q % 2 == 0 else -1)
    a[~r["valid"]] = 0.0
    total = pair.sum() if reduction != "mean" else (pair.mean() if P else np.nan)
    return dict(r, rewards=rewards, pairs=pair, loss=total, a=a, b=np.zeros(T),
                grad=gradient(r, labels, a, np.zeros(T), temperature))


# ---- e4m3 ---------------------------------------------------------------------------------------


def e4m3_values():
    """The 256 e4m3 values by their byte (two NaN, no infinities)."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = np.nan if e == 15 and m == 7 else (-v if b & 128 else v)
    return out


def to_e4m3(v):
    """fp64 values within +-448 rounded to the nearest e4m3 value, ties to the even mantissa."""
    v = np.asarray(v, np.float64)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    return np.rint(v / step) * step


def quantize(x, block_rows):
    """(values, scales) of a matrix, block by block."""
    R, D = x.shape
    nr, nd = -(-R // block_rows), -(-D // 128)
    out, scales = np.empty((R, D)), np.empty((nr, nd))
    for i in range(nr):
        for j in range(nd):
            cut = (slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
            top = np.abs(x[cut]).max()
            if not np.isfinite(top):
                scales[i, j], out[cut] = np.nan, np.nan
                continue
            k = -126
            if top > 0:
                k = int(np.floor(np.log2(top))) - 10
                while 448.0 * 2.0 ** k < top:
                    k += 1
                k = max(k, -126)
            scales[i, j] = 2.0 ** k if top > 0 else 1.0
            out[cut] = to_e4m3(x[cut] / scales[i, j])
    return out, scales


def linear(x, xs, w, ws):
    """The product of scaled e4m3 values, and the sum of its terms' magnitudes."""
    D, V = x.shape[1], w.shape[0]
    col = np.arange(D) // 128
    a = x * xs[:, col]
    b = w * ws[(np.arange(V) // 128)[:, None], col]
    return a @ b.T, np.abs(a) @ np.abs(b).T
