"""Tolerances of the post-training losses and the fp8 head, derived from the kernels' arithmetic.

E = 2^-24 is a rounding's half step.  d = lse_delta (tests/_logits_grading.py) bounds the relative error of a sum
of exponentials, Z = max |z| log2(e) / temperature.
  u = L' - x_t: one logarithm of such a sum and one product, D = lse_tol + 8 E (2 Z + 17) in all; the same bounds
      every log p_j
  log p_t = -softplus(u): D (1 - p_t), the slope of softplus, and 4 E of itself
  H: the sum of e y has the terms' errors d and y's own 3 Z E, |y| <= 2 Z; then the chain rule's factors, whose slope
      in u is at most p_t (1 - p_t) (|u| + H') <= (2 Z + 17) / 4
"""
import numpy as np

from tests._logits_grading import E24, lse_delta, lse_tol


def log_tol(zmax, tau):
    Z = zmax * 1.4426950408889634 / tau
    return lse_tol(zmax, tau) + 8 * E24 * (2 * Z + 17)


def lp_tol(r, zmax, tau):
    lp = np.where(np.isfinite(r["lp"]), r["lp"], 0.0)
    return log_tol(zmax, tau) * -np.expm1(lp) + 4 * E24 * np.abs(lp) + 1e-37


def ent_tol(zmax, tau):
    Z = zmax * 1.4426950408889634 / tau
    return lse_delta(zmax, tau) * (1 + 4 * Z) + log_tol(zmax, tau) * (1 + (2 * Z + 17) / 4) + 8 * E24 * (Z + 17)


def near(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    odd = ~np.isfinite(want)
    assert np.array_equal(got[odd], want[odd], equal_nan=True), f"{what}: infinities and NaN"
    tol = np.broadcast_to(tol, want.shape)[~odd]
    err = np.abs(got[~odd] - want[~odd])
    assert np.all(err <= tol), f"{what}: {np.sum(~(err <= tol))} off, worst {np.max(err / tol):.3g} of the tolerance"


def check_rows(lp, ent, r, zmax, tau):
    near(lp, r["lp"], lp_tol(r, zmax, tau), "log-probabilities")
    if ent is not None:
        near(ent, r["ent"], np.where(r["valid"], ent_tol(zmax, tau), 0.0), "entropies")


def check_grad(got, ref, ids, da, zmax, tau, eps):
    """ref: the oracle's dict with a, b and grad; da: the error of a.  g = (a (onehot - p) - b p (log p + H)) / tau
    moves by |a| (p + 1 - p_t at the token) 2 D e^D, by |b| p ((|log p + H| 2 + 1) D + dH), by da times its factor, by
    16 roundings of each term, and by the rounding to the output's type."""
    got = np.asarray(got, np.float64)
    p, a, b = ref["p"], np.abs(ref["a"])[:, None], np.abs(ref["b"])[:, None]
    D = log_tol(zmax, tau)
    hot = np.zeros(p.shape)
    for i in np.nonzero(ref["valid"])[0]:
        hot[i, ids[i]] = 1.0
    factor = np.where(hot > 0, 1 - p, p)
    factor = np.where(hot > 0, np.maximum(factor, np.abs(ref["grad"]) * tau / np.maximum(a, 1e-30) * (b == 0)), factor)
    inner = np.where(p > 0, np.abs(np.where(p > 0, ref["logp"], 0.0) + ref["ent"][:, None]), 0.0)
    tol = a * factor * (2 * D * np.exp(D) + 16 * E24) + b * p * ((2 * inner + 1) * D * np.exp(D) + ent_tol(zmax, tau) + 16 * E24 * inner)
    tol = (tol + np.asarray(da)[:, None] * factor) / tau + eps / 2 * np.abs(ref["grad"]) * 1.01 + 1e-37
    assert np.all(got[~ref["valid"]] == 0), "rows left out"
    near(got, ref["grad"], tol, "gradient")


def policy_errors(ref, adv, old, refp, w, kl, ent, zmax, tau, c):
    """(error of the rows' losses, error of a): ratios and exp(d) carry the log-probability's error."""
    lp, dlp = ref["lp"], lp_tol(ref, zmax, tau)
    w = np.ones_like(lp) if w is None else w
    r = np.ones_like(lp) if old is None else np.exp(lp - old)
    dr = r * (dlp * 1.01 + 8 * E24)
    loss = np.abs(adv) * dr + 4 * E24 * np.abs(adv) * (1 + r)
    a = np.abs(adv) * dr
    if kl:
        e = np.exp(refp - lp)
        loss = loss + kl * (np.abs(e - 1) * dlp + e * dlp ** 2 + 16 * E24 * (e + np.abs(refp - lp)))
        a = a + kl * e * (dlp * 1.01 + 8 * E24)
    if ent:
        loss = loss + abs(ent) * (ent_tol(zmax, tau) + 4 * E24 * ref["ent"])
    valid = ref["valid"]
    return np.where(valid, np.abs(w) * loss + 4 * E24 * np.abs(ref["loss_rows"]) + 1e-37, 0.0), np.where(
        valid, np.abs(w * c) * a + 4 * E24 * np.abs(ref["a"]), 0.0)


def preference_errors(ref, offsets, beta, kind, average, zmax, tau, c):
    """(error of the rewards, the pairs' losses, and a): sums of the rows' errors; their own additions are
    compensated, so a few roundings of the result (and of each difference's larger side, kept with it)."""
    P = (len(offsets) - 1) // 2
    dlp = np.where(ref["valid"], lp_tol(ref, zmax, tau), 0.0)
    rewards, share = np.zeros(2 * P), np.ones(2 * P)
    for q in range(2 * P):
        cut = slice(offsets[q], offsets[q + 1])
        n = ref["valid"][cut].sum()
        if average and n:
            share[q] = 1.0 / n
        rewards[q] = beta * share[q] * dlp[cut].sum() + 8 * E24 * np.abs(ref["rewards"][q])
    x = rewards[0::2] + rewards[1::2] + 4 * E24 * (np.abs(ref["rewards"][0::2]) + np.abs(ref["rewards"][1::2]) + 1)
    second = {"sigmoid": 0.25, "hinge": 0.0, "ipo": 2 / beta ** 2}[kind]
    first = {"sigmoid": 1.0, "hinge": 1.0, "ipo": 0.0}[kind]
    xs = ref["rewards"][0::2] - ref["rewards"][1::2]
    if kind == "ipo":
        first = 2 * (np.abs(xs) + 1) / beta ** 2
    pairs = first * x + second * x * x + 8 * E24 * np.abs(ref["pairs"]) + 1e-37
    da = np.zeros(len(ref["lp"]))
    for q in range(2 * P):
        cut = slice(offsets[q], offsets[q + 1])
        da[cut] = beta * share[q] * np.abs(c[q // 2]) * second * x[q // 2]
    return rewards + 1e-37, pairs, da + 16 * E24 * np.abs(ref["a"])


def check_linear(got, want, size, blocks, eps):
    """A block's 128 products are summed in fp32 on the tensor cores, in any order and with truncated additions (one
    step of 2^-23 of the running size each), and the blocks' sums with an fma each, the scale's product rounded."""
    tol = size * (128 * 2.0 ** -23 + (blocks + 2) * E24) + eps / 2 * np.abs(want) * 1.01 + 1e-37
    near(got, want, tol, "logits")
