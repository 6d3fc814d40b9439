"""Tolerances of the operators around the cross-entropy, derived from the kernels' arithmetic.

A log-sum-exp is a sum of 2^((z - m) k2), k2 = log2(e) / temperature, in fp32:
  exponent arguments: fma(z, k2, -m k2) with m k2 rounded: 2^-24 (|m k2| + |argument|) each, so at most
      3 Z 2^-24 in log2 units with Z = max |z| k2 (finite z); times ln 2 relative to the term
  2^x: 2^-22 relative (the hardware exponential's documented error)
  sums: a term passes at most 5 + 64 + 8 + 8 + 8 additions (its thread's tree, the stages of a slice, the
      warp's lanes and the warps, the cluster, the candidates left out), each 2^-24 relative; where the
      reference moves, the pair is rescaled by another exponential (2^-22 + 3 Z 2^-24): at most 32 times
so the sum's relative error, and the absolute error of its logarithm, is at most lse_delta below; the
logarithm and m * s + log S add three roundings of values no larger than Z + 16.
"""
import numpy as np

E24 = 2.0 ** -24


def lse_delta(zmax, temperature):
    Z = zmax * 1.4426950408889634 / temperature
    return 93 * E24 + 33 * (2.0 ** -22 + 3 * Z * E24)


def lse_tol(zmax, temperature):
    """Absolute tolerance of a log-sum-exp."""
    return lse_delta(zmax, temperature) + 3 * E24 * (zmax / temperature + 16)


def check_lse(got, want, zmax, temperature, what="lse"):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    none = want == -np.inf
    assert np.all(got[none] == -np.inf), f"{what}: not -inf"
    err = np.abs(got[~none] - want[~none])
    tol = lse_tol(zmax, temperature)
    assert np.all(err <= tol), f"{what}: off by {err.max():.3e}, tolerance {tol:.3e}"


def distill_delta(zmax, tmax, temperature):
    """Error of a log-probability ratio log(p / q) in the kernels: two log-sum-exps of each side (the
    tail's, the entries'; the latter, and q's, are shorter sums of the same kind)."""
    return 2 * lse_tol(zmax, temperature) + 2 * lse_tol(tmax, temperature)


def check_distill_loss(got, ref, zmax, tmax, temperature):
    """KL = sum q phi(log p/q) with phi(x) = e^x - 1 - x: an error d of x moves a term by
    q |e^x - 1| d = |p - q| d to first order and by max(p, q) e^d d^2 / 2 beyond it; the terms' own
    roundings are 8 of 2^-24 relative, and its sums 16 more."""
    got = np.asarray(got, np.float64)
    d = distill_delta(zmax, tmax, temperature)
    tv = np.abs(ref["p"] - ref["q"]).sum(1)
    tol = temperature ** 2 * (tv * d + 2 * d * d + 24 * E24 * ref["kl"]) + 1e-38
    valid = ref["valid"]
    assert np.all(got[~valid] == 0) and not np.any(np.signbit(got[~valid])), "ignored rows"
    inf = valid & ~np.isfinite(ref["loss_rows"])
    assert np.all(got[inf] == np.inf), "infinite losses"
    v = valid & ~inf
    err = np.abs(got[v] - ref["loss_rows"][v])
    assert np.all(err <= tol[v]), f"loss rows: worst {np.max(err / tol[v]):.2f} of the tolerance"


def check_distill_grad(got, ref, zmax, tmax, temperature, eps, c=None):
    """grad = c tau (p - q): errors d of the log-probabilities move it by |c| tau d (p + q) (twice, for the
    factor p_T - q_T and for the exponential), then a rounding of half an eps of the output's type."""
    got = np.asarray(got, np.float64)
    d = distill_delta(zmax, tmax, temperature)
    c = ref["c"] if c is None else c
    want = c[:, None] * (ref["p"] - ref["q"])
    tol = np.abs(c)[:, None] * (2 * d * np.exp(d) + 16 * E24) * (ref["p"] + ref["q"]) + eps / 2 * np.abs(want) * 1.01 + 1e-37
    assert np.all(got[~ref["valid"]] == 0) and not np.any(np.signbit(got[~ref["valid"]])), "ignored rows"
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"gradient: {bad.sum()} entries, worst {np.nanmax(err / tol):.2f} of the tolerance at "
                           f"{np.argwhere(bad)[:4].tolist()}")


def check_processed(got, want, size, eps):
    """A processed logit takes at most 7 fp32 operations on terms whose magnitudes add up to `size`, then
    a rounding to the output's type; masked entries are exact."""
    got = np.asarray(got, np.float64)
    inf = ~np.isfinite(want)
    assert np.array_equal(got[inf], want[inf]), "masked or infinite entries"
    tol = 8 * E24 * size[~inf] + eps / 2 * np.abs(want[~inf]) * 1.01 + 1e-37
    err = np.abs(got[~inf] - want[~inf])
    assert np.all(err <= tol), f"worst {np.max(err / tol):.2f} of the tolerance"
