"""What the log-probabilities are off by on the mean over many rows, which a sequence's sum or a step's ratios add up,
and the entropies of rows of few columns.

A row's own errors are of either sign: the result's rounding, at most 2^-21 at 8 to 16, is 2.8e-7 / sqrt(N) of the mean,
and 4 of those are allowed.  Beside it stand
  6e-8     the base-2 exponential's mean error over a row's terms (measured)
and 1e-9 for the 64-bit side and the sums' second order.  The temperature is what the calls take, an fp32 number.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def rows(T, V, tau, offset):
    """Logits, ids, and in 64 bits the log-probabilities and z_t - E z."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = 2 * torch.randn(T, V, generator=g, device="cuda") + offset
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    want, gap = torch.empty(2, T, dtype=torch.float64, device="cuda")
    for i in range(0, T, 256):
        x = z[i:i + 256].double() / tau
        logp = x.log_softmax(1)
        at = ids[i:i + 256, None]
        want[i:i + 256] = logp.gather(1, at)[:, 0]
        gap[i:i + 256] = (x.gather(1, at)[:, 0] - (logp.exp() * x).sum(1)) * tau
    return z, ids, want, gap


def bound(T):
    return 6e-8 + 4 * 2.8e-7 / math.sqrt(T) + 1e-9


CASES = [(T, V, tau, offset) for T, V in ((8192, 4000), (4096, 32000), (2048, 128256))
         for tau in (1.0, float(np.float32(1.3))) for offset in (0.0, 20.0, 100.0)]


@pytest.mark.parametrize("T,V,tau,offset", CASES)
def test_mean_error(vce, T, V, tau, offset):
    z, ids, want, _ = rows(T, V, tau, offset)
    adv = torch.ones(T, device="cuda")
    kw = dict(temperature=tau, reduction="sum")
    for name, lp in (
            ("forward", vce.ce_logprobs_forward(z, ids, tau, want_entropy=False)[0]),
            ("with entropies", vce.ce_logprobs_forward(z, ids, tau)[0]),
            ("policy forward", vce.policy_loss_forward(z, ids, adv, **kw)[2]),
            ("one pass with an entropy term", vce.policy_loss_forward_backward(z, ids, adv, entropy_coef=0.1, **kw)[2])):
        off = float((lp.double() - want).mean())
        print(f"{name} {T} x {V} at {tau:.3g} + {offset}: {off:.2e} of {bound(T):.2e}")
        assert abs(off) <= bound(T), name


@pytest.mark.parametrize("V", [2, 3, 9, 600])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("other", [0.0, 1.0, -2.0, 8.0])
def test_entropy_of_one_other_column(vce, V, tau, other):
    """A token of little probability beside one column (the rest masked): their entropy is all there is, and the other
    column's exponential is exactly 1.  A handful of roundings, 16 of 2^-24."""
    x = torch.tensor([-60.0, -30.0, -8.0, -1.0, 0.5, 9.0, 30.0])
    z = torch.full((len(x), V), float("-inf"))
    z[:, 0] = x
    z[:, V - 1] = other
    ids = torch.zeros(len(x), dtype=torch.int64)
    u = (other - x.double()) / tau
    p, q = torch.sigmoid(-u), torch.sigmoid(u)
    want = p * torch.nn.functional.softplus(u) + q * torch.nn.functional.softplus(-u)
    _, ent, _, _ = vce.ce_logprobs_forward(z.cuda(), ids.cuda(), tau)
    _, _, _, two, _, _ = vce.policy_loss_forward_backward(z.cuda(), ids.cuda(), torch.ones(len(x), device="cuda"),
                                                          temperature=tau, entropy_coef=0.1, want_entropy=True)
    for got in (ent, two):
        # the gap itself is exact (powers of two and their products), but for |u| roundings of 2^-24 in e^-|u|
        tol = (16 + 2 * u.abs()) * 2.0 ** -24 * want + 2.0 ** -126   # and fp32 ends there
        assert torch.all((got.double().cpu() - want).abs() <= tol)


@pytest.mark.parametrize("T,V,tau,offset", CASES)
def test_mean_error_of_the_one_pass(vce, T, V, tau, offset):
    """Without an entropy term the scale is rounded on both sides, ln 2 k_lo (z_t - E z): a common offset of the logits
    is not in it."""
    z, ids, want, gap = rows(T, V, tau, offset)
    k = 1.4426950408889634 / tau
    lost = math.log(2) * abs((k - float(np.float32(k))) * float(gap.mean()))
    lp = vce.policy_loss_forward_backward(z, ids, torch.ones(T, device="cuda"), temperature=tau, reduction="sum")[2]
    off = float((lp.double() - want).mean())
    print(f"{T} x {V} at {tau:.3g} + {offset}: {off:.2e} of {bound(T) + lost:.2e}")
    assert abs(off) <= bound(T) + lost
