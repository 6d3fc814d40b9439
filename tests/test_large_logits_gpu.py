"""Rows with logits of great size on the GPU: masks that are finite, from -1e10 to the type's lowest value, at several
temperatures, and logits of 1e12, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import policy_oracle as O
from tests import _policy_grading as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
FORMS = [(600, F32), (600, BF16), (20001, BF16), (40000, F32), (128256, BF16), (300001, F32)]


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def host(t):
    return t.detach().double().cpu().numpy()


def oracle_logits(z, tau):
    """In 64 bits; what passes fp32 when multiplied by log2(e) / temperature is -inf."""
    out = host(z)
    out[out * 1.4426950408889634 / tau < -float(torch.finfo(F32).max)] = -np.inf
    return out


def masked_rows(V, dtype, low, seed):
    """Every second column masked; the first half; all but three; all but the token and another; all; the token and the
    first half; all but the token; the last half."""
    g = torch.Generator().manual_seed(seed + V)
    z = (2 * torch.randn(8, V, generator=g)).to(dtype).cuda()
    ids = torch.randint(V // 2 + 1, V - 1, (8,), generator=g).cuda()
    z[0, ::2] = low
    z[1, : V // 2] = low
    keep = z[2, [V // 3, V // 2, V - 1]].clone()
    z[2] = low
    z[2, [V // 3, V // 2, V - 1]] = keep
    ids[2] = V // 3
    z[3] = low
    z[3, int(ids[3])] = 1.5
    z[3, 1] = -0.25
    z[4] = low
    z[5, : V // 2] = low
    z[5, int(ids[5])] = low
    z[6] = low
    z[6, int(ids[6])] = -3.0
    z[7, V // 2:] = low
    ids[7] = 3
    ids[0] |= 1
    return z, ids


def check_all(vce, z, ids, tau, zmax):
    """Log-probabilities, entropies and gradients of the calls and of the one pass with an entropy term and without."""
    T = z.shape[0]
    n = ids.cpu().numpy()
    z64 = oracle_logits(z, tau)
    dead = np.isneginf(z64).all(1)
    live = ~dead
    r = O.rows(z64[live], n[live], tau)
    zero = np.zeros(int(live.sum()))
    g = torch.Generator().manual_seed(5)
    ga, gb = torch.randn(2, T, generator=g).cuda()
    eps = torch.finfo(z.dtype).eps

    def gradients(got, a, b, da=zero):
        r["a"], r["b"] = a[live], b[live]
        r["grad"] = O.gradient(r, n[live], r["a"], r["b"], tau)
        G.check_grad(host(got)[live], r, n[live], da, zmax, tau, eps)
        assert np.all(host(got)[dead] == 0)

    for entropy in (True, False):
        lp, ent, stats, status = vce.ce_logprobs_forward(z, ids, tau, want_entropy=entropy)
        assert vce.vce_get_status(status) == 0
        G.check_rows(host(lp)[live], host(ent)[live] if entropy else None, r, zmax, tau)
        assert np.isnan(host(lp)[dead]).all()
        gradients(vce.ce_logprobs_backward(z, ids, stats, ga, gb if entropy else None, tau), host(ga),
                  host(gb) if entropy else np.zeros(T))
    adv = torch.linspace(0.5, 1.5, T).cuda()
    for ent in (0.0, 0.25):
        _, rows, lp, H, grad, status = vce.policy_loss_forward_backward(z, ids, adv, entropy_coef=ent, temperature=tau,
                                                                       reduction="none", want_entropy=ent != 0)
        assert vce.vce_get_status(status) == 0
        G.check_rows(host(lp)[live], host(H)[live] if ent else None, r, zmax, tau)
        want = -host(adv)[live] - ent * r["ent"]
        G.near(host(rows)[live], want, 4 * G.E24 * np.abs(want) + ent * G.ent_tol(zmax, tau), "losses")
        assert np.isnan(host(rows)[dead]).all()
        gradients(grad, -host(adv), np.full(T, -ent))


@pytest.mark.parametrize("V,dtype", FORMS)
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("low", [-1e10, -1e12, -1e20, -1e30, -1e37, None])
def test_finite_masks(vce, V, dtype, tau, low):
    low = torch.finfo(dtype).min if low is None else low
    z, ids = masked_rows(V, dtype, low, 0)
    check_all(vce, z, ids, tau, float(z.float()[z.float().abs() < 1e6].abs().max()))


@pytest.mark.parametrize("V,dtype", [(900, BF16), (1000, F32), (3000, BF16), (7001, BF16), (14000, BF16)])
@pytest.mark.parametrize("low", [-1e10, -1e30, None])
def test_finite_masks_of_many_rows(vce, V, dtype, low):
    """As many rows as there are SMs and more: the forms that hold a row in registers."""
    low = torch.finfo(dtype).min if low is None else low
    parts = [masked_rows(V, dtype, low, s) for s in range(24)]
    z, ids = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    check_all(vce, z, ids, 1.5, float(z.float()[z.float().abs() < 1e6].abs().max()))


@pytest.mark.parametrize("V,dtype", FORMS)
@pytest.mark.parametrize("tau", [1.0, 1.3])
@pytest.mark.parametrize("size", [1e11, -1e11, 1e30])
def test_great_logits(vce, V, dtype, tau, size):
    """Nothing but the rounding of z / tau is lost: equal logits share their mass, any other has all of it or none.  The
    log-probability of a token with none is off by its product's two roundings, the temperature's, the difference's
    and the result's: 5 half steps of 2^-24 of the largest."""
    g = torch.Generator().manual_seed(V)
    z = (2 * torch.randn(6, V, generator=g)).to(dtype).cuda()
    ids = torch.randint(4, V - 1, (6,), generator=g).cuda()
    top = abs(size)
    z[0, int(ids[0])] = top
    z[0, V - 1] = top                       # the token and one other
    z[1, 2] = z[1, 3] = z[1, V - 1] = top   # three others
    z[2, int(ids[2])] = top                 # the token alone
    z[3] = size                             # all alike
    z[4] = -top
    z[4, 0] = z[4, 1] = -top / 2            # two above the rest, the token not among them
    z[5] = size
    z[5, ::3] = size * 1.5                  # a third of the columns
    ids[5] = 3 if size > 0 else 4
    x = host(z) / tau
    p = np.zeros(x.shape)
    for i in range(6):
        p[i, x[i] == x[i].max()] = 1.0 / (x[i] == x[i].max()).sum()
    p[2] = 0.0
    p[2, int(ids[2])] = 1.0
    t = ids.cpu().numpy()
    pt = p[np.arange(6), t]
    want = np.where(pt > 0, np.log(np.maximum(pt, 1e-300)), x[np.arange(6), t] - x.max(1))
    ent = -np.log(p.max(1))
    tol = 5 * G.E24 * np.abs(x).max(1) * (pt == 0) + 16 * G.E24 * (1 + np.log(V))
    lp, H, stats, status = vce.ce_logprobs_forward(z, ids, tau)
    assert vce.vce_get_status(status) == 0
    one = vce.policy_loss_forward_backward(z, ids, torch.ones(6, device="cuda"), temperature=tau, reduction="none")
    two = vce.policy_loss_forward_backward(z, ids, torch.ones(6, device="cuda"), temperature=tau, reduction="none",
                                           entropy_coef=0.5, want_entropy=True)
    for l, h in ((lp, H), (one[2], None), (two[2], two[3])):
        G.near(host(l), want, tol, "log-probabilities")
        if h is not None:
            G.near(host(h), ent, np.full(6, 16 * G.E24 * (1 + np.log(V))), "entropies")
    hot = np.zeros(p.shape)
    hot[np.arange(6), t] = 1.0
    grad = (hot - p) / tau
    eps = torch.finfo(dtype).eps
    for got, g64 in ((vce.ce_logprobs_backward(z, ids, stats, torch.ones(6, device="cuda"), None, tau), grad),
                     (one[4], -grad), (two[4], -grad)):
        # 16 roundings of factors of size log V, and the output's
        G.near(host(got), g64, 16 * G.E24 * (1 + np.log(V)) * (p + hot) / tau + eps / 2 * np.abs(g64) * 1.01, "gradient")


@pytest.mark.parametrize("V,dtype", [(600, F32), (20001, BF16), (128256, BF16), (300001, F32)])
@pytest.mark.parametrize("tau", [1e-30, 1e-12, 1e-9, 1e-7, 1e-4, 1e6, 1e20, 1e37])
def test_temperatures_of_every_size(vce, V, dtype, tau):
    """The largest logits share all of the mass, or all columns do.  What a log-probability is off by: the products'
    roundings, as above, and an even row's handful."""
    tau = float(np.float32(tau))
    g = torch.Generator().manual_seed(V)
    z = (2 * torch.randn(5, V, generator=g)).to(dtype).cuda()
    ids = torch.randint(0, V, (5,), generator=g).cuda()
    ids[0] = z[0].argmax()
    z[1, 7] = z[1, int(ids[1])] = 12.0
    z[2, int(ids[2])] = 11.0
    z[3] = -3.0
    x = host(z) / tau
    x = x - x.max(1, keepdims=True)
    e = np.exp(x)
    p = e / e.sum(1, keepdims=True)
    t = ids.cpu().numpy()
    want = x[np.arange(5), t] - np.log(e.sum(1))
    size = np.abs(host(z) / tau).max(1)
    tol = 5 * G.E24 * np.maximum(np.abs(want), size * (p[np.arange(5), t] < 0.999)) + 16 * G.E24 * (1 + np.log(V))
    lp, H, stats, status = vce.ce_logprobs_forward(z, ids, tau)
    assert vce.vce_get_status(status) == 0
    one = vce.policy_loss_forward_backward(z, ids, torch.ones(5, device="cuda"), temperature=tau, reduction="none",
                                           grad_dtype=F32)
    hot = np.zeros(p.shape)
    hot[np.arange(5), t] = 1.0
    for l in (lp, one[2]):
        G.near(host(l), want, tol, "log-probabilities")
    # exponents up to 110 matter, each off by what z / tau rounds by
    rel = 5 * G.E24 * np.minimum(size, 110.0)[:, None] + 64 * G.E24 * (1 + np.log(V))
    got = vce.ce_logprobs_backward(z, ids, stats, torch.ones(5, device="cuda"), None, tau, grad_dtype=F32)
    for g64, sign in ((got, 1.0), (one[4], -1.0)):
        G.near(sign * host(g64) * tau, hot - p, rel * np.where(hot > 0, 1 - p + 1e-30, p) * 2 + 1e-37 * max(tau, 1.0) + 1e-30,
               "gradient")
    assert np.all(np.isfinite(host(H))) and np.all(host(H) >= 0) and np.all(host(H) <= np.log(V) * 1.000001)
