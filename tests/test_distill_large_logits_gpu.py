"""Distillation of students whose masks are finite, from -1e10 to the type's lowest value, at several temperatures, and
of logits of 1e11, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import logits_oracle as L
from tests import _logits_grading as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def student(T, V, K, dtype, seed):
    """Logits, and a teacher near them: ids in the row's second half, values, the others' log-sum-exp over tau."""
    g = torch.Generator().manual_seed(seed + V)
    z = (2 * torch.randn(T, V, generator=g)).to(dtype)
    ids = torch.stack([V // 2 + torch.randperm(V - V // 2, generator=g)[:K] for _ in range(T)])
    values = z.gather(1, ids).float() + torch.randn(T, K, generator=g)
    return z.cuda(), ids.cuda(), values.cuda(), torch.randn(T, generator=g).cuda()


def check(vce, z, ids, values, tail, tau, zmax, lost=()):
    """Masks count as -inf; rows of nothing else have no gradient; the rows `lost` are NaN throughout."""
    z64 = host(z)
    z64[z64 * 1.4426950408889634 / tau <= -2.0 ** 31] = -np.inf
    dead = np.isneginf(z64).all(1)
    live = ~dead
    live[list(lost)] = False
    n = lambda t: None if t is None else t[torch.from_numpy(live).cuda()]
    ref = L.distill(z64[live], n(ids).cpu().numpy(), host(n(values)), host(n(tail)), tau, None, "sum", 1.0)
    size = (zmax, max(float(values.abs().max()), 0.0 if tail is None else float(tail.abs().max()) * tau), tau)
    up = torch.ones(1, device="cuda")
    _, rows, stats, tops, status = vce.ce_distill_forward(z, ids, values, tail, tau, reduction="sum")
    two = vce.ce_distill_backward(z, ids, stats, tops, up, tau, "sum")
    _, r1, one, s1 = vce.ce_distill_forward_backward(z, ids, values, tail, tau, reduction="sum", grad_output=up)
    eps = torch.finfo(z.dtype).eps if z.dtype is BF16 else 2.0 ** -23
    for r, g, s in ((rows, two, status), (r1, one, s1)):
        assert vce.vce_get_status(s) == 0
        r, g = host(r), host(g)
        assert np.isnan(r[dead]).all() and np.all(g[dead] == 0)
        assert np.isnan(r[list(lost)]).all() and np.isnan(g[list(lost)]).all()
        G.check_distill_loss(r[live], ref, *size)
        G.check_distill_grad(g[live], ref, *size, eps)


def masked(V, dtype, low, seed):
    """The first half masked; every second column; all of the tail; the entries; one open column in the tail and none
    among the entries; everything; the entries and the tail's first half."""
    z, ids, values, tail = student(7, V, 4, dtype, seed)
    z[0, : V // 2] = low
    z[1, ::2] = low
    top = z.gather(1, ids)
    z[2] = low
    z[2, ids[2]] = top[2]
    z[3, ids[3]] = low
    z[4] = low
    z[4, 1] = 0.5
    z[5] = low
    z[6, : V // 2] = low
    z[6, ids[6]] = low
    return z, ids, values, tail


@pytest.mark.parametrize("V,dtype", [(300, F32), (20000, BF16), (70001, F32), (128256, BF16), (900001, BF16), (450000, F32)])
@pytest.mark.parametrize("tau", [0.7, 1.0, 2.0])
@pytest.mark.parametrize("low", [-1e10, -1e12, -1e30, None])
@pytest.mark.parametrize("with_tail", [True, False])
def test_finite_masks(vce, V, dtype, tau, low, with_tail):
    low = torch.finfo(dtype).min if low is None else low
    z, ids, values, tail = masked(V, dtype, low, 0)
    zmax = float(z.float()[z.float().abs() < 1e6].abs().max())
    check(vce, z, ids, values, tail if with_tail else None, tau, zmax)


@pytest.mark.parametrize("V,dtype", [(300, F32), (20000, BF16), (70001, F32), (900001, BF16)])
@pytest.mark.parametrize("size", [1e11, 1e30])
def test_great_logits(vce, V, dtype, size):
    """An entry far above the others has all the mass; among the other columns such a logit makes the row NaN."""
    z, ids, values, tail = student(4, V, 4, dtype, 1)
    z[0] = size
    z[1, int(ids[1, 2])] = size
    z[2, 3] = z[2, V // 2 - 2] = size
    z[3, 0] = size
    values[1, 2] = 500.0                    # which the teacher is sure of, too: else the loss is of that size
    check(vce, z, ids, values, tail, 1.0, 10.0, lost=(0, 2, 3))


@pytest.mark.parametrize("V,dtype", [(700, F32), (20000, BF16), (70001, F32)])
def test_products_below_the_border(vce, V, dtype):
    """A temperature whose products stay below 2^31: losses of the size of the logits' differences times it, off by 64
    roundings of the largest logit."""
    tau = float(np.float32(6e-9))
    g = torch.Generator().manual_seed(V)
    z = (2 * torch.randn(5, V, generator=g)).clamp(-8, 8).to(dtype).cuda()
    z[:, 1] = torch.tensor([7.75, -7.75, 7.5, 3.0, 8.0])
    z[1] -= 8 + z[1].max()
    z[1].clamp_(min=-8)
    ids = torch.stack([torch.randperm(V, generator=g)[:4] for _ in range(5)]).cuda()
    values = torch.randn(5, 4, generator=g).cuda()
    ref = L.distill(host(z), ids.cpu().numpy(), host(values), None, tau, None, "sum", 1.0)
    _, rows, stats, tops, status = vce.ce_distill_forward(z, ids, values, None, tau, reduction="sum")
    _, r1, one, s1 = vce.ce_distill_forward_backward(z, ids, values, None, tau, reduction="sum",
                                                    grad_output=torch.ones(1, device="cuda"))
    for r, s in ((rows, status), (r1, s1)):
        assert vce.vce_get_status(s) == 0
        assert np.all(np.abs(host(r) - ref["loss_rows"]) <= 64 * G.E24 * 8 * tau)
    assert torch.isfinite(one).all()
