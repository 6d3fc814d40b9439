"""The cross-entropy of rows with masked columns, -inf or finite: both calls, the one pass and chunks, against 64 bits.

A loss is off by at most lse_tol of the unmasked logits and 8 roundings of their size; a gradient p_j - [j = t] by twice
that of itself, and its output's rounding."""
import math

import pytest
import torch

from tests._logits_grading import E24, lse_tol

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def rows(V, dtype, low, T=7):
    """The first half masked; every second column; all but a few; all but the target; the target too; the last half; the
    first and last thirds."""
    g = torch.Generator().manual_seed(V)
    z = (2 * torch.randn(T, V, generator=g)).to(dtype).cuda()
    ids = torch.randint(V // 2 + 1, V - 1, (T,), generator=g).cuda()
    for i in range(0, T - 6, 7):
        z[i, : V // 2] = low
        z[i + 1, ::2] = low
        ids[i + 1] |= 1
        keep = z[i + 2, V // 2:V // 2 + 9].clone()
        z[i + 2] = low
        z[i + 2, V // 2:V // 2 + 9] = keep
        ids[i + 2] = V // 2 + 4
        z[i + 3] = low
        z[i + 3, int(ids[i + 3])] = 0.75
        z[i + 4, : V // 2] = low
        z[i + 4, int(ids[i + 4])] = low
        z[i + 5, V // 2:] = low
        ids[i + 5] = 3
        z[i + 6, : V // 3] = low
        z[i + 6, V - V // 3:] = low
        ids[i + 6] = V // 2
    return z, ids


@pytest.mark.parametrize("T,V,dtype", [(7, 40, F32), (7, 600, BF16), (7, 20001, BF16), (7, 40000, F32), (7, 128256, BF16),
                                       (7, 300001, F32), (700, 4003, BF16), (350, 32000, BF16), (700, 128, F32)])
@pytest.mark.parametrize("low", [-math.inf, -1e10, -1e12, -1e30, None])
def test_masked_columns(vce, T, V, dtype, low):
    low = torch.finfo(dtype).min if low is None else low
    z, ids = rows(V, dtype, low, T)
    z64 = z.double()
    logp = z64 - z64.logsumexp(1, keepdim=True)
    at = ids[:, None]
    want = -logp.gather(1, at)[:, 0]
    p = logp.exp()
    grad = p.clone()
    grad.scatter_add_(1, at, -torch.ones_like(want)[:, None])
    # a target that holds all of the mass: 1 - p_t
    zmax = float(z64[z64.abs() < 1e6].abs().max())
    tol = lse_tol(zmax, 1.0) + 8 * E24 * (2 * zmax + 17)
    big = want > 1e6
    eps = torch.finfo(dtype).eps
    one = torch.ones(T, device="cuda")
    loss, per_row, stats, status = vce.ce_forward(z, ids, reduction="none")
    two = vce.ce_backward(z, ids, stats, one, reduction="none")
    _, r1, _, g1, s1 = vce.ce_forward_backward(z, ids, reduction="none", grad_output=one)
    cut = V // 3
    chunks = [z[:, :cut].contiguous(), z[:, cut:2 * cut].contiguous(), z[:, 2 * cut:].contiguous()]
    _, rc, _, gc, _, sc = vce.ce_merge_chunks(chunks, ids, reduction="none", grad_output=one)
    for r, g, s in ((per_row, two, status), (r1, g1, s1), (rc, torch.cat(gc, 1), sc)):
        assert vce.vce_get_status(s) == 0
        r = r.double()
        assert torch.all((r - want).abs()[~big] <= tol)
        assert torch.all(((r - want).abs() <= 8 * E24 * want)[big] | torch.isinf(want[big]) & torch.isinf(r[big]))
        hot = torch.zeros_like(p)
        hot.scatter_(1, at, 1.0)
        bound = 2 * tol * p + tol * hot + (eps / 2 * 1.01) * grad.abs() + 1e-30
        assert torch.all((g.double() - grad).abs() <= bound)


@pytest.mark.parametrize("V,dtype", [(40, F32), (600, BF16), (20001, BF16), (40000, F32), (128256, BF16), (300001, F32)])
@pytest.mark.parametrize("low", [-1e10, -1e30, None])
def test_nothing_but_finite_masks_is_nan(vce, V, dtype, low):
    z = torch.full((3, V), torch.finfo(dtype).min if low is None else low, dtype=dtype, device="cuda")
    z[1] = torch.randn(V, device="cuda").to(dtype)
    ids = torch.tensor([V // 2, 1, V - 1], device="cuda")
    one = torch.ones(3, device="cuda")
    _, r, stats, status = vce.ce_forward(z, ids, reduction="none")
    g = vce.ce_backward(z, ids, stats, one, reduction="none")
    _, r1, _, g1, _ = vce.ce_forward_backward(z, ids, reduction="none", grad_output=one)
    for x, y in ((r, g), (r1, g1)):
        assert x.isnan().tolist() == [True, False, True]
        assert y[0].isnan().any() and y[2].isnan().any() and torch.isfinite(y[1]).all()
