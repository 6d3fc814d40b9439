"""Top K of rows whose masks are finite, from -1e10 to the type's lowest value, at several temperatures, and of logits of
1e11, against the fp64 oracle."""
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


def check(vce, z, k, tau):
    z64 = z.double().cpu().numpy()
    values, ids, lse, tail = L.topk(z64, k, tau)
    got = [t.double().cpu().numpy() for t in vce.ce_topk(z, k, tau)]
    assert np.array_equal(got[0], values) and np.array_equal(got[1], ids)
    normal = np.abs(z64[np.abs(z64) < 1e6])
    zmax = normal.max() if normal.size else 0.0
    for g, w in ((got[2], lse), (got[3], tail)):
        big = np.abs(w) > 1e6
        G.check_lse(g[~big], w[~big], zmax, tau)
        # of logits of that size: the roundings of log2(e) / temperature, the product, ln 2, and the result's
        low = w[big] < -float(torch.finfo(F32).max)
        assert np.all(np.isneginf(g[big][low]))
        assert np.all(np.abs(g[big] - w[big])[~low] <= 6 * G.E24 * np.abs(w[big])[~low])


@pytest.mark.parametrize("T,V,dtype", [(7, 90, F32), (7, 9001, BF16), (7, 128256, F32), (399, 20000, BF16), (399, 9001, F32)])
@pytest.mark.parametrize("tau", [0.7, 1.0, 2.0])
@pytest.mark.parametrize("low", [-1e10, -1e12, -1e30, None])
def test_finite_masks(vce, T, V, dtype, tau, low):
    """The first half masked; every second column; fewer than K left; one left; none; the last half; a block of them."""
    low = torch.finfo(dtype).min if low is None else low
    g = torch.Generator().manual_seed(V)
    z = (2 * torch.randn(T, V, generator=g)).to(dtype).cuda()
    for i in range(0, T, 7):
        z[i, : V // 2] = low
        z[i + 1, ::2] = low
        keep = z[i + 2, 3:12].clone()
        z[i + 2] = low
        z[i + 2, 3:12] = keep
        z[i + 3] = low
        z[i + 3, V // 3] = 1.25
        z[i + 4] = low
        z[i + 5, V // 2:] = low
        z[i + 6, V // 4: V // 2] = low
    check(vce, z, 20, tau)


@pytest.mark.parametrize("T,V,dtype", [(4, 90, F32), (4, 9001, BF16), (400, 20000, BF16)])
@pytest.mark.parametrize("size", [1e11, -1e11])
def test_great_logits(vce, T, V, dtype, size):
    """All alike; a few among the K; more than K of them; two sizes of them."""
    g = torch.Generator().manual_seed(V)
    z = (2 * torch.randn(T, V, generator=g)).to(dtype).cuda()
    for i in range(0, T, 4):
        z[i] = size
        z[i + 1, 2:9] = size
        z[i + 2, 10:60] = size
        z[i + 3] = size
        z[i + 3, 5:50] = size * 2
    check(vce, z, 20, 1.0)
