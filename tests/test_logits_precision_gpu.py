"""Top K and distillation against the fp64 oracle on inputs that leave rounding little room: tolerances
near what fp32 arithmetic does, so that a sum in fewer bits, a vector left out or one counted twice
shows, also in the partial vectors at a row's ends.

Inputs.  Temperature 1.  Odd columns hold 8, even ones values of [4, 8], the first and the last column of a
row 12.  So a kernel's partial sums (of a thread, a stage, a warp, a slice) refer to 8 or to 12, and
differences of references are exact (within a factor of two) or zero.

Units of 2^-24, relative error of a sum of 2^(z k2 - m), which is the absolute error of its logarithm:
  k2 rounded                        12   (max z)
  the fma's rounding                 8   (|z k2 - m| <= 8 log2 e, times ln 2)
  the hardware exponential          16   (2^-22 each; a term's own, and at most three rescalings: 4..8 -> 8 -> 12,
                                          and a group's to its thread's reference)
  a group's maximum times k2        12   (12 log2 e, times ln 2)
  additions                        100   (5 in a thread's tree, 64 stages, 5 lanes, 8 warps, 8 blocks, candidates)
SUM = 148.  A row's log-sum-exp is below 24; its logarithm, product and sum add 3 x 24: LSE = 220.
The average vector of eight columns among 128256 carries 1000 units, a row's first or last column
11000 among 128256 and 1600 among 900001.

Distillation without a teacher's tail, K entries elsewhere:
  ws = p_T / P    SUM + 40 (the entries' sum: its exponentials' arguments and K additions; one more factor)
  loss            x = log P, |x| <= 16: ws's error and 2 roundings of 16 in the logarithms; the entries' part
                  is a mean of (y, e^y) with y within 60; sums and products 30 of the loss
  tail gradient   SUM, 12, ws times P; bias = M + log2 S (below 40): 2 x 28 for its logarithm and sum; the
                  fma's argument below 30: 21; the exponential 4; products 6: 290 of p
  entries         Q (r - q) - p_T r, r = p / P: 60 (r + q) and ws's error of p
"""
import numpy as np
import pytest
import torch

from oracle import logits_oracle as L

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
UNIT = 2.0 ** -24
SUM, LSE = 148, 220
CASES = [(3, 128256, BF16, 0, 0), (3, 128257, F32, 2, 1), (330, 128256, BF16, 0, 0), (330, 33001, BF16, 4, 3),
         (330, 16385, F32, 3, 2), (2, 900001, BF16, 5, 5), (2, 450001, F32, 1, 0)]


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def flat(T, V, dtype, pad, left):
    g = torch.Generator(device="cuda").manual_seed(T + V)
    z = torch.empty(T, V + pad, dtype=dtype, device="cuda")[:, left:left + V]
    z.copy_(4.0 + 4.0 * torch.rand(T, V, generator=g, device="cuda"))
    z[:, 1::2] = 8.0
    z[:, 0] = z[:, V - 1] = 12.0
    return z


def sample(T):
    return sorted({0, 1, T // 2, T - 1})


@pytest.mark.parametrize("T,V,dtype,pad,left", CASES)
def test_topk_to_rounding(vce, T, V, dtype, pad, left):
    z = flat(T, V, dtype, pad, left)
    values, ids, lse, tail = vce.ce_topk(z, 16)
    rows = sample(T)
    rv, ri, rl, rt = L.topk(z[rows].double().cpu().numpy(), 16)
    assert np.array_equal(ids[rows].cpu().numpy(), ri)
    assert np.array_equal(values[rows].double().cpu().numpy(), rv)
    for got, want in ((lse, rl), (tail, rt)):
        err = np.abs(got[rows].double().cpu().numpy() - want)
        assert np.all(err <= LSE * UNIT), f"{err.max() / UNIT:.0f} units"


@pytest.mark.parametrize("T,V,dtype,pad,left", CASES)
def test_distill_to_rounding(vce, T, V, dtype, pad, left):
    K = 8
    z = flat(T, V, dtype, pad, left)
    g = torch.Generator().manual_seed(T + V)
    ids = (torch.randperm(V - 2, generator=g)[:T * K] if T * K < V - 2 else
           torch.stack([torch.randperm(V - 2, generator=g)[:K] for _ in range(T)])).reshape(T, K).add(1).cuda()
    values = torch.randn(T, K, generator=g).cuda()
    rows = sample(T)
    ref = L.distill(z[rows].double().cpu().numpy(), ids[rows].cpu().numpy(), values[rows].double().cpu().numpy(),
                    reduction="sum")
    at = np.arange(len(rows))[:, None], ids[rows].cpu().numpy()
    p, q, kl = ref["p"], ref["q"], ref["kl"]
    assert np.all(-np.log(p[at].sum(1)) < 16)
    tol = 290 * p
    P = p[at].sum(1, keepdims=True)
    tol[at] = 60 * (p[at] / P + q[at]) + 200 * p[at]
    loss_tol = UNIT * (SUM + 40 + 32 + 60 + 30 * kl)
    up = torch.ones(1, device="cuda")
    _, l2, stats, tops, _ = vce.ce_distill_forward(z, ids, values, reduction="sum")
    g2 = vce.ce_distill_backward(z, ids, stats, tops, up, reduction="sum", grad_dtype=F32)
    _, l1, g1, _ = vce.ce_distill_forward_backward(z, ids, values, reduction="sum", grad_output=up, grad_dtype=F32)
    for loss, grad in ((l2, g2), (l1, g1)):
        err = np.abs(loss[rows].double().cpu().numpy() - ref["loss_rows"])
        assert np.all(err <= loss_tol), f"loss: {np.max(err / loss_tol):.2f} of the tolerance"
        err = np.abs(grad[rows].double().cpu().numpy() - (p - q))
        assert np.all(err <= UNIT * tol), f"gradient: {np.max(err / (UNIT * tol)):.2f} of the tolerance"
