"""The fp64 oracle of the operators around the cross-entropy, pinned by closed forms, by the
cross-entropy oracle and by differences (no GPU), and the operators' refusals that need none."""
import ctypes
import inspect

import numpy as np
import pytest
import torch

from oracle import ce_oracle as CE
from oracle import logits_oracle as L


def test_topk_orders_ties_by_column_and_drops_minus_infinity():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0], [-np.inf] * 5, [0.0, 0.0, 0.0, 0.0, 0.0]])
    values, ids, full, tail = L.topk(z, 4)
    assert ids.tolist() == [[1, 2, 4, 0], [-1] * 4, [0, 1, 2, 3]]
    assert values[0].tolist() == [3, 3, 2, 1] and np.all(values[1] == -np.inf)
    assert tail[0] == -np.inf and full[1] == -np.inf and tail[2] == 0.0
    assert full[2] == pytest.approx(np.log(5.0))


def test_distill_with_one_entry_is_the_cross_entropy():
    rng = np.random.default_rng(1)
    z = rng.normal(size=(6, 40)) * 3
    labels = rng.integers(0, 40, 6)
    labels[2] = -100
    ref = CE.ce(z, labels, "mean")
    ids = labels[:, None].copy()
    ids[2] = -1
    got = L.distill(z, ids, rng.normal(size=(6, 1)))
    np.testing.assert_allclose(got["loss_rows"], ref["loss_rows"], rtol=1e-12, atol=1e-15)
    np.testing.assert_allclose(got["grad"], ref["grad"], rtol=1e-11, atol=1e-15)


def test_distill_of_the_teacher_itself_is_zero():
    rng = np.random.default_rng(2)
    z = rng.normal(size=(3, 50)) * 2
    values, ids, _, tail = L.topk(z, 7, 2.0)
    got = L.distill(z, ids, values, tail, 2.0)
    np.testing.assert_allclose(got["loss_rows"], 0.0, atol=1e-13)
    np.testing.assert_allclose(got["grad"], 0.0, atol=1e-15)


@pytest.mark.parametrize("with_tail,tau", [(True, 1.0), (True, 3.0), (False, 2.0)])
def test_distill_gradient_against_differences(with_tail, tau):
    rng = np.random.default_rng(3)
    T, V, K = 4, 23, 5
    z = rng.normal(size=(T, V)) * 2
    t, ids, _, tail = L.topk(rng.normal(size=(T, V)) * 2, K, tau)
    ids[1, 3:] = -1
    ids[2, 0] = -1
    tail = tail if with_tail else None
    g = L.distill(z, ids, t, tail, tau)["grad"]
    h = 1e-5
    for i in range(T):
        for j in range(V):
            up, down = z.copy(), z.copy()
            up[i, j] += h
            down[i, j] -= h
            d = (L.distill(up, ids, t, tail, tau)["loss_out"] - L.distill(down, ids, t, tail, tau)["loss_out"]) / (2 * h)
            assert abs(d - g[i, j]) < 1e-9, (i, j)
    np.testing.assert_allclose(g.sum(1), 0.0, atol=1e-14)


def test_process_against_hand_values_and_differences():
    z = np.array([[2.0, -2.0, 1.0, 0.5, 3.0]])
    kw = dict(temperature=[0.5], repetition=[2.0], history=[[0, 1, 1, 3]], prompt_lens=[1], allowed=np.array([[1, 1, 1, 1, 0]], bool))
    y, _ = L.process(z, frequency=[0.25], presence=[0.125], bias=[{2: 4.0}], **kw)
    # 0: prompt only; 1: twice behind it; 3: once
    assert y[0].tolist() == [2.0, (-4.0 - 0.5 - 0.125) / 0.5, 10.0, (0.25 - 0.25 - 0.125) / 0.5, -np.inf]
    up = np.array([[1.0, 1.0, 1.0, 1.0, 1.0]])
    g, _ = L.process(z, upstream=up, **kw)
    assert g[0].tolist() == [1.0, 4.0, 2.0, 1.0, 0.0]
    assert L.pack_mask(np.array([[1] * 31 + [0] + [0, 1]], bool)).tolist() == [[0x7FFFFFFF, 2]]


# ---- refusals that come before any CUDA call ---------------------------------------------------


@pytest.fixture(scope="module")
def vce():
    from vocab_cross_entropy_gb300 import build
    build.build()
    import vocab_cross_entropy_gb300 as v
    return v


def test_refusals_of_the_library(vce):
    x = 0x1000
    lib = vce.lib
    topk = lambda dt=1, T=4, V=64, ld=64, K=8, tau=1.0, p=x, v=x: lib.ce_topk(p, dt, T, V, ld, K, tau, v, x, x, x, None)
    assert topk(dt=3) == -2
    assert topk(T=-1) == -3 and topk(V=0) == -3 and topk(V=2097153, ld=2097153) == -3
    assert topk(K=0) == -8 and topk(K=65) == -8 and topk(V=1000, ld=1000, K=257) == -8
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-39):
        assert topk(tau=tau) == -8, tau
    assert topk(ld=63) == -4
    assert topk(T=0, p=None, v=None) == 0
    assert topk(p=None) == -1 and topk(v=x + 2) == -5

    def fwd(dt=1, T=4, V=64, ld=64, ids=x, tv=x, tdt=0, K=8, tau=1.0, red=2, loss_out=x, stats=x, top=x, status=x):
        return lib.ce_distill_forward(x, dt, T, V, ld, ids, tv, tdt, None, K, tau, None, -100, red, x, loss_out, stats,
                                      top, status, None)
    assert fwd(dt=2) == -2 and fwd(tdt=5) == -2 and fwd(red=3) == -2
    assert fwd(K=0) == -8 and fwd(K=65) == -8 and fwd(tau=0.0) == -8 and fwd(ld=1) == -4
    assert fwd(ids=None) == -1 and fwd(tv=None) == -1 and fwd(loss_out=None) == -1 and fwd(top=None) == -1
    assert fwd(status=None) == -1 and fwd(stats=x + 8) == -5 and fwd(T=8388609) == -3

    def bwd(ids=x, K=8, go=x, grad=0x900000, gdt=1, gld=64):
        return lib.ce_distill_backward(x, 1, 4, 64, 64, ids, K, 1.0, 2, x, x, go, grad, gdt, gld, None)
    assert bwd(gdt=7) == -2 and bwd(gld=63) == -4 and bwd(go=None) == -1 and bwd(K=300) == -8
    assert bwd(grad=x) == -8 and bwd(grad=x + 500) == -8        # over the logits

    def one(go=x, grad=0x900000, loss_out=x):
        return lib.ce_distill_forward_backward(x, 1, 4, 64, 64, x, x, 0, None, 8, 1.0, None, -100, 2, go, x, loss_out, x,
                                               grad, 1, 64, x, None)
    assert one(go=None) == -1 and one(loss_out=None) == -1 and one(grad=x) == -8

    def proc(dt=1, T=4, V=64, ld=64, temp=None, rep=None, hist=None, n=0, off=None, bias=None, bv=None, boff=None,
             mask=None, mld=2, out=0x900000, odt=1, old=64, rs=x):
        return lib.logits_process(x, dt, T, V, ld, temp, rep, None, None, hist, n, off, None, bias, bv, 0, boff, mask,
                                  mld, out, odt, old, rs, None)
    assert proc(dt=9) == -2 and proc(odt=9) == -2 and proc(V=0) == -3 and proc(ld=63) == -4 and proc(old=63) == -4
    assert proc(mask=x, mld=1) == -4 and proc(hist=x) == -1 and proc(bias=x, boff=x) == -1 and proc(off=x) == -1
    assert proc(rep=x) == -1                                     # a penalty without a history
    assert proc(out=x) == -8 and proc(out=x, odt=0) == -8 and proc(out=x + 2) == -8 and proc(out=x, old=65) == -8
    assert proc(rs=None) == -1 and proc(temp=x + 2) == -5 and proc(n=-1) == -3 and proc(T=0) == 0

    def procb(z=0x900000, grad=0x1900000, hist=x, off=x, ld=64):
        return lib.logits_process_backward(x, 1, 4, 64, 64, z, 1, ld, None, None, hist, 0, off, None, 0, grad, 1, 64, x,
                                           None)
    assert procb(z=None) == -1 and procb(ld=60) == -4 and procb(grad=0x900000) == -8 and procb(grad=x) == -8


def test_refusals_of_the_wrappers(vce):
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        vce.ce_topk(z, 2)
    with pytest.raises(TypeError, match="dtype"):
        vce.ce_topk(z.double(), 2)
    with pytest.raises(ValueError, match="2-D"):
        vce.logits_process(z[0])
    with pytest.raises(ValueError, match="unit column stride"):
        vce.ce_distill_forward(z.t(), torch.zeros(8, 1, dtype=torch.int64), torch.zeros(8, 1))
    with pytest.raises(TypeError, match="takes no out"):
        vce.process_logits(z, out=z)


def test_status_texts(vce):
    for code in (2, 3, 4):
        assert vce.vce_status_string(code) != "unknown status"


def test_exported(vce):
    for name in ("ce_topk", "ce_distill_forward", "ce_distill_backward", "ce_distill_forward_backward",
                 "distill_cross_entropy", "logits_process", "logits_process_backward", "process_logits"):
        assert name in vce.__all__ and inspect.getdoc(getattr(vce, name))
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_refusals_of_the_give_up_hooks(vce):
    x, lib = 0x1000, vce.lib
    topk = lambda ns=50_000_000, V=64: lib.vce_test_topk_stall(x, 4, V, 8, x, x, x, x, ns, None)
    assert topk(ns=999_999) == -8 and topk(ns=2_000_000_001) == -8 and topk(V=0) == -3
    one = lambda ns=50_000_000, status=x: lib.vce_test_distill_stall(x, 4, 64, x, x, 8, x, x, x, x, 0x900000, ns, status,
                                                                     None)
    assert one(ns=999_999) == -8 and one(ns=2_000_000_001) == -8 and one(status=None) == -1
    bwd = lambda ns=50_000_000, go=x: lib.vce_test_distill_bwd_stall(x, 4, 64, x, 8, x, x, go, 0x900000, ns, None)
    assert bwd(ns=999_999) == -8 and bwd(ns=2_000_000_001) == -8 and bwd(go=None) == -1


def test_teachers_of_more_entries_than_32_bits_are_refused(vce):
    """Entries beyond 2^31 (of tensors without storage) before anything else of the teacher is looked at."""
    from vocab_cross_entropy_gb300 import logits_ops
    ids = torch.empty(1, 2 ** 32 + 5, dtype=torch.int64, device="meta")
    with pytest.raises(ValueError, match="expected 1 to 256"):
        logits_ops._teacher(ids, ids.float(), None, 1, torch.device("cuda", 0))
