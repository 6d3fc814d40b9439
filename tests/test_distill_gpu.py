"""The distillation loss and its gradient on the GPU (two calls, one pass, autograd) against the fp64
oracle, within the tolerances derived in tests/_logits_grading.py."""
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


class Case:
    """Student logits (a matrix inside a wider one), teacher entries and labels; near: the teacher is
    the student plus noise of that size."""

    def __init__(self, T, V, K, dtype=BF16, tau=1.0, tail=True, near=1.0, tdtype=F32, pad=0, left=0, seed=0):
        g = torch.Generator().manual_seed(seed + T + V + K)
        full = (2.0 * torch.randn(T, V + pad, generator=g)).to(dtype)
        self.z = full.cuda()[:, left:left + V]
        t = full[:, left:left + V].double() + near * torch.randn(T, V, generator=g).double()
        tv, ids, _, rest = L.topk(t.numpy(), K, tau)
        self.values = torch.from_numpy(tv).to(tdtype).cuda()
        self.ids = torch.from_numpy(ids).cuda()
        self.tail = torch.from_numpy(rest).to(F32).cuda() if tail else None
        self.labels = None
        self.tau = tau

    def teacher(self):
        return self.ids, self.values, self.tail, self.tau, self.labels

    def oracle(self, reduction, go=1.0):
        host = lambda x: None if x is None else x.detach().double().cpu().numpy()
        v = host(self.values)
        v = np.where(self.ids.cpu().numpy() >= 0, v, -np.inf)
        return L.distill(host(self.z), self.ids.cpu().numpy(), v, host(self.tail), self.tau,
                         None if self.labels is None else self.labels.cpu().numpy(), reduction, go)

    def sizes(self):
        z, t = self.z.float(), self.values.float()
        fin = lambda x: float(x[torch.isfinite(x)].abs().max()) if torch.isfinite(x).any() else 0.0
        tmax = fin(t)
        if self.tail is not None:
            tmax = max(tmax, fin(self.tail) * self.tau)
        return fin(z), tmax, self.tau


def check(vce, c, reduction="mean", gdtype=None, go=None):
    """Both calls and the one pass against the oracle.  go: an upstream gradient per row or a number."""
    T = c.z.shape[0]
    per_row = reduction == "none"
    if go is None:
        go = np.linspace(0.5, 1.5, T) if per_row else 1.0
    up = torch.as_tensor(np.atleast_1d(go), dtype=F32, device="cuda")
    ref = c.oracle(reduction, up.cpu().double().numpy())
    gdtype = gdtype or c.z.dtype
    eps = torch.finfo(gdtype).eps if gdtype is BF16 else 2.0 ** -23
    loss, rows, stats, tops, status = vce.ce_distill_forward(c.z, *c.teacher(), reduction=reduction)
    assert vce.vce_get_status(status) == 0
    G.check_distill_loss(rows.cpu(), ref, *c.sizes())
    grad = vce.ce_distill_backward(c.z, c.ids, stats, tops, up, c.tau, reduction, grad_dtype=gdtype)
    G.check_distill_grad(grad.double().cpu(), ref, *c.sizes(), eps)
    l1, r1, g1, s1 = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction=reduction, grad_output=up,
                                                    grad_dtype=gdtype)
    assert vce.vce_get_status(s1) == 0
    G.check_distill_loss(r1.cpu(), ref, *c.sizes())
    G.check_distill_grad(g1.double().cpu(), ref, *c.sizes(), eps)
    if per_row:
        assert loss is None and l1 is None
        return
    for got, r in ((loss, rows), (l1, r1)):   # the sum of the rows it wrote: compensated, one rounding
        total = r.double().sum().item() / (max(ref["n"], 1) if reduction == "mean" else 1)
        if ref["n"] == 0 and reduction == "mean":
            assert np.isnan(got.item())
        else:
            assert abs(got.item() - total) <= 2.0 ** -23 * abs(total)


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("T,V,K,dtype,tau", [
    (1, 1, 1, F32, 1.0), (3, 2, 2, BF16, 1.0), (5, 9, 1, BF16, 2.0), (64, 1000, 8, F32, 1.0), (33, 1003, 256, BF16, 2.0),
    (6, 8192, 64, BF16, 4.0), (20, 32001, 100, BF16, 1.0), (2, 128256, 64, BF16, 2.0), (3, 70000, 32, F32, 1.0),
    (1, 300001, 20, F32, 1.0), (700, 600, 33, BF16, 1.0)])
def test_distill(vce, T, V, K, dtype, tau, tail):
    check(vce, Case(T, V, K, dtype, tau, tail))


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_distill_types_and_reductions(vce, dtype, gdtype, reduction):
    check(vce, Case(17, 5000, 12, dtype, 1.5, True, tdtype=BF16), reduction, gdtype)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("V,pad,left", [(4001, 0, 0), (4001, 6, 3), (4096, 1, 1), (4100, 4, 4), (33000, 5, 2)])
def test_distill_layouts(vce, V, pad, left, dtype, gdtype):
    check(vce, Case(7, V, 20, dtype, 1.0, True, pad=pad, left=left), "sum", gdtype, go=0.75)


@pytest.mark.parametrize("gdtype,pad,left", [(BF16, 3, 1), (F32, 2, 2), (BF16, 8, 0)])
def test_distill_gradient_layouts(vce, gdtype, pad, left):
    """A gradient inside a wider matrix, aligned unlike the logits: the columns around it stay."""
    T, V = 6, 9001
    c = Case(T, V, 10, BF16, 2.0, True)
    full = torch.full((T, V + pad), 7.0, dtype=gdtype, device="cuda")
    grad = full[:, left:left + V]
    up = torch.ones(1, device="cuda")
    ref = c.oracle("mean")
    eps = torch.finfo(gdtype).eps
    for one_pass in (False, True):
        full.fill_(7.0)
        if one_pass:
            vce.ce_distill_forward_backward(c.z, *c.teacher(), grad_output=up, grad_logits=grad)
        else:
            _, _, stats, tops, _ = vce.ce_distill_forward(c.z, *c.teacher())
            vce.ce_distill_backward(c.z, c.ids, stats, tops, up, c.tau, grad_logits=grad)
        G.check_distill_grad(grad.double().cpu(), ref, *c.sizes(), eps)
        assert torch.all(full[:, :left] == 7.0) and torch.all(full[:, left + V:] == 7.0)


@pytest.mark.parametrize("near", [0.0, 1e-3, 30.0])
@pytest.mark.parametrize("tail", [True, False])
def test_distill_near_and_far_teachers(vce, near, tail):
    """A student that matches its teacher (losses far below the rounding of its log-probabilities), and
    one that is far off."""
    check(vce, Case(9, 3000, 16, F32, 1.0, tail, near=near))


def test_distill_confident_student(vce):
    """One column with margins of 17 to 90: the tail's mass is far below fp32's resolution at 1, and the
    losses 1e-8 to 1e-39 keep their relative accuracy (K = 1: the cross-entropy's collapse regime)."""
    c = Case(8, 4000, 1, F32, 1.0, False)
    rows = torch.arange(8, device="cuda")
    margins = torch.linspace(17, 80, 8, device="cuda")
    c.z[rows, c.ids[:, 0]] = c.z.amax(1) + margins
    ref = c.oracle("none")
    loss = vce.ce_distill_forward(c.z, *c.teacher(), reduction="none")[1].double().cpu().numpy()
    assert np.all(np.abs(loss - ref["loss_rows"]) <= 1e-4 * ref["loss_rows"]) and np.all(loss > 0)
    ce = vce.ce_forward(c.z.contiguous(), c.ids[:, 0].contiguous(), reduction="none")[1].double().cpu().numpy()
    assert np.all(np.abs(loss - ce) <= 1e-4 * ce)
    g = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction="none")[2]
    top = g.gather(1, c.ids)[:, 0].double().cpu().numpy()
    assert np.all(np.abs(top + ref["loss_rows"]) <= 1e-4 * ref["loss_rows"])   # -(1 - p), p near 1
    check(vce, c, "sum")


def test_distill_ragged_and_ignored_rows(vce):
    c = Case(12, 2500, 9, BF16, 2.0, True)
    c.ids[1, 4:] = -1            # fewer entries
    c.ids[2, 1] = -1             # a gap
    c.ids[3] = -1                # no teacher
    c.ids[4, 1:] = -1            # one entry
    c.labels = torch.arange(12, device="cuda") % 50
    c.labels[[0, 7]] = -100
    c.z[3] = float("nan")        # an ignored row's logits do not matter
    c.z[7] = float("inf")
    keep = c.z.clone()
    c.z[3], c.z[7] = 0.0, 0.0
    refs = {r: c.oracle(r) for r in ("mean", "sum")}
    c.z.copy_(keep)
    size = (float(keep[0].float().abs().max()) + 8.0, 30.0, 2.0)
    for r, ref in refs.items():
        up = torch.ones(1, device="cuda")
        loss, rows, stats, tops, status = vce.ce_distill_forward(c.z, *c.teacher(), reduction=r)
        assert vce.vce_get_status(status) == 0
        G.check_distill_loss(rows.cpu(), ref, *size)
        assert abs(loss.item() - ref["loss_out"]) <= 1e-4 * ref["loss_out"]
        assert torch.all(tops[3] == 0) and torch.all(stats[3] == 0) and torch.all(stats[7] == 0)
        g = vce.ce_distill_backward(c.z, c.ids, stats, tops, up, c.tau, r)
        G.check_distill_grad(g.double().cpu(), ref, *size, 2.0 ** -7)
        g = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction=r)[2]
        G.check_distill_grad(g.double().cpu(), ref, *size, 2.0 ** -7)


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_distill_with_every_row_ignored(vce, reduction):
    c = Case(4, 300, 3)
    c.ids[:, 0] = -1
    check(vce, c, reduction)


def test_distill_masked_students(vce):
    """-inf logits: among the tail, on entries (infinite loss where q > 0), all of the tail, all of the
    entries, and a row of nothing else."""
    inf = float("inf")
    c = Case(7, 600, 4, F32, 1.0, True)
    cols = torch.arange(600, device="cuda")
    c.z[0, ::3] = -inf
    c.z[0, c.ids[0]] = 1.0
    c.z[1, c.ids[1, 2]] = -inf
    c.values[2, 1:] = -inf                          # a teacher entry without mass on a masked logit
    c.z[2, c.ids[2, 1]] = -inf
    is_top = torch.zeros(600, dtype=torch.bool, device="cuda")
    is_top[c.ids[3]] = True
    c.z[3][~is_top] = -inf                          # nothing left in the tail, which has mass
    c.z[4, c.ids[4]] = -inf                         # nothing left among the entries
    c.tail[5] = -inf
    is_top = torch.zeros(600, dtype=torch.bool, device="cuda")
    is_top[c.ids[5]] = True
    c.z[5][~is_top] = -inf                          # nothing left in a tail without mass: finite
    assert cols.numel() == 600
    rows = [0, 1, 2, 3, 4, 5]
    live = Case.__new__(Case)
    live.z, live.ids, live.values, live.tail = c.z[rows], c.ids[rows], c.values[rows], c.tail[rows]
    live.labels, live.tau = None, 1.0
    ref = live.oracle("sum")
    loss, r, stats, tops, status = vce.ce_distill_forward(live.z, *live.teacher(), reduction="sum")
    assert vce.vce_get_status(status) == 0 and loss.item() == inf
    G.check_distill_loss(r.cpu(), ref, *live.sizes())
    assert [bool(np.isinf(x)) for x in ref["loss_rows"]] == [False, True, False, True, True, False]
    up = torch.ones(1, device="cuda")
    g2 = vce.ce_distill_backward(live.z, live.ids, stats, tops, up, 1.0, "sum")
    g1 = vce.ce_distill_forward_backward(live.z, *live.teacher(), reduction="sum")[2]
    for g in (g1, g2):
        G.check_distill_grad(g.double().cpu(), ref, *live.sizes(), 2.0 ** -23)
    c.z[6] = -inf                                   # no student at all: NaN, and no gradient
    loss, r, g, status = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction="sum")
    assert vce.vce_get_status(status) == 0
    assert torch.isnan(r[6]) and torch.all(g[6] == 0)


def test_distill_bad_teachers(vce):
    """Ids out of range or twice in a row, and teachers without finite mass: a status, a NaN loss, no
    gradient; the other rows are not touched by it."""
    good = Case(8, 20000, 6, BF16, 1.0, True)
    ref = good.oracle("sum")
    for what in range(6):
        c = Case(8, 20000, 6, BF16, 1.0, True)
        if what == 0:
            c.ids[3, 2] = 20000
        elif what == 1:
            c.ids[3, 0] = -2
        elif what == 2:
            c.ids[3, 5] = c.ids[3, 1]
        elif what == 3:
            c.values[3] = -float("inf")
            c.tail[3] = -float("inf")
        elif what == 4:
            c.values[3, 1] = float("nan")
        else:
            c.tail[3] = float("inf")
        loss, rows, stats, tops, status = vce.ce_distill_forward(c.z, *c.teacher(), reduction="sum")
        assert vce.vce_get_status(status) == 2 and torch.isnan(loss).all(), what
        assert torch.isnan(rows).nonzero().flatten().tolist() == [3]
        up = torch.ones(1, device="cuda")
        g2 = vce.ce_distill_backward(c.z, c.ids, stats, tops, up, 1.0, "sum")
        l1, r1, g1, s1 = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction="sum")
        assert vce.vce_get_status(s1) == 2 and torch.isnan(r1).nonzero().flatten().tolist() == [3]
        others = [0, 1, 2, 4, 5, 6, 7]
        part = {k: (v[others] if isinstance(v, np.ndarray) else v) for k, v in ref.items()}
        for g in (g1, g2):
            assert torch.all(g[3] == 0), what
            G.check_distill_grad(g[others].double().cpu(), part, *good.sizes(), 2.0 ** -7)


@pytest.mark.parametrize("T,V,K,dtype,pad,left", [
    (700, 20000, 256, BF16, 0, 0),     # short rows of several stages, most entries
    (650, 17001, 40, F32, 3, 1), (1300, 2500, 7, BF16, 1, 0),
    (330, 70001, 100, BF16, 0, 0), (320, 40000, 200, F32, 2, 1)])   # rows of 128 KB and more
def test_distill_several_rows_a_block(vce, T, V, K, dtype, pad, left):
    c = Case(T, V, K, dtype, 2.0, True, pad=pad, left=left)
    c.labels = torch.arange(T, device="cuda") % 50 + 1
    c.labels[::7] = -100
    c.labels[40:80] = -100             # more ignored rows in a row than a warp looks ahead
    c.ids[5::11, K // 2:] = -1
    c.ids[3::13] = -1
    check(vce, c)
    check(vce, c, "none", BF16 if dtype is F32 else F32)


@pytest.mark.parametrize("V,dtype", [(900001, BF16), (450000, F32)])
def test_distill_rows_longer_than_shared_memory(vce, V, dtype):
    check(vce, Case(3, V, 40, dtype, 1.0, True))
    c = Case(2, V, 3, dtype, 1.0, True)
    c.ids[0, 2] = c.ids[0, 1]               # a refused row of that length ends cleanly too
    _, rows, g, status = vce.ce_distill_forward_backward(c.z, *c.teacher())
    assert vce.vce_get_status(status) == 2 and torch.isnan(rows[0]) and torch.all(g[0] == 0)


def test_distill_same_bits_every_time(vce):
    c = Case(200, 40001, 64, BF16, 2.0, True)
    up = torch.ones(1, device="cuda")
    def both():
        loss, rows, stats, tops, _ = vce.ce_distill_forward(c.z, *c.teacher())
        return (loss, rows, stats, tops, vce.ce_distill_backward(c.z, c.ids, stats, tops, up, c.tau),
                *vce.ce_distill_forward_backward(c.z, *c.teacher(), grad_output=up)[:3])
    first = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(both(), first))


def test_distill_autograd(vce):
    for reduction in ("mean", "sum", "none"):
        c = Case(10, 3001, 7, F32, 2.0, True)
        z = c.z.clone().requires_grad_(True)
        loss = vce.distill_cross_entropy(z, *c.teacher(), reduction=reduction)
        up = torch.linspace(0.5, 2, 10, device="cuda") if reduction == "none" else torch.tensor(0.7, device="cuda")
        loss.backward(up.expand(loss.shape))
        ref = c.oracle(reduction, up.double().cpu().numpy())
        G.check_distill_grad(z.grad.double().cpu(), ref, *c.sizes(), 2.0 ** -23)
    # against differences of the fp64 loss
    want = c.z.double().cpu().numpy()
    i, j, h = 3, int(c.ids[3, 2]), 1e-4
    f = lambda d: (lambda zz: (zz.__setitem__((i, j), zz[i, j] + d), L.distill(
        zz, c.ids.cpu().numpy(), c.values.double().cpu().numpy(), c.tail.double().cpu().numpy(), 2.0)["loss_rows"][i])[1])(want.copy())
    diff = (f(h) - f(-h)) / (2 * h) * float(up[i])
    assert abs(z.grad[i, j].item() - diff) <= 1e-4 * abs(diff) + 1e-7


def test_distill_streams_and_graphs(vce):
    c, d = Case(30, 30001, 16, BF16, 1.0, True), Case(30, 30001, 16, BF16, 1.0, True, seed=9)
    up = torch.ones(1, device="cuda")
    want = {id(x): vce.ce_distill_forward_backward(x.z, *x.teacher(), grad_output=up) for x in (c, d)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [(x, vce.ce_distill_forward_backward(x.z, *x.teacher(), grad_output=up, stream=s))
           for x, s in zip((c, d, c, d), streams)]
    torch.cuda.synchronize()
    for x, g in got:
        assert all(torch.equal(a, b) for a, b in zip(g[:3], want[id(x)][:3]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, rows, stats, tops, status = vce.ce_distill_forward(c.z, *c.teacher())
        grad = vce.ce_distill_backward(c.z, c.ids, stats, tops, up)
    for name in ("ids", "values", "tail"):
        getattr(c, name).copy_(getattr(d, name))
    c.z.copy_(d.z)
    graph.replay()
    fresh = vce.ce_distill_forward(d.z, *d.teacher())
    assert torch.equal(loss, fresh[0]) and torch.equal(rows, fresh[1])
    assert torch.equal(grad, vce.ce_distill_backward(d.z, d.ids, fresh[2], fresh[3], up))


def test_distill_autograd_in_a_graph(vce):
    """Forward and backward captured together, replayed with new contents."""
    c, d = Case(9, 3001, 7, BF16, 2.0, True), Case(9, 3001, 7, BF16, 2.0, True, seed=9)
    z = c.z.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        vce.distill_cross_entropy(z, *c.teacher()).backward()
    torch.cuda.current_stream().wait_stream(side)
    z.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = vce.distill_cross_entropy(z, *c.teacher())
        loss.backward()
    with torch.no_grad():
        z.copy_(d.z)
    for name in ("ids", "values", "tail"):
        getattr(c, name).copy_(getattr(d, name))
    graph.replay()
    fresh = d.z.clone().requires_grad_(True)
    want = vce.distill_cross_entropy(fresh, *d.teacher())
    want.backward()
    assert torch.equal(loss, want) and torch.equal(z.grad, fresh.grad)


def test_distill_refusals(vce):
    c = Case(4, 100, 5)
    go = torch.ones(1, device="cuda")
    with pytest.raises(vce.VceError):
        vce.ce_distill_forward(c.z, c.ids, c.values, temperature=0.0)
    with pytest.raises(TypeError):
        vce.ce_distill_forward(c.z, c.ids.int(), c.values)
    with pytest.raises(ValueError):
        vce.ce_distill_forward(c.z, c.ids, c.values[:, :4])
    with pytest.raises(ValueError):
        vce.ce_distill_forward(c.z, c.ids, c.values, c.tail[:3])
    with pytest.raises(TypeError):
        vce.ce_distill_forward(c.z, c.ids, c.values.half())
    with pytest.raises(ValueError):
        vce.ce_distill_forward_backward(c.z, c.ids, c.values, grad_output=torch.ones(4, device="cuda"))
    with pytest.raises(vce.VceError):
        vce.ce_distill_forward_backward(c.z, c.ids, c.values, grad_output=go, grad_logits=c.z)
    with pytest.raises(ValueError):
        vce.ce_distill_forward(c.z, c.ids.cpu(), c.values)
    out = vce.ce_distill_forward_backward(c.z[:0], c.ids[:0], c.values[:0], reduction="sum")
    assert out[0].item() == 0 and out[2].shape == (0, 100) and vce.vce_get_status(out[3]) == 0


@pytest.mark.parametrize("V,dtype", [(600, F32), (20000, BF16), (70001, BF16), (900001, BF16), (450000, F32)])
@pytest.mark.parametrize("tail", [True, False])
def test_distill_nan_and_infinite_students(vce, V, dtype, tail):
    """NaN or +inf among a student's logits, in the tail or on an entry, alone among -inf too: the row's
    loss and its whole gradient are NaN, whatever kernel takes it, and the other rows are as they were."""
    nan, inf = float("nan"), float("inf")
    c = Case(8, V, 5, dtype, 1.0, tail)
    ref = c.oracle("sum")
    free = [next(j for j in range(V // 2 + 7, V) if j not in c.ids[i].tolist()) for i in range(8)]
    c.z[1, free[1]] = nan
    c.z[2, c.ids[2, 3]] = nan
    c.z[3, free[3]] = inf
    c.z[4, c.ids[4, 0]] = inf
    keep = c.z[5, c.ids[5]].clone()
    c.z[5] = -inf                                   # NaN, and nothing else, in the tail
    c.z[5, c.ids[5]] = keep
    c.z[5, free[5]] = nan
    c.z[6, c.ids[6]] = nan                          # every entry
    bad, good = [1, 2, 3, 4, 5, 6], [0, 7]
    up = torch.ones(1, device="cuda")
    loss, rows, stats, tops, status = vce.ce_distill_forward(c.z, *c.teacher(), reduction="sum")
    g2 = vce.ce_distill_backward(c.z, c.ids, stats, tops, up, c.tau, "sum")
    l1, r1, g1, s1 = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction="sum", grad_output=up)
    size = (float(c.z[good].float().abs().max()), *c.sizes()[1:])
    part = {k: (v[good] if isinstance(v, np.ndarray) and v.ndim else v) for k, v in ref.items()}
    for l, r, g, s in ((loss, rows, g2, status), (l1, r1, g1, s1)):
        assert vce.vce_get_status(s) == 0 and torch.isnan(l).all()
        assert torch.isnan(r).nonzero().flatten().tolist() == bad
        assert torch.isnan(g[bad]).all()
        G.check_distill_loss(r[good].cpu(), part, *size)
        G.check_distill_grad(g[good].double().cpu(), part, *size, 2.0 ** -7 if dtype is BF16 else 2.0 ** -23)
    assert torch.isnan(tops[bad]).all() and not torch.isnan(tops[good]).any()


@pytest.mark.parametrize("V,dtype", [(300, F32), (20000, BF16), (70001, F32), (900001, BF16), (450000, F32)])
@pytest.mark.parametrize("tail", [True, False])
def test_distill_students_of_the_lowest_value(vce, V, dtype, tail):
    """A student row whose mask (the type's lowest value) leaves nothing is a row of nothing else, as one
    of -inf: NaN loss, no gradient.  Such masks beside open columns carry no mass."""
    low = torch.finfo(dtype).min
    c = Case(4, V, 4, dtype, 1.0, tail)
    c.z[1] = low
    c.z[2, ::2] = low
    c.z[2, c.ids[2]] = 1.0
    clean = c.z.clone()
    c.z[1] = 0.0
    c.z[2] = torch.where(c.z[2] == low, -float("inf"), c.z[2])
    ref, size = c.oracle("sum"), c.sizes()
    c.z.copy_(clean)
    good = [0, 2, 3]
    part = {k: (v[good] if isinstance(v, np.ndarray) and v.ndim else v) for k, v in ref.items()}
    up = torch.ones(1, device="cuda")
    loss, rows, stats, tops, status = vce.ce_distill_forward(c.z, *c.teacher(), reduction="sum")
    g2 = vce.ce_distill_backward(c.z, c.ids, stats, tops, up, c.tau, "sum")
    l1, r1, g1, s1 = vce.ce_distill_forward_backward(c.z, *c.teacher(), reduction="sum", grad_output=up)
    for r, g, s in ((rows, g2, status), (r1, g1, s1)):
        assert vce.vce_get_status(s) == 0
        assert torch.isnan(r).nonzero().flatten().tolist() == [1] and torch.all(g[1] == 0)
        G.check_distill_loss(r[good].cpu(), part, *size)
        G.check_distill_grad(g[good].double().cpu(), part, *size, 2.0 ** -7 if dtype is BF16 else 2.0 ** -23)


@pytest.mark.parametrize("T", [1, 2, 9])
@pytest.mark.parametrize("V,dtype", [(900001, BF16), (450000, F32)])
def test_distill_long_rows_that_are_all_ignored_or_refused(vce, V, dtype, T):
    """MEAN over rows longer than shared memory none of which has a gradient: NaN whatever ran when, not
    the count's 1 / N, which uses the same word before."""
    g = torch.Generator().manual_seed(V + T)
    z = torch.randn(T, V, generator=g).to(dtype).cuda()
    ids = torch.randint(0, V // 2, (T, 3), generator=g).cuda()
    ids[:, 1] = ids[:, 0] + V // 4
    values = torch.randn(T, 3, generator=g).cuda()
    grad = torch.empty_like(z)
    loss = torch.empty(1, device="cuda")
    for first, status in ((-1, 0), (V, 2)):
        bad = ids.clone()
        bad[:, 0] = first
        for _ in range(20):
            loss.fill_(5.0)
            grad.fill_(5.0)
            out = vce.ce_distill_forward_backward(z, bad, values, loss_out=loss, grad_logits=grad)
            assert torch.isnan(loss).all() and vce.vce_get_status(out[3]) == status
            assert torch.all(grad == 0)
            assert torch.all(out[1] == 0) if first == -1 else torch.isnan(out[1]).all()


@pytest.mark.parametrize("T,V", [(3, 70000), (2, 20000), (400, 9000), (2, 900000)])
def test_distill_waits_that_give_up_are_reported(vce, T, V):
    """The last block of every cluster waits in vain for what its gradient needs, once the statistics
    have been exchanged and the first block has its losses: a status, NaN losses, and a context that
    stays usable."""
    c = Case(T, V, 5, BF16, 1.0, False)
    z = c.z.contiguous()
    loss, rows, _, status = vce.vce_test_distill_stall(z, c.ids, c.values)
    code = vce.vce_get_status(status)
    assert 105 <= code <= 109 and "gave up" in vce.vce_status_string(code)
    assert torch.isnan(rows).all() and torch.isnan(loss).all()
    check(vce, c, "sum")


@pytest.mark.parametrize("T,V", [(3, 20000), (5, 100000)])
def test_distill_backward_waits_that_give_up_leave_nan(vce, T, V):
    c = Case(T, V, 5, BF16, 1.0, False)
    z = c.z.contiguous()
    _, _, stats, tops, _ = vce.ce_distill_forward(z, *c.teacher(), reduction="sum")
    want = vce.ce_distill_backward(z, c.ids, stats, tops, torch.ones(1, device="cuda"), 1.0, "sum")
    got = vce.vce_test_distill_bwd_stall(z, c.ids, stats, tops)
    vectors = V // 8                                  # both are multiples of 8: rows of whole vectors
    parts = -(-vectors // 4096)
    last = -(-vectors // parts) * (parts - 1) * 8     # the first column of the last block
    assert torch.isnan(got[:, last:]).all() and torch.equal(got[:, :last], want[:, :last])
    again = vce.ce_distill_backward(z, c.ids, stats, tops, torch.ones(1, device="cuda"), 1.0, "sum")
    assert torch.equal(again, want)


@pytest.mark.parametrize("T,V,dtype,gdtype,pad,left", [
    (2, 900001, BF16, BF16, 5, 5), (2, 900001, BF16, F32, 5, 5), (3, 450001, F32, BF16, 2, 1),
    (300, 70001, BF16, F32, 1, 0), (700, 20001, BF16, BF16, 4, 3)])
def test_distill_gradients_whose_stores_back_up(vce, T, V, dtype, gdtype, pad, left):
    """Rows that no vector store fits keep a thread's reads of a stage waiting behind its stores: no
    stage may be copied over before they are done.  The one pass against the two calls, again and again."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.empty(T, V + pad, dtype=dtype, device="cuda")[:, left:left + V]
    z.copy_(4.0 + 4.0 * torch.rand(T, V, generator=g, device="cuda"))
    ids = torch.randint(0, V // 8, (T, 8), generator=g, device="cuda") * 8 + torch.arange(8, device="cuda")
    values = torch.randn(T, 8, generator=g, device="cuda")
    up = torch.ones(1, device="cuda")
    _, _, stats, tops, status = vce.ce_distill_forward(z, ids, values, reduction="sum")
    assert vce.vce_get_status(status) == 0
    want = vce.ce_distill_backward(z, ids, stats, tops, up, reduction="sum", grad_dtype=gdtype).float()
    # p = e^(z - L') p_T of both, in fp32, their log-sum-exps by other kernels: 2e-5 relative (the two sums' 2 x
    # 150 units of 2^-24, as in the tests to rounding), and a rounding of each to the gradient's type
    tol = (2e-5 + (torch.finfo(gdtype).eps if gdtype is BF16 else 0.0)) * want.abs() + 1e-12
    # the entries are differences: within 2e-5 of the larger of p and q, at most 1
    tol.scatter_(1, ids, 2e-5 + (torch.finfo(gdtype).eps if gdtype is BF16 else 0.0) * want.gather(1, ids).abs())
    for _ in range(12):
        got = vce.ce_distill_forward_backward(z, ids, values, reduction="sum", grad_output=up, grad_dtype=gdtype)[2]
        assert torch.all((got.float() - want).abs() <= tol)
