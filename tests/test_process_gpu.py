"""logits_process and its gradient on the GPU against the fp64 oracle, and the operators in a row: a
teacher's masked top K into a student's distillation, and a decoded token."""
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
    def __init__(self, T, V, dtype=BF16, history=40, bias=5, mask=True, params=True, pad=0, left=0, seed=0):
        rng = np.random.default_rng(seed + T + V)
        full = torch.from_numpy(rng.normal(size=(T, V + pad)) * 2).to(dtype).cuda()
        self.z = full[:, left:left + V]
        self.T, self.V = T, V
        f32 = lambda x: x.astype(np.float32)
        self.temp, self.rep = f32(rng.uniform(0.5, 1.5, T)), f32(rng.uniform(1.0, 1.5, T))
        self.freq, self.pres = f32(rng.uniform(-0.2, 0.5, T)), f32(rng.uniform(0, 0.4, T))
        if not params:
            self.temp = self.rep = self.freq = self.pres = None
        self.hist = self.prompt = self.bias = self.allowed = None
        if history:
            lens = rng.integers(0, history + 1, T)
            lens[-1] = history
            pool = rng.integers(0, V, 12)
            pool[0], pool[1] = 0, V - 1
            self.hist = [np.where(rng.random(n) < 0.6, rng.choice(pool, n), rng.integers(0, V, n)) for n in lens]
            self.prompt = np.minimum(rng.integers(0, history, T), lens)
        if bias:
            self.bias = []
            for i in range(T):
                cols = set(rng.choice(V, min(V, rng.integers(0, bias + 1)), replace=False).tolist())
                if self.hist is not None and len(self.hist[i]):
                    cols.add(int(self.hist[i][0]))          # a biased column with a history
                self.bias.append({c: float(np.float32(rng.normal() * 3)) for c in sorted(cols)})
        if mask:
            p = np.where(np.arange(T) % 3 == 0, 0.95, 20 / V)[:, None]
            self.allowed = rng.random((T, V)) < p
            if T > 4:
                self.allowed[4] = False

    def kwargs(self, backward=False):
        dev = lambda x, t=None: None if x is None else torch.as_tensor(x, dtype=t).cuda()
        kw = dict(temperature=dev(self.temp))
        if self.hist is not None:
            kw.update(repetition_penalty=dev(self.rep), history_ids=dev(np.concatenate(self.hist), torch.int64),
                      history_offsets=dev(np.concatenate([[0], np.cumsum([len(h) for h in self.hist])]), torch.int64))
            if not backward:
                kw.update(frequency_penalty=dev(self.freq), presence_penalty=dev(self.pres),
                          prompt_lens=dev(self.prompt, torch.int64))
        if self.bias is not None and not backward:
            ids = [c for b in self.bias for c in b]
            kw.update(bias_ids=dev(np.array(ids, np.int64)),
                      bias_values=dev(np.array([v for b in self.bias for v in b.values()], np.float32)),
                      bias_offsets=dev(np.concatenate([[0], np.cumsum([len(b) for b in self.bias])]), torch.int64))
        if self.allowed is not None:
            kw.update(mask=torch.from_numpy(L.pack_mask(self.allowed)).cuda())
        return kw

    def oracle(self, upstream=None, z=None):
        z = (self.z if z is None else z).double().cpu().numpy()
        up = None if upstream is None else upstream.double().cpu().numpy()
        return L.process(z, temperature=self.temp, repetition=self.rep, frequency=self.freq, presence=self.pres,
                         history=self.hist, prompt_lens=self.prompt, bias=self.bias, allowed=self.allowed, upstream=up)


EPS = {BF16: 2.0 ** -7, F32: 2.0 ** -23}


def check(vce, c, odtype=None):
    odtype = odtype or c.z.dtype
    want, size = c.oracle()
    out, status = vce.logits_process(c.z, out_dtype=odtype, **c.kwargs())
    assert out.dtype is odtype and torch.all(status == 0)
    G.check_processed(out.double().cpu().numpy(), want, size, EPS[odtype])


@pytest.mark.parametrize("T,V,history,bias,mask", [
    (1, 1, 3, 1, False), (2, 5, 9, 2, True), (6, 33, 50, 4, True), (9, 1000, 0, 0, True), (9, 1000, 0, 0, False),
    (9, 1000, 30, 0, False), (9, 1000, 0, 6, False), (1, 128256, 1777, 16, True), (5, 32001, 5000, 40, True),
    (300, 2000, 60, 3, True), (2, 300000, 900, 100, True), (1, 1050001, 2000, 20, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_process(vce, T, V, history, bias, mask, dtype):
    check(vce, Case(T, V, dtype, history, bias, mask))


@pytest.mark.parametrize("dtype,odtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("V,pad,left", [(4000, 0, 0), (4001, 0, 0), (4001, 5, 3), (4096, 3, 1), (20000, 4, 4)])
def test_process_layouts(vce, V, pad, left, dtype, odtype):
    check(vce, Case(7, V, dtype, 100, 10, True, pad=pad, left=left), odtype)


def test_process_history_lengths(vce):
    """Rows of no token to many in one call: hash tables of every size, and windows of columns for the
    rows that are too long for them."""
    for V, lens in ((40000, [0, 1, 47, 48, 49, 383, 384, 385, 3000, 12288, 12289, 60000]), (70001, [0] * 40 + [9000]),
                    (33, [0, 500, 2000]), (9000, [5000, 30000])):
        c = Case(len(lens), V, BF16, 8, 3, True)
        rng = np.random.default_rng(V)
        c.hist = [rng.integers(0, V, n) if i % 2 else rng.integers(0, min(V, 700), n) for i, n in enumerate(lens)]
        c.prompt = np.array([n // 3 for n in lens])
        check(vce, c, F32)
        up = torch.randn(c.T, V, device="cuda").to(BF16)
        want, size = c.oracle(up)
        g, status = vce.logits_process_backward(up, c.z, grad_dtype=F32, **c.kwargs(backward=True))
        assert torch.all(status == 0)
        G.check_processed(g.double().cpu().numpy(), want, size, EPS[F32])


@pytest.mark.parametrize("dtype,odtype", [(BF16, F32), (F32, BF16), (F32, F32)])
def test_process_output_inside_a_wider_matrix(vce, dtype, odtype):
    T, V = 5, 3001
    c = Case(T, V, dtype, 50, 5, True)
    want, size = c.oracle()
    full = torch.full((T, V + 9), 7.0, dtype=odtype, device="cuda")
    out, _ = vce.logits_process(c.z, out=full[:, 4:4 + V], **c.kwargs())
    G.check_processed(out.double().cpu().numpy(), want, size, EPS[odtype])
    assert torch.all(full[:, :4] == 7) and torch.all(full[:, 4 + V:] == 7)


def test_process_masked_logits_do_not_matter(vce):
    """NaN and infinities in masked columns, the type's lowest value in open ones."""
    c = Case(6, 3000, F32, 30, 4, True)
    masked = torch.from_numpy(~c.allowed).cuda()
    clean = c.z.clone()
    c.z[masked] = float("nan")
    c.z[:, 1::2] = torch.where(masked[:, 1::2], float("inf"), c.z[:, 1::2])
    want, size = c.oracle(z=torch.where(masked, 0.0, clean))
    out, _ = vce.logits_process(c.z, **c.kwargs())
    G.check_processed(out.double().cpu().numpy(), want, size, EPS[F32])
    low = torch.full((2, 100), -float("inf"), device="cuda")
    out, _ = vce.logits_process(low, temperature=torch.tensor([0.5, 2.0], device="cuda"))
    assert torch.all(out == -float("inf"))


@pytest.mark.parametrize("T,V,history,mask,dtype,gdtype", [
    (3, 7, 9, True, F32, F32), (40, 1001, 30, True, BF16, BF16), (5, 32001, 3000, True, BF16, F32),
    (5, 32000, 0, True, F32, BF16), (2, 128256, 500, False, BF16, BF16)])
def test_process_backward(vce, T, V, history, mask, dtype, gdtype):
    c = Case(T, V, dtype, history, 0, mask)
    up = torch.randn(T, V, generator=torch.Generator().manual_seed(V)).to(gdtype).cuda()
    want, size = c.oracle(up)
    g, status = vce.logits_process_backward(up, c.z, **c.kwargs(backward=True))
    assert g.dtype is dtype and torch.all(status == 0)
    G.check_processed(g.double().cpu().numpy(), want, size, EPS[dtype])


def test_process_autograd(vce):
    for history, bias in ((50, 4), (0, 0), (0, 4)):
        c = Case(8, 901, F32, history, bias, True)
        z = c.z.clone().requires_grad_(True)
        y = vce.process_logits(z, **c.kwargs())
        w = torch.randn(901, device="cuda")
        open_ = torch.from_numpy(c.allowed).cuda()
        torch.where(open_, y * w, 0.0).sum().backward()
        want, size = c.oracle((open_ * w).float())
        G.check_processed(z.grad.double().cpu().numpy(), want, size, EPS[F32])
    z = c.z.clone().requires_grad_(True)
    vce.process_logits(z, temperature=torch.full((8,), 2.0, device="cuda")).sum().backward()   # an expanded gradient
    assert torch.all(z.grad == 0.5)


def test_process_row_statuses(vce):
    T, V = 7, 5000
    c = Case(T, V, F32, 20, 3, False)
    want, size = c.oracle()
    kw = c.kwargs()
    off = kw["history_offsets"].tolist()
    rows = {}
    if off[2] > off[1]:
        kw["history_ids"][off[1]] = V
        rows[1] = 1
    kw["temperature"][2], rows[2] = 0.0, 3
    kw["temperature"][3], rows[3] = float("nan"), 3
    kw["repetition_penalty"][4], rows[4] = -1.0, 3
    out, status = vce.logits_process(c.z, **kw)
    assert {i: s for i, s in enumerate(status.tolist()) if s} == rows
    good = [i for i in range(T) if i not in rows]
    G.check_processed(out[good].double().cpu().numpy(), want[good], size[good], EPS[F32])

    kw = c.kwargs()
    b = kw["bias_offsets"].tolist()
    i = next(i for i in range(T) if b[i + 1] - b[i] >= 2)
    kw["bias_ids"][b[i] + 1] = kw["bias_ids"][b[i]]            # the same column twice
    _, status = vce.logits_process(c.z, **kw)
    assert {j: s for j, s in enumerate(status.tolist()) if s} == {i: 1}

    kw = c.kwargs()
    kw["history_offsets"][T] = 10 ** 15                         # past the list
    kw["history_offsets"][0] = -5
    _, status = vce.logits_process(c.z, **kw)
    assert status.tolist() == [4, 0, 0, 0, 0, 0, 4]


def test_process_streams_graphs_and_order(vce):
    """At once on several streams, replayed from a graph with new contents, and the same bits each time
    (the counts are integers)."""
    c, d = Case(20, 32001, BF16, 3000, 20, True), Case(20, 32001, BF16, 3000, 20, True, seed=1)
    kw = c.kwargs()
    want = vce.logits_process(c.z, **kw)[0]
    torch.cuda.synchronize()
    outs = [vce.logits_process(c.z, stream=torch.cuda.Stream(), **kw)[0] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held, status = vce.logits_process(c.z, **kw)
    c.z.copy_(d.z)
    kw["temperature"].fill_(2.0)
    graph.replay()
    assert torch.equal(held, vce.logits_process(d.z, **kw)[0]) and torch.all(status == 0)


def test_process_refusals(vce):
    c = Case(4, 100, F32, 10, 2, True)
    kw = c.kwargs()
    bad = lambda **k: dict(kw, **k)
    with pytest.raises(ValueError):
        vce.logits_process(c.z, **bad(history_offsets=None))
    with pytest.raises(ValueError):
        vce.logits_process(c.z, **bad(bias_values=None))
    with pytest.raises(ValueError):
        vce.logits_process(c.z, **bad(mask=kw["mask"][:, :3]))
    with pytest.raises(TypeError):
        vce.logits_process(c.z, **bad(mask=kw["mask"].to(torch.int64)))
    with pytest.raises(TypeError):
        vce.logits_process(c.z, **bad(history_ids=kw["history_ids"].int()))
    with pytest.raises(ValueError):
        vce.logits_process(c.z, **bad(temperature=kw["temperature"][:2]))
    with pytest.raises(vce.VceError):
        vce.logits_process(c.z, repetition_penalty=kw["repetition_penalty"])
    for over in (c.z, torch.cat([c.z, c.z])[2:6]):
        with pytest.raises(vce.VceError):
            vce.logits_process(over, out=over)
    with pytest.raises(vce.VceError):
        vce.logits_process_backward(c.z, c.z.clone(), grad_logits=c.z)
    with pytest.raises(vce.VceError):
        vce.logits_process(c.z, out=c.z.view(-1).view(BF16)[:400].view(4, 100))
    with pytest.raises(vce.VceError):
        vce.logits_process_backward(c.z, None, **c.kwargs(backward=True))
    out, status = vce.logits_process(c.z[:0], temperature=kw["temperature"][:0])
    assert out.shape == (0, 100) and status.shape == (0,)


def test_a_teachers_masked_top_k_into_a_student(vce):
    """Teacher logits processed and reduced to their top K, the student distilled from them and trained
    through its own temperature and mask: every step against the oracle of its own inputs."""
    T, V, K, tau = 24, 8003, 30, 2.0
    teacher, student = Case(T, V, BF16, 0, 0, True, seed=3), Case(T, V, BF16, 0, 0, False, seed=4)
    teacher.allowed[:, :2000] = True
    teacher.allowed[4] = False                    # a teacher without a column left
    zt, status = vce.logits_process(teacher.z, out_dtype=F32, mask=teacher.kwargs()["mask"])
    values, ids, _, tail = vce.ce_topk(zt, K, tau)
    rv, ri, _, rt = L.topk(zt.double().cpu().numpy(), K, tau)
    assert np.array_equal(ids.cpu().numpy(), ri) and torch.all(ids[4] == -1) and torch.all(status == 0)
    z = student.z.clone().requires_grad_(True)
    y = vce.process_logits(z, temperature=torch.full((T,), 0.8, device="cuda"), out_dtype=F32)
    y.retain_grad()
    loss = vce.distill_cross_entropy(y, ids, values, tail, tau)
    loss.backward()
    ref = L.distill(y.detach().double().cpu().numpy(), ri, rv, tail.double().cpu().numpy(), tau)
    assert ref["n"] == T - 1
    zmax = float(y.detach().abs().max())
    tmax = max(float(zt[torch.isfinite(zt)].abs().max()), float(tail[torch.isfinite(tail)].abs().max()) * tau)
    assert abs(loss.item() - ref["loss_out"]) <= 1e-4 * ref["loss_out"]
    G.check_distill_grad(y.grad.double().cpu(), ref, zmax, tmax, tau, 2.0 ** -23)
    want = y.grad.double().cpu().numpy() / float(np.float32(0.8))
    G.check_processed(z.grad.double().cpu().numpy(), want, np.abs(want), EPS[BF16])


def test_a_decoded_token(vce):
    """One token of a batch: its processed logits, then the best tokens with their log-probabilities."""
    c = Case(6, 128256, BF16, 500, 10, True, seed=5)
    out, status = vce.logits_process(c.z, out_dtype=F32, **c.kwargs())
    values, ids, lse, _ = vce.ce_topk(out, 5)
    host = out.double().cpu().numpy()
    rv, ri, rl, _ = L.topk(host, 5)
    assert np.array_equal(ids.cpu().numpy(), ri) and np.array_equal(values.double().cpu().numpy(), rv)
    open_ = np.isfinite(rl)
    assert (~open_).sum() == 1 and torch.all(status == 0)          # the row with nothing allowed
    logp = (values - lse[:, None]).double().cpu().numpy()[open_]
    tol = G.lse_tol(np.abs(host[np.isfinite(host)]).max(), 1.0) + 2.0 ** -23 * 16
    there = np.isfinite(rv[open_])
    want = rv[open_] - rl[open_][:, None]
    assert np.all(np.abs(logp[there] - want[there]) <= tol)


@pytest.mark.parametrize("V,history", [(1000, 30), (32001, 3000), (40000, 20000), (128256, 500)])
@pytest.mark.parametrize("mask", [True, False])
def test_process_rows_with_an_error_show_it(vce, V, history, mask):
    """A bad id, bias ids out of order, bad offsets or a bad parameter: that row is NaN, its gradient +0.0,
    also where nobody looks at row_status (autograd); the other rows are as they were."""
    c = Case(8, V, F32, history, 5, mask)
    want, size = c.oracle()
    kw = c.kwargs()
    off, b = kw["history_offsets"].tolist(), kw["bias_offsets"].tolist()
    rows = {}
    i = next(i for i in range(8) if off[i + 1] > off[i])
    kw["history_ids"][off[i + 1] - 1] = V
    rows[i] = 1
    j = next(j for j in range(8) if j not in rows and b[j + 1] - b[j] >= 2)
    kw["bias_ids"][b[j]] = V + 7
    rows[j] = 1
    k = [x for x in range(7) if x not in rows]
    kw["temperature"][k[0]], rows[k[0]] = -1.0, 3
    kw["repetition_penalty"][k[1]], rows[k[1]] = 0.0, 3
    rows[7] = 4
    kw["history_offsets"][8] += 1
    z = c.z.clone().requires_grad_(True)
    y = vce.process_logits(z, **kw)
    out, status = vce.logits_process(c.z, **kw)
    assert {r: s for r, s in enumerate(status.tolist()) if s} == rows
    good = [r for r in range(8) if r not in rows]
    bad = list(rows)
    for o in (y.detach(), out):
        assert torch.isnan(o[bad]).all()
        G.check_processed(o[good].double().cpu().numpy(), want[good], size[good], EPS[F32])
    up = torch.randn(8, V, device="cuda")
    y.backward(up)
    back = {r for r, s in rows.items() if r != j}        # the backward does not read the biases
    wantg, sizeg = c.oracle(up)
    assert torch.all(z.grad[list(back)] == 0) and not torch.signbit(z.grad[list(back)]).any()
    fine = good + [j]
    G.check_processed(z.grad[fine].double().cpu().numpy(), wantg[fine], sizeg[fine], EPS[F32])


def test_process_bad_temperatures_without_lists(vce):
    c = Case(4, 5001, BF16, 0, 0, True)
    kw = c.kwargs()
    kw["temperature"][2] = 0.0
    out, status = vce.logits_process(c.z, **kw)
    assert status.tolist() == [0, 0, 3, 0]
    assert torch.isnan(out[2]).all() and not torch.isnan(out[[0, 1, 3]]).any()
    g, status = vce.logits_process_backward(torch.ones_like(c.z), temperature=kw["temperature"], mask=kw["mask"])
    assert status.tolist() == [0, 0, 3, 0] and torch.all(g[2] == 0)
