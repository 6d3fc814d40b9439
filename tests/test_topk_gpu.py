"""ce_topk on the GPU against the fp64 oracle: ids and values exactly, log-sum-exps within the
tolerance derived in tests/_logits_grading.py."""
import numpy as np
import pytest
import torch

from oracle import logits_oracle as L
from tests import _logits_grading as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def logits_of(T, V, dtype, seed, pad=0, left=0, std=2.0):
    """[T, V] logits on the GPU inside a matrix of pad more columns, left of them before the first."""
    g = torch.Generator().manual_seed(seed)
    full = (std * torch.randn(T, V + pad, generator=g)).to(dtype).cuda()
    return full[:, left:left + V]


def check(vce, z, k, tau=1.0):
    values, ids, lse, tail = [x.cpu().numpy() for x in vce.ce_topk(z, k, tau)]
    host = z.double().cpu().numpy()
    rv, ri, rl, rt = L.topk(host, k, tau)
    assert np.array_equal(ids, ri)
    assert np.array_equal(values.astype(np.float64), rv)
    zmax = np.abs(host[np.isfinite(host)]).max(initial=0.0)
    G.check_lse(lse, rl, zmax, tau)
    G.check_lse(tail, rt, zmax, tau, "tail")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,k", [(1, 1, 1), (3, 7, 7), (5, 33, 4), (64, 1000, 8), (2, 1000, 256), (1, 8192, 256),
                                   (7, 8193, 1), (1, 128256, 20), (19, 32001, 64), (400, 5003, 50), (2, 300001, 100)])
def test_topk(vce, T, V, k, dtype):
    check(vce, logits_of(T, V, dtype, T + V + k), k, 0.7 if V % 2 else 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,left", [(1, 0), (1, 1), (13, 5), (8, 0), (7, 7)])
def test_topk_layouts(vce, pad, left, dtype):
    check(vce, logits_of(9, 4001, dtype, pad + left, pad, left), 40, 2.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_topk_ties(vce, dtype):
    """Constant rows, rows of few distinct values, sorted rows: equal logits in column order."""
    V = 20011
    z = torch.zeros(6, V, dtype=dtype)
    z[1] = (torch.arange(V) % 3).to(dtype)
    z[2] = torch.linspace(-4, 4, V).to(dtype)
    z[3] = torch.linspace(4, -4, V).to(dtype)
    z[4, ::2] = -0.0
    z[5] = torch.where(torch.arange(V) % 977 == 5, 1.0, -1.0).to(dtype)
    for k in (1, 17, 256):
        check(vce, z.cuda(), k)


@pytest.mark.parametrize("V", [77, 5000, 128256])
def test_topk_masked_rows(vce, V):
    """-inf entries are never among the K: rows with nothing, one logit, and fewer than K."""
    z = logits_of(5, V, torch.float32, V)
    z[0] = -float("inf")
    z[1] = -float("inf")
    z[1, V // 2] = 1.5
    z[2, 9:] = -float("inf")
    z[3, ::2] = -float("inf")
    z[4] = torch.finfo(torch.float32).min
    z[4, 3] = 2.0
    check(vce, z, 30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(4, 90), (4, 9001), (400, 20000)])
def test_topk_masks_of_the_lowest_value(vce, T, V, dtype):
    """Columns masked with the type's lowest value, whose product with log2(e) / temperature passes
    fp32: they take no part where anything else is left, and are the log-sum-exp where nothing is."""
    low = torch.finfo(dtype).min
    z = torch.full((T, V), low, dtype=dtype, device="cuda")
    z[1, 7] = 2.0
    z[2, 5:25] = 1.0
    values, ids, lse, tail = [x.double().cpu().numpy() for x in vce.ce_topk(z, 20)]
    want_lse, want_tail = [low, 2.0, 1.0 + np.log(20.0), low], [low, low, low, low]
    np.testing.assert_allclose(lse[:4], want_lse, rtol=1e-6)
    np.testing.assert_allclose(tail[:4], want_tail, rtol=1e-6)
    assert ids[0].tolist() == list(range(20)) and ids[1].tolist() == [7] + list(range(7)) + list(range(8, 20))
    assert ids[2].tolist() == list(range(5, 25)) and np.all(lse[4:] == lse[0])
    # as a teacher and as a student: the masked columns carry no mass
    student = torch.randn(T, V, device="cuda")
    out = vce.ce_distill_forward(student, ids_ := vce.ce_topk(z, 20)[1], vce.ce_topk(z, 20)[0], vce.ce_topk(z, 20)[3])
    want = -torch.log_softmax(student[1], 0)[7].item()
    assert vce.vce_get_status(out[4]) == 0 and abs(out[1][1].item() - want) <= 1e-5 * want and ids_.shape == (T, 20)


def test_topk_one_value_far_above(vce):
    """The tail is summed without the K: with a margin of 60 it would cancel to nothing as a difference,
    and as part of a group whose maximum is the large logit it would underflow at a margin of 150."""
    z = logits_of(3, 40000, torch.float32, 5)
    z[0, 17] = 60.0
    z[1, 39999] = 150.0
    z[2] -= 120.0
    z[2, 20000] = 30.0
    check(vce, z, 1)
    check(vce, z, 5)


def test_topk_many_rows_and_wide(vce):
    z = logits_of(2000, 1500, torch.bfloat16, 8)
    check(vce, z, 33)
    check(vce, logits_of(2, 2000003, torch.bfloat16, 9), 256, 4.0)


@pytest.mark.parametrize("dtype,V,pad,left", [(torch.bfloat16, 20011, 0, 0), (torch.bfloat16, 70000, 8, 8),
                                              (torch.float32, 16385, 3, 1), (torch.bfloat16, 131000, 0, 0)])
@pytest.mark.parametrize("k", [1, 64, 256])
def test_topk_rows_enough_for_every_sm(vce, dtype, V, pad, left, k):
    """More rows than two an SM: sampled rows against the oracle, and rows of ties, of -inf and with
    one value far above among them."""
    T = 330
    z = logits_of(T, V, dtype, V + k, pad, left)
    z[5] = 0.25
    z[17] = -float("inf")
    z[18, 3:] = -float("inf")
    z[170, V - 1] = 90.0
    z[171] = (torch.arange(V, device="cuda") % 5).to(dtype)
    values, ids, lse, tail = [x.cpu().numpy() for x in vce.ce_topk(z, k, 0.9)]
    rows = np.array([0, 5, 17, 18, 151, 152, 153, 170, 171, 303, 304, 329])
    host = z[torch.from_numpy(rows).cuda()].double().cpu().numpy()
    rv, ri, rl, rt = L.topk(host, k, 0.9)
    assert np.array_equal(ids[rows], ri) and np.array_equal(values[rows].astype(np.float64), rv)
    zmax = np.abs(host[np.isfinite(host)]).max()
    G.check_lse(lse[rows], rl, zmax, 0.9)
    G.check_lse(tail[rows], rt, zmax, 0.9, "tail")
    # every row against the few-rows path, which takes another kernel
    for r in range(0, T, 110):
        v2, i2, _, _ = vce.ce_topk(z[r:r + 110], k, 0.9)
        assert np.array_equal(i2.cpu().numpy(), ids[r:r + 110]) and np.array_equal(v2.cpu().numpy(), values[r:r + 110])


def test_topk_same_bits_every_time(vce):
    z = logits_of(400, 128256, torch.bfloat16, 10)
    first = [x.clone() for x in vce.ce_topk(z, 64, 2.0)]
    for _ in range(5):
        for a, b in zip(vce.ce_topk(z, 64, 2.0), first):
            assert torch.equal(a, b)


def test_topk_streams_and_graphs(vce):
    z = logits_of(40, 50001, torch.bfloat16, 11)
    want = vce.ce_topk(z, 20)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [vce.ce_topk(z, 20, stream=s) for s in streams]       # at once, on three streams
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = vce.ce_topk(z, 20)
    other = logits_of(40, 50001, torch.bfloat16, 12)
    want = [x.clone() for x in vce.ce_topk(other, 20)]
    z.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_topk_leaves_what_is_behind_its_outputs(vce):
    T, k = 5, 9
    z = logits_of(T, 999, torch.bfloat16, 13)
    bufs = [torch.full((T * k + 8,), -7.0, device="cuda"), torch.full((T * k + 8,), -7, dtype=torch.int64, device="cuda"),
            torch.full((T + 8,), -7.0, device="cuda"), torch.full((T + 8,), -7.0, device="cuda")]
    vce.ce_topk(z, k, values=bufs[0][:T * k].view(T, k), ids=bufs[1][:T * k].view(T, k), lse=bufs[2][:T],
                tail_lse=bufs[3][:T])
    for b, n in zip(bufs, (T * k, T * k, T, T)):
        assert torch.all(b[n:] == -7)


def test_topk_refusals(vce):
    z = logits_of(4, 100, torch.float32, 1)
    with pytest.raises(ValueError):
        vce.ce_topk(z, 0)
    for kw in (dict(k=101), dict(k=257), dict(k=5, temperature=0.0), dict(k=5, temperature=float("nan"))):
        with pytest.raises(vce.VceError):
            vce.ce_topk(z, **kw)
    with pytest.raises(TypeError):
        vce.ce_topk(z, 5, ids=torch.empty(4, 5, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        vce.ce_topk(z, 5, values=torch.empty(4, 6, device="cuda"))
    out = vce.ce_topk(z[:0], 5)
    assert [tuple(x.shape) for x in out] == [(0, 5), (0, 5), (0,), (0,)]


@pytest.mark.parametrize("V,pad", [(2097150, 0), (2097151, 0), (2097152, 1)])
def test_topk_the_longest_fp32_rows(vce, V, pad):
    """Unaligned rows of the most columns have one vector more than eight times 64 stages: the largest
    logits in the last vector of each block's slice, and everywhere else."""
    T = 4
    z = logits_of(T, V, torch.float32, V, pad)
    for i in range(T):
        shift = z[i].data_ptr() % 16 // 4
        vectors = (V + shift + 3) // 4
        per = -(-vectors // 8)                      # vectors of a slice
        for p in range(8):
            last = min((p + 1) * per, vectors) - 1
            for q in range(4):
                c = last * 4 - shift + q
                if 0 <= c < V:
                    z[i, c] = 12.0 + (p * 5 + i) % 8 + q / 8
    check(vce, z, 1)
    check(vce, z, 20)
    check(vce, z, 256, 2.0)


@pytest.mark.parametrize("T,V", [(3, 50001), (40, 5000), (330, 20000)])
def test_topk_waits_that_give_up_leave_nan(vce, T, V):
    """Slices whose last stage is never copied: NaN and -1 in every output, and a context that stays
    usable."""
    z = logits_of(T, V, torch.bfloat16, T + V).contiguous()
    values, ids, lse, tail = vce.vce_test_topk_stall(z, 9)
    assert torch.isnan(values).all() and torch.all(ids == -1) and torch.isnan(lse).all() and torch.isnan(tail).all()
    check(vce, z[:3], 9)


def test_topk_counts_beyond_32_bits_are_refused(vce):
    """2^32 + 5 is not 5."""
    z = logits_of(1, 100, torch.float32, 1)
    held = torch.cuda.memory_allocated()
    for k in (2 ** 32 + 5, 2 ** 31, -2 ** 32 + 5):
        with pytest.raises(ValueError):
            vce.ce_topk(z, k)
    assert torch.cuda.memory_allocated() == held
