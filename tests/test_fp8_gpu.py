"""The fp8 head on the GPU: block quantisation bit for bit, the product against the fp64 oracle, and the head as it
is used, its logits going into the other operators."""
import numpy as np
import pytest
import torch

from oracle import policy_oracle as O
from tests import _policy_grading as G

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def host(t):
    return t.detach().double().cpu().numpy()


def check_quantize(vce, x, rows):
    q, s = vce.quantize_fp8(x, rows)
    want, scales = O.quantize(host(x), rows)
    assert np.array_equal(host(s), scales, equal_nan=True)
    assert np.array_equal(host(q), want, equal_nan=True)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,D", [(1, 1), (1, 16), (3, 127), (5, 128), (130, 129), (128, 256), (257, 1000), (2, 4096), (1000, 40)])
def test_quantize(vce, R, D, dtype, rows):
    g = torch.Generator().manual_seed(R + D)
    x = torch.randn(R, D, generator=g) * torch.exp(4 * torch.randn(R, 1, generator=g))
    check_quantize(vce, x.to(dtype).cuda(), rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_edges(vce, rows, dtype):
    """Zeros, the largest and smallest magnitudes, 448 and its neighbours, ties, NaN and infinities."""
    x = torch.zeros(6, 520, dtype=dtype, device="cuda")
    x[0, :128] = torch.finfo(dtype).max
    x[1, :4] = torch.tensor([448.0, 449.0, 447.0, -448.0])
    x[1, 128:132] = torch.tensor([450.0, -1.0, 0.01, 17.0])
    x[2, :3] = torch.tensor([1e-38, -2e-39, 1e-45])
    x[2, 128] = torch.finfo(dtype).tiny
    x[3, 256:264] = torch.tensor([1.0625, 1.1875, 1.3125, -1.4375, 2.0 ** -10, 3 * 2.0 ** -11, 1.75, 1.5])
    x[3, 400] = 0.875
    check_quantize(vce, x, rows)
    x[4, 5], x[4, 200], x[4, 300] = float("nan"), float("inf"), float("-inf")
    check_quantize(vce, x, rows)


def test_quantize_layouts(vce):
    """A matrix inside a wider one, at every alignment; caller's outputs."""
    g = torch.Generator().manual_seed(1)
    for dtype in (BF16, F32):
        full = torch.randn(133, 1100, generator=g).to(dtype).cuda()
        for left, D in ((0, 1024), (1, 1024), (3, 700), (8, 512), (4, 1096)):
            for rows in (1, 128):
                check_quantize(vce, full[:, left:left + D], rows)
    q, s = torch.zeros(133, 64, dtype=E4M3, device="cuda"), torch.zeros(2, 1, device="cuda")
    a, b = vce.quantize_fp8(full[:, :64], 128, q=q, scales=s)
    assert a is q and b is s
    e = torch.empty(0, 64, device="cuda")
    q, s = vce.quantize_fp8(e, 128)
    assert q.shape == (0, 64) and s.shape == (0, 1)


def operands(T, D, V, seed=0):
    g = torch.Generator().manual_seed(seed + T + D + V)
    x = torch.randn(T, D, generator=g) * torch.exp(torch.randn(D, generator=g))
    w = torch.randn(V, D, generator=g) / D ** 0.5
    q = []
    for m, rows in ((x, 1), (w, 128)):
        # any e4m3 values, and scales that are no powers of two
        amax = torch.zeros(-(-m.shape[0] // rows), -(-D // 128))
        for i in range(amax.shape[0]):
            for j in range(amax.shape[1]):
                amax[i, j] = m[i * rows:(i + 1) * rows, 128 * j:128 * (j + 1)].abs().max()
        s = (amax / 448).clamp(min=1e-6)
        wide = s.repeat_interleave(rows, 0)[:m.shape[0]].repeat_interleave(128, 1)[:, :D]
        q += [(m / wide).clamp(-448, 448).to(E4M3).cuda(), s.cuda()]
    return q


def check_linear(vce, ops, dtype, out=None):
    x, xs, w, ws = ops
    want, size = O.linear(host(x), host(xs), host(w), host(ws))
    got = vce.linear_fp8(x, xs, w, ws, out=out, out_dtype=dtype)
    G.check_linear(host(got), want, size, xs.shape[1], torch.finfo(dtype).eps)
    return got


@pytest.mark.parametrize("T", [1, 2, 7, 16, 33, 64, 100, 128, 129, 200, 256, 300])
@pytest.mark.parametrize("D,V", [(16, 1), (128, 128), (144, 1000), (1040, 257), (512, 5003)])
def test_linear(vce, T, D, V):
    check_linear(vce, operands(T, D, V), BF16 if (T + V) % 2 else F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D,V", [(1, 4096, 20000), (5, 2064, 32001), (70, 8192, 3000), (600, 1024, 2049), (1000, 256, 513),
                                   (257, 65536, 130)])
def test_linear_sizes(vce, T, D, V, dtype):
    check_linear(vce, operands(T, D, V), dtype)


@pytest.mark.parametrize("T", [1, 40, 100, 128])
@pytest.mark.parametrize("D,V", [(4096, 1000), (4096, 1300), (2160, 300), (2048, 128), (1152, 2500), (400, 9000)])
def test_linear_parts_of_k(vce, T, D, V):
    """Few tiles of w: clusters of two, four and eight CTAs share K, some with blocks left over or none at all."""
    check_linear(vce, operands(T, D, V), F32 if T == 40 else BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,left", [(0, 0), (1, 0), (3, 1), (8, 8), (12, 4)])
@pytest.mark.parametrize("T,V", [(3, 1000), (40, 777), (300, 1024)])
def test_linear_output_layouts(vce, T, V, pad, left, dtype):
    """Rows of a wider matrix: nothing beside them is written."""
    ops = operands(T, 272, V)
    full = torch.full((T + 2, V + pad), 7.0, dtype=dtype, device="cuda")
    check_linear(vce, ops, dtype, full[1:T + 1, left:left + V] if left + V <= V + pad else full[1:T + 1, :V])
    keep = torch.ones_like(full, dtype=torch.bool)
    keep[1:T + 1, left:left + V] = False
    assert torch.all(full[keep] == 7)


@pytest.mark.parametrize("T", [1, 20, 200])
def test_linear_nan_stays_in_its_row_and_column(vce, T):
    x, xs, w, ws = operands(T, 400, 900)
    x.view(torch.uint8)[0, 390] = 0x7F
    w.view(torch.uint8)[333, 17] = 0xFF
    got = vce.linear_fp8(x, xs, w, ws).float()
    assert torch.isnan(got[0]).all() and torch.isnan(got[:, 333]).all()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[0], rest[:, 333] = False, False
    assert torch.isfinite(got[rest]).all()
    xs[T - 1, 2] = float("inf")
    got = vce.linear_fp8(x, xs, w, ws).float()
    assert not torch.isfinite(got[T - 1]).any()


def test_linear_no_rows_and_refusals(vce):
    x, xs, w, ws = operands(4, 256, 300)
    assert vce.linear_fp8(x[:0], xs[:0], w, ws).shape == (0, 300)
    with pytest.raises(TypeError):
        vce.linear_fp8(x.to(BF16), xs, w, ws)
    with pytest.raises(TypeError):
        vce.linear_fp8(x, xs, w, ws, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        vce.linear_fp8(x, xs[:, :1], w, ws)
    with pytest.raises(ValueError):
        vce.linear_fp8(x, xs, w[:, :128], ws)
    with pytest.raises(ValueError):
        vce.linear_fp8(x, xs, w, ws, out=torch.empty(4, 299, device="cuda"))
    with pytest.raises(ValueError):
        vce.linear_fp8(x.cpu(), xs, w, ws)
    y, ys, v, vs = operands(4, 136, 300)
    with pytest.raises(vce.VceError):       # D not a multiple of 16
        vce.linear_fp8(y, ys, v, vs)
    flat = torch.zeros(4 * 256 + 8, dtype=torch.uint8, device="cuda").view(E4M3)
    with pytest.raises(vce.VceError):       # not on a 16-byte boundary
        vce.linear_fp8(flat[8:].view(4, 256), xs, w, ws)
    with pytest.raises(ValueError):
        vce.quantize_fp8(torch.zeros(4, 4, device="cuda"), 64)
    with pytest.raises(TypeError):
        vce.quantize_fp8(torch.zeros(4, 4, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,D,V", [(1, 1024, 9000), (40, 512, 5003), (300, 1024, 2049)])
def test_linear_same_bits_on_streams_and_in_graphs(vce, T, D, V):
    x, xs, w, ws = operands(T, D, V)
    want = vce.linear_fp8(x, xs, w, ws, out_dtype=F32).clone()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [vce.linear_fp8(x, xs, w, ws, out_dtype=F32, stream=s) for s in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vce.linear_fp8(x, xs, w, ws, out_dtype=F32))
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("T", [1, 20, 50, 200, 700])
def test_linear_waits_that_give_up_leave_nan(vce, T):
    ops = operands(T, 400, 900)
    want = vce.linear_fp8(*ops, out_dtype=F32)
    assert torch.isnan(vce.vce_test_linear_fp8_stall(*ops)).all()
    assert torch.equal(vce.linear_fp8(*ops, out_dtype=F32), want)


def test_head_into_the_losses(vce):
    """As they are used together: a frozen head's logits from quantised hidden states and weights, the reference's
    and the old policy's log-probabilities from those, and the losses of a policy near it; top K of the same logits."""
    T, D, V = 48, 256, 4099
    g = torch.Generator().manual_seed(3)
    hidden, weight = torch.randn(T, D, generator=g).to(BF16).cuda(), (torch.randn(V, D, generator=g) / 4).to(BF16).cuda()
    x, xs = vce.quantize_fp8(hidden)
    w, ws = vce.quantize_fp8(weight, 128)
    frozen = vce.linear_fp8(x, xs, w, ws, out_dtype=F32)
    wide = lambda q, s, r: host(q) * np.repeat(np.repeat(host(s), r, 0)[:q.shape[0]], 128, 1)[:, :D]
    a, b = wide(x, xs, 1), wide(w, ws, 128)
    G.check_linear(host(frozen), a @ b.T, np.abs(a) @ np.abs(b).T, 2, torch.finfo(F32).eps)
    values, ids, _, _ = vce.ce_topk(frozen, 4)
    tokens = ids[:, 1].contiguous()
    ref, _, _, status = vce.ce_logprobs_forward(frozen, tokens)
    assert vce.vce_get_status(status) == 0
    z = (frozen + 0.05 * torch.randn(T, V, generator=g).cuda()).to(BF16)
    z.requires_grad_(True)
    adv = torch.randn(T, generator=g).cuda()
    r = O.rows(host(frozen), tokens.cpu().numpy())
    zm = float(max(frozen.abs().max(), z.detach().abs().max()))
    G.check_rows(host(ref), None, r, zm, 1.0)
    loss = vce.policy_loss(z, tokens, adv, ref, ref, clip_low=0.9, clip_high=9.0, kl_coef=0.1, entropy_coef=0.01)
    loss.backward()
    want = O.policy(host(z), tokens.cpu().numpy(), host(adv), host(ref), host(ref), None, 0.9, 9.0, 0.0, 0.1, 0.01)
    tol, da = G.policy_errors(want, host(adv), host(ref), host(ref), None, 0.1, 0.01, zm, 1.0, np.full(T, 1.0 / T))
    assert abs(float(loss) - want["loss"]) <= tol.mean() + 1e-6 * abs(want["loss"])
    G.check_grad(host(z.grad), want, tokens.cpu().numpy(), da, zm, 1.0, torch.finfo(BF16).eps)
    z.grad = None
    off = [0, 12, 20, 33, 48]
    loss = vce.preference_loss(z, tokens, torch.tensor(off).cuda(), ref)
    loss.backward()
    want = O.preference(host(z), tokens.cpu().numpy(), off, host(ref))
    _, tp, da = G.preference_errors(want, off, 0.1, "sigmoid", False, zm, 1.0, np.full(2, 0.5))
    assert abs(float(loss) - want["loss"]) <= tp.mean() + 1e-6 * abs(want["loss"])
    G.check_grad(host(z.grad), want, tokens.cpu().numpy(), da, zm, 1.0, torch.finfo(BF16).eps)
