"""Token log-probabilities, the policy loss and the preference loss on the GPU against the fp64 oracle, within the
tolerances derived in tests/_policy_grading.py."""
import numpy as np
import pytest
import torch

from oracle import policy_oracle as O
from tests import _policy_grading as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


def logits(T, V, dtype, seed=0, pad=0, left=0, scale=2.0):
    g = torch.Generator().manual_seed(seed + 31 * T + V)
    full = (scale * torch.randn(T, V + pad, generator=g)).to(dtype).cuda()
    return full[:, left:left + V]


def tokens(T, V, seed=0, ignored=()):
    g = torch.Generator().manual_seed(seed + T)
    ids = torch.randint(0, V, (T,), generator=g)
    for i in ignored:
        ids[i] = IGNORE
    return ids.cuda()


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def zmax(z):
    f = z.float()
    f = f[torch.isfinite(f) & (f.abs() < 1e30)]
    return float(f.abs().max()) if f.numel() else 0.0


def eps_of(dtype):
    return torch.finfo(dtype).eps


def check_logprobs(vce, z, ids, tau, gdtype=None, entropy=True):
    T = z.shape[0]
    r = O.rows(host(z), ids.cpu().numpy(), tau)
    lp, ent, stats, status = vce.ce_logprobs_forward(z, ids, tau, want_entropy=entropy)
    assert vce.vce_get_status(status) == 0
    G.check_rows(host(lp), host(ent), r, zmax(z), tau)
    g = torch.Generator().manual_seed(5)
    ga, gb = torch.randn(2, T, generator=g).cuda()
    gdtype = gdtype or z.dtype
    for a, b in ((ga, gb if entropy else None), (ga, None)) + (((None, gb),) if entropy else ()):
        got = vce.ce_logprobs_backward(z, ids, stats, a, b, tau, grad_dtype=gdtype)
        r["a"] = np.where(r["valid"], 0.0 if a is None else host(a), 0.0)
        r["b"] = np.where(r["valid"], 0.0 if b is None else host(b), 0.0)
        r["grad"] = O.gradient(r, ids.cpu().numpy(), r["a"], r["b"], tau)
        G.check_grad(host(got), r, ids.cpu().numpy(), np.zeros(T), zmax(z), tau, eps_of(gdtype))


@pytest.mark.parametrize("T,V,dtype,tau", [
    (1, 1, BF16, 1.0), (1, 2, F32, 1.0), (3, 7, BF16, 0.5), (5, 1000, F32, 1.0), (9, 4001, BF16, 0.7), (2, 4096, F32, 2.0),
    (300, 513, BF16, 1.0), (4, 33001, F32, 1.0), (1, 128256, BF16, 1.0), (17, 50257, BF16, 1.3), (3, 262147, BF16, 1.0),
    (2, 140001, F32, 1.0)])
@pytest.mark.parametrize("entropy", [True, False])
def test_logprobs(vce, T, V, dtype, tau, entropy):
    check_logprobs(vce, logits(T, V, dtype), tokens(T, V), tau, entropy=entropy)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("V,pad,left", [(4001, 6, 3), (4096, 1, 1), (33000, 5, 2), (20000, 8, 8)])
def test_logprobs_layouts(vce, V, pad, left, dtype, gdtype):
    check_logprobs(vce, logits(7, V, dtype, 0, pad, left), tokens(7, V, ignored=[2, 6]), 1.0, gdtype)


@pytest.mark.parametrize("V,dtype", [(700, F32), (20000, BF16), (128256, BF16)])
def test_logprobs_of_confident_rows(vce, V, dtype):
    """The token far above the rest, the rest far above the token, another column with all the mass."""
    z = logits(6, V, dtype, 3)
    ids = torch.arange(6).cuda() * 3 + 1
    for i in range(6):
        z[i, int(ids[i])] = [40.0, -40.0, 12.0, 200.0, -3.0, 90.0][i]
    z[4, 0] = 60.0
    r = O.rows(host(z), ids.cpu().numpy())
    assert r["lp"][3] > -1e-60
    check_logprobs(vce, z, ids, 1.0)


@pytest.mark.parametrize("V,dtype", [(600, F32), (20001, BF16), (128256, BF16), (300000, F32)])
@pytest.mark.parametrize("low", [float("-inf"), None])
def test_logprobs_with_masks(vce, V, dtype, low):
    """Masked columns, a masked token, only the token left, one other left, nothing left."""
    low = torch.finfo(dtype).min if low is None else low
    z = logits(6, V, dtype, 4)
    ids = tokens(6, V, 1)
    z[0, ::2] = low
    ids[0] = 1
    z[1, int(ids[1])] = low
    z[2] = low
    z[2, int(ids[2])] = 1.5
    z[3] = low
    z[3, (int(ids[3]) + 1) % V] = -2.0
    z[4] = low
    z[5, : V // 2] = low
    ids[5] = V - 1
    lp, ent, stats, status = vce.ce_logprobs_forward(z, ids)
    assert vce.vce_get_status(status) == 0
    z64 = host(z)
    z64[z64 < -1e38] = -np.inf
    keep = [0, 1, 2, 3, 5]
    r = O.rows(z64[keep], ids.cpu().numpy()[keep])
    G.check_rows(host(lp)[keep], host(ent)[keep], r, zmax(z), 1.0)
    assert torch.isnan(lp[4]) and torch.isnan(ent[4])
    ones = torch.ones(6, device="cuda")
    g = vce.ce_logprobs_backward(z, ids, stats, ones, ones)
    assert torch.all(g[4] == 0)
    r["a"] = r["b"] = np.ones(5)
    r["grad"] = O.gradient(r, ids.cpu().numpy()[keep], r["a"], r["b"])
    G.check_grad(host(g)[keep], r, ids.cpu().numpy()[keep], np.zeros(5), zmax(z), 1.0, eps_of(dtype))


@pytest.mark.parametrize("V,dtype", [(600, F32), (20001, BF16), (300000, F32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("place", ["token", "first", "last", "middle"])
def test_logprobs_with_nan_and_infinity(vce, V, dtype, bad, place):
    z = logits(3, V, dtype, 5)
    ids = torch.tensor([V // 3, V // 3, 5], device="cuda")
    z[1, dict(token=V // 3, first=0, last=V - 1, middle=V // 2)[place]] = bad
    lp, ent, stats, status = vce.ce_logprobs_forward(z, ids)
    assert vce.vce_get_status(status) == 0
    assert torch.isnan(lp[1]) and torch.isnan(ent[1])
    g = vce.ce_logprobs_backward(z, ids, stats, torch.ones(3, device="cuda"), torch.ones(3, device="cuda"))
    assert torch.isnan(g[1]).all() and torch.isfinite(g[0]).all() and torch.isfinite(g[2]).all()
    r = O.rows(host(z)[[0, 2]], ids.cpu().numpy()[[0, 2]])
    G.check_rows(host(lp)[[0, 2]], host(ent)[[0, 2]], r, zmax(z), 1.0)


@pytest.mark.parametrize("V", [600, 20001, 128256])
def test_left_out_rows_are_not_read_and_bad_tokens_reported(vce, V):
    z = logits(5, V, BF16, 6)
    z[1] = float("nan")
    z[3] = float("inf")
    ids = tokens(5, V, ignored=[1, 3])
    lp, ent, stats, status = vce.ce_logprobs_forward(z, ids)
    assert vce.vce_get_status(status) == 0
    ones = torch.ones(5, device="cuda")
    g = vce.ce_logprobs_backward(z, ids, stats, ones, ones)
    for t in (lp[[1, 3]], ent[[1, 3]], g[[1, 3]]):
        assert torch.all(t == 0)
    ids[2], ids[4] = V, -1
    lp, ent, stats, status = vce.ce_logprobs_forward(z, ids)
    assert vce.vce_get_status(status) == 1
    assert torch.isnan(lp[[2, 4]]).all() and torch.isnan(ent[[2, 4]]).all() and torch.isfinite(lp[[0, 1, 3]]).all()
    g = vce.ce_logprobs_backward(z, ids, stats, ones, ones)
    assert torch.all(g[[2, 4]] == 0)
    loss, rows, lp2, _, _, status = vce.policy_loss_forward(z, ids, ones)
    assert vce.vce_get_status(status) == 1 and torch.isnan(loss).all() and torch.isnan(rows[[2, 4]]).all()
    out = vce.policy_loss_forward_backward(z, ids, ones, entropy_coef=0.1)
    assert vce.vce_get_status(out[5]) == 1 and torch.isnan(out[0]).all() and torch.all(out[4][1:] == 0)
    assert torch.isfinite(out[4][0]).all()


# ---- policy loss --------------------------------------------------------------------------------


def policy_case(T, V, dtype, tau, seed=0, ref=True, weights=True, ignored=(), pad=0, left=0):
    g = torch.Generator().manual_seed(seed + T + V)
    z, ids = logits(T, V, dtype, seed, pad, left), tokens(T, V, seed, ignored)
    lp = O.rows(host(z), np.where(ids.cpu().numpy() < 0, 0, ids.cpu().numpy()), tau)["lp"]
    # ratios well away from where the loss is clipped (0.8, 1.3) and bounded (2.5), on every side of them
    step = torch.tensor([0.0, 0.1, -0.1, 0.5, -0.5, 1.2, -1.2])[torch.randint(0, 7, (T,), generator=g)]
    old = torch.from_numpy(lp).float() + step
    adv = torch.randn(T, generator=g)
    adv[adv.abs() < 0.05] = 0.0
    return dict(z=z, ids=ids, adv=adv.cuda(), old=old.cuda(),
                ref=(torch.from_numpy(lp).float() + 0.6 * torch.randn(T, generator=g)).cuda() if ref else None,
                w=(torch.rand(T, generator=g) + 0.1).cuda() if weights else None)


def check_policy(vce, c, tau=1.0, kl=0.05, ent=0.02, dual=2.5, reduction="mean", gdtype=None, entropy=True):
    z, ids = c["z"], c["ids"]
    T = z.shape[0]
    gdtype = gdtype or z.dtype
    kl = kl if c["ref"] is not None else 0.0
    up = torch.linspace(0.5, 1.5, T).cuda() if reduction == "none" else torch.full((1,), 0.75, device="cuda")
    want = O.policy(host(z), ids.cpu().numpy(), host(c["adv"]), host(c["old"]), host(c["ref"]), host(c["w"]), 0.2, 0.3, dual,
                    kl, ent, tau, reduction, host(up) if reduction == "none" else 0.75)
    scale = host(up) * np.ones(T) * (1.0 / want["n"] if reduction == "mean" and want["n"] else 1.0)
    tol, da = G.policy_errors(want, host(c["adv"]), host(c["old"]), host(c["ref"]), host(c["w"]), kl, ent, zmax(z), tau, scale)
    kw = dict(clip_low=0.2, clip_high=0.3, dual_clip=dual, kl_coef=kl, entropy_coef=ent, temperature=tau,
              reduction=reduction, want_entropy=entropy)
    args = (z, ids, c["adv"], c["old"], c["ref"], c["w"])
    loss, rows, lp, H, stats, status = vce.policy_loss_forward(*args, **kw)
    assert vce.vce_get_status(status) == 0
    grad = vce.policy_loss_backward(z, ids, stats, up, tau, reduction, grad_dtype=gdtype)
    one = vce.policy_loss_forward_backward(*args, grad_output=up, grad_dtype=gdtype, **kw)
    assert vce.vce_get_status(one[5]) == 0
    for l, r, p, h, g in ((loss, rows, lp, H, grad), one[:5]):
        G.check_rows(host(p), host(h) if entropy else None, want, zmax(z), tau)
        G.near(host(r), want["loss_rows"], tol, "loss rows")
        G.check_grad(host(g), want, ids.cpu().numpy(), da, zmax(z), tau, eps_of(gdtype))
        if reduction == "none":
            assert l is None
        else:   # the sum of the rows it wrote: compensated, a rounding or two
            s = float(r.double().sum()) / (want["n"] if reduction == "mean" else 1)
            assert abs(float(l) - s) <= 4 * G.E24 * (abs(s) + 2.0 ** -20 * float(r.double().abs().sum()))


@pytest.mark.parametrize("T,V,dtype,tau", [
    (1, 2, F32, 1.0), (7, 33, BF16, 1.0), (40, 1000, F32, 0.7), (30, 4001, BF16, 1.0), (5, 33001, BF16, 1.3),
    (3, 128256, BF16, 1.0), (9, 20000, F32, 1.0), (2, 300001, BF16, 1.0)])
@pytest.mark.parametrize("ent", [0.0, 0.02])
def test_policy(vce, T, V, dtype, tau, ent):
    check_policy(vce, policy_case(T, V, dtype, tau, ignored=[0] if T > 5 else []), tau, ent=ent)


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_policy_types_and_reductions(vce, dtype, gdtype, reduction):
    check_policy(vce, policy_case(11, 6007, dtype, 1.0, 2, ignored=[3, 10]), reduction=reduction, gdtype=gdtype)


@pytest.mark.parametrize("ref,weights,dual,entropy", [(False, False, 0.0, False), (True, False, 0.0, True), (False, True, 2.5, False)])
@pytest.mark.parametrize("pad,left", [(0, 0), (6, 3), (8, 8)])
def test_policy_options_and_layouts(vce, ref, weights, dual, entropy, pad, left):
    check_policy(vce, policy_case(13, 9001 - pad, BF16, 1.0, 3, ref, weights, [1], pad, left), dual=dual, entropy=entropy,
                 ent=0.0 if not entropy else 0.01)


def test_policy_many_rows(vce):
    """More rows than a launch has blocks, several to each."""
    check_policy(vce, policy_case(700, 1003, BF16, 1.0, 4, ignored=list(range(5, 700, 7))))
    check_policy(vce, policy_case(400, 9000, F32, 1.0, 4, ignored=list(range(100, 250))), ent=0.0)


def test_policy_on_policy_and_degenerate(vce):
    """No old log-probabilities: a ratio of 1; zero advantages; every row left out; no rows."""
    c = policy_case(6, 500, F32, 1.0)
    c["old"] = None
    check_policy(vce, c)
    c["adv"].zero_()
    check_policy(vce, c, ent=0.0)
    c["ids"][:] = IGNORE
    out = vce.policy_loss_forward_backward(c["z"], c["ids"], c["adv"])
    assert torch.isnan(out[0]).all() and torch.all(out[1] == 0) and torch.all(out[4] == 0)
    out = vce.policy_loss_forward_backward(c["z"], c["ids"], c["adv"], reduction="sum")
    assert float(out[0]) == 0
    e = torch.empty(0, 500, device="cuda")
    out = vce.policy_loss_forward(e, c["ids"][:0], c["adv"][:0], reduction="sum")
    assert float(out[0]) == 0 and vce.vce_get_status(out[5]) == 0
    out = vce.policy_loss_forward_backward(e, c["ids"][:0], c["adv"][:0])
    assert torch.isnan(out[0]).all() and vce.vce_get_status(out[5]) == 0
    lp, ent, _, status = vce.ce_logprobs_forward(e, c["ids"][:0])
    assert lp.numel() == 0 and vce.vce_get_status(status) == 0


# ---- preference loss ------------------------------------------------------------------------------


def check_preference(vce, T, V, offsets, dtype=BF16, tau=1.0, kind="sigmoid", average=False, ref=True, reduction="mean",
                     ignored=(), gdtype=None, seed=0):
    z, ids = logits(T, V, dtype, seed), tokens(T, V, seed, ignored)
    z[: offsets[0]] = float("nan")          # padding is not read
    z[offsets[-1]:] = float("nan")
    P = (len(offsets) - 1) // 2
    g = torch.Generator().manual_seed(seed)
    lp = O.rows(np.nan_to_num(host(z)), np.where(ids.cpu().numpy() < 0, 0, ids.cpu().numpy()), tau)["lp"]
    refp = (torch.from_numpy(lp).float() + 0.4 * torch.randn(T, generator=g)).cuda() if ref else None
    eps = 0.1 if kind == "sigmoid" else 0.0
    up = torch.linspace(0.5, 1.5, P).cuda() if reduction == "none" else torch.full((1,), 0.75, device="cuda")
    go = host(up) if reduction == "none" else 0.75
    want = O.preference(host(z), ids.cpu().numpy(), offsets, host(refp), 0.1, kind, eps, 0.05, average, tau, reduction, go)
    c = np.broadcast_to(go, (P,)) * (1.0 / P if reduction == "mean" else 1.0)
    zm = zmax(z)
    trew, tpair, da = G.preference_errors(want, offsets, 0.1, kind, average, zm, tau, c)
    off = torch.tensor(offsets).cuda()
    kw = dict(beta=0.1, kind=kind, label_smoothing=eps, margin=0.05, average=average, temperature=tau, reduction=reduction)
    loss, pairs, rewards, got, stats, status = vce.preference_loss_forward(z, ids, off, refp, **kw)
    assert vce.vce_get_status(status) == 0
    G.check_rows(host(got), None, want, zm, tau)
    G.near(host(rewards), want["rewards"], trew, "rewards")
    G.near(host(pairs), want["pairs"], tpair, "pair losses")
    grad = vce.preference_loss_backward(z, ids, stats, up, P, tau, reduction, grad_dtype=gdtype)
    G.check_grad(host(grad), want, ids.cpu().numpy(), da, zm, tau, eps_of(gdtype or dtype))
    if reduction != "none":
        s = float(pairs.double().sum()) / (P if reduction == "mean" else 1)
        assert abs(float(loss) - s) <= 4 * G.E24 * abs(s)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("ref", [False, True])
def test_preference_kinds(vce, kind, average, ref):
    check_preference(vce, 40, 3001, [2, 9, 20, 21, 37], kind=kind, average=average, ref=ref, ignored=[5, 12])


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("dtype,gdtype", [(BF16, F32), (F32, BF16), (F32, F32)])
def test_preference_types_and_reductions(vce, dtype, gdtype, reduction):
    check_preference(vce, 30, 1001, [0, 3, 9, 14, 14, 27, 28], dtype, 0.7, reduction=reduction, gdtype=gdtype)


@pytest.mark.parametrize("T,V,offsets", [
    (2, 5, [0, 1, 2]), (1, 9, [0, 0, 1]), (4, 20000, [0, 0, 0, 1, 4]), (600, 513, [0, 300, 600]), (7, 128256, [1, 3, 6])])
def test_preference_sequences(vce, T, V, offsets):
    """Single tokens, empty sequences, empty pairs, long ones, long rows."""
    check_preference(vce, T, V, offsets)


def test_preference_bad_inputs(vce):
    z, ids = logits(12, 400, F32), tokens(12, 400)
    for bad in ([0, 5, 3, 8, 12], [-1, 5, 6, 8, 12], [0, 5, 6, 8, 13]):
        loss, pairs, rewards, lp, stats, status = vce.preference_loss_forward(z, ids, torch.tensor(bad).cuda())
        assert vce.vce_get_status(status) == 4
        assert torch.isnan(loss).all() and torch.isnan(pairs).all() and torch.isnan(rewards).all()
        g = vce.preference_loss_backward(z, ids, stats, torch.ones(1, device="cuda"), 2)
        assert torch.all(g == 0)
    off = torch.tensor([0, 3, 6, 9, 12]).cuda()
    ids[7] = 400
    loss, pairs, rewards, lp, stats, status = vce.preference_loss_forward(z, ids, off, reduction="none")
    assert vce.vce_get_status(status) == 1 and torch.isnan(pairs[1]) and torch.isfinite(pairs[0]) and torch.isnan(lp[7])
    g = vce.preference_loss_backward(z, ids, stats, torch.ones(2, device="cuda"), 2, reduction="none")
    assert torch.all(g[6:] == 0) and (g[:6] != 0).any()
    ids[7] = 3
    z[10] = float("-inf")
    loss, pairs, rewards, lp, stats, status = vce.preference_loss_forward(z, ids, off, reduction="none")
    assert vce.vce_get_status(status) == 0 and torch.isnan(pairs[1]) and torch.isfinite(pairs[0])
    g = vce.preference_loss_backward(z, ids, stats, torch.ones(2, device="cuda"), 2, reduction="none")
    assert torch.all(g[6:] == 0) and torch.isfinite(g).all()


def test_preference_statistics_of_another_call_name_no_pair(vce):
    """Rows whose saved pair is not among the call's have no gradient, and read no upstream one."""
    z, ids = logits(12, 400, F32), tokens(12, 400)
    off = torch.tensor([0, 3, 6, 9, 12]).cuda()
    stats = vce.preference_loss_forward(z, ids, off, reduction="none")[4]
    two = vce.preference_loss_backward(z, ids, stats, torch.ones(2, device="cuda"), 2, reduction="none")
    one = vce.preference_loss_backward(z, ids, stats, torch.ones(1, device="cuda"), 1, reduction="none")
    assert torch.equal(one[:6], two[:6]) and (two[6:] != 0).any() and torch.all(one[6:] == 0)


def test_preference_without_pairs(vce):
    z, ids = logits(3, 50, F32), tokens(3, 50)
    off = torch.tensor([1]).cuda()
    loss, pairs, rewards, lp, stats, status = vce.preference_loss_forward(z, ids, off)
    assert vce.vce_get_status(status) == 0 and torch.isnan(loss).all() and pairs.numel() == 0 and torch.all(lp == 0)
    g = vce.preference_loss_backward(z, ids, stats, torch.ones(1, device="cuda"), 0)
    assert torch.all(g == 0)


# ---- autograd, streams, graphs ------------------------------------------------------------------


def test_autograd_matches_the_calls(vce):
    c = policy_case(12, 3001, BF16, 0.8, 9, ignored=[4])
    z = c["z"].clone().requires_grad_(True)
    lp, ent = vce.token_logprobs(z, c["ids"], 0.8)
    ga, gb = torch.randn(2, 12, device="cuda")
    torch.autograd.backward((lp, ent), (ga, gb))
    _, _, stats, _ = vce.ce_logprobs_forward(c["z"], c["ids"], 0.8)
    assert torch.equal(z.grad, vce.ce_logprobs_backward(c["z"], c["ids"], stats, ga, gb, 0.8))
    z.grad = None
    lp, none = vce.token_logprobs(z, c["ids"], 0.8, want_entropy=False)
    assert none is None
    lp.sum().backward()
    assert torch.equal(z.grad, vce.ce_logprobs_backward(c["z"], c["ids"], stats, torch.ones_like(lp), None, 0.8))
    z.grad = None
    _, ent = vce.token_logprobs(z, c["ids"], 0.8)
    ent.sum().backward()
    assert torch.equal(z.grad, vce.ce_logprobs_backward(c["z"], c["ids"], stats, None, torch.ones_like(lp), 0.8))
    kw = dict(kl_coef=0.1, entropy_coef=0.01, temperature=0.8)
    for reduction in ("mean", "sum", "none"):
        z.grad = None
        loss = vce.policy_loss(z, c["ids"], c["adv"], c["old"], c["ref"], c["w"], reduction=reduction, **kw)
        up = torch.rand_like(loss) + 0.5
        loss.backward(up)
        out = vce.policy_loss_forward(c["z"], c["ids"], c["adv"], c["old"], c["ref"], c["w"], reduction=reduction, **kw)
        assert torch.equal(loss.detach().reshape(-1), out[1] if reduction == "none" else out[0])
        assert torch.equal(z.grad, vce.policy_loss_backward(c["z"], c["ids"], out[4], up.reshape(-1), 0.8, reduction))
    off = torch.tensor([0, 4, 6, 9, 12]).cuda()
    for reduction in ("mean", "sum", "none"):
        z.grad = None
        loss = vce.preference_loss(z, c["ids"], off, c["ref"], reduction=reduction)
        up = torch.rand_like(loss) + 0.5
        loss.backward(up)
        out = vce.preference_loss_forward(c["z"], c["ids"], off, c["ref"], reduction=reduction)
        assert torch.equal(loss.detach().reshape(-1), out[1] if reduction == "none" else out[0])
        assert torch.equal(z.grad, vce.preference_loss_backward(c["z"], c["ids"], out[4], up.reshape(-1), 2, 1.0, reduction))


def _everything(vce, c, off, stream=None):
    kw = dict(kl_coef=0.05, entropy_coef=0.01)
    args = (c["z"], c["ids"], c["adv"], c["old"], c["ref"], c["w"])
    up = torch.full((1,), 0.5, device="cuda") if stream is None else c["up"]
    out = list(vce.ce_logprobs_forward(c["z"], c["ids"], stream=stream))
    out.append(vce.ce_logprobs_backward(c["z"], c["ids"], out[2], c["adv"], c["old"], stream=stream))
    f = vce.policy_loss_forward(*args, stream=stream, **kw)
    out += [t for t in f if t is not None]
    out.append(vce.policy_loss_backward(c["z"], c["ids"], f[4], up, stream=stream))
    out += [t for t in vce.policy_loss_forward_backward(*args, grad_output=up, stream=stream, **kw) if t is not None]
    f = vce.preference_loss_forward(c["z"], c["ids"], off, c["ref"], stream=stream)
    out += list(f)
    out.append(vce.preference_loss_backward(c["z"], c["ids"], f[4], up, 2, stream=stream))
    return out


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("T,V,dtype", [(12, 3001, BF16), (400, 9000, BF16), (14, 70000, F32)])
def test_same_bits_every_time_on_any_stream_and_in_graphs(vce, T, V, dtype):
    c = policy_case(T, V, dtype, 1.0, 11, ignored=[4])
    c["up"] = torch.full((1,), 0.5, device="cuda")
    off = torch.tensor([0, 4, 6, 9, T]).cuda()
    want = [t.clone() for t in _everything(vce, c, off)]
    torch.cuda.synchronize()
    for _ in range(3):
        assert _same(_everything(vce, c, off), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _everything(vce, c, off, s)
    s.synchronize()
    assert _same(got, want)
    graphs, outs = [], []
    for _ in range(2):                      # two graphs that run at once
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_everything(vce, c, off))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got in outs:
        assert _same(got, want)


def test_two_calls_at_once(vce):
    a, b = policy_case(300, 20000, BF16, 1.0, 1), policy_case(200, 30001, BF16, 1.0, 2)
    off = torch.tensor([0, 4, 6, 9, 12]).cuda()
    for c in (a, b):
        c["up"] = torch.full((1,), 0.5, device="cuda")
    want = [[t.clone() for t in _everything(vce, c, off)] for c in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [_everything(vce, c, off, s) for c, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert _same(got[0], want[0]) and _same(got[1], want[1])


def test_autograd_in_a_graph(vce):
    c = policy_case(20, 5000, BF16, 1.0, 12)
    z = c["z"].clone().requires_grad_(True)
    off = torch.tensor([0, 4, 6, 9, 20]).cuda()

    def step():
        z.grad = None
        lp, ent = vce.token_logprobs(z, c["ids"])
        loss = vce.policy_loss(z, c["ids"], c["adv"], c["old"], c["ref"], kl_coef=0.1, entropy_coef=0.1)
        loss = loss + vce.preference_loss(z, c["ids"], off, c["ref"]) + (lp * c["adv"]).sum() + ent.mean()
        loss.backward()
        return loss.detach()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = step().clone()
        wg = z.grad.clone()
        z.grad = None
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(z.grad, wg)


# ---- refusals ---------------------------------------------------------------------------------------


def test_refusals(vce):
    z, ids = logits(6, 300, BF16), tokens(6, 300)
    ones = torch.ones(6, device="cuda")
    one = torch.ones(1, device="cuda")
    off = torch.tensor([0, 2, 6]).cuda()
    with pytest.raises(ValueError):
        vce.ce_logprobs_forward(z[0], ids)
    with pytest.raises(TypeError):
        vce.ce_logprobs_forward(z.half(), ids)
    with pytest.raises(TypeError):
        vce.ce_logprobs_forward(z, ids.int())
    with pytest.raises(TypeError):
        vce.ce_logprobs_forward(z, None)
    with pytest.raises(ValueError):
        vce.ce_logprobs_forward(z, ids[:5])
    with pytest.raises(ValueError):
        vce.ce_logprobs_forward(z.t()[:6], ids)
    with pytest.raises(ValueError):
        vce.ce_logprobs_forward(z, ids.cpu())
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(vce.VceError):
            vce.ce_logprobs_forward(z, ids, tau)
    _, _, stats, _ = vce.ce_logprobs_forward(z, ids)
    with pytest.raises(vce.VceError):   # in place
        vce.ce_logprobs_backward(z, ids, stats, ones, grad_logits=z)
    with pytest.raises(TypeError):
        vce.policy_loss_forward(z, ids, None)
    for kw in (dict(clip_low=-0.1), dict(clip_high=float("nan")), dict(dual_clip=0.5), dict(kl_coef=0.1),
               dict(entropy_coef=float("inf")), dict(kl_coef=float("nan"))):
        with pytest.raises(vce.VceError):
            vce.policy_loss_forward(z, ids, ones, **kw)
        with pytest.raises(vce.VceError):
            vce.policy_loss_forward_backward(z, ids, ones, **kw)
    with pytest.raises(KeyError):
        vce.policy_loss_forward(z, ids, ones, reduction="median")
    with pytest.raises(ValueError):
        vce.policy_loss_forward_backward(z, ids, ones, grad_output=ones)
    with pytest.raises(vce.VceError):
        vce.policy_loss_forward_backward(z, ids, ones, grad_logits=z)
    with pytest.raises(ValueError):
        vce.preference_loss_forward(z, ids, off[:2])
    with pytest.raises(KeyError):
        vce.preference_loss_forward(z, ids, off, kind="linear")
    for kw in (dict(beta=0.0), dict(beta=float("inf")), dict(label_smoothing=0.6), dict(kind="ipo", label_smoothing=0.1),
               dict(margin=float("nan"))):
        with pytest.raises(vce.VceError):
            vce.preference_loss_forward(z, ids, off, **kw)
    stats = vce.preference_loss_forward(z, ids, off)[4]
    with pytest.raises(ValueError):
        vce.preference_loss_backward(z, ids, stats, one, 1, reduction="none", grad_logits=torch.empty(6, 299, device="cuda"))
    torch.cuda.synchronize()


# ---- waits that give up -----------------------------------------------------------------------------


@pytest.mark.parametrize("T,V", [(3, 70000), (2, 20000), (400, 9000), (2, 200000), (170, 128256)])
def test_waits_that_give_up_are_reported(vce, T, V):
    """The last block of every cluster waits in vain for its gradient's coefficients, once the statistics have been
    exchanged and the first block has its results: a status, NaN, and a context that stays usable."""
    z, ids = logits(T, V, BF16).contiguous(), tokens(T, V)
    adv = torch.linspace(-1, 1, T).cuda()
    loss, rows, lp, _, status = vce.vce_test_policy_stall(z, ids, adv)
    code = vce.vce_get_status(status)
    assert 105 <= code <= 109 and "gave up" in vce.vce_status_string(code)
    assert torch.isnan(rows).all() and torch.isnan(lp).all() and torch.isnan(loss).all()
    one = vce.policy_loss_forward_backward(z, ids, adv, reduction="sum")
    assert vce.vce_get_status(one[5]) == 0 and torch.isfinite(one[4]).all() and torch.isfinite(one[2]).all()


@pytest.mark.parametrize("T,V", [(3, 20000), (5, 100000)])
def test_backward_waits_that_give_up_leave_nan(vce, T, V):
    z, ids = logits(T, V, BF16).contiguous(), tokens(T, V)
    stats = vce.policy_loss_forward(z, ids, torch.ones(T, device="cuda"), reduction="sum")[4]
    one = torch.ones(1, device="cuda")
    want = vce.policy_loss_backward(z, ids, stats, one, reduction="sum")
    got = vce.vce_test_policy_bwd_stall(z, ids, stats)
    vectors = V // 8                                  # both are multiples of 8: rows of whole vectors
    parts = -(-vectors // 4096)
    last = -(-vectors // parts) * (parts - 1) * 8     # the first column of the last block
    assert torch.isnan(got[:, last:]).all() and torch.equal(got[:, :last], want[:, :last])
    assert torch.equal(vce.policy_loss_backward(z, ids, stats, one, reduction="sum"), want)
