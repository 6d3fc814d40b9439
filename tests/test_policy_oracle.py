"""The fp64 oracle of the post-training losses and the fp8 head, against closed forms, differences and torch."""
import numpy as np
import pytest
import torch

from oracle import policy_oracle as O


def _case(T=6, V=11, seed=0):
    g = np.random.default_rng(seed)
    z = 2 * g.standard_normal((T, V))
    ids = g.integers(0, V, T)
    return g, z, ids


def test_rows_against_torch():
    g, z, ids = _case()
    ids[2] = O.IGNORE_INDEX
    r = O.rows(z, ids, 0.7)
    logp = torch.log_softmax(torch.from_numpy(z) / 0.7, 1)
    for i in range(len(ids)):
        if ids[i] == O.IGNORE_INDEX:
            assert r["lp"][i] == 0 and r["ent"][i] == 0
            continue
        assert abs(r["lp"][i] - float(logp[i, ids[i]])) < 1e-13
        assert abs(r["ent"][i] + float((logp[i].exp() * logp[i]).sum())) < 1e-13


def test_rows_with_masks_and_certainty():
    z = np.array([[0.0, -np.inf, -np.inf], [0.0, 1.0, -np.inf], [800.0, 0.0, 0.0]])
    r = O.rows(z, np.array([0, 2, 0]))
    assert r["lp"][0] == 0 and r["ent"][0] == 0
    assert r["lp"][1] == -np.inf and r["ent"][1] > 0.5
    assert r["lp"][2] <= 0 and r["ent"][2] >= 0 and r["lp"][2] > -1e-300


def _difference(f, z, grad, tol):
    h = 1e-6
    for i in range(z.shape[0]):
        for j in range(z.shape[1]):
            up, down = z.copy(), z.copy()
            up[i, j] += h
            down[i, j] -= h
            assert abs((f(up) - f(down)) / (2 * h) - grad[i, j]) < tol


@pytest.mark.parametrize("kl,ent,dual,weights", [(0, 0, 0, False), (0.3, 0.2, 0, True), (0.1, 0.0, 2.0, False)])
def test_policy_gradient_against_differences(kl, ent, dual, weights):
    g, z, ids = _case()
    ids[1] = O.IGNORE_INDEX
    lp = O.rows(z, np.where(ids < 0, 0, ids), 1.3)["lp"]
    old, ref = lp + 0.4 * g.standard_normal(6), lp + 0.4 * g.standard_normal(6)
    adv = g.standard_normal(6)
    w = g.random(6) if weights else None
    f = lambda x: O.policy(x, ids, adv, old, ref, w, 0.2, 0.3, dual, kl, ent, 1.3)
    _difference(lambda x: f(x)["loss"], z, f(z)["grad"], 1e-8)


@pytest.mark.parametrize("kind,average", [("sigmoid", False), ("hinge", True), ("ipo", False), ("sigmoid", True)])
def test_preference_gradient_against_differences(kind, average):
    g, z, ids = _case(9)
    ids[3] = O.IGNORE_INDEX
    offsets = np.array([1, 3, 6, 6, 8])
    ref = O.rows(z, np.where(ids < 0, 0, ids), 0.9)["lp"] + 0.3 * g.standard_normal(9)
    f = lambda x: O.preference(x, ids, offsets, ref, 0.2, kind, 0.1 if kind == "sigmoid" else 0.0, 0.05, average, 0.9)
    _difference(lambda x: f(x)["loss"], z, f(z)["grad"], 1e-6)


def test_e4m3_against_torch():
    table = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_values(), table, equal_nan=True)
    g = np.random.default_rng(1)
    v = np.concatenate([g.uniform(-448, 448, 4000), g.uniform(-0.02, 0.02, 4000), np.arange(-448, 449) / 2.0 ** 10,
                        table[np.isfinite(table)]]).astype(np.float32)
    assert np.array_equal(O.to_e4m3(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())


def test_quantize_keeps_blocks_within_range():
    g = np.random.default_rng(2)
    x = g.standard_normal((130, 200)) * np.exp(3 * g.standard_normal((130, 1)))
    x[128:, :128] = 0
    for rows in (1, 128):
        q, s = O.quantize(x, rows)
        assert np.all(np.abs(q) <= 448) and np.all(np.log2(s) == np.rint(np.log2(s)))
        wide = np.repeat(np.repeat(s, rows, 0)[:130], 128, 1)[:, :200]
        assert np.all(np.abs(q * wide - x) <= np.maximum(2.0 ** -4 * np.abs(x), wide * 2.0 ** -10))
        assert s[-1, 0] == 1.0


def test_argument_errors_need_no_gpu():
    """The C entry points refuse what they can see before any CUDA call."""
    import ctypes
    from vocab_cross_entropy_gb300 import build
    lib = ctypes.CDLL(build.build())
    P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    x, rows = P(0x1000), [P, i32, i64, i64, i64]
    f = lib.ce_logprobs_forward
    f.argtypes = rows + [P, i64, f32, P, P, P, P, P]
    call = lambda dt=1, T=4, V=8, ld=8, ids=x, tau=1.0, stats=x, status=x: f(x, dt, T, V, ld, ids, -100, tau, x, None, stats, status, None)
    assert call(dt=7) == -2 and call(V=0) == -3 and call(T=-1) == -3 and call(T=1 << 24) == -3 and call(V=1 << 22, ld=1 << 22) == -3
    assert call(ld=7) == -4 and call(ids=None) == -1 and call(status=None) == -1
    assert call(tau=0.0) == call(tau=float("nan")) == call(tau=-1.0) == -8
    assert call(ids=P(0x1004)) == -5 and call(stats=P(0x1008)) == -5
    b = lib.ce_logprobs_backward
    b.argtypes = rows + [P, f32, P, P, P, P, i32, i64, P]
    assert b(x, 1, 4, 8, 8, x, 1.0, x, x, None, x, 1, 8, None) == -8          # in place
    assert b(x, 1, 4, 8, 8, x, 1.0, None, x, None, P(0x9000), 1, 8, None) == -1
    assert b(x, 1, 4, 8, 8, x, 1.0, x, x, None, P(0x9000), 1, 7, None) == -4
    params = (f32 * 5)(0.2, 0.2, 0.0, 0.0, 0.0)
    g = lib.policy_loss_forward
    g.argtypes = rows + [P, i64, f32, P, P, P, P, P, i32, P, P, P, P, P, P, P]
    call = lambda p=params, red=2, adv=x, ref=None, loss=x: g(x, 1, 4, 8, 8, x, -100, 1.0, None, adv, ref, None, p, red, x, loss, x, None, x, x, None)
    assert call(p=None) == -1 and call(red=3) == -2 and call(adv=None) == -1 and call(loss=None) == -1
    for bad in ((-0.1, 0.2, 0, 0, 0), (0.2, -1, 0, 0, 0), (0.2, 0.2, 0.5, 0, 0), (0.2, 0.2, 0, 0.1, 0), (0.2, 0.2, 0, 0, float("inf"))):
        assert call(p=(f32 * 5)(*bad)) == -8
    class Pref(ctypes.Structure):
        _fields_ = [("kind", i32), ("beta", f32), ("eps", f32), ("margin", f32), ("average", i32)]
    h = lib.preference_loss_forward
    h.argtypes = rows + [P, i64, f32, P, i64, P, P, i32, P, P, P, P, P, P, P]
    call = lambda p, n=2, off=x: h(x, 1, 4, 8, 8, x, -100, 1.0, off, n, None, ctypes.byref(p), 2, x, x, x, x, x, x, None)
    ok = (0, 0.1, 0.0, 0.0, 0)
    assert call(Pref(*ok), n=-1) == -3 and call(Pref(*ok), off=None) == -1
    for bad in ((3, 0.1, 0, 0, 0), (0, 0.0, 0, 0, 0), (0, 0.1, 0.6, 0, 0), (1, 0.1, 0.1, 0, 0), (0, 0.1, 0, float("nan"), 0), (0, 0.1, 0, 0, 2)):
        assert call(Pref(*bad)) == -8
    q = lib.vce_quantize_fp8
    q.argtypes = rows + [i32, P, P, P]
    assert q(x, 1, 4, 0, 8, 1, x, x, None) == -3 and q(x, 1, 4, 8, 8, 64, x, x, None) == -8 and q(x, 1, 4, 8, 7, 1, x, x, None) == -4
    assert q(x, 5, 4, 8, 8, 1, x, x, None) == -2 and q(x, 1, 4, 8, 8, 1, None, x, None) == -1
    l = lib.vce_linear_fp8
    l.argtypes = [P, P, P, P, i64, i64, i64, P, i32, i64, P]
    assert l(x, x, x, x, 4, 24, 8, x, 1, 8, None) == -3 and l(x, x, x, x, 4, 32, 8, x, 1, 7, None) == -4
    assert l(P(0x1008), x, x, x, 4, 32, 8, x, 1, 8, None) == -5 and l(x, None, x, x, 4, 32, 8, x, 1, 8, None) == -1
    assert l(x, x, x, x, 4, 32, 8, x, 9, 8, None) == -2
