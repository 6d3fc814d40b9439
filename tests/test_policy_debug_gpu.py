"""The post-training losses and the fp8 head in the debug build (device-side index checks): no check fails on valid
inputs of every kernel, and every output equals the release build's bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def debug_library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    from vocab_cross_entropy_gb300 import build as b
    return b.build(debug_checks=True)


def _run_everything(vce):
    g = torch.Generator().manual_seed(7)
    out = []
    for T, V, dtype in ((5, 401, torch.float32), (300, 4001, torch.bfloat16), (340, 20000, torch.bfloat16),
                        (9, 70001, torch.float32), (160, 70001, torch.bfloat16), (2, 530001, torch.bfloat16)):
        full = torch.randn(T, V + 5, generator=g).to(dtype).cuda()
        z = full[:, 3:V + 3]
        ids = torch.randint(0, V, (T,), generator=g).cuda()
        ids[T // 2] = -100
        adv, old = torch.randn(2, T, generator=g).cuda()
        up = torch.ones(1, device="cuda")
        for ent in (True, False):
            f = vce.ce_logprobs_forward(z, ids, 0.9, want_entropy=ent)
            out += [t for t in f if t is not None]
            out.append(vce.ce_logprobs_backward(z, ids, f[2], adv, old if ent else None, 0.9))
            kw = dict(entropy_coef=0.1 if ent else 0.0)
            f = vce.policy_loss_forward(z, ids, adv, old - 9, **kw)
            out += [t for t in f if t is not None]
            out.append(vce.policy_loss_backward(z, ids, f[4], up, grad_dtype=torch.float32))
            out += [t for t in vce.policy_loss_forward_backward(z, ids, adv, old - 9, **kw) if t is not None]
        off = torch.tensor([0, T // 3, T // 2, T - 1, T]).cuda()
        f = vce.preference_loss_forward(z, ids, off, old)
        out += list(f) + [vce.preference_loss_backward(z, ids, f[4], up, 2)]
    for T, D, V in ((1, 400, 900), (40, 272, 3001), (300, 512, 1024), (129, 144, 777)):
        x, xs = vce.quantize_fp8(torch.randn(T, D, generator=g).cuda())
        w, ws = vce.quantize_fp8(torch.randn(V, D, generator=g).cuda(), 128)
        out += [x.view(torch.uint8), xs, w.view(torch.uint8), ws, vce.linear_fp8(x, xs, w, ws),
                vce.linear_fp8(x, xs, w, ws, out_dtype=torch.float32)]
    torch.cuda.synchronize()
    return [t.clone() for t in out]


def test_debug_build_checks_nothing_wrong_and_changes_no_bit(debug_library):
    import vocab_cross_entropy_gb300 as vce
    want = _run_everything(vce)
    prev = vce.use_library(debug_library)
    try:
        assert vce.vce_debug_checks()
        vce.vce_debug_status()
        got = _run_everything(vce)
        assert vce.vce_debug_status() == 0
    finally:
        vce.restore_library(prev)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
