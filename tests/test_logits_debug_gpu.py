"""The operators around the cross-entropy in the debug build (device-side index checks): no check fails
on valid inputs of every kernel, and every output equals the release build's bit for bit."""
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
    for T, V, dtype, k in ((5, 4001, torch.float32, 9), (340, 20000, torch.bfloat16, 40), (2, 530001, torch.bfloat16, 12)):
        z = torch.randn(T, V, generator=g).to(dtype).cuda()
        teacher = torch.randn(T, V, generator=g).to(dtype).cuda()
        values, ids, lse, tail = vce.ce_topk(teacher, k, 2.0)
        fwd = vce.ce_distill_forward(z, ids, values, tail, 2.0)
        up = torch.ones(1, device="cuda")
        out += [values, ids, lse, tail, *fwd[:4], vce.ce_distill_backward(z, ids, fwd[2], fwd[3], up, 2.0)]
        out += list(vce.ce_distill_forward_backward(z, ids, values, tail, 2.0)[:3])
        mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, (V + 31) // 32), generator=g, dtype=torch.int64).to(torch.int32).cuda()
        history = torch.randint(0, V, (T * 50,), generator=g).cuda()
        kw = dict(history_ids=history, history_offsets=torch.arange(T + 1, device="cuda") * 50, mask=mask,
                  repetition_penalty=torch.full((T,), 1.3, device="cuda"))
        out += list(vce.logits_process(z, **kw)) + list(vce.logits_process_backward(z, teacher, **kw))
        out += list(vce.logits_process(z, mask=mask))
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
        assert torch.equal(a, b) or torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
