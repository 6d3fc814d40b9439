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


def _process_everything(vce):
    """logits_process and its gradient on every way through its kernel: no lists, a word for every column,
    hash tables, windows after a full table; aligned and not; masked, biased."""
    g = torch.Generator().manual_seed(11)
    out = []
    for T, V, dtype, lens in ((5, 4001, torch.float32, [0, 7, 900, 40, 3]), (3, 128256, torch.bfloat16, [3000, 0, 500]),
                              (300, 20000, torch.bfloat16, [50] * 300), (41, 70001, torch.bfloat16, [0] * 40 + [9000]),
                              (2, 32000, torch.float32, [20000, 9000])):
        z = (2.0 * torch.randn(T, V, generator=g)).to(dtype).cuda()
        up = torch.randn(T, V, generator=g).to(dtype).cuda()
        mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (T, (V + 31) // 32), generator=g, dtype=torch.int64).to(torch.int32).cuda()
        offsets = torch.tensor([0] + lens).cumsum(0).cuda()
        kw = dict(temperature=torch.full((T,), 0.7, device="cuda"), repetition_penalty=torch.full((T,), 1.3, device="cuda"),
                  history_ids=torch.randint(0, V, (sum(lens),), generator=g).cuda(), history_offsets=offsets)
        bias = dict(bias_ids=torch.arange(10, device="cuda").mul(V // 10).repeat(T), bias_values=torch.randn(10 * T, generator=g).cuda(),
                    bias_offsets=torch.arange(T + 1, device="cuda") * 10)
        for m in (None, mask):
            out += list(vce.logits_process(z, mask=m, frequency_penalty=torch.full((T,), 0.2, device="cuda"), **kw, **bias))
            out += list(vce.logits_process_backward(up, z, mask=m, **kw))
            out += list(vce.logits_process(z, mask=m, temperature=kw["temperature"]))
    torch.cuda.synchronize()
    return [t.clone() for t in out]


def test_debug_build_of_the_processing_checks_nothing_wrong(debug_library):
    import vocab_cross_entropy_gb300 as vce
    want = _process_everything(vce)
    prev = vce.use_library(debug_library)
    try:
        vce.vce_debug_status()
        got = _process_everything(vce)
        assert vce.vce_debug_status() == 0
    finally:
        vce.restore_library(prev)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_debug_build_changes_no_bit_nor_a_nan(debug_library):
    """The other operators bit for bit, NaN for NaN."""
    import vocab_cross_entropy_gb300 as vce
    want = _run_everything(vce)
    prev = vce.use_library(debug_library)
    try:
        got = _run_everything(vce)
        assert vce.vce_debug_status() == 0
    finally:
        vce.restore_library(prev)
    for a, b in zip(got, want):
        assert torch.equal(torch.isnan(a.float()), torch.isnan(b.float()))
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
