"""The rewards of sequences with a row that has no log-probability: NaN, and of no other sequence."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("what", ["token", "masked", "nan"])
@pytest.mark.parametrize("row,seq", [(0, 0), (4, 1), (11, 3)])
def test_reward_of_a_sequence_with_an_error_is_nan(vce, row, seq, what, average):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(12, 400, generator=g).cuda()
    ids = torch.randint(0, 400, (12,), generator=g).cuda()
    off = torch.tensor([0, 3, 6, 9, 12]).cuda()
    _, pairs, want, _, _, _ = vce.preference_loss_forward(z, ids, off, average=average, reduction="none")
    if what == "token":
        ids[row] = 400
    else:
        z[row] = float("nan") if what == "nan" else float("-inf")
    _, got_pairs, got, _, _, status = vce.preference_loss_forward(z, ids, off, average=average, reduction="none")
    assert vce.vce_get_status(status) == (1 if what == "token" else 0)
    assert torch.isnan(got[seq]) and torch.isnan(got_pairs[seq // 2])
    rest = torch.arange(4) != seq
    assert torch.equal(got[rest.cuda()], want[rest.cuda()])
    assert torch.equal(got_pairs[1 - seq // 2], pairs[1 - seq // 2])
