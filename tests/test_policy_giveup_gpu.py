"""The one pass where a wait gave up: no gradient keeps what the buffer held before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vce():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")
    import vocab_cross_entropy_gb300 as v
    return v


@pytest.mark.parametrize("T,V", [(3, 70000), (2, 20000), (400, 9000), (2, 200000), (170, 128256)])
def test_gradients_behind_a_wait_that_gave_up_are_nan(vce, T, V):
    """The hook's buffer holds zeros, and no gradient of these rows is 0: the last block of every cluster waits in vain,
    in all of its rows, and the others are right or have waited in vain too."""
    g = torch.Generator().manual_seed(T + V)
    z = torch.randn(T, V, generator=g).bfloat16().cuda()
    ids = torch.randint(0, V, (T,), generator=g).cuda()
    _, _, _, grad, status = vce.vce_test_policy_stall(z, ids, torch.ones(T, device="cuda"))
    assert 105 <= vce.vce_get_status(status) <= 109
    assert (grad != 0).all() and grad.isnan().any(1).all()
    want = vce.policy_loss_forward_backward(z, ids, torch.ones(T, device="cuda"), reduction="sum")[4]
    assert torch.equal(torch.where(grad.isnan(), want, grad), want)
