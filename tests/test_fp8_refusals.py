"""The fp8 calls refuse operands that lie over one another, before anything is enqueued (no GPU: the addresses are never
followed, and what is not refused is the device's turn)."""
import pytest

KB = 1024
ARG = -8
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def vce():
    from vocab_cross_entropy_gb300 import build
    build.build()
    import vocab_cross_entropy_gb300 as v
    return v


@pytest.fixture()
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses that are not memory")


def quantize(vce, x, q, s, R=16, D=256, ld=256, dt=BF16, rows=1):
    return vce.lib.vce_quantize_fp8(x, dt, R, D, ld, rows, q, s, None)


def linear(vce, x, xs, w, ws, out, T=4, D=256, V=64, dt=BF16, ld=64):
    return vce.lib.vce_linear_fp8(x, xs, w, ws, T, D, V, out, dt, ld, None)


def test_quantize_refuses_overlap(vce, no_gpu):
    # x 8 KB from 64 KB, q 4 KB, scales 16 x 2 x 4 = 128 bytes
    x, q, s = 64 * KB, 128 * KB, 192 * KB
    assert quantize(vce, x, q, s) != ARG
    assert quantize(vce, x, x + 8 * KB, s) != ARG and quantize(vce, x, x - 4 * KB, s) != ARG
    for over in (x, x + 8 * KB - 16, x - 4 * KB + 16, x + 2 * KB):
        assert quantize(vce, x, over, s) == ARG
    for over in (x, x + 8 * KB - 4, x - 124):
        assert quantize(vce, x, q, over) == ARG
    assert quantize(vce, x, q, x - 128) != ARG and quantize(vce, x, q, x + 8 * KB) != ARG
    for over in (q, q + 4 * KB - 4, q - 124):
        assert quantize(vce, x, q, over) == ARG
    # rows of a wider matrix: its extent ends with the last row's columns
    assert quantize(vce, x, x + (15 * 512 + 256) * 2, s, ld=512) != ARG
    assert quantize(vce, x, x + (15 * 512 + 256) * 2 - 16, s, ld=512) == ARG
    assert quantize(vce, x, x, s, R=0) == 0


def test_linear_refuses_overlap(vce, no_gpu):
    # x 1 KB, its scales 32 bytes, w 16 KB, its scales 8 bytes, out 512 bytes
    x, xs, w, ws, out = 64 * KB, 96 * KB, 128 * KB, 192 * KB, 256 * KB
    assert linear(vce, x, xs, w, ws, out) != ARG
    for at, n in ((x, KB), (xs, 32), (w, 16 * KB), (ws, 8)):
        for over in (at, at + n - 4, at - 508):
            assert linear(vce, x, xs, w, ws, over) == ARG
        assert linear(vce, x, xs, w, ws, at + n) != ARG and linear(vce, x, xs, w, ws, at - 512) != ARG
    assert linear(vce, x, xs, x, ws, out) != ARG      # operands may share what nothing writes
    assert linear(vce, x, xs, w, ws, x, T=0) == 0


@pytest.mark.gpu
def test_on_the_gpu(vce):
    import torch
    x = torch.zeros(16, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(vce.VceError):
        vce.quantize_fp8(x, q=x.view(torch.float8_e4m3fn).view(-1)[:16 * 256].view(16, 256))
    q, s = vce.quantize_fp8(x)
    w, ws = vce.quantize_fp8(x, 128)
    with pytest.raises(vce.VceError):
        vce.linear_fp8(q, s, w, ws, out=w.view(torch.bfloat16).view(-1)[:256].view(16, 16))
