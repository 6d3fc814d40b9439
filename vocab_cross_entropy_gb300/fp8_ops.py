"""The head in 8-bit floating point (``include/vce_fp8.h``): a matrix to e4m3 with a scale for each block of
128, and the logits of hidden states and weights held so.  Argument checks and marshalling only, as in
``logits_ops``."""
from __future__ import annotations

import torch

from . import _DT
from .logits_ops import _F32, _flat, _matrix, _matrix_out, _out, _run

_E4M3 = torch.float8_e4m3fn
FP8_BLOCK = 128


def _blocks(n):
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def quantize_fp8(x, block_rows=1, *, q=None, scales=None, stream=None):
    """A [R, D] float32 or bfloat16 matrix as e4m3 values and a power of two for each block of block_rows x
    128 elements (block_rows 1: hidden states; 128: weights), the least that keeps the block within +-448.

    Returns (q [R, D] float8_e4m3fn, scales [ceil(R / block_rows), ceil(D / 128)] float32): x is q times
    its block's scale, to a rounding of q.
    """
    dt, R, D, ld = _matrix(x, "x")
    if block_rows not in (1, FP8_BLOCK):
        raise ValueError(f"block_rows: {block_rows}, expected 1 or {FP8_BLOCK}")
    dev = x.device
    q, p_q = _out(q, "q", _E4M3, (R, D), dev, stream)
    scales, p_s = _out(scales, "scales", _F32, (-(-R // block_rows), _blocks(D)), dev, stream)
    _run("vce_quantize_fp8", dev, stream, x.data_ptr(), dt, R, D, ld, block_rows, p_q, p_s)
    return q, scales


def linear_fp8(x, x_scales, w, w_scales, *, out=None, out_dtype=torch.bfloat16, stream=None):
    """Logits [T, V] of hidden states x [T, D] with a scale for each row and block of 128 columns, and weights w
    [V, D] with one for each block of 128 x 128 (``quantize_fp8``'s results, or any e4m3 values and float32
    scales).  D a multiple of 16.  No gradient: the head is frozen.  Returns out (float32 or bfloat16)."""
    for t, name in ((x, "x"), (w, "w")):
        if t.dim() != 2:
            raise ValueError(f"{name}: expected a 2-D tensor")
    if x.device.type != "cuda":
        raise ValueError(f"x: on {x.device}, expected a CUDA device")
    (T, D), V, dev = x.shape, w.shape[0], x.device
    if out is None and out_dtype not in _DT:
        raise TypeError(f"out_dtype: unsupported dtype {out_dtype}; use float32 or bfloat16")
    p = (_flat(x, "x", _E4M3, (T, D), dev), _flat(x_scales, "x_scales", _F32, (T, _blocks(D)), dev),
         _flat(w, "w", _E4M3, (V, D), dev), _flat(w_scales, "w_scales", _F32, (_blocks(V), _blocks(D)), dev))
    out, p_out, odt, ld = _matrix_out(out, "out", T, V, out_dtype, dev, stream)
    _run("vce_linear_fp8", dev, stream, *p, T, D, V, p_out, odt, ld)
    return out


def vce_test_linear_fp8_stall(x, x_scales, w, w_scales, wait_ns=50_000_000, *, stream=None):
    """Test hook: linear_fp8 whose stages never complete.  Returns out (float32)."""
    (T, D), V = x.shape, w.shape[0]
    out = torch.zeros(T, V, device=x.device)
    _run("vce_test_linear_fp8_stall", x.device, stream, x.data_ptr(), x_scales.data_ptr(), w.data_ptr(),
         w_scales.data_ptr(), T, D, V, out.data_ptr(), int(wait_ns))
    return out
