"""Block-FP8 linear layer in numpy float64.

TEST INFRASTRUCTURE ONLY.  Weights: e4m3 codes [N, K], one fp32 scale per block
of 128 outputs x 128 inputs.  Tokens are quantised per 128 inputs: scale
max|x| * (1 / 448) (1 for zeros), codes e4m3(x / scale); 1 / 448, the product
and the division each rounded to fp32.  Sums in float64.
"""
import numpy as np

from .lmhead_ref import e4m3_decode, e4m3_encode

BLOCK = 128


def quantize_tokens(x_f32):
    """[T, K] -> (codes [T, K], scales [T, ceil(K / 128)])."""
    x = np.asarray(x_f32, np.float32)
    T, K = x.shape
    kb = -(-K // BLOCK)
    p = np.zeros((T, kb * BLOCK), np.float32)
    p[:, :K] = x
    p = p.reshape(T, kb, BLOCK)
    amax = np.abs(p).max(axis=2)
    s = np.where(amax > 0, amax * (np.float32(1) / np.float32(448)), np.float32(1)).astype(np.float32)
    codes = e4m3_encode((p / s[:, :, None]).astype(np.float32))
    return codes.reshape(T, kb * BLOCK)[:, :K], s


def linear(x_f32, w_codes, w_scales):
    """(y [T, N], sum of magnitudes [T, N]) in float64."""
    codes, sx = quantize_tokens(x_f32)
    N, K = w_codes.shape
    y = np.zeros((codes.shape[0], N))
    mag = np.zeros_like(y)
    for b in range(sx.shape[1]):
        cols = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        s = sx[:, b].astype(np.float64)[:, None] * np.repeat(w_scales[:, b].astype(np.float64), BLOCK)[None, :N]
        xd, wd = e4m3_decode(codes[:, cols]), e4m3_decode(w_codes[:, cols])
        y += (xd @ wd.T) * s
        mag += (np.abs(xd) @ np.abs(wd).T) * s
    return y, mag
