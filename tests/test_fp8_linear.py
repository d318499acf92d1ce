"""The block-FP8 linear layer without a GPU: the oracle against brute force and
against torch's e4m3, and the refusals of the entry points and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.fp8_linear_ref as F
import oracle.lmhead_ref as L
import weight_only_int4_fp32_b200 as lm

BAD = lm.LING_MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (2, 3, 130), (3, 129, 256), (2, 130, 300)])
def test_oracle_is_the_sum_over_dequantised_weights(T, N, K):
    rng = np.random.default_rng(T + N + K)
    x = rng.normal(size=(T, K)).astype(np.float32)
    w = rng.integers(0, 0x7E, size=(N, K)).astype(np.uint8) | (rng.integers(0, 2, size=(N, K)) << 7).astype(np.uint8)
    s = rng.random((-(-N // 128), -(-K // 128))).astype(np.float32) + 0.1
    y, mag = F.linear(x, w, s)
    codes, sx = F.quantize_tokens(x)
    for t in range(T):
        for n in range(0, N, max(1, N // 5)):
            want = sum(float(L.e4m3_decode(codes[t, k])) * float(sx[t, k // 128]) * float(L.e4m3_decode(w[n, k]))
                       * float(s[n // 128, k // 128]) for k in range(K))
            assert abs(y[t, n] - want) <= 1e-12 * mag[t, n] + 1e-300


def test_oracle_token_codes_are_torchs():
    x = torch.randn(5, 300, generator=torch.Generator().manual_seed(0)).bfloat16().float()
    x[1, 128:256] = 0.0
    codes, sx = F.quantize_tokens(x.numpy())
    for b in range(3):
        blk = x[:, b * 128:(b + 1) * 128]
        s = blk.abs().amax(1, keepdim=True) * (torch.ones(1) / torch.full((1,), 448.0))
        s[s == 0] = 1.0
        assert np.array_equal(s[:, 0].numpy(), sx[:, b])
        q = (blk / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(q, codes[:, b * 128:(b + 1) * 128])


def _create(codes=0x100000, scales=0x200000, N=256, K=256, T=8):
    h = ctypes.c_void_p()
    return lm.lib.ling_moe_fp8_linear_create(codes, scales, N, K, T, ctypes.byref(h)), h.value


@pytest.mark.parametrize("kw,code", [
    (dict(codes=None), BAD), (dict(scales=None), BAD), (dict(scales=0x200002), BAD), (dict(N=0), BAD), (dict(K=-1), BAD),
    (dict(T=0), BAD), (dict(N=(1 << 24) + 1), lm.LING_MOE_ERR_UNSUPPORTED),
    (dict(K=(1 << 22) + 1), lm.LING_MOE_ERR_UNSUPPORTED), (dict(T=(1 << 24) + 1), lm.LING_MOE_ERR_UNSUPPORTED)])
def test_create_refuses(kw, code):
    assert _create(**kw) == (code, None)
    assert lm.lib.ling_moe_fp8_linear_create(0x100000, 0x200000, 8, 8, 8, None) == BAD


def test_null_handle():
    assert lm.lib.ling_moe_fp8_linear_forward(None, 16, 8, 1, 32, 0, 8, None) == BAD
    assert lm.lib.ling_moe_fp8_linear_status(None, None) == BAD
    assert lm.lib.ling_moe_fp8_linear_test_set_wait(None, 0, 0) == BAD
    assert lm.lib.ling_moe_fp8_linear_launch_count(None) == 0
    lm.lib.ling_moe_fp8_linear_destroy(None)


def test_binding_refuses_wrong_tensors():
    with pytest.raises(ValueError):
        lm.BlockFP8Linear(torch.zeros(8, 8), torch.zeros(1, 1), 4)                       # not e4m3
    with pytest.raises(ValueError):
        lm.BlockFP8Linear(torch.zeros(8, 8, dtype=torch.uint8), torch.zeros(1, 1), 4)    # not on the GPU
    f = object.__new__(lm.BlockFP8Linear)
    f.out_features, f.in_features, f.handle, f._torch = 8, 16, None, torch
    with pytest.raises(ValueError):
        f.forward(torch.zeros(2, 16, dtype=torch.bfloat16))
