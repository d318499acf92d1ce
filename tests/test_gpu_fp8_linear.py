"""The block-FP8 linear layer on the GPU against the 64-bit oracle.

Tolerance, u = 2^-24, M = sum of |products| scaled.  A block's sum of exact
products: mma.sync takes 8 chained instructions per block, tcgen05 4, each
taken as its exact result rounded once, possibly toward zero (2 u of the
block's magnitudes): at most 16 u M over all blocks.  The scales' product
rounds once (1 u), its product with the block sum and the addition once per
block (kb u), the 8 warps' sums of the streaming kernel 8 times.  So
|gpu - exact| <= (16 + 1 + kb + 8) u M, and for a bf16 output half a step,
2^-8 |exact|, more.
"""
import numpy as np
import pytest
import torch

import oracle.fp8_linear_ref as F
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0**-24


def weights(N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(N, K, generator=g, device=DEV) * 60.0
    codes = w.clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.rand(-(-N // 128), -(-K // 128), generator=g, device=DEV) * 1e-3 + 1e-4
    return codes, scales


def tokens(T, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(T, K, generator=g, device=DEV).bfloat16()


def check(y, x, codes, scales, rows=None):
    """Compare rows of y (all, or the given ones) with the oracle."""
    rows = np.arange(x.shape[0]) if rows is None else np.asarray(rows)
    want, mag = F.linear(x[rows].float().cpu().numpy(), codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy())
    got = y[rows].double().cpu().numpy()
    tol = (25 + scales.shape[1]) * U * mag + 1e-37
    if y.dtype == torch.bfloat16:
        tol = tol + 2.0**-8 * np.abs(want)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.max(np.abs(got - want) / tol):.2f} of the bound"
    return float(np.max(np.abs(got - want) / tol))


SHAPES = [(1, 1), (7, 130), (128, 128), (130, 257), (256, 2560), (1536, 384), (2560, 768), (1000, 1001), (4100, 640)]


@pytest.mark.parametrize("N,K", SHAPES)
def test_matches_the_oracle(N, K):
    codes, scales = weights(N, K, N + K)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=700)
    for T in (1, 2, 7, 8, 9, 16, 33, 128, 129, 300):
        x = tokens(T, K, T)
        rows = np.unique(np.linspace(0, T - 1, 40).astype(int))
        for dt in (torch.float32, torch.bfloat16):
            y = f.forward(x, out_dtype=dt)
            assert f.status() == lm.LING_MOE_OK
            worst = check(y, x, codes, scales, rows)
        print(f"N={N} K={K} T={T}: {worst:.3f} of the bound")
    f.close()


def test_several_waves_of_tiles():
    codes, scales = weights(4096, 512, 3)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=4000)
    for T in (4000, 1111):
        x = tokens(T, 512, T)
        y = f.forward(x)
        check(y, x, codes, scales, np.unique(np.linspace(0, T - 1, 60).astype(int)))
        assert torch.equal(y, f.forward(x))  # the same call gives the same bits
    f.close()


def test_strided_rows_and_untouched_surroundings():
    N, K = 300, 260
    codes, scales = weights(N, K, 9)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=64)
    for T in (3, 40):
        for off, pad in ((0, 0), (1, 3), (8, 28)):
            buf = tokens(T, K + off + pad, T)
            x = buf[:, off:off + K]
            for dt in (torch.float32, torch.bfloat16):
                ob = torch.full((T + 1, N + off + pad), 7.0, dtype=dt, device=DEV)
                out = ob[:T, off:off + N]
                assert f.forward(x, out=out) is out
                check(out, x, codes, scales)
                assert (ob[T] == 7).all() and (ob[:, :off] == 7).all() and (ob[:, off + N:] == 7).all()
    f.close()


def test_extreme_and_zero_tokens():
    N, K = 200, 384
    codes, scales = weights(N, K, 4)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=32)
    for T in (6, 30):
        x = tokens(T, K, 1).float()
        x[0] = 0.0
        x[1, 128:256] = 0.0
        x[2] *= 2.0**100
        x[3] *= 2.0**-120                # scales near the bottom of fp32
        x[4] = 0.0
        x[4, 5] = 3.0
        x = x.bfloat16()
        y = f.forward(x, out_dtype=torch.float32)
        keep = [i for i in range(T) if i != 3]
        check(y, x, codes, scales, keep)
        # row 3's scales are subnormal: both sides take the same fp32 steps, products below 2^-126 flush
        assert torch.isfinite(y[3]).all() and y[3].abs().max() < 2.0**-100
        assert (y[0] == 0).all()
        # a non-finite token spoils itself only
        z = x.clone()
        z[2, 7], z[5, 300] = float("nan"), float("inf")
        w = f.forward(z, out_dtype=torch.float32)
        assert torch.isnan(w[2]).all() and torch.isnan(w[5]).all()
        for i in (0, 1, 3, 4):
            assert torch.equal(w[i], y[i])
    f.close()


def test_stream_graph_and_two_handles():
    (c1, s1), (c2, s2) = weights(512, 640, 1), weights(640, 512, 2)
    a, b = lm.BlockFP8Linear(c1, s1, 64), lm.BlockFP8Linear(c2, s2, 64)
    for T in (1, 40):
        x = tokens(T, 640, 5)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            want = b.forward(a.forward(x))
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = b.forward(a.forward(x))
        for seed in (5, 6):
            x.copy_(tokens(T, 640, seed))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want) == (seed == 5)
            assert torch.equal(y, b.forward(a.forward(x)))
    a.close(), b.close()


def test_refusals_and_wait_timeout():
    codes, scales = weights(256, 256, 1)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=64)
    x = tokens(64, 256, 1)
    n = f.launch_count()
    with pytest.raises(lm.LingMoEError):
        f.forward(tokens(65, 256, 1))
    with pytest.raises(ValueError):
        f.forward(x.float())
    with pytest.raises(ValueError):
        f.forward(x[:, :255])
    with pytest.raises(ValueError):
        f.forward(x.t())
    with pytest.raises(ValueError):
        f.forward(x, out=torch.empty(64, 256, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        lm.BlockFP8Linear(codes, scales[:1], 4)
    with pytest.raises(lm.LingMoEError):
        f.forward(x, out=x)  # overlap
    for stride in (255, -256):
        assert lm.lib.ling_moe_fp8_linear_forward(f.handle, x.data_ptr(), stride, 2, codes.data_ptr(), 1, 256, None) == \
            lm.LING_MOE_ERR_INVALID_ARG
    assert f.forward(x[:0]).shape == (0, 256) and f.launch_count() == n
    y = f.forward(x)
    f.test_set_wait(0, 2_000_000)  # CTA 0 loads nothing: its waits run out after 2 ms
    f.forward(x)
    assert f.status() == lm.LING_MOE_ERR_DEVICE_TIMEOUT
    f.test_set_wait(-1)
    assert torch.equal(f.forward(x), y) and f.status() == lm.LING_MOE_OK
    f.close()


def test_long_rows_take_the_separate_quantisation():
    """K = 13100: eight tokens' codes no longer fit a CTA's shared memory; seven and fewer do."""
    N, K = 40, 13100
    codes, scales = weights(N, K, 11)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=8)
    for T, launches in ((8, 2), (7, 1), (1, 1)):
        n = f.launch_count()
        x = tokens(T, K, T)
        check(f.forward(x, out_dtype=torch.float32), x, codes, scales)
        check(f.forward(x, out_dtype=torch.float32), x, codes, scales)
        assert f.launch_count() == n + 2 * launches
    f.close()


@pytest.mark.parametrize("T", [1, 8, 40])
def test_token_codes_at_the_borders_between_codes(T):
    """Weights are the identity, so outputs show the codes: quotients on, and a step beside, the borders."""
    N = K = 128
    codes = torch.eye(N, device=DEV).to(torch.float8_e4m3fn)
    f = lm.BlockFP8Linear(codes, torch.ones(1, 1, device=DEV), max_tokens=T)
    mids = torch.tensor([m * 2.0**e for e in range(-11, 5) for m in (17, 19, 21, 23, 25, 27, 29)])[:110]
    for top in (448.0, 447.0, 450.0, 3.0, 1e-3, 2.0**-100, 2.0**-120):
        x = torch.zeros(T, K)
        x[:, 1:111] = (mids * (top / 448.0)).bfloat16().float()
        x[:, 0] = top
        x = x.bfloat16().to(DEV)
        y = f.forward(x, out_dtype=torch.float32)
        c, s = F.quantize_tokens(x.float().cpu().numpy())
        want = F.e4m3_decode(c) * s.astype(np.float64)
        # one product of a code with the scale, rounded once; below 2^-126 it may flush
        assert (np.abs(y.double().cpu().numpy() - want) <= U * np.abs(want) + 2.0**-126).all()
    f.close()


@pytest.mark.parametrize("T,N,K", [(3900, 4100, 300), (4000, 4096, 1024), (3841, 3970, 129)])
def test_wide_tiles(T, N, K):
    """Sizes whose tiles are 256 outputs wide, in several waves; the last ones partly empty."""
    codes, scales = weights(N, K, T)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=T)
    x = tokens(T, K, 1)
    rows = np.unique(np.concatenate([np.linspace(0, T - 1, 30).astype(int), np.arange(T - 70, T, 3)]))
    for dt in (torch.float32, torch.bfloat16):
        ob = torch.full((T + 1, N), 7.0, dtype=dt, device=DEV)
        f.forward(x, out=ob[:T])
        assert f.status() == lm.LING_MOE_OK
        check(ob[:T], x, codes, scales, rows)
        assert (ob[T] == 7).all() and torch.equal(f.forward(x, out_dtype=dt), ob[:T])
    y = f.forward(x)
    for cta in (0, 1, 5):  # this CTA loads nothing: its waits run out after 2 ms
        f.test_set_wait(cta, 2_000_000)
        f.forward(x)
        assert f.status() == lm.LING_MOE_ERR_DEVICE_TIMEOUT
    f.test_set_wait(-1)
    assert torch.equal(f.forward(x), y) and f.status() == lm.LING_MOE_OK
    f.close()
