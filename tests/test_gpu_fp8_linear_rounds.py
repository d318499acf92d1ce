"""The streaming linear kernel where the 16-lane groups that quantise tokens end after different numbers of rounds, and
the layer on another stream than the current one."""
import pytest
import torch

import tests.test_gpu_fp8_linear as base
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,blocks", [(1, 49), (1, 48), (1, 97), (5, 21), (7, 15), (3, 33), (8, 13), (2, 81), (8, 31)])
@pytest.mark.parametrize("N", [10, 700])
def test_quantisation_in_uneven_rounds(T, blocks, N):
    """48 pairs of token and block to a round of one CTA, 96 of two."""
    K = blocks * 128 - 5
    codes, scales = base.weights(N, K, 1)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=T)
    for seed in (1, 2):
        x = base.tokens(T, K, seed)
        for dt in (torch.float32, torch.bfloat16):
            base.check(f.forward(x, out_dtype=dt), x, codes, scales)
    f.close()


@pytest.mark.parametrize("T", [3, 50])
def test_on_another_stream(T):
    codes, scales = base.weights(500, 640, 2)
    f = lm.BlockFP8Linear(codes, scales, max_tokens=64)
    x = base.tokens(T, 640, 3)
    want = f.forward(x)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for given in (False, True):
            o = torch.empty_like(want) if given else None
            side.wait_stream(torch.cuda.current_stream())
            got = f.forward(x, out=o, stream=stream)
            assert f.status(stream=stream) == lm.LING_MOE_OK
            assert torch.equal(got, want)
    f.close()
