"""Beam search on another stream than the current one."""
import numpy as np
import pytest
import torch

import oracle.beam_ref as B
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_on_another_stream():
    G, W, V = 3, 4, 30000
    g = torch.Generator(device=DEV).manual_seed(3)
    z = 2.0 * torch.randn(G, W, V, generator=g, device=DEV)
    c = -torch.rand(G, W, generator=g, device=DEV)
    fin = torch.zeros(G, W, dtype=torch.bool, device=DEV)
    fin[1, 2] = True
    bs = lm.BeamSearch(G, W, V)
    want = bs.select(z, c, fin, 5)
    states = torch.randn(G * W, 1000, generator=g, device=DEV)
    moved = B.reorder(states.cpu().numpy(), want[1].cpu().numpy())
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        st = states.clone()
        side.wait_stream(torch.cuda.current_stream())
        got = bs.select(z, c, fin, 5, stream=stream)
        bs.reorder(st, got[1], stream=stream)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert np.array_equal(st.cpu().numpy(), moved)
    bs.close()
