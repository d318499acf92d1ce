"""Prefill of values near the top of fp32 under decays that the solution divides by."""
import pytest
import torch

import oracle.delta_ref as D
import tests.test_gpu_delta as base
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rate", [0.0, 0.3, 0.65, 2.0])
@pytest.mark.parametrize("size", [2.0**90, 2.0**105, 2.0**120, 2.0**-110])
def test_large_and_small_values(size, rate, d):
    """One head's values at the size, the other's ordinary; both stay within their own bounds."""
    T, H = 130, 2
    f = lm.GatedDeltaRule(H, H, d, d, T, 1)
    q, k, v, g, beta = [t.clone() for t in base.make(T, H, H, d, d, False, 3)]
    v[:, 0] = (v[:, 0].double() * size).to(torch.bfloat16)
    g = 0.1 * g - rate
    st = base.pool(1, H, d, d, 3)
    st[0, 0] *= size
    s0 = base.np64(st[0])
    a = (q, k, v, g, beta)
    out = f.prefill(*a, st, torch.tensor([0, T], dtype=torch.int32, device=DEV))
    assert f.status() == lm.LING_MOE_OK
    for h in (slice(0, 1), slice(1, 2)):
        x = base.sub(a, slice(0, T), h)
        want, states = D.rule(*x, s0[h], d**-0.5)
        eo, es = D.prefill_bound(*x, s0[h], d**-0.5)
        base.close_out(base.np64(out[:, h]), want, eo)
        base.close_state(base.np64(st[0, h]), states[-1], es)
    f.close()
