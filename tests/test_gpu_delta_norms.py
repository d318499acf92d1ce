"""The gated delta rule with queries and keys whose squares pass the range of fp32."""
import pytest
import torch

import oracle.delta_ref as D
import tests.test_gpu_delta as base
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def both(f, a, st, n, scale, step_tokens=3):
    """A prefill of the first n tokens and a step of the ones behind them, each against the oracle."""
    s0 = base.np64(st[0])
    out = f.prefill(*[t[:n] for t in a], st, i32([0, n]))
    x = base.sub(a, slice(0, n))
    want, states = D.rule(*x, s0, scale)
    eo, es = D.prefill_bound(*x, s0, scale)
    base.close_out(base.np64(out), want, eo)
    base.close_state(base.np64(st[0]), states[-1], es)
    s1 = base.np64(st[0])
    o2 = f.step(*[t[n:n + step_tokens].unsqueeze(0) for t in a], st)
    x = base.sub(a, slice(n, n + step_tokens))
    want, states = D.rule(*x, s1, scale)
    eo, es = D.step_bound(*x, s1, scale)
    base.close_out(base.np64(o2[0]), want, eo)
    base.close_state(base.np64(st[0]), states[-1], es[-1])
    return out, o2


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("size", [1e18, 1e19, 1e25, 1e37, 1e-19, 1e-38])
def test_large_and_small_queries_and_keys(dk, size):
    """Every finite query and key is divided by its norm, also where its squares pass the largest (or fall below the
    smallest) fp32 number."""
    T, H, dv = 90, 2, 64
    f = lm.GatedDeltaRule(H, H, dk, dv, T, 1)
    for which in ((0,), (1,), (0, 1)):
        a = [t.clone() for t in base.make(T, H, H, dk, dv, True, 60)]
        for i in which:
            a[i][3::2] = (a[i][3::2].double() * size).to(torch.bfloat16)  # beside ordinary ones
        a[1][5, :, 1:] = 0  # one channel alone
        both(f, a, base.pool(1, H, dk, dv, 60), 80, dk**-0.5)
    f.close()


def test_one_large_channel():
    """The largest bf16 number in one channel, ordinary ones beside it."""
    T, H, d = 70, 2, 64
    f = lm.GatedDeltaRule(H, H, d, d, T, 1)
    a = [t.clone() for t in base.make(T, H, H, d, d, True, 61)]
    a[0][::3, :, 5] = torch.finfo(torch.bfloat16).max
    a[1][1::3, :, 60] = -torch.finfo(torch.bfloat16).max
    a[1][2::9] = torch.finfo(torch.bfloat16).max
    both(f, a, base.pool(1, H, d, d, 61), 65, d**-0.5)
    f.close()
