"""Packed prompts of the gated delta rule with boundaries out of order or out of range: the bits of a call with the
boundaries that they count as, and the oracle's results."""
import numpy as np
import pytest
import torch

import oracle.delta_ref as D
import tests.test_gpu_delta as base
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run(f, a, st, cu, **kw):
    out = torch.full((a[0].shape[0], f.v_heads, f.head_v), 7.0, dtype=torch.bfloat16, device=DEV)
    f.prefill(*a, st, i32(cu), out=out, **kw)
    assert f.status() == lm.LING_MOE_OK
    return out


@pytest.mark.parametrize("cu", [[0, 300, 0, 300], [0, 100, 50, 250], [120, 20, 300, 290, 310], [-7, 64, 10, 64, 65, 1, 300],
                                [300, 0, 300, 0], [0, 1, 0, 1, 0, 1, 0, 1, 0, 300]])
def test_boundaries_never_run_back(cu):
    """A boundary below an earlier one counts as that one: sequences are disjoint."""
    T, H, d = 300, 2, 64
    n = len(cu) - 1
    f = lm.GatedDeltaRule(H, H, d, d, T, n)
    a = base.make(T, H, H, d, d, True, 30)
    st = base.pool(n, H, d, d, 30)
    st0, ref = st.clone(), st.clone()
    clean = np.maximum.accumulate(np.clip(cu, 0, T)).tolist()
    got, want = run(f, a, st, cu), run(f, a, ref, clean)
    assert torch.equal(got, want) and torch.equal(st, ref)
    for i in range(n):
        lo, hi = clean[i], clean[i + 1]
        if lo == hi:
            assert torch.equal(st[i], st0[i])
            continue
        x = base.sub(a, slice(lo, hi))
        o, states = D.rule(*x, base.np64(st0[i]), d**-0.5)
        eo, es = D.prefill_bound(*x, base.np64(st0[i]), d**-0.5)
        base.close_out(base.np64(got[lo:hi]), o, eo)
        base.close_state(base.np64(st[i]), states[-1], es)
    f.close()


@pytest.mark.parametrize("seed", range(4))
def test_many_boundaries_out_of_order(seed):
    """More sequences than a warp looks at together, over several segments of the workspace."""
    T, H, d, n = 700, 64, 64, 101
    r = np.random.default_rng(seed)
    cu = np.sort(r.integers(0, T + 1, n + 1)) + r.integers(-40, 41, n + 1) * (r.random(n + 1) < 0.5)
    clean = np.maximum.accumulate(np.clip(cu, 0, T))
    f = lm.GatedDeltaRule(H, H, d, d, T, n)
    a = base.make(T, H, H, d, d, True, 31 + seed)
    st = base.pool(n, H, d, d, 31)
    ref = st.clone()
    got, want = run(f, a, st, cu.tolist()), run(f, a, ref, clean.tolist())
    assert torch.equal(got, want) and torch.equal(st, ref)
    f.close()
