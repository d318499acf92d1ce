"""Packed prompts of the gated delta rule: padding slots before and between live sequences, several segments of the
workspace with 128 x 128 heads.  A sequence's results do not depend on its neighbours, so all comparisons between
calls are bit for bit."""
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


@pytest.mark.parametrize("slots", [[1, -1, 0], [-1, 1, 0], [2, 0, -1], [-1, 3, 1], [9, -5, 2]])
@pytest.mark.parametrize("lengths", [[60, 30, 60], [200, 65, 3], [1, 700, 470], [64, 0, 1100]])
def test_live_sequences_around_padding(slots, lengths):
    """Those whose slot is outside the pool take up their tokens and nothing else; 64 heads, so that the longer ones span
    several segments."""
    T, H, d = sum(lengths), 64, 64
    f = lm.GatedDeltaRule(H, H, d, d, T, 3)
    a = base.make(T, H, H, d, d, True, 40)
    st = base.pool(3, H, d, d, 40)
    want_s = st.clone()
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    got = run(f, a, st, cu, slots=i32(slots))
    for i, s in enumerate(slots):
        sl = slice(cu[i], cu[i + 1])
        if not 0 <= s < 3:
            assert (got[sl] == 7).all()
        elif lengths[i]:
            alone = [t[sl] for t in a]
            assert torch.equal(run(f, alone, want_s, [0, lengths[i]], slots=i32([s])), got[sl])
    assert torch.equal(st, want_s)
    f.close()


@pytest.mark.parametrize("lengths", [[2600], [900, 1, 1699]])
def test_segments_of_wide_heads(lengths):
    """128 x 128 heads, 64 of them: 18 chunks to a segment, three segments."""
    T, n, H, d = sum(lengths), len(lengths), 64, 128
    f = lm.GatedDeltaRule(16, H, d, d, T, n)
    a = base.make(T, 16, H, d, d, True, 50)
    st = base.pool(n, H, d, d, 50)
    st0 = st.clone()
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    out = run(f, a, st, cu)
    assert f.launch_count() >= 6
    for i in range(n):
        for h in (slice(0, 1), slice(63, 64)):
            x, s0 = base.sub(a, slice(cu[i], cu[i + 1]), h), base.np64(st0[i][h])
            want, states = D.rule(*x, s0, d**-0.5)
            eo, es = D.prefill_bound(*x, s0, d**-0.5)
            base.close_out(base.np64(out[cu[i]:cu[i + 1], h]), want, eo)
            base.close_state(base.np64(st[i][h]), states[-1], es)
    f.close()
