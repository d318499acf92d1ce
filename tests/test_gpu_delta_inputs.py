"""Inputs of the gated delta rule that the other tests do not make: decays of any alignment or expanded along
their channels, strided write strengths, another scale, another stream."""
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
def test_decays_off_alignment_and_expanded(dk):
    T, H, dv = 90, 4, 128
    f = lm.GatedDeltaRule(2, H, dk, dv, T, 1)
    q, k, v, g, beta = base.make(T, 2, H, dk, dv, True, 70)
    want = both(f, (q, k, v, g, beta), base.pool(1, H, dk, dv, 70), 80, dk**-0.5)
    wide = torch.zeros(T, H, dk + 3, device=DEV)
    for off in (0, 1, 3):
        w = wide[:, :, off:off + dk]
        w.copy_(g)
        got = both(f, (q, k, v, w, beta), base.pool(1, H, dk, dv, 70), 80, dk**-0.5)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a decay per head, as such and expanded along the channels
    h = g[:, :, 0].contiguous()
    want = both(f, (q, k, v, h, beta), base.pool(1, H, dk, dv, 70), 80, dk**-0.5)
    got = both(f, (q, k, v, h.unsqueeze(-1).expand(T, H, dk), beta), base.pool(1, H, dk, dv, 70), 80, dk**-0.5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # write strengths and decays with gaps, one of them for all heads
    b2 = torch.zeros(T, H, 5, device=DEV)
    b2[:, :, 2] = beta
    g2 = torch.zeros(T, 3, H, device=DEV)
    g2[:, 1] = h
    got = both(f, (q, k, v, g2[:, 1], b2[:, :, 2]), base.pool(1, H, dk, dv, 70), 80, dk**-0.5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = beta[:, :1].expand(T, H)
    both(f, (q, k, v, g[:, :1].expand(T, H, dk), one), base.pool(1, H, dk, dv, 70), 80, dk**-0.5)
    f.close()


@pytest.mark.parametrize("scale", [1.0, -0.25, 1e-6, 300.0])
def test_another_scale(scale):
    T, H, d = 90, 2, 128
    f = lm.GatedDeltaRule(H, H, d, d, T, 1, scale=scale)
    s32 = float(np.float32(scale))
    both(f, base.make(T, H, H, d, d, True, 80), base.pool(1, H, d, d, 80), 80, s32)
    f.close()


def test_a_handle_that_only_steps():
    """max_tokens sizes the prefill alone: 1 is enough for windows of many sequences."""
    H, d, B, n = 32, 128, 20, 8
    small, large = lm.GatedDeltaRule(H, H, d, d, 1, B), lm.GatedDeltaRule(H, H, d, d, 500, B)
    a = [t.view(B, n, *t.shape[1:]) for t in base.make(B * n, H, H, d, d, True, 85)]
    s1 = base.pool(B, H, d, d, 85)
    s2 = s1.clone()
    assert torch.equal(small.step(*a, s1), large.step(*a, s2)) and torch.equal(s1, s2)
    with pytest.raises(lm.LingMoEError):
        small.prefill(*[t[0] for t in a], s1, i32([0, n]))
    small.close(), large.close()


def test_on_another_stream():
    """stream= as a torch stream and as its raw handle, while another one is current; outputs given and allocated."""
    T, H, d = 100, 4, 128
    f = lm.GatedDeltaRule(H, H, d, d, T, 1)
    a = base.make(T, H, H, d, d, True, 90)
    win = [t[:4].unsqueeze(0) for t in a]
    s0 = base.pool(1, H, d, d, 90)
    ws = s0.clone()
    want = f.prefill(*a, ws, i32([0, T]))
    want_w = f.step(*win, ws)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for given in (False, True):
            st, cu = s0.clone(), i32([0, T])
            o = torch.empty_like(want) if given else None
            side.wait_stream(torch.cuda.current_stream())
            got = f.prefill(*a, st, cu, out=o, stream=stream)
            got_w = f.step(*win, st, stream=stream)
            assert f.status(stream=stream) == lm.LING_MOE_OK
            assert torch.equal(got, want) and torch.equal(got_w, want_w) and torch.equal(st, ws)
    f.close()
