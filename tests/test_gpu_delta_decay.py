"""Prefill under decays that leave little of what was written: the state against the 64-bit oracle, relative to itself.

With G_t the running sum over tokens of each token's slowest log-decay (the largest
over its channels, 0 at most), S_t = exp(G_t) S'_t, where S' follows the same
recurrence with the log-decays g - (its slowest) and the values v_t exp(-G_t).  The
kernel takes the factors exp(G) out of every operand that feeds the state
and carries them in fp32, so its error is the one that oracle/delta_ref.py derives for
S', times exp(G).  Each such factor adds 3 u (u = 2^-24: an exponential rounded once
and two products), less than the 360 u that the bound gives each decay.
"""
import numpy as np
import pytest
import torch

import oracle.delta_ref as D
import tests.test_gpu_delta as base
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def relative_bound(q, k, v, g, beta, s0, scale):
    """2-norm of the state's error by column, decays common to all channels taken out."""
    g = np.minimum(g, 0.0)
    slow = g if g.ndim == 2 else g.max(-1)                     # [T, Hv]
    G = np.cumsum(slow, 0)
    vp = np.where(v == 0.0, 0.0, v * np.exp(-G)[:, :, None])
    rest = g - slow if g.ndim == 2 else g - slow[..., None]
    _, e = D.prefill_bound(q, k, vp, rest, beta, s0, scale)
    return e * np.exp(G[-1])[:, None]


@pytest.mark.parametrize("tail", ["beta", "v"])
@pytest.mark.parametrize("channel", [False, True])
@pytest.mark.parametrize("T,rate", [(64, 0.3), (64, 1.1), (30, 2.5), (64, 0.05), (150, 0.4), (17, 4.0)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_a_few_writes_and_a_long_decay(T, rate, dk, dv, channel, tail):
    """Five tokens write; after them nothing is written (beta 0), or nothing but corrections (v 0)."""
    H = 2
    f = lm.GatedDeltaRule(H, H, dk, dv, T, 1)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    for seed, start in ((1, 0.0), (2, 1.0)):
        q, k, v, g, beta = [t.clone() for t in base.make(T, H, H, dk, dv, channel, seed)]
        g = 0.2 * g - rate
        v[5:] = 0.0
        if tail == "beta":
            beta[5:] = 0.0
        a = (q, k, v, g, beta)
        st = start * base.pool(1, H, dk, dv, seed)
        s0 = base.np64(st[0])
        out = f.prefill(*a, st, cu)
        assert f.status() == lm.LING_MOE_OK
        x = base.sub(a, slice(0, T))
        want, states = D.rule(*x, s0, dk**-0.5)
        size = np.linalg.norm(states[-1], axis=-2)
        e = relative_bound(*x, s0, dk**-0.5)
        assert (e < (2e-3 if tail == "beta" else 0.5) * size).all(), "the bound says little"
        worst = base.close_state(base.np64(st[0]), states[-1], e)
        rel = np.linalg.norm(base.np64(st[0]) - states[-1]) / np.linalg.norm(states[-1])
        print(f"start {start}: {worst:.4f} of the bound, relative error {rel:.1e}")
        eo, _ = D.prefill_bound(*x, s0, dk**-0.5)
        base.close_out(base.np64(out), want, eo)
    f.close()


def test_decays_from_none_to_all():
    """Per-head decays from 0 to -inf in one prompt, tokens that write all along."""
    T, H, d = 200, 8, 128
    f = lm.GatedDeltaRule(H, H, d, d, T, 1)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    q, k, v, g, beta = [t.clone() for t in base.make(T, H, H, d, d, False, 3)]
    g = g * torch.tensor([0.0, 1e-3, 0.1, 1.0, 10.0, 100.0, 1e4, 1e30], device=DEV)
    g[60, 1], g[64:70, 2], g[3] = -float("inf"), -float("inf"), 5.0
    a = (q, k, v, g, beta)
    st = base.pool(1, H, d, d, 3)
    s0 = base.np64(st[0])
    out = f.prefill(*a, st, cu)
    x = base.sub(a, slice(0, T))
    want, states = D.rule(*x, s0, d**-0.5)
    eo, es = D.prefill_bound(*x, s0, d**-0.5)
    base.close_out(base.np64(out), want, eo)
    base.close_state(base.np64(st[0]), states[-1], es)
    f.close()


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("T,rate,w", [(15, 6.0, 5), (30, 2.0, 5), (40, 1.5, 5), (64, 0.8, 5), (100, 0.5, 5), (8, 12.0, 5),
                                      (8, 12.0, 1), (16, 5.0, 1), (60, 1.0, 1)])
def test_first_writes_survive_whatever_the_channels_decay(T, rate, w, dk):
    """w tokens write under mild decays; then every channel of every token decays at random and nothing is written,
    so that all channels fall far below the slowest decays' product.  Those tokens' state has the error e of
    oracle/delta_ref.py, of which each channel keeps its decays' part; a row of k exp(..) is off by
    2^-22 and 360 u of itself and 2^-38 of its largest, its channels' decays once more by 360 u."""
    H, dv = 2, 64
    f = lm.GatedDeltaRule(H, H, dk, dv, T, 1)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    for seed, start in ((5, 0.0), (6, 1.0)):
        q, k, v, g, beta = [t.clone() for t in base.make(T, H, H, dk, dv, True, seed)]
        r = torch.Generator(device=DEV).manual_seed(seed)
        g[w:] = -rate * torch.rand(T - w, H, dk, generator=r, device=DEV)
        beta[w:] = 0.0
        st = start * base.pool(1, H, dk, dv, seed)
        s0 = base.np64(st[0])
        f.prefill(q, k, v, g, beta, st, cu)
        assert f.status() == lm.LING_MOE_OK
        x = base.sub((q, k, v, g, beta), slice(0, T))
        _, states = D.rule(*x, s0, dk**-0.5)
        _, e = D.prefill_bound(*[t[:w] for t in x], s0, dk**-0.5)
        left = np.exp(x[3][w:].sum(0)).max(-1)[:, None]      # [H, 1]: the channel that decays least
        written = np.abs(np.stack([states[0] - np.exp(x[3][0])[..., None] * s0]
                                  + [states[t] - np.exp(x[3][t])[..., None] * states[t - 1] for t in range(1, w)]))
        tol = left * (e + (2.0**-22 + 720 * D.U + 2.0**-38 * dk) * (np.linalg.norm(written, axis=-2).sum(0)
                                                                    + np.linalg.norm(s0, axis=-2)))
        size = np.linalg.norm(states[-1], axis=-2)
        assert np.linalg.norm(tol) < 0.05 * np.linalg.norm(size), "the bound says little"
        worst = base.close_state(base.np64(st[0]), states[-1], tol)
        rel = np.linalg.norm(base.np64(st[0]) - states[-1]) / np.linalg.norm(states[-1])
        print(f"start {start}: {worst:.4f} of the bound, relative error {rel:.1e}, state {size.max():.1e}")
    f.close()
