"""The gated delta rule without a GPU: the oracle against loops and against the
chunk form, its error bounds, and the refusals of the entry points and the binding."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.delta_ref as D
import weight_only_int4_fp32_b200 as lm

BAD, UNSUP = lm.LING_MOE_ERR_INVALID_ARG, lm.LING_MOE_ERR_UNSUPPORTED


def inputs(T, Hk, Hv, dk, dv, channel, seed):
    r = np.random.default_rng(seed)
    f = lambda *s: r.normal(size=s).astype(np.float32)  # noqa: E731
    g = -np.abs(f(T, Hv, dk) if channel else f(T, Hv)) * 0.3
    return (f(T, Hk, dk), f(T, Hk, dk), f(T, Hv, dv), g, r.random((T, Hv)).astype(np.float32)), f(Hv, dk, dv)


@pytest.mark.parametrize("channel", [True, False])
def test_oracle_is_the_recurrence(channel):
    (q, k, v, g, b), s0 = inputs(5, 2, 4, 6, 3, channel, 1)
    g[2] = 0.7            # above 0: counts as 0
    g[3, 1] = -np.inf     # forgets everything
    out, states = D.rule(q, k, v, g, b, s0, 0.5)
    S = s0.astype(np.float64)
    for t in range(5):
        for h in range(4):
            kk = k[t, h // 2] / np.sqrt(float((k[t, h // 2].astype(np.float64) ** 2).sum()) + 1e-6)
            qq = q[t, h // 2] / np.sqrt(float((q[t, h // 2].astype(np.float64) ** 2).sum()) + 1e-6)
            for c in range(6):
                S[h, c] *= np.exp(min(float(g[t, h, c] if channel else g[t, h]), 0.0))
            for j in range(3):
                u = b[t, h] * (v[t, h, j] - sum(S[h, c, j] * kk[c] for c in range(6)))
                for c in range(6):
                    S[h, c, j] += kk[c] * u
                assert abs(out[t, h, j] - 0.5 * sum(S[h, c, j] * qq[c] for c in range(6))) < 1e-12
        assert np.allclose(states[t], S, rtol=0, atol=1e-12)


@pytest.mark.parametrize("T", [1, 63, 64, 65, 130])
def test_bounds_are_positive_and_cover_fp32(T):
    """The recurrence in fp32 stays within the step's bound; the prefill's bound is finite and not below bf16's worth."""
    (q, k, v, g, b), s0 = inputs(T, 1, 2, 64, 8, True, T)
    out, states = D.rule(q, k, v, g, b, s0, 0.125)
    o, e = D.step_bound(q, k, v, g, b, s0, 0.125)
    qn, kn, vn, a, bn = (x.astype(np.float32) for x in D.heads(q, k, v, g, b))
    S = s0.copy()
    for t in range(T):
        S = S * a[t][:, :, None]
        u = bn[t][:, None] * (vn[t] - np.einsum("hkv,hk->hv", S, kn[t]))
        S = S + kn[t][:, :, None] * u[:, None]
        assert (np.linalg.norm(S - states[t], axis=1) <= e[t]).all()
        assert (np.abs(0.125 * np.einsum("hkv,hk->hv", S, qn[t]) - out[t]) <= o[t]).all()
    po, pe = D.prefill_bound(q, k, v, g, b, s0, 0.125)
    assert np.isfinite(po).all() and (po > 0).all() and (pe > 0).all()
    assert pe.max() < 0.01 * np.linalg.norm(states[-1], axis=1).max()


def _create(**kw):
    c = dict(k_heads=2, v_heads=4, head_k=64, head_v=128, max_tokens=64, max_seqs=4, scale=0.0)
    c.update(kw)
    h = ctypes.c_void_p()
    return lm.lib.ling_moe_delta_create(ctypes.byref(lm.ling_moe_delta_config_t(**c)), ctypes.byref(h)), h.value


@pytest.mark.parametrize("kw,code", [
    (dict(k_heads=0), BAD), (dict(v_heads=-4), BAD), (dict(v_heads=3), BAD), (dict(max_tokens=0), BAD), (dict(max_seqs=0), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(head_k=96), UNSUP), (dict(head_v=256), UNSUP),
    (dict(k_heads=1, v_heads=1025), UNSUP), (dict(max_tokens=(1 << 24) + 1), UNSUP), (dict(max_seqs=(1 << 18) + 1), UNSUP)])
def test_create_refuses(kw, code):
    assert _create(**kw) == (code, None)


def test_null_arguments():
    h = ctypes.c_void_p()
    assert lm.lib.ling_moe_delta_create(None, ctypes.byref(h)) == BAD
    assert lm.lib.ling_moe_delta_create(ctypes.byref(lm.ling_moe_delta_config_t(1, 1, 64, 64, 1, 1, 0.0)), None) == BAD
    io = lm.ling_moe_delta_io_t()
    assert lm.lib.ling_moe_delta_step(None, ctypes.byref(io), 1, 1, None, None) == BAD
    assert lm.lib.ling_moe_delta_prefill(None, ctypes.byref(io), 1, None, 1, None, None) == BAD
    assert lm.lib.ling_moe_delta_status(None, None) == BAD
    assert lm.lib.ling_moe_delta_test_set_wait(None, 1, 0) == BAD
    assert lm.lib.ling_moe_delta_launch_count(None) == 0
    lm.lib.ling_moe_delta_destroy(None)


def test_binding_refuses_wrong_tensors():
    f = object.__new__(lm.GatedDeltaRule)
    f.k_heads, f.v_heads, f.head_k, f.head_v, f.max_tokens, f.max_seqs, f.handle, f._torch = 1, 2, 64, 64, 8, 2, None, torch
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    st, cu = torch.zeros(2, 2, 64, 64), torch.zeros(3, dtype=torch.int32)
    a = [bf(2, 1, 1, 64), bf(2, 1, 1, 64), bf(2, 1, 2, 64), torch.zeros(2, 1, 2, 64), torch.zeros(2, 1, 2)]
    with pytest.raises(ValueError, match="q must be a CUDA"):
        f.step(*a, st)  # on the host
    with pytest.raises(ValueError, match="4-D"):
        f.step(a[0][0], *a[1:], st)
    with pytest.raises(ValueError, match="3-D"):
        f.prefill(*a, st, cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        f.prefill(*[t[0] for t in a], st, cu.view(3, 1))
    with pytest.raises(ValueError):
        f.prefill(*[t[0] for t in a], st, cu)  # on the host
    with pytest.raises(ValueError, match="scale"):
        lm.GatedDeltaRule(1, 1, 64, 64, 8, 1, scale=0.0)
