"""The gated delta rule on the GPU against the 64-bit oracle.

The bounds on the state's error (per column, 2-norm) and on the output before
its rounding are derived in oracle/delta_ref.py; a bf16 output adds half a
step, 2^-8 of its value, and 2^-134 below bf16's normal range.
"""
import numpy as np
import pytest
import torch

import oracle.delta_ref as D
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(tokens, Hk, Hv, dk, dv, channel, seed, strong=0.0, pad=0):
    """q, k, v as slices of one projection's rows (`pad` elements wider), g, beta."""
    r = torch.Generator(device=DEV).manual_seed(seed)
    w = [Hk * dk, Hk * dk, Hv * dv]
    rows = torch.randn(tokens, sum(w) + pad, generator=r, device=DEV).to(torch.bfloat16)
    q, k, v = rows[:, pad:].split(w, 1)
    g = -torch.rand(tokens, Hv, dk if channel else 1, generator=r, device=DEV).exp().sub(1).mul(0.2)
    if strong:  # some channels forget (almost) everything at once
        hit = torch.rand(g.shape, generator=r, device=DEV) < strong
        g = torch.where(hit, g * 500.0 - 30.0, g)
    beta = torch.rand(tokens, Hv, generator=r, device=DEV)
    return [q.view(tokens, Hk, dk), k.view(tokens, Hk, dk), v.view(tokens, Hv, dv), g if channel else g[..., 0], beta]


def pool(slots, Hv, dk, dv, seed):
    r = torch.Generator(device=DEV).manual_seed(seed + 1000)
    return 0.5 * torch.randn(slots, Hv, dk, dv, generator=r, device=DEV)


def np64(t):
    return t.double().cpu().numpy()


def sub(a, sl, heads=None):
    """The tokens `sl` of the inputs on the host, of value heads `heads` (a slice) only."""
    q, k, v, g, b = [np64(t[sl]) for t in a]
    if heads is not None:
        r = v.shape[1] // k.shape[1]
        at = np.arange(v.shape[1])[heads]
        q, k, v, g, b = q[:, at // r], k[:, at // r], v[:, at], g[:, at], b[:, at]
    return q, k, v, g, b


def close_out(got, want, bound):
    tol = bound + 2.0**-8 * (np.abs(want) + bound) + 2.0**-134
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1, f"output off by {worst:.2f} of the bound"
    return worst


def close_state(got, want, e):
    worst = np.max(np.linalg.norm(got - want, axis=-2) / (e + 2.0**-24 * np.linalg.norm(want, axis=-2)))
    assert worst <= 1, f"state off by {worst:.2f} of the bound"
    return worst


# ------------------------------------------------------------------ step
STEP = [(1, 1, 1, 1, 64, 64, True), (3, 2, 1, 2, 64, 128, False), (2, 8, 2, 4, 128, 64, True), (5, 4, 4, 4, 128, 128, True),
        (2, 3, 1, 8, 128, 128, False), (1, 7, 3, 3, 64, 64, True), (70, 1, 2, 2, 128, 128, True)]


@pytest.mark.parametrize("B,n,Hk,Hv,dk,dv,channel", STEP)
def test_step_matches_the_oracle(B, n, Hk, Hv, dk, dv, channel):
    f = lm.GatedDeltaRule(Hk, Hv, dk, dv, max_tokens=8, max_seqs=B)
    for seed, (strong, pad) in enumerate([(0.0, 0), (0.1, 3), (0.0, 8)]):
        a = make(B * n, Hk, Hv, dk, dv, channel, seed, strong, pad)
        shape = lambda t: t.view(B, n, *t.shape[1:])  # noqa: E731
        st = pool(B + 2, Hv, dk, dv, seed)
        slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(seed))[:B].int().to(DEV)
        st0 = st.clone()
        out = f.step(*map(shape, a), st, slots=slots)
        worst = [0.0, 0.0]
        for i in range(B):
            x = sub(a, slice(i * n, i * n + n))
            s0 = np64(st0[slots[i]])
            want, states = D.rule(*x, s0, dk**-0.5)
            eo, es = D.step_bound(*x, s0, dk**-0.5)
            worst[0] = max(worst[0], close_out(np64(out[i]), want, eo))
            worst[1] = max(worst[1], close_state(np64(st[slots[i]]), states[-1], es[-1]))
        rest = [s for s in range(B + 2) if s not in slots.tolist()]
        assert torch.equal(st[rest], st0[rest])
        print(f"seed {seed}: output {worst[0]:.3f}, state {worst[1]:.3f} of the bound")
    assert f.launch_count() == 3
    f.close()


def test_step_by_step_is_the_window_bit_for_bit():
    B, n, H, d = 3, 6, 2, 128
    f = lm.GatedDeltaRule(H, H, d, d, 8, B)
    a = [t.view(B, n, *t.shape[1:]) for t in make(B * n, H, H, d, d, True, 1)]
    st = pool(B, H, d, d, 1)
    one, win = st.clone(), st.clone()
    outs = torch.cat([f.step(*[t[:, i:i + 1] for t in a], one) for i in range(n)], 1)
    assert torch.equal(f.step(*a, win), outs) and torch.equal(win, one)
    # accepted counts (clamped): the state of the accepted part, all outputs
    part = st.clone()
    acc = torch.tensor([0, 4, 9], dtype=torch.int32, device=DEV)
    assert torch.equal(f.step(*a, part, accepted=acc), outs)
    assert torch.equal(part[0], st[0]) and torch.equal(part[2], win[2])
    four = st.clone()
    f.step(*[t[:, :4] for t in a], four)
    assert torch.equal(part[1], four[1])
    neg = st.clone()
    f.step(*a, neg, accepted=torch.full((B,), -5, dtype=torch.int32, device=DEV))
    assert torch.equal(neg, st)
    f.close()


def test_step_padding_slots_leave_everything():
    B, H, d = 4, 2, 64
    f = lm.GatedDeltaRule(H, H, d, d, 8, B)
    a = [t.view(B, 1, *t.shape[1:]) for t in make(B, H, H, d, d, True, 2)]
    st = pool(3, H, d, d, 2)
    st0, out = st.clone(), torch.full((B, 1, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    f.step(*a, st, slots=torch.tensor([-1, 2, 3, 0], dtype=torch.int32, device=DEV), out=out)
    assert (out[0] == 7).all() and (out[2] == 7).all() and torch.equal(st[1], st0[1])
    ref = st0.clone()
    want = f.step(*[t[[1, 3]].contiguous() for t in a], ref, slots=torch.tensor([2, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(out[[1, 3]], want) and torch.equal(ref, st)
    f.close()


def test_far_offsets():
    """Strides that pass 2^31 elements and a pool that passes 2^32 bytes."""
    H, d = 32, 128
    f = lm.GatedDeltaRule(1, H, d, d, 8, 2)
    st = torch.zeros(2200, H, d, d, device=DEV)  # 4.6 GB
    a = make(4, 1, H, d, d, True, 5)
    big = torch.empty(2**31 + 4096, dtype=torch.bfloat16, device=DEV)
    k = big.as_strided((2, 2, 1, d), (2**31, d, d, 1))
    k.copy_(a[1].view(2, 2, 1, d))
    x = [t.view(2, 2, *t.shape[1:]) for t in a]
    slots = torch.tensor([2199, 1], dtype=torch.int32, device=DEV)
    out = f.step(x[0], k, *x[2:], st, slots=slots)
    small = torch.zeros(2, H, d, d, device=DEV)
    assert torch.equal(out, f.step(*x, small)) and torch.equal(st[2199], small[0]) and torch.equal(st[1], small[1])
    f.close()


# ------------------------------------------------------------------ prefill
PREFILL = [  # lengths, Hk, Hv, dk, dv, channel
    ([1], 1, 1, 64, 64, True), ([64], 1, 2, 128, 64, False), ([65, 0, 63], 2, 2, 64, 128, True),
    ([0, 200, 1, 129], 1, 2, 128, 128, True), ([7, 300, 64, 2], 2, 4, 128, 128, False), ([515], 1, 1, 128, 128, True)]


@pytest.mark.parametrize("lengths,Hk,Hv,dk,dv,channel", PREFILL)
def test_prefill_matches_the_oracle(lengths, Hk, Hv, dk, dv, channel):
    T, n = sum(lengths), len(lengths)
    f = lm.GatedDeltaRule(Hk, Hv, dk, dv, max_tokens=T + 5, max_seqs=n)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    for seed, (strong, pad) in enumerate([(0.0, 0), (0.05, 1), (0.6, 8)]):
        a = make(T + 5, Hk, Hv, dk, dv, channel, seed, strong, pad)  # five rows behind the last sequence
        st = pool(n + 1, Hv, dk, dv, seed)
        st0, out = st.clone(), torch.full((T + 5, Hv, dv), 7.0, dtype=torch.bfloat16, device=DEV)
        slots = torch.arange(n, 0, -1, dtype=torch.int32, device=DEV)
        fresh = torch.tensor([i % 2 == 1 for i in range(n)], device=DEV)
        f.prefill(*a, st, torch.tensor(cu, dtype=torch.int32, device=DEV), slots=slots, fresh=fresh, out=out)
        assert f.status() == lm.LING_MOE_OK
        assert (out[T:] == 7).all() and torch.equal(st[0], st0[0])
        worst = [0.0, 0.0]
        for i in range(n):
            if lengths[i] == 0:
                assert torch.equal(st[n - i], st0[n - i])
                continue
            x = sub(a, slice(cu[i], cu[i + 1]))
            s0 = np64(st0[n - i]) * (0.0 if i % 2 else 1.0)
            want, states = D.rule(*x, s0, dk**-0.5)
            eo, es = D.prefill_bound(*x, s0, dk**-0.5)
            worst[0] = max(worst[0], close_out(np64(out[cu[i]:cu[i + 1]]), want, eo))
            worst[1] = max(worst[1], close_state(np64(st[n - i]), states[-1], es))
            rel = np.linalg.norm(np64(st[n - i]) - states[-1]) / np.linalg.norm(states[-1])
        print(f"seed {seed}: output {worst[0]:.3f}, state {worst[1]:.3f} of the bound; state rel {rel:.1e}")
    f.close()


@pytest.mark.parametrize("lengths", [[2500], [100, 3, 2397], [1152, 0, 1348], [1200, 1300]])
def test_prefill_over_several_segments(lengths):
    """64 heads: a segment of the workspace holds 18 chunks (8 records per SM), so these take three:
    the halves of the workspace are used in turn, and again."""
    Hk, Hv, dk, dv, T, n = 32, 64, 64, 64, sum(lengths), len(lengths)
    f = lm.GatedDeltaRule(Hk, Hv, dk, dv, max_tokens=T, max_seqs=n)
    a = make(T, Hk, Hv, dk, dv, True, 4)
    st = pool(n, Hv, dk, dv, 4)
    st0 = st.clone()
    cu = np.concatenate([[0], np.cumsum(lengths)])
    out = f.prefill(*a, st, torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert f.status() == lm.LING_MOE_OK and f.launch_count() >= 6
    for i in range(n):
        if not lengths[i]:
            continue
        for h in (slice(0, 2), slice(62, 64)):
            x, s0 = sub(a, slice(cu[i], cu[i + 1]), h), np64(st0[i][h])
            want, states = D.rule(*x, s0, dk**-0.5)
            eo, es = D.prefill_bound(*x, s0, dk**-0.5)
            close_out(np64(out[cu[i]:cu[i + 1], h]), want, eo)
            close_state(np64(st[i][h]), states[-1], es)
    f.close()


def test_prefill_then_step_then_prefill():
    """A prompt, a window of tokens, a further prompt chunk on the same states."""
    H, d = 2, 128
    f = lm.GatedDeltaRule(H, H, d, d, 200, 1)
    a = make(180, H, H, d, d, True, 6)
    st = torch.zeros(1, H, d, d, device=DEV)
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=DEV)  # noqa: E731
    o1 = f.prefill(*[t[:100] for t in a], st, cu(100))
    o2 = f.step(*[t[100:104].unsqueeze(0) for t in a], st)
    o3 = f.prefill(*[t[104:] for t in a], st, cu(76))
    x = sub(a, slice(0, 180))
    s0 = np.zeros((H, d, d))
    want, states = D.rule(*x, s0, d**-0.5)
    # the pieces' errors add: three times the prefill's whole bound holds them
    eo, es = D.prefill_bound(*x, s0, d**-0.5)
    close_out(np64(torch.cat([o1, o2[0], o3])), want, 3 * eo)
    close_state(np64(st[0]), states[-1], 3 * es)
    f.close()


def test_alike_keys_and_strong_writes():
    """All keys equal and beta 1 or 2: A is full, T alternates; decay 0."""
    T, d = 150, 64
    f = lm.GatedDeltaRule(1, 1, d, d, T, 1)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    for b in (1.0, 2.0):
        q, k, v, g, beta = make(T, 1, 1, d, d, True, 8)
        k = k[:1].expand(T, 1, d)
        g, beta = torch.zeros_like(g), torch.full_like(beta, b)
        st = pool(1, 1, d, d, 8)
        x, s0 = sub([q, k, v, g, beta], slice(0, T)), np64(st[0])
        out = f.prefill(q, k, v, g, beta, st, cu)
        want, states = D.rule(*x, s0, d**-0.5)
        eo, es = D.prefill_bound(*x, s0, d**-0.5)
        close_out(np64(out), want, eo)
        close_state(np64(st[0]), states[-1], es)
        # The worst-case bound is wide here.  Roundings of about 20 u in A's 64 x 64 / 2
        # entries that do not conspire add as the root of their number: 45 x 20 u = 5e-5
        # of the largest write per chunk, three chunks, beta 2: below 1e-3 of it.
        top = np.abs(states - np.concatenate([s0[None], states[:-1]])).max()
        assert np.abs(np64(st[0]) - states[-1]).max() < 1e-3 * max(top, np.abs(states[-1]).max())
    f.close()


def test_zeros_infinities_and_nan():
    T, H, d = 140, 3, 64
    f = lm.GatedDeltaRule(H, H, d, d, T, 2)
    a = make(T, H, H, d, d, True, 9)
    q, k, v, g, beta = [t.clone() for t in a]
    k[5], q[6], v[7], beta[8] = 0, 0, 0, 0
    g[9], g[10, :, :3], g[70], g[71] = float("-inf"), float("-inf"), 3.0, -1e30
    cu = torch.tensor([0, 80, T], dtype=torch.int32, device=DEV)
    st = pool(2, H, d, d, 9)
    st0 = st.clone()
    out = f.prefill(q, k, v, g, beta, st, cu)
    for i, sl in enumerate((slice(0, 80), slice(80, T))):
        x, s0 = sub([q, k, v, g, beta], sl), np64(st0[i])
        want, states = D.rule(*x, s0, d**-0.5)
        eo, es = D.prefill_bound(*x, s0, d**-0.5)
        close_out(np64(out[sl]), want, eo)
        close_state(np64(st[i]), states[-1], es)
    # steps over the same special tokens
    for t in (5, 6, 7, 8, 9, 10, 70, 71):
        s1 = st0[:1].clone()
        x = sub([q, k, v, g, beta], slice(t, t + 1))
        o = f.step(*[z[t:t + 1].unsqueeze(0) for z in (q, k, v, g, beta)], s1)
        want, states = D.rule(*x, np64(st0[0]), d**-0.5)
        eo, es = D.step_bound(*x, np64(st0[0]), d**-0.5)
        close_out(np64(o[0]), want, eo)
        close_state(np64(s1[0]), states[-1], es[-1])
    # a bad value spoils its own sequence and head, nothing else
    for j, bad in enumerate((float("nan"), float("inf"))):
        for m, t in enumerate((q, k, v, g, beta)):
            if m == 3 and j == 1:
                continue  # +inf as a log-decay counts as 0
            w = [z.clone() for z in (q, k, v, g, beta)]
            w[m][(20, 1) if w[m].dim() == 2 else (20, 1, 4)] = bad
            sb = st0.clone()
            ob = f.prefill(*w, sb, cu)
            keep = [0, 2]
            assert torch.equal(ob[:, keep], out[:, keep]) and torch.equal(sb[:, keep], st[:, keep])
            assert torch.equal(ob[80:], out[80:]) and torch.equal(sb[1], st[1])
            assert not torch.isfinite(ob[20:80, 1]).all()
            if m:
                assert not torch.isfinite(sb[0, 1]).all()
            so = st0[:1].clone()
            oo = f.step(*[z[20:21].unsqueeze(0) for z in w], so)
            assert torch.isfinite(oo[:, :, keep]).all() and not torch.isfinite(oo[:, :, 1]).all()
            assert torch.isfinite(so[:, keep]).all() and (m == 0 or not torch.isfinite(so[:, 1]).all())
    f.close()


def test_bad_boundaries_are_clamped():
    T, H, d = 100, 1, 64
    f = lm.GatedDeltaRule(H, H, d, d, T, 3)
    a = make(T, H, H, d, d, True, 10)
    for cu in ([-5, 40, 1000, 20], [50, 10, 60, 2**31 - 1], [0, 0, 0, 0], [-(2**31), -1, 100, 100]):
        st = pool(3, H, d, d, 10)
        st0 = st.clone()
        guard = torch.full((T + 8, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        f.prefill(*a, st, torch.tensor(cu, dtype=torch.int32, device=DEV), out=guard[4:T + 4])
        assert f.status() == lm.LING_MOE_OK
        assert (guard[:4] == 7).all() and (guard[T + 4:] == 7).all()
        lo = [min(max(c, 0), T) for c in cu[:3]]
        hi = [min(max(c, l), T) for c, l in zip(cu[1:], lo)]
        for i in range(3):
            if hi[i] <= lo[i]:
                assert torch.equal(st[i], st0[i])
    f.close()


def test_padding_slots_in_a_prefill():
    T, H, d = 150, 2, 64
    f = lm.GatedDeltaRule(H, H, d, d, T, 3)
    a = make(T, H, H, d, d, True, 11)
    cu = torch.tensor([0, 60, 90, T], dtype=torch.int32, device=DEV)
    st = pool(2, H, d, d, 11)
    st0 = st.clone()
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    f.prefill(*a, st, cu, slots=torch.tensor([1, -1, 2], dtype=torch.int32, device=DEV), out=out)
    assert (out[60:] == 7).all() and torch.equal(st[0], st0[0]) and not torch.equal(st[1], st0[1])
    f.close()


def test_streams_graphs_and_repeats():
    T, H, d = 300, 4, 128
    f = lm.GatedDeltaRule(H, H, d, d, T, 2)
    a = [t.clone() for t in make(T, H, H, d, d, True, 12)]
    cu = torch.tensor([0, 170, T], dtype=torch.int32, device=DEV)
    s0 = pool(2, H, d, d, 12)
    want_s = s0.clone()
    want = f.prefill(*a, want_s, cu)
    two = [t[:8].view(2, 4, *t.shape[1:]) for t in a]
    want_w = f.step(*two, want_s)
    side, st = torch.cuda.Stream(), s0.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, w = f.prefill(*a, st, cu), f.step(*two, st)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(w, want_w) and torch.equal(st, want_s)
    graph = torch.cuda.CUDAGraph()
    st.copy_(s0)
    with torch.cuda.graph(graph):
        o, w = f.prefill(*a, st, cu), f.step(*two, st)
    for _ in range(2):
        st.copy_(s0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(w, want_w) and torch.equal(st, want_s)
    a[2].mul_(2.0)  # other values, same graph
    st.copy_(s0)
    graph.replay()
    s1 = s0.clone()
    assert torch.equal(f.prefill(*a, s1, cu), o) and not torch.equal(o, want)
    f.close()


def test_refusals_and_wait_timeout():
    T, H, d = 130, 1, 64
    f = lm.GatedDeltaRule(H, 2 * H, d, d, T, 2)
    a = make(T, H, 2 * H, d, d, True, 13)
    st = pool(2, 2 * H, d, d, 13)
    cu = torch.tensor([0, 100, T], dtype=torch.int32, device=DEV)
    win = lambda n, B=2: [t[:B * n].reshape(B, n, *t.shape[1:]) for t in a]  # noqa: E731
    n0 = f.launch_count()
    with pytest.raises(lm.LingMoEError):
        f.step(*win(9), st)                                   # more than 8 tokens
    with pytest.raises(lm.LingMoEError):
        f.step(*win(1, 3), st)                                # more sequences than the handle takes
    with pytest.raises(lm.LingMoEError):
        f.step(*win(1), st[:1])                               # fewer slots than sequences
    with pytest.raises(lm.LingMoEError):
        f.prefill(*make(T + 1, H, 2 * H, d, d, True, 1), st, cu)
    w = [t.contiguous() for t in win(1)]
    with pytest.raises(lm.LingMoEError):
        f.step(*w, st, out=w[2])                              # out is v
    for i, t in enumerate((a[0].float(), a[1][..., :32], a[2][:, :1], a[3].half(), a[4][:1])):
        bad = list(a)
        bad[i] = t
        with pytest.raises(ValueError):
            f.prefill(*bad, st, cu)
    with pytest.raises(ValueError):
        f.prefill(*a, st.transpose(2, 3), cu)
    with pytest.raises(ValueError):
        f.prefill(*a, st, cu.long())
    with pytest.raises(ValueError):
        f.prefill(*a, st, cu, slots=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        f.prefill(*a, st, cu, fresh=torch.zeros(2, device=DEV))
    with pytest.raises(ValueError):
        f.prefill(*a, st, cu, out=torch.empty(T, 2, d, device=DEV))
    with pytest.raises(ValueError):
        f.step(*win(1), st, accepted=torch.zeros(2, dtype=torch.int64, device=DEV))
    z = [t[:0] for t in a]
    assert f.prefill(*z, st, cu).shape == (0, 2, d) and f.step(*[t.view(2, 0, *t.shape[1:]) for t in z], st).shape == (2, 0, 2, d)
    assert f.launch_count() == n0
    s1, s2 = st.clone(), st.clone()
    y = f.prefill(*a, s1, cu)
    f.test_set_wait(True, 2_000_000)  # no copies are issued: the waits run out after 2 ms
    f.prefill(*a, st.clone(), cu)
    assert f.status() == lm.LING_MOE_ERR_DEVICE_TIMEOUT
    f.test_set_wait(False)
    assert torch.equal(f.prefill(*a, s2, cu), y) and torch.equal(s1, s2) and f.status() == lm.LING_MOE_OK
    f.close()


@pytest.mark.parametrize("dk,dv,n", [(64, 64, 1), (128, 128, 4), (128, 64, 8), (64, 128, 5)])
def test_step_of_many_heads(dk, dv, n):
    """More heads than fit the GPU at once: the same bits as a few sequences at a time, padding and all."""
    Hk, Hv, B = 2, 8, 130
    f = lm.GatedDeltaRule(Hk, Hv, dk, dv, 8, B)
    a = [t.view(B, n, *t.shape[1:]) for t in make(B * n, Hk, Hv, dk, dv, True, 20)]
    st = pool(B, Hv, dk, dv, 20)
    slots = torch.randperm(B, generator=torch.Generator().manual_seed(1)).int()
    slots[[0, 5, 37, 38, 39, 40, 129]] = torch.tensor([-1, B, -7, -7, 2**31 - 1, -(2**31), -1], dtype=torch.int32)
    slots = slots.to(DEV)
    acc = (torch.arange(B, device=DEV) % (n + 1)).int()
    big, small = st.clone(), st.clone()
    o1 = torch.full((B, n, Hv, dv), 7.0, dtype=torch.bfloat16, device=DEV)
    o2 = o1.clone()
    f.step(*a, big, slots=slots, accepted=acc, out=o1)
    for i in range(0, B, 10):
        f.step(*[t[i:i + 10] for t in a], small, slots=slots[i:i + 10], accepted=acc[i:i + 10], out=o2[i:i + 10])
    assert torch.equal(o1, o2) and torch.equal(big, small) and f.status() == lm.LING_MOE_OK
    assert (o1[[0, 5, 37, 129]] == 7).all() and not torch.equal(big, st)
    x = sub([t[77] for t in a], slice(0, n))
    s0 = np64(st[slots[77]])
    want, states = D.rule(*x, s0, dk**-0.5)
    eo, es = D.step_bound(*x, s0, dk**-0.5)
    close_out(np64(o1[77]), want, eo)
    if acc[77]:
        close_state(np64(big[slots[77]]), states[acc[77] - 1], es[acc[77] - 1])
    assert torch.equal(f.step(*a, st.clone(), slots=slots, accepted=acc, out=o2), o1)
    f.test_set_wait(True, 2_000_000)  # the copies of later heads are not issued: the waits run out
    f.step(*a, st.clone(), slots=slots)
    assert f.status() == lm.LING_MOE_ERR_DEVICE_TIMEOUT
    f.test_set_wait(False)
    f.step(*a, small.copy_(st), slots=slots, accepted=acc, out=o2)
    assert torch.equal(o1, o2) and torch.equal(big, small) and f.status() == lm.LING_MOE_OK
    f.close()
