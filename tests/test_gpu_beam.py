"""Beam search on the GPU against the 64-bit oracle: tokens, parents and
finished flags equal, scores within one fp32 rounding plus the kernel's sum.

Score tolerance.  |score - exact| <= 2^-24 |score| (the final rounding) + the
error of log sum exp.  A term exp(z - m) takes z - m rounded (2^-25 |z - m|),
its product with log2 e (two roundings, 2^-24 |z - m| log2 e) and a 2-ulp
exponential: relative error below (|z - m| + 4) 2^-23, weighted by
exp(z - m) <= 1 whose mean of |z - m| is below 32 for these inputs: 36 * 2^-23
< 5e-6; fp32 partial sums of n <= 700 terms: n 2^-24 < 5e-5 at worst.  The
bound below uses 6e-5 absolute on lse for every case.
"""
import numpy as np
import pytest
import torch

import oracle.beam_ref as B
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


def check(bs, logits, scores, finished=None, eos=-1, **kw):
    t, p, s, d = bs.select(logits, scores, finished, eos, **kw)
    z = logits.float().cpu().numpy()
    z = z.reshape(-1, bs.beams, bs.vocab)
    wt, wp, ws, wd = B.select(z, scores.cpu().numpy(), None if finished is None else finished.cpu().numpy(), eos)
    assert np.array_equal(t.cpu().numpy(), wt), "tokens"
    assert np.array_equal(p.cpu().numpy(), wp), "parents"
    assert np.array_equal(d.cpu().numpy(), wd), "finished"
    s = s.cpu().numpy().astype(np.float64)
    fine = np.isfinite(ws)
    assert np.array_equal(fine, np.isfinite(s)) and np.isneginf(s[~fine]).all()
    assert (np.abs(s - ws)[fine] <= 2.0**-24 * np.abs(ws[fine]) + 6e-5).all()
    return t, p, s, d


def make(G, W, V, dtype, seed, scale=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = (scale * torch.randn(G, W, V, generator=g, device=DEV)).to(dtype)
    c = -torch.sort(torch.rand(G, W, generator=g, device=DEV) * 8)[0]
    return z, c


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,W,V", [(1, 1, 1), (1, 1, 5), (2, 16, 3), (3, 5, 1000), (1, 4, 4096), (2, 3, 4097), (1, 16, 20000),
                                   (40, 8, 12289), (1, 2, 157184), (70, 16, 300)])
def test_select_matches_the_oracle(G, W, V, dtype):
    bs = lm.BeamSearch(G, W, V)
    z, c = make(G, W, V, dtype, G * 1000 + V)
    check(bs, z, c)
    fin = torch.rand(G, W, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)) < 0.4
    check(bs, z, c, fin, eos=V // 2)
    c[:, 1:] = -INF  # the first step
    check(bs, z, c, None, eos=V - 1)
    bs.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_select_ties_masks_and_infinities(dtype):
    G, W, V = 3, 6, 9000
    bs = lm.BeamSearch(G, W, V)
    lowest = torch.finfo(dtype).min
    z, c = make(G, W, V, dtype, 5)
    for fill in (0.0, -INF, lowest, float("nan")):
        y = z.clone()
        y[0] = fill                        # every logit of the group
        y[1, 2] = fill                     # one beam's row
        y[2, :, 100:] = fill               # all but a few tokens
        check(bs, y, c)
        y[2, :, 3:] = fill                 # fewer live tokens than beams (where fill is no candidate)
        check(bs, y, c)
    y = z.clone()
    y[0, 1, 77] = INF                      # no softmax: the row has no candidate
    y[1, :, ::2] = float("nan")
    y[2, :, 1::3] = -INF
    check(bs, y, c)
    # whole numbers: ties everywhere, -0 equal to +0
    check(bs, z.round(), c.round())
    y = torch.zeros_like(z)
    y[:, :, ::2] = -0.0
    check(bs, y, torch.zeros_like(c))
    # rows in ascending and descending order; large offsets
    up = torch.arange(V, device=DEV, dtype=torch.float32) * 2**-9
    check(bs, up.expand(G, W, V).to(dtype).contiguous(), c)
    check(bs, up.flip(0).expand(G, W, V).to(dtype).contiguous(), c)
    if dtype == torch.float32:
        check(bs, z + 40.0, c - 1000.0)
    # dead, NaN-scored and finished beams of a group at once
    c2 = c.clone()
    c2[0, 0], c2[0, 1], c2[1] = float("nan"), -INF, -INF
    fin = torch.zeros(G, W, dtype=torch.bool, device=DEV)
    fin[2], fin[0, 3], fin[1, 2] = True, True, True
    check(bs, z, c2, fin, eos=7)
    bs.close()


def test_equal_beams_score_equally_whatever_their_alignment():
    """Rows of an odd length start at every alignment; the first step copies one row to all beams."""
    G, W, V = 2, 8, 30011
    bs = lm.BeamSearch(G, W, V)
    z, c = make(G, 1, V, torch.float32, 9)
    z = z.expand(G, W, V).contiguous()
    t, p, s, _ = check(bs, z, torch.zeros(G, W, device=DEV))
    assert (p.cpu().numpy() == np.arange(W)).all() and (s == s[:, :1]).all()
    # strided logits: a slice of a wider buffer, beams and groups apart
    buf = torch.full((G, W + 1, V + 13), 99.0, device=DEV)
    view = buf[:, :W, 5:5 + V]
    view.copy_(z)
    check(bs, view, c.expand(G, W).contiguous() - torch.arange(W, device=DEV))
    check(bs, z.view(G * W, V), torch.zeros(G, W, device=DEV))
    bs.close()


def test_select_in_place_graph_and_streams():
    G, W, V = 4, 4, 50000
    bs = lm.BeamSearch(8, W, V)
    z, c = make(G, W, V, torch.float32, 21)
    want = B.select(z.cpu().numpy(), c.cpu().numpy(), np.zeros((G, W), bool), 3)
    fin = torch.zeros(G, W, dtype=torch.bool, device=DEV)
    t, p = (torch.empty(G, W, dtype=torch.int32, device=DEV) for _ in range(2))
    cc = c.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    lm._check(lm.lib.ling_moe_beam_select(bs.handle, z.data_ptr(), 0, W * V, V, G, cc.data_ptr(), fin.data_ptr(), 3,
                                          t.data_ptr(), p.data_ptr(), cc.data_ptr(), fin.data_ptr(), st.cuda_stream))
    st.synchronize()
    assert np.array_equal(t.cpu().numpy(), want[0]) and np.allclose(cc.cpu().numpy(), want[2], atol=1e-4)
    assert np.array_equal(fin.cpu().numpy(), want[3])
    bs.select(z, c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = bs.select(z, c, torch.zeros(G, W, dtype=torch.bool, device=DEV), 3)
    for seed in (31, 32):
        z2, c2 = make(G, W, V, torch.float32, seed)
        z.copy_(z2)
        c.copy_(c2)
        g.replay()
        torch.cuda.synchronize()
        want = B.select(z.cpu().numpy(), c.cpu().numpy(), None, 3)
        assert np.array_equal(out[0].cpu().numpy(), want[0]) and np.array_equal(out[1].cpu().numpy(), want[1])
    bs.close()


def test_select_refusals():
    W, V = 4, 100
    bs = lm.BeamSearch(2, W, V)
    z, c = make(2, W, V, torch.float32, 1)
    fin = torch.zeros(2, W, dtype=torch.bool, device=DEV)
    n = bs.launch_count()
    for bad in (lambda: bs.select(z, c, fin), lambda: bs.select(z, c, fin, eos=V), lambda: bs.select(z, c, eos=-2),
                lambda: bs.select(torch.cat([z, z]), torch.cat([c, c]))):
        with pytest.raises(lm.LingMoEError) as e:
            bad()
        assert e.value.code == lm.LING_MOE_ERR_INVALID_ARG
    for bad in (lambda: bs.select(z.half(), c), lambda: bs.select(z.transpose(0, 1), c),
                lambda: bs.select(z, c.double()), lambda: bs.select(z, c[:1]), lambda: bs.select(z, c, fin.int(), 3),
                lambda: bs.select(z[:, :, ::2], c)):
        with pytest.raises(ValueError):
            bad()
    one = torch.empty(2 * W, dtype=torch.int32, device=DEV)
    f = torch.empty(2 * W, device=DEV)
    d = torch.empty(2 * W, dtype=torch.uint8, device=DEV)
    for t, p, s in ((one, one, f), (one, c, f), (z, one, f)):  # outputs that overlap
        assert lm.lib.ling_moe_beam_select(bs.handle, z.data_ptr(), 0, W * V, V, 2, c.data_ptr(), None, -1, t.data_ptr(),
                                           p.data_ptr(), s.data_ptr(), d.data_ptr(), None) == lm.LING_MOE_ERR_INVALID_ARG
    assert lm.lib.ling_moe_beam_select(bs.handle, z.data_ptr(), 7, W * V, V, 2, c.data_ptr(), None, -1, 16, 32, 48, 64,
                                       None) == lm.LING_MOE_ERR_INVALID_ARG
    t, _, _, _ = bs.select(z[:0], c[:0])
    assert t.shape == (0, W) and bs.launch_count() == n
    bs.close()


@pytest.mark.parametrize("G,W,shape,dtype", [
    (1, 1, (4,), torch.float32), (3, 2, (5,), torch.float32), (2, 4, (3, 7), torch.bfloat16), (5, 5, (64, 33), torch.float32),
    (2, 8, (128, 128), torch.float32), (1, 16, (4, 128, 128), torch.float32), (3, 16, (1,), torch.uint8),
    (2, 9, (301,), torch.uint8)])
def test_reorder_moves_rows(G, W, shape, dtype):
    rng = np.random.default_rng(G * 100 + W)
    bs = lm.BeamSearch(G, W, 10)
    raw = lambda n, sh: torch.from_numpy(rng.integers(0, 100, size=(n, *sh))).to(DEV).to(dtype)  # noqa: E731
    for kind in range(4):
        parents = np.stack([[np.roll(np.arange(W), 1), rng.permutation(W), rng.integers(0, W, W),
                             rng.integers(-2, W + 2, W)][kind] for _ in range(G)]).astype(np.int32)
        states = [raw(G * W, shape), raw(G * W, (3,)), raw(G * W, (16,))]
        want = [B.reorder(s.float().cpu().numpy(), parents) for s in states]
        bs.reorder(states, torch.from_numpy(parents).to(DEV))
        for s, x in zip(states, want):
            assert np.array_equal(s.float().cpu().numpy(), x)
        # rows of a pool, some out of range; rows nobody names stay
        pool = raw(G * W + 5, shape)
        slots = rng.permutation(G * W + 5)[:G * W].reshape(G, W).astype(np.int32)
        slots[0, 0] = -1 if kind % 2 else G * W + 5
        want = B.reorder(pool.float().cpu().numpy(), parents, slots)
        bs.reorder(pool, torch.from_numpy(parents).to(DEV), torch.from_numpy(slots).to(DEV))
        assert np.array_equal(pool.float().cpu().numpy(), want)
    bs.close()


def test_reorder_many_tensors_and_refusals():
    G, W = 2, 4
    bs = lm.BeamSearch(G, W, 10)
    parents = torch.tensor([[1, 0, 3, 2], [2, 2, 1, 3]], dtype=torch.int32, device=DEV)
    states = [torch.randn(G * W, 8 + i, device=DEV) for i in range(70)]
    want = [B.reorder(s.cpu().numpy(), parents.cpu().numpy()) for s in states]
    bs.reorder(states, parents)
    assert all(np.array_equal(s.cpu().numpy(), x) for s, x in zip(states, want))
    s = torch.zeros(G * W, 8, device=DEV)
    for bad in (lambda: bs.reorder([s, s[:4]], parents), lambda: bs.reorder(s.t(), parents),
                lambda: bs.reorder(s, parents.long()), lambda: bs.reorder(s, parents[:, :3])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lm.LingMoEError):
        bs.reorder([s, s], parents)      # the same rows twice
    with pytest.raises(lm.LingMoEError):
        bs.reorder(s[:7], parents)       # too few rows
    bs.reorder([], parents)
    bs.reorder([torch.zeros(G * W, 0, device=DEV)], parents)
    bs.close()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_select_more_equal_logits_than_the_candidates_fit(dtype):
    """600 rows in one piece each, the largest logit of a row on the tokens of 30 of a CTA's 256 threads: few enough
    threads to be looked at once more, but more candidates than their buffer takes."""
    G, W, V = 100, 6, 40000
    bs = lm.BeamSearch(G, W, V)
    z, c = make(G, W, V, dtype, 21, scale=0.5)
    z.clamp_(max=5.0)
    vec = 8 if dtype == torch.bfloat16 else 4
    t = torch.arange(V, device=DEV)
    own = (t % (256 * vec)) // vec
    z[:, :, own < 30] = 7.0
    z[::2, 3] = z[::2, 2]      # equal rows
    z[1::3, :, 5] = 8.0        # one above them
    check(bs, z, c)
    bs.close()
