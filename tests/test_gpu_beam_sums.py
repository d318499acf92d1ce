"""Beam search over long vocabularies: the selection's sums against closed forms."""
import math

import numpy as np
import pytest
import torch

import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("V,rows", [(1 << 24, 304), ((1 << 22) + 5, 304), (1 << 24, 16), (157184, 304)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_long_sums_keep_their_last_terms(V, rows, dtype):
    """The first 8192 logits 0, all others -1.1: log sum exp in closed form.  With many rows one CTA walks a whole row, 16
    or 32 logits of a tile per thread, each thread with a 0 among its first.  A term exp(z - m) is off by (|z - m| + 4) 2^-23 =
    6.1e-7 of itself, a tile's sum of at most 32 terms in four chains of 8 and two joins by 10 2^-24 = 6.0e-7; tiles
    are added in 64 bits, so however many they are, the logarithm is off by 1.3e-6 (and by a fp32 exponential that
    joins threads and pieces of different largest logits, 0 and -1.1: (1.1 + 2) 2^-23 = 3.7e-7 more)."""
    W, G = 16, rows // 16
    z = torch.full((V,), -1.1, device=DEV).to(dtype)
    x = float(z[0])
    z[:8192] = 0.0
    c = torch.full((G, W), -math.inf, device=DEV)
    c[:, 3] = -2.0
    bs = lm.BeamSearch(G, W, V)
    t, p, s, d = bs.select(z.expand(G, W, V), c)
    want = np.full(W, -2.0 - math.log(8192 + (V - 8192) * math.exp(x)))
    got = s.double().cpu().numpy()
    err = np.abs(got - want).max()
    print(f"V {V}, {rows} rows: scores off by {err:.2e}")
    assert (np.abs(got - want) <= 1.7e-6 + 2.0**-24 * np.abs(want)).all(), err
    assert t.tolist() == [list(range(W))] * G and (p == 3).all() and not d.any()
    bs.close()


@pytest.mark.parametrize("V", [1 << 24, 157184])
def test_rows_that_rise_slowly(V):
    """Logits i / 2^22 (whole numbers of 24 bits, so exact), the largest of every tile a little above the last one's: the
    sums are rescaled all along, if by little.  The bound of the test above with terms up to 4 and on average 1 below the largest, its reference up
    to 1 below that ((1 + 1 + 4) 2^-23 = 7.2e-7), and 2^-22 / (1 - 1 / e) = 3.8e-7 for the rescalings."""
    W, G = 16, 19
    z = torch.arange(V, device=DEV, dtype=torch.float32) * 2.0**-22
    c = torch.full((G, W), -math.inf, device=DEV)
    c[:, 0] = 0.5
    bs = lm.BeamSearch(G, W, V)
    t, p, s, _ = bs.select(z.expand(G, W, V), c)
    lse = math.log(math.expm1(V * 2.0**-22) / math.expm1(2.0**-22))
    want = 0.5 + (V - 1 - np.arange(W)) * 2.0**-22 - lse
    err = np.abs(s.double().cpu().numpy() - want)
    print(f"V {V}: scores off by {err.max():.2e}")
    assert (err <= 2.1e-6 + 2.0**-24 * np.abs(want)).all(), err.max()
    assert t.tolist() == [list(range(V - 1, V - 1 - W, -1))] * G and (p == 0).all()
    bs.close()
