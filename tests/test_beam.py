"""Beam search without a GPU: the oracle against a brute force over every
candidate, and the refusals of the C entry points and the binding."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

import oracle.beam_ref as B
import weight_only_int4_fp32_b200 as lm

BAD = lm.LING_MOE_ERR_INVALID_ARG


def brute(z, c, fin, eos):
    """Every candidate of one group scored in Python floats and sorted."""
    W, V = z.shape
    cand = []
    for w, t in itertools.product(range(W), range(V)):
        if fin[w]:
            if t == eos:
                cand.append((-c[w], w, t))
            continue
        lse = math.log(math.fsum(math.exp(x) for x in z[w]))
        cand.append((-(c[w] + z[w, t] - lse), w, t))
    cand.sort()
    return [(t, w, -s) for s, w, t in cand[:W]]


@pytest.mark.parametrize("W,V", [(1, 1), (1, 7), (3, 2), (4, 50), (7, 13)])
def test_oracle_select_is_a_sort_of_every_candidate(W, V):
    rng = np.random.default_rng(W * 100 + V)
    z = rng.normal(size=(2, W, V))
    c = -np.sort(rng.random((2, W)) * 3)
    fin = rng.random((2, W)) < 0.3
    t, p, s, d = B.select(z, c, fin, eos=V - 1)
    for g in range(2):
        want = brute(z[g], c[g], fin[g], V - 1)
        for i, (wt, wp, ws) in enumerate(want):
            assert (t[g, i], p[g, i]) == (wt, wp) and abs(s[g, i] - ws) < 1e-12
            assert d[g, i] == (wt == V - 1)
        assert (t[g, len(want):] == -1).all() and np.isneginf(s[g, len(want):]).all()


def test_oracle_select_ties_go_to_the_lower_beam_then_the_lower_token():
    t, p, s, _ = B.select(np.zeros((1, 3, 5)), np.zeros((1, 3)))
    assert t.tolist() == [[0, 1, 2]] and p.tolist() == [[0, 0, 0]]
    z = np.zeros((1, 2, 4))
    z[0, :, 2] = 1.0
    t, p, _, _ = B.select(z, np.zeros((1, 2)))
    assert t.tolist() == [[2, 2]] and p.tolist() == [[0, 1]]


def test_oracle_reorder_moves_all_places_at_once():
    s = np.arange(6)[:, None]
    assert B.reorder(s, np.array([[1, 2, 0], [0, 0, 2]])).ravel().tolist() == [1, 2, 0, 3, 3, 5]
    slots = np.array([[4, 2, 9], [0, -1, 5]])
    assert B.reorder(s, np.array([[1, 0, 0], [2, 0, 7]]), slots).ravel().tolist() == [5, 1, 4, 3, 2, 5]


def _create(groups, beams, vocab, out=True):
    h = ctypes.c_void_p()
    return lm.lib.ling_moe_beam_create(groups, beams, vocab, ctypes.byref(h) if out else None), h.value


@pytest.mark.parametrize("groups,beams,vocab,code", [
    (0, 4, 100, BAD), (1, 0, 100, BAD), (1, 4, 0, BAD), (1, 17, 100, lm.LING_MOE_ERR_UNSUPPORTED),
    (65536, 4, 100, lm.LING_MOE_ERR_UNSUPPORTED), (1, 4, (1 << 30) + 1, lm.LING_MOE_ERR_UNSUPPORTED)])
def test_create_refuses(groups, beams, vocab, code):
    assert _create(groups, beams, vocab) == (code, None)
    assert _create(1, 4, 100, out=False)[0] == BAD


def test_null_handle():
    assert lm.lib.ling_moe_beam_select(None, 16, 0, 1, 1, 1, 16, None, -1, 16, 16, 16, 16, None) == BAD
    assert lm.lib.ling_moe_beam_launch_count(None) == 0
    lm.lib.ling_moe_beam_destroy(None)


def _reorder(states=((0x100000, 64),), rows=8, slots=None, parents=0x900000, groups=2, beams=4):
    ptr = (ctypes.c_void_p * len(states))(*[a for a, _ in states])
    nb = (ctypes.c_size_t * len(states))(*[b for _, b in states])
    return lm.lib.ling_moe_beam_reorder(ptr, nb, len(states), rows, slots, parents, groups, beams, None)


@pytest.mark.parametrize("kw", [
    dict(beams=0), dict(beams=17), dict(groups=-1), dict(groups=65536), dict(rows=-1), dict(rows=7),
    dict(parents=None), dict(parents=0x900002), dict(slots=0x800001), dict(states=((None, 64),)),
    dict(parents=0x100000 + 64), dict(slots=0x100000),
    dict(states=((0x100000, 64), (0x100000 + 500, 64)))])
def test_reorder_refuses(kw):
    assert _reorder(**kw) == BAD
    assert lm.ling_moe_last_error()


def test_reorder_of_nothing_is_ok():
    assert _reorder(groups=0) == lm.LING_MOE_OK and _reorder(states=()) == lm.LING_MOE_OK
    assert _reorder(rows=0, slots=0x800000) == lm.LING_MOE_OK


def test_binding_refuses_wrong_tensors():
    b = object.__new__(lm.BeamSearch)  # no handle: the checks run before the library is called
    b.beams, b.vocab, b.handle, b._torch = 4, 100, None, torch
    with pytest.raises(ValueError):
        b.select(torch.zeros(1, 4, 100), torch.zeros(1, 4))               # not on the GPU
    with pytest.raises(ValueError):
        b.select(torch.zeros(3, 100), torch.zeros(1, 4))                  # rows do not fill groups
    with pytest.raises(ValueError):
        b.reorder([torch.zeros(4, 3)], torch.zeros(1, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.reorder([torch.zeros(4, 3)], torch.zeros(4, dtype=torch.int32))
