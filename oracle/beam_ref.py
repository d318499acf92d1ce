"""Beam search's selection and reordering in numpy float64.

Candidates of group g: c_w + z_w[t] - log sum exp z_w for the tokens of a live
beam, (eos, c_w) for a finished one; the W best in order, ties to the lower
beam and (inside a beam, the larger logit, then) the lower token.  NaN and
-inf logits are no candidates; a row with +inf has none.
"""
import numpy as np


def select(logits, scores, finished=None, eos=-1):
    """(tokens, parents, scores float64, finished) [G, W] of logits [G, W, V]."""
    z = np.asarray(logits, np.float64)
    G, W, V = z.shape
    z = np.where(np.isnan(z), -np.inf, z)
    tokens = np.full((G, W), -1, np.int64)
    parents = np.tile(np.arange(W), (G, 1))
    out = np.full((G, W), -np.inf)
    done = np.ones((G, W), bool)
    for g in range(G):
        cand = []  # (score, beam, logit, token)
        for w in range(W):
            c = float(scores[g][w])
            if not c > -np.inf:
                continue
            if finished is not None and finished[g][w]:
                cand.append((c, w, 0.0, eos))
                continue
            row = z[g, w]
            m = row.max()
            if not np.isfinite(m):
                continue
            lse = m + np.log(np.exp(row - m).sum())
            keep = np.lexsort((np.arange(V), -row))[:W]
            cand += [(row[t] - lse + c, w, row[t], int(t)) for t in keep if row[t] > -np.inf]
        cand.sort(key=lambda x: (-x[0], x[1], -x[2], x[3]))
        for i, (s, w, _, t) in enumerate(cand[:W]):
            tokens[g, i], parents[g, i], out[g, i], done[g, i] = t, w, s, t == eos
    return tokens, parents, out, done


def reorder(state, parents, slots=None):
    """The rows of `state` after the move (a new array)."""
    G, W = parents.shape
    n = state.shape[0]
    slots = np.arange(G * W).reshape(G, W) if slots is None else slots
    new = state.copy()
    for g in range(G):
        for w in range(W):
            p = parents[g, w]
            if 0 <= p < W and 0 <= slots[g, p] < n and 0 <= slots[g, w] < n:
                new[slots[g, w]] = state[slots[g, p]]
    return new
