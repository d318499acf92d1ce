"""Gated delta rule in numpy float64, and bounds on what the kernels may be off.

TEST INFRASTRUCTURE ONLY.  Per value head, with k and q divided by
sqrt(sum of squares + 1e-6):
  S <- diag(exp min(g, 0)) S;  u = beta (v - S^T k);  S <- S + k u^T;
  out = scale S^T q
Arrays: q, k [T, Hk, dk], v [T, Hv, dv], g [T, Hv, dk] or [T, Hv],
beta [T, Hv], state [Hv, dk, dv].

The bounds carry, per head and state column, the 2-norm e of the state's error.
One token maps an error by (I - beta k k^T) diag(a), whose norm is at most
max(a) for unit keys and 0 <= beta <= 2, so e <- max(a) e + (what the token's
own rounding adds).  u = 2^-24 below.
"""
import numpy as np

U = 2.0**-24
CHUNK = 64


def _unit(x):
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)


def heads(q, k, v, g, beta):
    """float64, one row per value head: unit q and k, decays exp(min(g, 0)) per channel."""
    r = v.shape[1] // k.shape[1]
    q, k = np.repeat(_unit(q), r, 1), np.repeat(_unit(k), r, 1)
    g = np.asarray(g, np.float64)
    g = g if g.ndim == 3 else np.broadcast_to(g[:, :, None], k.shape)
    a = np.exp(np.where(g > 0, 0.0, g))
    return q, k, np.asarray(v, np.float64), a, np.asarray(beta, np.float64)


def rule(q, k, v, g, beta, state, scale):
    """(out [T, Hv, dv], states after every token [T, Hv, dk, dv])."""
    q, k, v, a, b = heads(q, k, v, g, beta)
    S = np.asarray(state, np.float64).copy()
    out = np.empty(v.shape)
    states = np.empty((v.shape[0], *S.shape))
    for t in range(v.shape[0]):
        S = S * a[t][:, :, None]
        u = b[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        out[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
        states[t] = S
    return out, states


def step_bound(q, k, v, g, beta, state, scale):
    """(error of out before its rounding [T, Hv, dv], 2-norm of the state's error by column after every token [T, Hv, dv]).

    exp is off by 2 ulp (4 u) and its product by 1 u; a unit key by 9 u (a sum of
    squares in 9 additions, halved by the root; root, sum with the 1e-6, quotient,
    product); S^T k adds 19 u in its chain of 16 products and 3 joins, so it is
    off by 33 u |S|; v - x and beta by 2 u (|v| + |S|); k u^T by the key's 9 u,
    and its sum by 1 u more.  The output takes S^T q (33 u) and k.q (9 + 18 u)
    with three more roundings."""
    q, k, v, a, b = heads(q, k, v, g, beta)
    S = np.asarray(state, np.float64).copy()
    e = np.zeros((S.shape[0], S.shape[2]))
    out, es = np.empty(v.shape), np.empty(v.shape)
    for t in range(v.shape[0]):
        S0 = np.linalg.norm(S, axis=1)
        S = S * a[t][:, :, None]
        bt = np.abs(b[t])[:, None]
        u = b[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        size = S0 + np.abs(v[t])
        du = 35 * U * bt * size
        e = a[t].max(-1)[:, None] * e + 6 * U * S0 + du + 11 * U * np.abs(u) + 1e-37
        out[t] = abs(scale) * (e + 36 * U * S0 + du + 32 * U * np.abs(u)) * (1 + 4 * U)
        es[t] = e
    return out, es


def prefill_bound(q, k, v, g, beta, state, scale):
    """The same for the chunked prefill of one sequence: (out's error [T, Hv, dv], the last state's by column [Hv, dv]).

    Chunks of 64 tokens:  (I + A) [W, U~] = diag(b) [Kt, V],  U = U~ - W S0,
    O = Qt S0 + B U,  S1 = D S0 + Kh^T U.  Every decay is a product of at most
    64 exps (5 u each with its product), a key's norm 9 u, the joins a few more:
    eta = 360 u.  Operands that feed the state are two fp16 terms (2^-22 of the
    value, at least 2^-35 at the fixed scale of 2^10; scaled by their largest at
    least 2^-37 of it), with the product of the two low terms left out and 16 u
    of fp32 sums: mm = 3 2^-22 + 16 u of the magnitudes.  The fp16 operands of
    the output: 2^-11 each.

    The solution Z of (I + A) Z = R by 16-row blocks: what is computed solves the
    system up to the residual of  A's error E and its products (E + mm |A|) |Z|,
    R's error, 8 u of the sums, and the diagonal blocks' inverses Td, formed by
    16 steps of substitution (32 u |Td| |Ld| |Td|), split and multiplied:
    |Ld| (32 u |Td| |Ld| |Td| + (2^-22 + mm) |Td|) |Ld| |Z|.  Its error is |(I + A)^-1|
    times that, and 2^-22 |Z| for the terms that are kept."""
    q, k, v, a, b = heads(q, k, v, g, beta)
    T_, H = b.shape
    S = np.asarray(state, np.float64).copy()
    e = np.zeros((H, S.shape[2]))
    out = np.empty(v.shape)
    eta, mm, h16, tiny = 360 * U, 3 * 2.0**-22 + 16 * U, 2.0**-11, 2.0**-35
    ab = np.abs
    with np.errstate(divide="ignore"):
        la = np.log(a)
    for c in range(0, T_, CHUNK):
        sl = slice(c, min(T_, c + CHUNK))
        n = sl.stop - c
        tr = lambda x: np.swapaxes(x[sl], 0, 1)  # noqa: E731  [H, n, ...]
        qc, kc, vc, bc, lc = tr(q), tr(k), tr(v), tr(b), tr(la)
        # decays between tokens: products of the factors, zeros included
        dec = np.zeros((H, n, n, a.shape[2]))  # [h, i, j, c] = prod a over (j, i]
        for j in range(n):
            dec[:, j, j] = 1.0
            for i in range(j + 1, n):
                dec[:, i, j] = dec[:, i - 1, j] * np.exp(lc[:, i])
        first = dec[:, :, 0] * np.exp(lc[:, :1])     # [h, i, c] = prod a over the chunk's first i + 1
        to_end = dec[:, n - 1]                       # [h, j, c]
        low, strict, eye = np.tril(np.ones((n, n))), np.tril(np.ones((n, n)), -1), np.eye(n)
        A = np.einsum("hic,hijc,hjc->hij", kc, dec, kc) * strict * bc[:, :, None]
        Am = np.einsum("hic,hijc,hjc->hij", ab(kc), dec, ab(kc)) * strict * ab(bc)[:, :, None]
        B = np.einsum("hic,hijc,hjc->hij", qc, dec, kc) * low
        Bm = np.einsum("hic,hijc,hjc->hij", ab(qc), dec, ab(kc)) * low
        del dec
        Ti = np.linalg.inv(eye + A) * low
        Ta = ab(Ti)
        blocks = (np.arange(n)[:, None] // 16 == np.arange(n)[None, :] // 16) * low
        Ld, Td = ab(eye + A) * blocks, Ta * blocks  # a triangular inverse's diagonal blocks are its blocks' inverses
        Kt, Qt, Kh, D = kc * first, qc * first, kc * to_end, first[:, n - 1]
        E = (eta + mm) * Am + tiny * strict
        inv = Ld @ (32 * U * Td @ Ld @ Td + (2.0**-22 + mm) * Td + tiny * blocks) @ Ld

        def solve(R, r_err):
            Z = Ti @ (bc[:, :, None] * R)
            za = ab(Z) + 2.0**-36 * (ab(eye + A) @ ab(Z)).max(axis=1, keepdims=True)
            resid = r_err * ab(bc)[:, :, None] * ab(R) + (E + mm * ab(A)) @ za + inv @ za \
                + 8 * U * (ab(bc)[:, :, None] * ab(R) + ab(A) @ ab(Z))
            return Z, Ta @ resid + 2.0**-22 * ab(Z)

        W, dW = solve(Kt, eta)
        Ut, dUt = solve(vc, 2 * U)
        dW = dW + tiny
        Uc = Ut - W @ S
        O = Qt @ S + B @ Uc
        S1 = D[:, :, None] * S + np.swapaxes(Kh, 1, 2) @ Uc
        top = lambda x: ab(x).max(axis=1, keepdims=True) * 2.0**-37  # noqa: E731  by column
        Sa, Ua = ab(S) + top(S), ab(Uc) + top(Uc)
        dU = (dW + mm * ab(W)) @ Sa + dUt + 8 * U * (ab(Ut) + ab(W) @ ab(S))
        dS = 330 * U * D[:, :, None] * ab(S) + np.swapaxes(ab(Kh), 1, 2) @ dU \
            + np.swapaxes((eta + mm) * ab(Kh) + tiny, 1, 2) @ Ua + 10 * U * (ab(S1) + D[:, :, None] * ab(S))
        dUe = dU + ab(bc)[:, :, None] * e[:, None, :]
        dO = ((2 * h16 + eta + 16 * U) * ab(Qt) + tiny) @ Sa + np.linalg.norm(Qt, axis=2)[:, :, None] * e[:, None, :] \
            + ab(B) @ dUe + ((2 * h16 + eta + 16 * U) * Bm + 2 * h16 * ab(B) + tiny) @ Ua + 8 * U * ab(O)
        out[sl] = np.swapaxes(abs(scale) * dO, 0, 1)
        shrink = np.prod(np.swapaxes(np.exp(lc), 1, 2).max(1), axis=1)  # [H]: product over tokens of max(a)
        e = shrink[:, None] * e + np.linalg.norm(dS, axis=1) + 1e-37
        S = S1
    return out, e
