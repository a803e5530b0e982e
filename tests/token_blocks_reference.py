"""The delta rule over several tokens from its recurrence in 64 bits, with a bound that follows how it is computed
in blocks of eight tokens (u = 2^-24, half a unit of fp32's last place, relative):

- A decay: e^g by expf, off by 4 u; a sigmoid by (10 + 2.4 |z|) u (its exponential is off by (4 + 2.4 |z|) u, the
  sum and the quotient by 6 u); e^(lower s) by that times |lower s|, one rounding of the product, and
  (4 + 2.4 |lower s|) u of the exponential. A product of decays is off by the sum of its factors' and u for each.
- Products on split operands: x = hi + lo with |lo| <= 2^-11 |x|, of 12 bits cut off to 11 (2^-23 of x); two
  of these, and lo lo left out (2^-22): 8 u, 9 with what is of higher order. An MMA adds 8 products to its sum,
  each of the nine and the result cut off at a unit of fp32 (2 u) of the largest: 20 u of the sum of magnitudes.
- P = S^T (G k), R = S^T (G s q): d / 16 MMAs a warp and two additions (1 u for the small products' own sums): with
  w = G k off by e_w, sum |w| E + (9 + 20 d / 16 + 3 + e_w) u sum |w| |S|, E bounding the state's error.
- A, H (sums over channels in fp32): 4 in a lane, 5 levels of shuffles and the products: 12 u, scale 2 u, decays.
- 1 / |k|: half of the sum's 12 u and of eps, rsqrt's 4 u: 16 u.
- u = P + sum A e, e = r (beta (v - r u)), o = r (R + sum H e): every product and addition 1 u of its magnitude.
- S = G S + sum w e: three MMAs on one sum: 9 + 60 u and w's, the sum with the state one rounding.
"""
import numpy as np

from tests.layer_reference import FLUSH, U

BLOCK = 8


def decay_error(g, kind, lower):
    """What a decay may be off by, in u, relative."""
    if kind == "none":
        return np.zeros_like(g)
    if kind == "log":
        return np.full_like(g, 4.0)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    es = 10 + 2.4 * np.abs(g)
    return es if kind == "logsigmoid" else np.abs(lower * s) * (es + 1) + 4 + 2.4 * np.abs(lower * s)


def tokens(q, k, v, a, ea, beta, scale, S, count, l2norm):
    """One row and head: q, k, a, ea [K, d] (ea: the decays' errors in u), v [K, d], beta [K], S [d, d], its first
    `count` tokens. Returns out [K, d] and the state, with bounds."""
    K, d = q.shape
    out, tol, S, E = np.zeros((K, d)), np.zeros((K, d)), S.copy(), np.zeros_like(S)
    ea = ea + 1
    for lo in range(0, count, BLOCK):
        S0, C = S.copy(), min(BLOCK, count - lo)
        e, err = np.zeros((C, d)), np.zeros((C, d))  # as they are kept: with k's factor
        span = np.ones((C, d))                         # G_{j:t} of every earlier token, and what it is off by
        espan = np.zeros((C, d))
        G, eG = np.ones(d), np.zeros(d)
        for t in range(C):
            i = lo + t
            G, eG = G * a[i], eG + ea[i]
            span[:t], espan[:t] = span[:t] * a[i], espan[:t] + ea[i]
            r = rq = 1.0
            er = 0.0
            if l2norm:
                r, rq, er = 1 / np.sqrt((k[i] ** 2).sum() + 1e-6), 1 / np.sqrt((q[i] ** 2).sum() + 1e-6), 16.0
            # The definition, one token at a time.
            S = a[i][:, None] * S
            e[t] = r * beta[i] * (v[i] - r * (k[i] @ S))
            S = S + k[i][:, None] * e[t][None]
            out[i] = scale * rq * (q[i] @ S)

            def read(w, ew, past):
                """The magnitudes that meet in S0^T w + sum_j (w . k_j G_{j:t}) e_j, and their error."""
                fixed = 9 + 20 * d / 16 + 3
                mag = np.abs(w * G) @ np.abs(S0)
                bad = np.abs(w * G) @ E + U * (((fixed + ew + eG) * np.abs(w * G)) @ np.abs(S0))
                for j in range(past):
                    p = np.abs(w * k[lo + j] * span[j])
                    m = p.sum() * np.abs(e[j])
                    bad = bad + p.sum() * err[j] + U * ((12 + ew + espan[j]) * p).sum() * np.abs(e[j]) + 2 * U * m
                    mag = mag + m
                return mag, bad + (past + 1) * U * mag

            mag, bad = read(k[i], 1, t)
            err[t] = r * beta[i] * (r * bad + U * (er + 4) * r * mag + 4 * U * np.abs(v[i])) + U * (er + 2) * np.abs(e[t])
            mag, bad = read(scale * q[i], 2, t + 1)
            tol[i] = rq * (bad + U * (er + 2) * mag)
        # w_j e_j, and G S0.
        bad = G[:, None] * E + U * ((eG + 1) * G)[:, None] * np.abs(S0) + U * np.abs(S)
        for j in range(C):
            w = np.abs(k[lo + j] * span[j])
            bad = bad + w[:, None] * err[j][None] + U * ((69 + 2 + espan[j]) * w)[:, None] * np.abs(e[j])[None]
        E = bad
    return dict(out=out, tol_out=tol + FLUSH, state=S, tol_state=E + FLUSH)
