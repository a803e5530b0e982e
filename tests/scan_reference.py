"""The gated linear recurrence and its gradient from their definitions, in 64
bits and token by token, with bounds on what fp32 arithmetic may add.

The bounds. Let m_t = a_t m_{t-1} + |w_t x_t| (m_0 = |h_0|), the recurrence of
the magnitudes, and u = 2^-24. A computed a_t is off by at most 8 u (an exp2 of
2 units of 2^-23, its rounded argument, a reciprocal and a few products), a
computed w_t by 24 u (1 - a keeps its relative accuracy; where it comes from
1 - e^x with e^x < 0.71 the 4 u of e^x grow by 0.71 / 0.29), and each product
and sum adds u. So the error of h obeys err_t <= a_t err_{t-1} + 40 u m_t, i.e.
err_t <= 40 u S_t with S_t = a_t S_{t-1} + m_t. Where pieces of the sequence are
composed, the maps of up to 18 pieces meet on the way to a token, one product
and sum each: at most 40 u m_t more, once. Hence 40 u (S_t + m_t); the backward
recurrence obeys the same with dout for w x. What is rounded to bf16 adds 2^-8
of its value (half a step). FLUSH covers numbers below the smallest normal fp32
number, 1.2e-38, which the kernels may flush to zero: under "norm" the weight is
the square root of such a one (up to sqrt(10 x 1.2e-38) = 3.5e-19), and inputs of
up to 5 carry it into sums of some tens.
"""
import numpy as np

U = 2.0 ** -24
BF16 = 2.0 ** -8
FLUSH = 1e-16


def gate(g, kind, lower):
    """log a and dlog a/dg."""
    g = np.asarray(g, np.float64)
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        c = 1.0 / (1.0 + np.exp(g))
    if kind == "log":
        return g, np.ones_like(g)
    if kind == "logsigmoid":
        return -np.logaddexp(0.0, -g), c
    return lower * s, lower * s * c


def weight(la, kind):
    """w and dw/dlog a (0 where w is 0 under "norm")."""
    if kind == "plain":
        return np.ones_like(la), np.zeros_like(la)
    if kind == "complement":
        return -np.expm1(la), -np.exp(la)
    w = np.sqrt(-np.expm1(2 * la))
    slope = np.zeros_like(w)
    np.divide(-np.exp(2 * la), w, out=slope, where=w > 0)
    return w, slope


def scan(x, g, init=None, kind="log", lower=-5.0, write="plain", dout=None, dfinal=None):
    """One sequence: x, g [T, D]; init, dfinal [D]. Returns a dict of value arrays and, under
    "tol_" + name, the fp32 bounds: out, final, and with dout: dx, dg, dinit."""
    x = np.asarray(x, np.float64)
    T, D = x.shape
    la, slope = gate(g, kind, lower)
    a = np.exp(la)
    w, dw = weight(la, write)
    with np.errstate(invalid="ignore"):
        wslope = np.where(dw == 0, 0.0, dw * slope)  # dw/dg; a slope of 0 wins over -0 / 0
    h0 = np.zeros(D) if init is None else np.asarray(init, np.float64)
    h, m, s = h0.copy(), np.abs(h0), np.abs(h0)
    H, M, TH = (np.empty((T, D)) for _ in range(3))
    before, tbefore = np.empty((T, D)), np.empty((T, D))
    t_h = np.zeros(D)
    for t in range(T):
        before[t], tbefore[t] = h, t_h
        b = w[t] * x[t]
        h = a[t] * h + b
        m = a[t] * m + np.abs(b)
        s = a[t] * s + m
        t_h = 40 * U * (s + m)
        H[t], M[t], TH[t] = h, m, t_h
    r = dict(out=H, final=h, tol_out=TH + FLUSH, tol_final=t_h + FLUSH)
    if dout is None:
        return r
    dout = np.asarray(dout, np.float64)
    u = np.zeros(D) if dfinal is None else np.asarray(dfinal, np.float64)
    um, us = np.abs(u), np.abs(u)
    E, TE, EM = (np.empty((T, D)) for _ in range(3))
    for t in range(T - 1, -1, -1):
        e = dout[t] + u
        em = np.abs(dout[t]) + um
        es = us + em
        E[t], EM[t], TE[t] = e, em, 40 * U * (es + em)
        u, um, us = a[t] * e, a[t] * em, a[t] * es
    mbefore = np.vstack([np.abs(h0)[None], M[:-1]]) if T else M
    inner = a * before * slope + x * wslope
    inner_m = a * mbefore * np.abs(slope) + np.abs(x * wslope)
    r.update(dx=w * E, tol_dx=w * (TE + 30 * U * EM) + FLUSH, dinit=u,
             tol_dinit=40 * U * (us + um) + FLUSH, dg=E * inner,
             tol_dg=TE * inner_m + EM * (tbefore * a * np.abs(slope) + 64 * U * inner_m) + FLUSH)
    return r


def spans(B, T, cu):
    return [(b * T, (b + 1) * T) for b in range(B)] if cu is None else list(zip(cu[:-1], cu[1:]))
