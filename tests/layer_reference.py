"""The norms, their gradients, 8-bit states and the delta rule over several tokens from their definitions,
in 64 bits, each with a bound on what fp32 arithmetic may add (name "tol_" + output's).

The bounds, with u = 2^-24 (half a unit of fp32's last place, relative):
- A sum of products over a row: a thread adds at most 32 of them in turn, then come at most 10 levels of
  shuffles and warps and a division: at most 48 u of the sum of the magnitudes. A mean of squares is
  positive, so its relative error is at most 48 u and its root's half of that; rsqrt adds 4 u (2 units of
  2^-23): r is off by at most 28 u, n = h r by 29 u, y = w n by 30 u.
- Gradients: u = w dy (1 u) and n (29 u) give a mean off by at most (48 + 30 + 2) u of mean|u n|; then
  n times it, the difference and the product with r add 29 + 3 + 28 u of the magnitudes: in all
  r (64 u |u| + 144 u |n| mean|u n|), and dh adds its own rounding.
- A weight's gradient: `rows` summands in any order are off by at most rows u of the sum of magnitudes, and
  each summand by 40 u.
- sigmoid(z): e^-z by the fast exponential is off by (2 + 1.2 |z|) 2^-23 = (4 + 2.4 |z|) u, the sum and the
  quotient add 6 u: (10 + 2.4 |z|) u for s, and twice that for 1 - s = e^-z s.
- decode over tokens: see `tokens`.
What is rounded to bf16 adds 2^-8 of its value (half a step), e4m3 2^-4 of it, or half its smallest step.
"""
import numpy as np

U = 2.0 ** -24
BF16 = 2.0 ** -8
E4M3 = 2.0 ** -4
FLUSH = 1e-30  # numbers that fp32 may flush to zero, with room


def f64(t):
    import torch
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def half_step(value, bf16):
    return BF16 * np.abs(value) if bf16 else U * np.abs(value)


def norm(h, w, eps):
    """y, rstd of rows h [rows, D]."""
    r = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    y = h * r[:, None] * (1.0 if w is None else w)
    return dict(y=y, tol_y=30 * U * np.abs(y) + FLUSH, rstd=r, tol_rstd=28 * U * r)


def norm_grad(dy, h, w, eps, dh=None):
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n = h * r
    u = dy * (1.0 if w is None else w)
    dx = r * (u - n * (u * n).mean(-1, keepdims=True))
    tol = r * U * (64 * np.abs(u) + 144 * np.abs(n) * np.abs(u * n).mean(-1, keepdims=True))
    if dh is not None:
        dx = dx + dh
        tol = tol + U * np.abs(dx)
    rows = h.shape[0]
    return dict(dx=dx, tol_dx=tol + FLUSH, dw=(dy * n).sum(0),
                tol_dw=(rows + 40) * U * np.abs(dy * n).sum(0) + FLUSH)


def gate(o, z, w, eps):
    r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    return o * r * (1.0 if w is None else w) / (1.0 + np.exp(-z))


def gate_grad(dout, o, z, w, eps):
    """o [rows, dv]."""
    w = np.ones(o.shape[-1]) if w is None else w
    r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    n = o * r
    with np.errstate(over="ignore"):
        s, c = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    es = (10 + 2.4 * np.abs(z)) * U
    u = dout * s * w
    mean = np.abs(u * n).mean(-1, keepdims=True)
    emean = (80 * U * np.abs(u * n) + es * np.abs(u * n)).mean(-1, keepdims=True)
    do = r * (u - n * (u * n).mean(-1, keepdims=True))
    dz = u * n * c
    rows = o.shape[0]
    return dict(do=do, tol_do=r * ((64 * U + es) * np.abs(u) + np.abs(n) * (64 * U * mean + emean)) + FLUSH,
                dz=dz, tol_dz=(40 * U + 3 * es) * np.abs(dz) + FLUSH, dw=(dout * s * n).sum(0),
                tol_dw=((rows + 40) * U * np.abs(dout * s * n) + es * np.abs(dout * s * n)).sum(0) + FLUSH)


def blocks_top(y, size):
    """The largest magnitude of every block of `size` values of a row, the last one what is left."""
    return np.stack([np.abs(y[:, i:i + size]).max(-1) for i in range(0, y.shape[1], size)], 1)


def decay(g, kind, lower):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return np.exp(g) if kind == "log" else s if kind == "logsigmoid" else np.exp(lower * s)


def tokens(q, k, v, a, beta, scale, S, count, l2norm):
    """One row and head: q, k, a [K, d], v [K, d], beta [K], S [d, d], its first `count` tokens. Returns
    out [K, d] and the state, with bounds.

    The bound follows the recurrence. A decay is off by at most 200 u (for the bounded gate, log a up to 10
    in magnitude times the 16 u of its sigmoid, and the exponential's 28 u; less for the others); with
    normalisation, k and q by 70 u. E bounds the state's error: S~ = a S has a E + 201 u |S~|; the read
    S~^T k, a sum over d channels (at most 32 in a thread, then two shuffles, over products of rounded a k:
    48 u), has sum |k| E~ + 320 u sum |k| |S~|; e = beta (v - read) has beta times that and 3 u of
    beta (|v| + |read|); S = S~ + k e has E~ + |k| err(e) + 73 u |k e| + u |S|. The output is
    (a q)^T S + (q.k) e: sum |q| E~ + 320 u sum |q| |S~| + sum |q k| (err(e) + 200 u |e|)."""
    K, d = q.shape
    out, tol = np.zeros((K, d)), np.zeros((K, d))
    S = S.copy()
    E = np.zeros_like(S)
    for t in range(count):
        kk, qq = k[t], q[t]
        if l2norm:
            kk, qq = kk / np.sqrt((kk * kk).sum() + 1e-6), qq / np.sqrt((qq * qq).sum() + 1e-6)
        qq = scale * qq
        S = a[t][:, None] * S
        E = a[t][:, None] * E + 201 * U * np.abs(S)
        read, mag = kk @ S, np.abs(kk) @ np.abs(S)
        err = np.abs(kk) @ E + 320 * U * mag
        e = beta[t] * (v[t] - read)
        err = beta[t] * (err + 3 * U * (np.abs(v[t]) + np.abs(read)))
        tol[t] = np.abs(qq) @ E + 320 * U * (np.abs(qq) @ np.abs(S)) + np.abs(qq * kk).sum() * (err + 200 * U * np.abs(e))
        S = S + kk[:, None] * e[None]
        E = E + np.abs(kk)[:, None] * err[None] + 73 * U * np.abs(kk[:, None] * e[None]) + U * np.abs(S)
        out[t] = qq @ S
    return dict(out=out, tol_out=tol + FLUSH, state=S, tol_state=E + FLUSH)
