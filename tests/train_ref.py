"""Plain 64-bit definitions of the training calls (numpy), with bounds on what
fp32 and fp16 arithmetic may add.  Written from the formulas; shares nothing
with the library."""
from __future__ import annotations

import numpy as np

import oracle

U32 = 2.0 ** -24        # half a step of fp32, relative
UBF = 2.0 ** -8         # of bf16
U16 = 2.0 ** -11        # of fp16


# ------------------------------------------------------ 8-bit checkpoints
def act8(x):
    """x [T, H] float -> (codes int8, scales uint8, values float64)."""
    b = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    e = np.frexp(safe)[1] - 7
    e = e + (np.rint(np.ldexp(safe, -e)) > 127)
    e = np.where(amax == 0, -126, np.clip(e, -126, 121))
    q = np.clip(np.rint(np.ldexp(np.where(bad[..., None], 0.0, b), -e[..., None])), -127, 127)
    v = np.where(bad[..., None], np.nan, np.ldexp(q, e[..., None]))
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return q.astype(np.int8).reshape(x.shape), s, v.reshape(x.shape)


# ----------------------------------------------- balance loss and routing
def balance(logits, ids, mask, E, balance_coef, z_coef):
    """(counts int [E+1], losses [4], gradient [T, E] for d_loss = 1)."""
    l = np.asarray(logits, np.float64)
    T, k = ids.shape
    keep = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    N = int(keep.sum())
    counts = np.zeros(E + 1, np.int64)
    np.add.at(counts, ids[keep].ravel(), 1)
    counts[E] = N
    grad = np.zeros((T, E))
    if N == 0:
        return counts, np.zeros(4), grad
    f = counts[:E] / (N * k)
    P, z = np.zeros(E), 0.0
    for t in np.nonzero(keep)[0]:
        m = l[t].max()
        if m == -np.inf:
            continue
        e = np.exp(l[t] - m)
        p, lse = e / e.sum(), m + np.log(e.sum())
        P += p / N
        z += lse * lse / N
        grad[t] = balance_coef * E / N * p * (f - (f * p).sum()) + z_coef * 2 * lse / N * p
    b = E * (f * P).sum()
    return counts, np.array([balance_coef * b + z_coef * z, b, z, N]), grad


def gates(ids, w, dw, E, keep=None):
    """The gates' gradient, [T, E]."""
    T, k = ids.shape
    w, dw = np.asarray(w, np.float64), np.asarray(dw, np.float64)
    v = w * (dw - (w * dw).sum(1, keepdims=True))
    g = np.zeros((T, E))
    for t in range(T):
        if keep is None or keep[t]:
            np.add.at(g[t], ids[t], v[t])
    return g


def spread(logits, keep):
    """Largest distance of a finite logit of a counted row from its row's maximum."""
    l = np.asarray(logits, np.float64)[keep]
    if l.size == 0:
        return 0.0
    m = l.max(1, keepdims=True)
    d = np.where(np.isfinite(l) & np.isfinite(m), np.where(np.isfinite(m), m, 0) - np.where(np.isfinite(l), l, 0), 0)
    return float(np.abs(d).max(initial=0.0))


# ---------------------------------------------------------------- experts
def matrices(bits, H, I, blob):
    """(Wg [I,H], Wu [I,H], Wd [H,I]) of a blob, float64."""
    return oracle.expert_weights(bits, H, I, blob)


def ffn_forward(W, x):
    g, u = x @ W[0].T, x @ W[1].T
    return (g / (1 + np.exp(-g)) * u) @ W[2].T


def ffn_backward(W, x, dy, ua, ub):
    """One expert on rows x, dy [n, H]: (dxp, dw, bound on |dxp| errors, bound
    on |dw| errors).  ua: half a step of the products' operands (weights, x,
    dy, the gradients of g and u), 0 for exact operands; ub: of the sums."""
    Wg, Wu, Wd = W
    H, I = Wg.shape[1], Wg.shape[0]
    g, u, q = x @ Wg.T, x @ Wu.T, dy @ Wd
    s = 1 / (1 + np.exp(-g))
    a = g * s
    F = s + a * (1 - s)
    dg, du = q * u * F, q * a
    dxp, dw = dg @ Wg + du @ Wu, (q * a * u).sum(1)
    # an fp16 operand below 2^-14 of its row's scale is off by up to 2^-25 of that scale
    def tiny(v):
        return np.abs(v).max(1, keepdims=True) * 2.0 ** -25 if ua else 0.0

    def r(n):
        return 2 * ua + (n + 8) * ub
    ax, ay = np.abs(x), np.abs(dy)
    eg = r(H) * (ax @ np.abs(Wg).T) + tiny(x) * np.abs(Wg).sum(1)
    eu = r(H) * (ax @ np.abs(Wu).T) + tiny(x) * np.abs(Wu).sum(1)
    eq = r(H) * (ay @ np.abs(Wd)) + tiny(dy) * np.abs(Wd).sum(0)
    # F and silu vary by at most 0.5 and 1.1 per unit of g; |F| <= 1.1
    small = 1.1                                       # room for the products of two errors
    edg = small * (np.abs(u * F) * eq + np.abs(q * F) * eu + np.abs(q * u) * 0.5 * eg) + (ua + 12 * U32) * np.abs(q * u) * 1.1
    edu = small * (np.abs(a) * eq + np.abs(q) * 1.1 * eg) + (ua + 12 * U32) * np.abs(du)
    if ua:                                            # the stored gradients' own smallest steps
        top = np.abs(x).max(1, keepdims=True) * np.abs(dy).max(1, keepdims=True)
        edg, edu = edg + 2.0 ** -25 * top, edu + 2.0 ** -25 * top
    ex = small * (edg @ np.abs(Wg) + edu @ np.abs(Wu)) + (ua + (2 * I + 8) * ub) * (np.abs(dg) @ np.abs(Wg) + np.abs(du) @ np.abs(Wu))
    ew = small * (np.abs(a * u) * eq + np.abs(q * a) * eu + np.abs(q * u) * 1.1 * eg).sum(1) + (I + 8) * U32 * np.abs(q * a * u).sum(1)
    return dxp, dw, ex, ew


def experts_backward(bits, H, I, blobs, shared, ids, w, x, dy, ua=0.0, ub=U32, skip=()):
    """(dx, dw, bounds of both) of the whole step in float64; experts in `skip`
    add nothing."""
    T, k = ids.shape
    dx, dw = np.zeros((T, H)), np.zeros((T, k))
    ex, ew = np.zeros((T, H)), np.zeros((T, k))
    size = np.zeros((T, H))
    w = np.asarray(w, np.float64)
    for e in np.unique(ids):
        if e in skip or e < 0:
            continue
        t, j = np.nonzero(ids == e)
        d, v, bx, bw = ffn_backward(matrices(bits, H, I, blobs[e]), x[t], dy[t], ua, ub)
        wt = w[t, j][:, None]
        np.add.at(dx, t, d * wt)
        np.add.at(ex, t, bx * np.abs(wt))
        np.add.at(size, t, np.abs(d * wt))
        dw[t, j], ew[t, j] = v, bw
    if shared is not None:
        d, _, bx, _ = ffn_backward(matrices(bits, H, I, shared), x, dy, ua, ub)
        dx += d
        ex += bx
        size += np.abs(d)
    return dx, dw, 1.05 * ex + (k + 4) * U32 * size, 1.05 * ew
