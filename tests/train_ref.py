"""Plain 64-bit implementations of the training step's operators, and the
error bounds their float32 kernels are held to.

A kernel's output is a float32 evaluation of a sum of products, rounded once
to the output's type.  With u the type's unit roundoff (2^-8 bf16, 2^-24
float32) and n terms of magnitude sum S = sum |a_i b_i|,
    |got - exact| <= u |exact| + (n + 8) 2^-23 S
holds for any order of addition and for additions that truncate (each of the
n steps loses at most 2^-23 of a partial sum, which is at most S); the 8 covers
the products, the scale factors and the rounding of the bound itself.
Everything below works on exact float64 copies of the inputs.
"""
from __future__ import annotations

import numpy as np

ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
STEP = 2.0 ** -23


def bound(exact, terms, magnitude, kind):
    """Largest |got - exact| of a sum of `terms` products of absolute sum
    `magnitude`, rounded to `kind`; float32's smallest normal stands in for
    what underflows."""
    acc = (np.asarray(terms) + 8) * STEP * magnitude
    return ROUND[kind] * (np.abs(exact) + acc) + acc + 2.0 ** -126


def check(got, exact, limit, what):
    got = np.asarray(got, np.float64)
    assert got.shape == exact.shape, what
    bad = ~(np.abs(got - exact) <= limit)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} values outside the bound, the worst "
                           f"{np.max(np.where(bad, np.abs(got - exact) / limit, 0)):.3g} times")


def sort_slots(idx, N, capacity):
    """expert_offsets, perm, inv_perm of idx [T, k], slot by slot."""
    flat = idx.reshape(-1)
    mine = [[] for _ in range(N)]
    none = []
    for slot, e in enumerate(flat.tolist()):
        if 0 <= e < N and (capacity == 0 or len(mine[e]) < capacity):
            mine[e].append(slot)
        else:
            none.append(slot)
    off = np.concatenate([[0], np.cumsum([len(m) for m in mine])]).astype(np.int32)
    kept = [s for m in mine for s in m]
    perm = np.array(kept + [-1] * len(none), np.int32)
    inv = np.zeros(flat.size, np.int32)
    for pos, s in enumerate(kept):
        inv[s] = pos
    for i, s in enumerate(none):
        inv[s] = -2 - (len(kept) + i)
    return off, perm, inv.reshape(idx.shape)


def dispatch(x, perm, k):
    out = np.zeros((perm.size, x.shape[1]), x.dtype)
    live = perm >= 0
    out[live] = x[perm[live] // k]
    return out


def combine(y, gate, inv, add):
    """(exact, sum of magnitudes)"""
    T, k = inv.shape
    out = np.zeros((T, y.shape[1])) if add is None else add.copy()
    mag = np.abs(out)
    for t in range(T):
        for s in range(k):
            if inv[t, s] >= 0:
                r = (1.0 if gate is None else gate[t, s]) * y[inv[t, s]]
                out[t] += r
                mag[t] += np.abs(r)
    return out, mag


def combine_grad(dout, y, gate, inv):
    """(dy, dgate, sum of magnitudes of dgate)"""
    T, k = inv.shape
    dy = np.zeros_like(y)
    dgate, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            if inv[t, s] >= 0:
                dy[inv[t, s]] = (1.0 if gate is None else gate[t, s]) * dout[t]
                dgate[t, s] = dout[t] @ y[inv[t, s]]
                mag[t, s] = np.abs(dout[t]) @ np.abs(y[inv[t, s]])
    return dy, dgate, mag


def gates(prob, idx, renorm):
    """The gates of the chosen experts (zero for a slot without one)."""
    here = idx >= 0
    p = np.where(here, np.take_along_axis(prob, np.where(here, idx, 0), 1), 0.0)
    if renorm:
        total = p.sum(1, keepdims=True)
        p = np.where(total > 0, p / np.where(total > 0, total, 1.0), 0.0)
    return p


def balance_loss(prob, load, c):
    return c * prob.shape[1] * float(load @ prob.mean(0))


def load_of(idx, N):
    return np.bincount(idx[idx >= 0], minlength=N) / idx.size


def gate_grad(prob, idx, dgate, renorm, c):
    """(dlogits, loss, sum of magnitudes of dlogits)"""
    T, N = prob.shape
    v, mag_v = np.zeros((T, N)), np.zeros((T, N))
    for t in range(T):
        live = [s for s in range(idx.shape[1]) if idx[t, s] >= 0]
        p = np.array([prob[t, idx[t, s]] for s in live])
        dg = dgate[t, live]
        if renorm and live:
            total = p.sum()
            mean = (dg * p).sum() / total if total > 0 else 0.0
            size = (np.abs(dg) + (np.abs(dg) * p).sum() / total) / total if total > 0 else np.zeros(len(live))
            dg = (dg - mean) / total if total > 0 else np.zeros(len(live))
        else:
            size = np.abs(dg)
        for s, a, b in zip(live, dg, size):
            v[t, idx[t, s]] += a
            mag_v[t, idx[t, s]] += b
    load = load_of(idx, N)
    v += c * N / T * load
    mag_v += c * N / T * load
    dl = prob * (v - (prob * v).sum(1, keepdims=True))
    return dl, balance_loss(prob, load, c), prob * (mag_v + (prob * mag_v).sum(1, keepdims=True))


def sigmoid(g):
    return 1.0 / (1.0 + np.exp(-g))


def by_expert(off):
    return ((e, slice(int(off[e]), int(off[e + 1]))) for e in range(len(off) - 1))


def experts_up(x, off, wg, wu):
    """{"g", "u", "h"}: (exact, (terms, magnitude) or its propagated error bound)"""
    M, I, d = x.shape[0], wg.shape[1], wg.shape[2]
    g, u, mg, mu = (np.zeros((M, I)) for _ in range(4))
    for e, r in by_expert(off):
        g[r], u[r] = x[r] @ wg[e].T, x[r] @ wu[e].T
        mg[r], mu[r] = np.abs(x[r]) @ np.abs(wg[e]).T, np.abs(x[r]) @ np.abs(wu[e]).T
    return g, u, g * sigmoid(g) * u, mg, mu


def up_h_limit(g, u, h, mg, mu, d, kind):
    """h = g s(g) u from g, u off by at most eg, eu: |d silu| <= 1.1 |dg|, and
    the exponential, the division and the products within 16 steps."""
    eg, eu = (d + 8) * STEP * mg, (d + 8) * STEP * mu
    silu = np.abs(g * sigmoid(g))
    off = 1.1 * eg * (np.abs(u) + eu) + (silu + 1.1 * eg) * eu + 16 * STEP * np.abs(h)
    return ROUND[kind] * (np.abs(h) + off) + off + 2.0 ** -126


def experts_down(h, off, wd):
    y, mag = np.zeros((h.shape[0], wd.shape[2])), np.zeros((h.shape[0], wd.shape[2]))
    for e, r in by_expert(off):
        y[r], mag[r] = h[r] @ wd[e], np.abs(h[r]) @ np.abs(wd[e])
    return y, mag


def experts_dx(dg, du, off, wg, wu):
    dx, mag = np.zeros((dg.shape[0], wg.shape[2])), np.zeros((dg.shape[0], wg.shape[2]))
    for e, r in by_expert(off):
        dx[r] = dg[r] @ wg[e] + du[r] @ wu[e]
        mag[r] = np.abs(dg[r]) @ np.abs(wg[e]) + np.abs(du[r]) @ np.abs(wu[e])
    return dx, mag


def experts_dw(a, b, off, N):
    """(dW, magnitude, terms): a^T b over every expert's rows"""
    dw, mag = np.zeros((N, a.shape[1], b.shape[1])), np.zeros((N, a.shape[1], b.shape[1]))
    terms = np.zeros((N, 1, 1))
    for e, r in by_expert(off):
        dw[e], mag[e], terms[e] = a[r].T @ b[r], np.abs(a[r]).T @ np.abs(b[r]), r.stop - r.start
    return dw, mag, terms


def experts_dh(dy, g, u, off, wd):
    """dg, du and the largest error of each before rounding"""
    M, I, d = dy.shape[0], wd.shape[1], wd.shape[2]
    dh, mag = np.zeros((M, I)), np.zeros((M, I))
    for e, r in by_expert(off):
        dh[r], mag[r] = dy[r] @ wd[e].T, np.abs(dy[r]) @ np.abs(wd[e]).T
    s = sigmoid(g)
    fg, fu = u * s * (1 + g * (1 - s)), g * s
    size = np.abs(u) * s * (1 + np.abs(g) * (1 - s))  # the factor's terms in absolute value
    eh = (d + 8) * STEP * mag
    og = eh * np.abs(fg) + 16 * STEP * (np.abs(dh) + eh) * size
    ou = eh * np.abs(fu) + 16 * STEP * (np.abs(dh) + eh) * np.abs(fu)
    return dh * fg, dh * fu, og, ou


def rounded(exact, off, kind):
    return ROUND[kind] * (np.abs(exact) + off) + off + 2.0 ** -126
