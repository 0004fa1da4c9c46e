"""Plain 64-bit implementations of the block's norms and of packed rows, and
the error bounds that the float32 kernels are held to.

STEP = 2^-23 and ROUND are train_ref's: a float32 sum of n terms of absolute sum
S is off by at most (n + 8) STEP S whatever its order, a product or quotient by
STEP of itself.  Each function returns exact values and, before the rounding to
the output's type, the largest error; train_ref.rounded adds that rounding.
Bounds count the error of every factor once; products of two errors are below
2^-40 of the value and are covered by the constants.
"""
from __future__ import annotations

import numpy as np

from train_ref import STEP

GATES = ("none", "token", "channel", "full")


def rstd(x, eps):
    return 1.0 / np.sqrt((x * x).mean(1) + eps)


def rstd_off(d):
    """Relative error of a float32 rstd: half of the sum's, and the root, the division and eps."""
    return ((d + 8) / 2 + 8) * STEP


def norm(x, w, eps, offset):
    """n, its error, rstd, its error (w None = zeros)"""
    r = rstd(x, eps)
    f = offset + (0.0 if w is None else w)
    n = x * r[:, None] * f
    # offset + w is rounded too, relative to the larger of the two
    off = np.abs(n) * (rstd_off(x.shape[1]) + 4 * STEP) + np.abs(x * r[:, None]) * (abs(offset) + np.abs(f)) * STEP
    return n, off, r, r * rstd_off(x.shape[1])


def spread(gate, kind):
    return 1.0 if kind == "none" else gate[:, None] if kind == "token" else gate


def block(y, res, gate, kind, w_post, w_next, eps, offset, scale, post):
    """{"out", "next", "rstd_post", "rstd_next"}: (exact, error)"""
    p, off, got = y, 0.0, {}
    if post:
        p, off, r, roff = norm(y, w_post, eps, offset)
        got["rstd_post"] = r, roff
    g = scale * spread(gate, kind)
    out = res + g * p
    eo = np.abs(g) * off + 4 * STEP * (np.abs(g * p) + np.abs(res))
    got["out"] = out, eo
    n, noff, r, roff = norm(out, w_next, eps, offset)
    # the relative error of rstd from out's own: sum |out| eo over sum out^2 + d eps
    rel = (np.abs(out) * eo).sum(1) / ((out * out).sum(1) + out.shape[1] * eps)
    f = np.abs(offset + (0.0 if w_next is None else w_next))
    got["next"] = n, noff + np.abs(n) * rel[:, None] + r[:, None] * f * eo
    got["rstd_next"] = r, roff + r * rel
    return got


def block_grad(dout, dnext, y, out, gate, kind, w_post, w_next, a, b, offset, scale, post):
    """Gradients by name: (exact, error).  dout or dnext may be None (zero); a, b: rstd_post, rstd_next."""
    some = dout if dout is not None else dnext
    T, d = some.shape
    n = (d + 8) * STEP
    D0 = np.zeros((T, d)) if dout is None else dout
    got = {}
    if dnext is not None:
        wn = offset + (0.0 if w_next is None else w_next)
        wmag = abs(offset) + np.abs(wn)
        xo, g = out * b[:, None], dnext * wn
        s0 = (g * xo).sum(1)
        c = b * s0 / d
        ec = b / d * (n + 4 * STEP) * (np.abs(dnext * xo) * wmag).sum(1) + 4 * STEP * np.abs(c)
        bg = b[:, None] * g
        D = D0 + bg - xo * c[:, None]
        eD = np.abs(xo) * ec[:, None] + 6 * STEP * (np.abs(D0) + np.abs(b[:, None] * dnext * wmag) + np.abs(xo * c[:, None]))
        got["dw_next"] = (dnext * xo).sum(0), (T + 8) * STEP * np.abs(dnext * xo).sum(0)
    else:
        D, eD, xo, c, ec, bg, wmag = D0, np.zeros((T, d)), np.zeros((T, d)), np.zeros(T), np.zeros(T), np.zeros((T, d)), 1.0
    got["dresidual"] = D, eD
    if y is None:
        return got
    wp = offset + (0.0 if w_post is None else w_post) if post else 1.0
    pmag = abs(offset) + np.abs(wp) if post else 1.0
    yn = y * a[:, None] if post else y
    gt = gate if kind == "token" else np.ones(T)
    gc = gate if kind in ("channel", "full") else 1.0
    v, vm = yn * wp * gc, np.abs(yn * gc) * pmag          # without a token's gate; its terms in absolute value
    dv = (D * v).sum(1)
    edv = (n + 8 * STEP) * ((np.abs(D0) + np.abs(bg)) * vm + np.abs(xo * c[:, None]) * vm).sum(1) + ec * np.abs((xo * v).sum(1)) + \
        (n + 8 * STEP) * np.abs(c) * (np.abs(xo) * vm).sum(1)
    gate_all = gt[:, None] * gc * np.ones((T, d))
    if kind == "token":
        got["dgate"] = scale * dv, abs(scale) * (edv + 4 * STEP * np.abs(dv))
    elif kind == "full":
        got["dgate"] = scale * D * yn * wp, abs(scale) * np.abs(yn) * (np.abs(wp) * eD + 6 * STEP * np.abs(D) * pmag)
    elif kind == "channel":
        s = (D * yn).sum(0)
        es = (eD * np.abs(yn)).sum(0) + (T + 12) * STEP * np.abs(D * yn).sum(0)
        got["dgate"] = scale * wp * s, abs(scale) * (np.abs(wp) * es + 4 * STEP * pmag * np.abs(s))
    dp = scale * D * gate_all
    if post:
        m = scale * gt * dv / d
        em = abs(scale) * np.abs(gt) / d * edv + 4 * STEP * np.abs(m)
        dy = a[:, None] * (dp * wp - yn * m[:, None])
        edy = a[:, None] * (abs(scale) * np.abs(gate_all * wp) * eD + np.abs(yn) * em[:, None] +
                            8 * STEP * (np.abs(dp) * pmag + np.abs(yn * m[:, None])))
        s = (D * gate_all * yn).sum(0)
        es = (eD * np.abs(gate_all * yn)).sum(0) + (T + 12) * STEP * np.abs(D * gate_all * yn).sum(0)
        got["dw_post"] = scale * s, abs(scale) * (es + 4 * STEP * np.abs(s))
    else:
        dy, edy = dp, abs(scale) * np.abs(gate_all) * (eD + 6 * STEP * np.abs(D))
    got["dy"] = dy, edy
    return got


# ---------------------------------------------------------------- packed rows


def pack(x):
    """x [rows, cols] (float64 copies of float32 values) -> q [rows, nb, 32] in column order, E [rows, nb]:
    value by value, the least E whose steps hold every magnitude."""
    rows, cols = x.shape
    nb = (cols + 31) // 32
    b = np.zeros((rows, nb * 32))
    b[:, :cols] = x
    b = b.reshape(rows, nb, 32)
    q, E = np.zeros(b.shape, np.int64), np.zeros((rows, nb), np.int64)
    for r in range(rows):
        for j in range(nb):
            v = b[r, j]
            if not np.isfinite(v).all():
                E[r, j] = 255
                continue
            big = np.abs(v).max()
            e = 0 if big < 2.0 ** -126 else max(0, int(np.floor(np.log2(big))) + 127 - 9)
            while np.rint(big * 2.0 ** (127 - e)) > 127:
                e += 1
            E[r, j] = min(e, 248)  # a step of 2^122 would take the largest values to 2^128
            q[r, j] = np.clip(np.rint(v * 2.0 ** (127 - E[r, j])), -127, 127)
    return q, E


def unpack(q, E, cols):
    """Values of q [rows, nb, 32] in column order."""
    with np.errstate(invalid="ignore"):
        v = q * np.where(E == 255, np.nan, 2.0 ** (E - 127.0))[:, :, None]
    return v.reshape(q.shape[0], -1)[:, :cols]


def columns(kept, nb):
    """The bytes as they are kept -> [rows, nb, 32] in column order."""
    kept = np.asarray(kept).reshape(-1, nb, 32)
    c = np.arange(32)
    return kept[:, :, 4 * (c % 8) + c // 8]


def kept(q):
    """[rows, nb, 32] in column order -> bytes as they are kept [rows, 32 nb]."""
    c = np.arange(32)
    out = np.zeros(q.shape, np.int8)
    out[:, :, 4 * (c % 8) + c // 8] = q
    return out.reshape(q.shape[0], -1)
