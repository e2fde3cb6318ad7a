"""CPU oracle of the expert products and of the head's loss
(include/muon_experts.h, include/muon_head.h), in float64, row by row from the
definitions, with bounds of what rounding may do to each result.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24       # half a step of binary32, relative
TINY = 2.0 ** -126   # results below this may be taken as zero: binary32 has no more full precision there


def experts(x, w, offsets):
    """(y, reach): y[r] = W_e x[r], zero for rows of no expert; reach = sum |w| |x|, what the rounding of sums scales with."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = np.zeros((x.shape[0], w.shape[1]))
    reach = np.zeros_like(y)
    for e in range(w.shape[0]):
        r = slice(offsets[e], offsets[e + 1])
        y[r] = x[r] @ w[e].T
        reach[r] = np.abs(x[r]) @ np.abs(w[e]).T
    return y, reach


def experts_grad_w(x, gy, offsets):
    """(grad_w, reach) of <experts(x, w), gy>."""
    x, gy = np.asarray(x, np.float64), np.asarray(gy, np.float64)
    n = len(offsets) - 1
    g = np.zeros((n, gy.shape[1], x.shape[1]))
    reach = np.zeros_like(g)
    for e in range(n):
        r = slice(offsets[e], offsets[e + 1])
        g[e] = gy[r].T @ x[r]
        reach[e] = np.abs(gy[r]).T @ np.abs(x[r])
    return g, reach


def head(x, w, targets, softcap=0.0, ignore_index=-100, grad_loss=None, grad_lse=None, half_step=U):
    """loss, lse and, with grad_loss, grad_x and grad_w, as a dict, each with a bound of its error under "tol_*" before
    the result itself is rounded.

    A logit is a sum of `dim` products in binary32: off by (dim + 4) u sum |x| |w| at most (four more for operands that
    are multiplied in parts).  The soft cap has slope 1 at most and is itself evaluated to 6 u cap, and but for bfloat16
    operands with caps up to 32 also to 18 u |z|: below |l / cap| = 0.3 by a series (0.9 u for what it leaves out, 6 u for
    its roundings), above by 1 - 2 / (1 + e^(2 l / cap)), whose numerator's 4.2 u is most against 0.29 (14.4 u, and 3 u for
    the constants).  exp of an argument a is off by (|a| + 4) u, relative; sums of at most 256 terms in turn and a tree
    above them by (256 + 64) u.  The gradient with respect to a logit is rounded to the operands' type (half_step), and summed over by products again.
    """
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    rows, dim = x.shape
    vocab = w.shape[0]
    targets = np.asarray(targets)
    seen = (targets != ignore_index) & (targets >= 0) & (targets < vocab)
    out = {"loss": np.zeros(rows), "lse": np.zeros(rows), "tol_loss": np.zeros(rows), "tol_lse": np.zeros(rows)}
    bad = ~seen & (targets != ignore_index)
    out["loss"][bad] = out["lse"][bad] = np.nan
    xs, t = x[seen], targets[seen]
    l = xs @ w.T
    tol_z = (dim + 4) * U * (np.abs(xs) @ np.abs(w).T)
    z = l
    if softcap:
        z = softcap * np.tanh(l / softcap)
        tol_z = tol_z + U * (6 * softcap if half_step > U and softcap <= 32 else np.minimum(6 * softcap, 18 * np.abs(z)))
    top = z.max(1, keepdims=True) if len(xs) else z
    lse = top + np.log(np.exp(z - top).sum(1, keepdims=True))
    p = np.exp(z - lse)
    away = (p * (tol_z + (np.abs(z - top) + 4) * U)).sum(1, keepdims=True)
    tol_lse = away + (256 + 64) * U + 2 * U * np.abs(lse)
    at = np.arange(len(xs))
    out["lse"][seen], out["loss"][seen] = lse[:, 0], lse[:, 0] - z[at, t]
    out["tol_lse"][seen] = tol_lse[:, 0]
    out["tol_loss"][seen] = tol_lse[:, 0] + tol_z[at, t] + 2 * U * np.abs(z[at, t])
    if grad_loss is None:
        return out
    g = np.asarray(grad_loss, np.float64)[seen, None]
    h = np.zeros_like(g) if grad_lse is None else np.asarray(grad_lse, np.float64)[seen, None]
    d = (g + h) * p
    tol = np.abs(d) * (tol_z + tol_lse + (np.abs(z - lse) + 8) * U) + np.abs(d) * U + (np.abs(g) + np.abs(h)) * p * U
    d[at, t] -= g[:, 0]
    tol[at, t] += 2 * U * np.abs(g[:, 0])
    if softcap:
        slope = 1 - (z / softcap) ** 2
        tol = tol * slope + np.abs(d) * (2 * np.abs(z) / softcap ** 2 * tol_z + 6 * U)
        d = d * slope
    rounding = np.full(d.shape, half_step)
    if half_step > U:
        rounding[at, t] = half_step ** 2
    tol = tol + rounding * (np.abs(d) + tol) + TINY * (np.abs(g) + np.abs(h) + 2)
    out["grad_x"], out["tol_grad_x"] = np.zeros((rows, dim)), np.zeros((rows, dim))
    out["grad_x"][seen] = d @ w
    # sums over the vocabulary, then over its pieces (64 of them at most)
    out["tol_grad_x"][seen] = tol @ np.abs(w) + (vocab + 68) * U * (np.abs(d) @ np.abs(w)) + vocab * TINY
    out["grad_w"] = d.T @ xs
    out["tol_grad_w"] = tol.T @ np.abs(xs) + (len(xs) + 4) * U * (np.abs(d).T @ np.abs(xs)) + len(xs) * TINY
    return out
