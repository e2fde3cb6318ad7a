"""CPU oracle of the block operators (include/muon_blocks.h), in float64: the
gradient of the orthogonalisation, written as the reverse of the iteration on
X itself.  The library instead differentiates the m x m recursion, so the two
share no formula.
"""
from __future__ import annotations

import numpy as np

from .muon_oracle import EPS, normalise, orient, schedule


def orthogonalise_vjp(u, y, coeffs, steps: int, eps: float = EPS) -> np.ndarray:
    """d<orthogonalise(u), y>/du.

    X' = a X + (b A + c A A) X with A = X X^T, so with Y the cotangent of X':
    S = Y X^T + X Y^T is the cotangent of (b A + c A A) made symmetric, T =
    b S + c (S A + A S) that of A, and X has the cotangent a Y + B Y + T X.
    X_0 = u / (|u| + eps) adds its own term; |u| has no gradient at u = 0.
    """
    uw, tr = orient(np.asarray(u, dtype=np.float64))
    yw = np.asarray(y, dtype=np.float64)
    yw = yw.T if tr else yw
    xs = [normalise(uw, eps)]
    sched = schedule(coeffs, steps)
    for a, b, c in sched:
        x = xs[-1]
        g = x @ x.T
        xs.append(a * x + (b * g + c * (g @ g)) @ x)
    for (a, b, c), x in zip(reversed(sched), reversed(xs[:-1])):
        g = x @ x.T
        s = yw @ x.T
        s = s + s.T
        t = b * s + c * (s @ g + g @ s)
        yw = a * yw + (b * g + c * (g @ g)) @ yw + t @ x
    norm = np.sqrt((uw * uw).sum())
    d = yw / (norm + eps)
    if norm > 0:
        d = d - uw * ((yw * uw).sum() / ((norm + eps) ** 2 * norm))
    return d.T if tr else d
