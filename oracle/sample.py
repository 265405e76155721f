"""fp64 / exact reference of the token draw: one row, one filter after the other.

Weights are fixed-point integers, as the operator defines them; they come from
``decimal`` at 40 digits, one per distinct logit, so every cut and the draw are
exact.  ``u`` and the parameters are the fp32 values as given.
"""
from __future__ import annotations

from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np

ONE = 1 << 45


def weights(values, top, T):
    """round(2^45 * exp((x - top) / T)) for each of `values` (floats), T > 0; and how far
    the unrounded value is from the nearest tie of that rounding."""
    getcontext().prec = 40
    t = Decimal(float(T))
    out = []
    for x in values:
        y = (Decimal(float(x)) - Decimal(float(top))) / t
        out.append(0 if y < -40 else int((y.exp() * ONE).to_integral_value()))
    return out


def draw(x, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-prob) of one row of logits (fp64 array of bf16 values)."""
    x = np.asarray(x, dtype=np.float64) + 0.0
    T, top_p, min_p, u = (float(np.float32(a)) for a in (T, top_p, min_p, u))
    if np.isnan(x).any() or not np.isfinite(x.max()):
        return -1, float("nan")
    if any(np.isnan(a) for a in (T, top_p, min_p, u)) or T < 0 or np.isinf(T):
        return -1, float("nan")
    top = x.max()
    first = int(np.argmax(x))
    over = np.log1p(np.exp(np.delete(x, first) - top).sum())     # lse - top
    if T == 0:
        return first, float(-over)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if top_k > 0:
        order = order[:top_k]
    distinct, back = np.unique(x[order], return_inverse=True)
    w = np.array(weights(distinct, top, T), dtype=object)[back]
    cum = np.cumsum(w)
    if top_p < 1:
        need = Fraction(max(top_p, 0.0)) * int(cum[-1])
        n = next(i for i in range(len(cum)) if cum[i] >= need and i + 1 >= 1) + 1
        order, w, cum = order[:n], w[:n], cum[:n]
    if min_p > 0:
        keep = sum(1 for a in w if a >= Fraction(min(min_p, 1.0)) * ONE)
        order, w, cum = order[:keep], w[:keep], cum[:keep]
    total = int(cum[-1])
    if u >= 1:
        i = max(j for j in range(len(w)) if w[j] > 0)
    else:
        goal = Fraction(max(u, 0.0)) * total
        i = next(j for j in range(len(cum)) if cum[j] > goal)
    t = int(order[i])
    return t, float((x[t] - top) - over)
