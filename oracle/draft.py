"""Verification of drafted tokens, in exact rational arithmetic.

Test infrastructure: only the tests use this module; the GPU path never does.

Speculative sampling's published rule: drafted token x_i stays while
u_i q_i(x_i) < p_i(x_i); at the first refusal the next token is drawn from
max(p - q, 0) (from p where all stay) by inverse distribution: the lowest v
whose running sum passes u_next times the total. q = None stands for tokens
drafted without sampling (all of q on the drafted token). Entries that are
not positive and finite count as zero; an empty rest falls back to p, an empty
p to the last entry.
"""

import math
from fractions import Fraction

import numpy as np


def _positive(v):
    return v if math.isfinite(v) and v > 0 else 0.0


def verify(p, q, drafted, length, u, u_next):
    """One sequence: p [D+1, V], q [D, V] or None, drafted [D] ints, length,
    u [D], u_next -> (tokens list of D+1, accepted)."""
    D, V = p.shape[0] - 1, p.shape[1]
    length = min(max(int(length), 0), D)
    n = 0
    while n < length:
        x = int(drafted[n])
        if not 0 <= x < V:
            break
        qx = 1.0 if q is None else float(q[n, x])
        px = float(p[n, x])
        if math.isnan(px) or math.isnan(qx):
            break
        if not (math.isinf(px) or math.isinf(qx)):
            if not Fraction(float(u[n])) * Fraction(qx) < Fraction(px):
                break
        elif not float(u[n]) * qx < px:
            break
        n += 1
    row = [float(v) for v in p[n]]
    all_ = [Fraction(_positive(v)) for v in row]
    if n == length:
        rest = all_
    elif q is None:
        rest = [Fraction(0) if v == int(drafted[n]) else a for v, a in enumerate(all_)]
    else:
        rest = []
        for a, b in zip(row, q[n]):
            b = float(b)
            d = (Fraction(a) - Fraction(b)) if math.isfinite(a) and math.isfinite(b) else None
            if d is None:                      # infinities and NaN: as float64 subtracts them
                rest.append(Fraction(_positive(float(np.float64(a) - np.float64(b)))))
            else:
                rest.append(d if d > 0 else Fraction(0))
    if not any(rest):
        rest = all_
    nxt = V - 1
    if any(rest):
        target = Fraction(float(u_next)) * sum(rest)
        run = Fraction(0)
        for v, r in enumerate(rest):
            run += r
            if run > target:
                nxt = v
                break
    return [int(t) for t in drafted[:n]] + [nxt] + [-1] * (D - n), n


def verify_batch(p, q, drafted, length, u, u_next):
    out = [verify(p[b], None if q is None else q[b], drafted[b], p.shape[1] - 1 if length is None else length[b],
                  u[b], u_next[b]) for b in range(p.shape[0])]
    return np.array([t for t, _ in out], dtype=np.int32), np.array([n for _, n in out], dtype=np.int32)
