"""Experts by scores: softmax or sigmoid, bias, groups, top-k, weights (fp64).

Test infrastructure: only the tests use this module; the GPU path never does.

A token at a time, from the definition: scores s, choice values c = s + bias
(without a bias the order of the logits themselves), a group's worth the sum
of its `top` largest values, the groups of most worth, the experts of largest
c among them. NaN ranks after every number, ties go to the lower index.
"""

import math

import numpy as np

from . import router


def _score(l, score):
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        numbers = l[~np.isnan(l)]
        m = numbers.max() if numbers.size else math.nan
        e = np.where(l == -math.inf, 0.0, np.exp(l - m))
        total = e.sum()
        return np.zeros_like(l) if total == 0 else e / total


def _before(values):
    """Indices from the first choice on: larger first, NaN last, then the lower index."""
    return sorted(range(len(values)), key=lambda i: (math.isnan(values[i]), -values[i] if values[i] == values[i] else 0, i))


def choose(l, k, score, bias, groups, keep, top, renormalize, scale):
    """One token's logits [E] (fp64) -> (ids [k], weights [k], scores [E])."""
    E = len(l)
    s = _score(l, score)
    with np.errstate(invalid="ignore"):
        c = l if bias is None else s + bias
    size = E // groups
    stay = range(groups)
    if keep < groups:
        worth = []
        for g in range(groups):
            part = (s if bias is None and top == 2 else c)[g * size:(g + 1) * size]
            best = [part[i] for i in _before(part)[:top]]
            with np.errstate(invalid="ignore"):
                worth.append(best[0] if top == 1 else best[0] + best[1])
        stay = _before(worth)[:keep]
    ids = [e for e in _before(c) if e // size in set(stay)][:k]
    w = s[ids]
    if renormalize:
        total = w.sum()
        w = np.zeros(k) if total == 0 else w / total
    return ids, w * scale, s


def route(logits, k, score="softmax", bias=None, groups=1, keep=1, top=1, renormalize=True, scale=1.0):
    """logits [T, E] -> dict as router.route's (weights fp64)."""
    lg = np.asarray(logits, dtype=np.float64)
    b = None if bias is None else np.asarray(bias, dtype=np.float64)
    rows = [choose(l, k, score, b, groups, keep, top, renormalize, scale) for l in lg]
    ids = np.array([r[0] for r in rows], dtype=np.int32).reshape(len(rows), k)
    off, sorted_pairs, pos = router.permute(ids, lg.shape[1])
    return {"topk_ids": ids, "topk_w": np.array([r[1] for r in rows]).reshape(len(rows), k), "expert_off": off,
            "sorted_pairs": sorted_pairs, "pair_pos": pos}
