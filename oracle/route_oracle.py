"""Float64 oracle of expert routing from scores: one token at a time, sorted lists, no array tricks.

    s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  v_e = s_e + b_e,  key_e = v_e with a bias, l_e without
    a group's score is the sum of its `group_top` largest v_e; the best `top_groups` groups stay
    ids = the k first experts of the groups that stay, by (-key, id);  w_i = scale s_i (/ sum s_j)

A logit of -inf masks an expert: score 0, no part in its group's score, behind every other expert.  A NaN key is
ordered like a masked expert's, and a NaN v_e has no part in a group's score."""

from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np

NINF = float("-inf")


@dataclass
class RouteShape:
    n_experts: int
    top_k: int
    score: str = "softmax"
    n_groups: int = 1
    top_groups: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0


def scores(row, kind: str) -> list[float]:
    if kind == "sigmoid":
        return [0.0 if l == NINF else (1 / (1 + math.exp(-l)) if l > -700 else math.exp(l)) if l == l else math.nan
                for l in row]
    if any(l != l or l == math.inf for l in row):   # exp(inf - inf), and with it the denominator
        return [math.nan] * len(row)
    m = max(row)
    if m == NINF:
        return [0.0] * len(row)
    e = [0.0 if l == NINF else math.exp(l - m) for l in row]
    total = math.fsum(e)
    return [x / total for x in e]


def route_row(sh: RouteShape, row, bias=None):
    """(ids, weights) of one token."""
    row = [float(l) for l in row]
    s = scores(row, sh.score)
    v = [a + (0.0 if bias is None else float(b)) for a, b in zip(s, bias if bias is not None else row)]
    key = []
    for e, l in enumerate(row):
        x = l if bias is None else v[e]
        key.append(NINF if l == NINF or x != x else x)
    size = sh.n_experts // sh.n_groups
    ranked = []
    for g in range(sh.n_groups):
        vals = sorted((v[e] for e in range(g * size, (g + 1) * size) if row[e] != NINF and v[e] == v[e] and v[e] != NINF),
                      reverse=True)[:sh.group_top]
        ranked.append((-(sum(vals) if vals else NINF), g))
    stay = {g for _, g in sorted(ranked)[:sh.top_groups]}
    order = sorted((e for e in range(sh.n_experts) if e // size in stay), key=lambda e: (-key[e], e))
    ids = order[:sh.top_k]
    w = [s[e] for e in ids]
    if sh.renormalize:
        total = math.fsum(w) if all(x == x for x in w) else math.nan
        w = [0.0 if total == 0 else x / total for x in w]
    return ids, [x * sh.scale for x in w]


def route(sh: RouteShape, logits: np.ndarray, bias=None):
    """ids int32 [T, k] and weights float64 [T, k]."""
    rows = [route_row(sh, r, bias) for r in np.asarray(logits, dtype=np.float64)]
    return (np.array([i for i, _ in rows], dtype=np.int32).reshape(-1, sh.top_k),
            np.array([w for _, w in rows], dtype=np.float64).reshape(-1, sh.top_k))
