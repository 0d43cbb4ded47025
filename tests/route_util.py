"""How far apart the routing oracle's group scores lie, so that comparing ids exactly means something.

Both sides form scores in double precision (u = 2^-53, half an ulp at 1).  A sigmoid: an exp of at most one ulp, a sum and a
quotient, 4 u of itself.  A softmax: an exp of a rounded difference d, (|d| + 2) u, and a quotient, together (|d| + 3) u
of itself; and a denominator, the same for all experts of the row, of up to 1024 terms in sums of 16 and 6 steps (22 u)
that are off by (mean |d| + 2) u with mean |d| <= log 1024 < 7: 31 u, which scales all scores alike.  A bias and the
sum of two values add u |v| each, and u of the sum.  Of the difference of two groups' scores a side is therefore off by
at most  sum over both of ((|d| + 4) u s + u |v|) + u |totals| + 31 u |difference of the sums of s|."""

import math

import numpy as np

from oracle import route_oracle as R

U = 2.0 ** -53


def group_gaps(sh, row, bias):
    """(gap, need) of each two different groups whose scores are next to each other in the row's order."""
    s = R.scores(row, sh.score)
    b = [0.0] * len(row) if bias is None else [float(x) for x in bias]
    v = [x + y for x, y in zip(s, b)]
    top = max((l for l in row if l == l), default=R.NINF)
    size = sh.n_experts // sh.n_groups
    groups = []
    for g in range(sh.n_groups):
        at = sorted((e for e in range(g * size, (g + 1) * size) if row[e] != R.NINF and math.isfinite(v[e])),
                    key=lambda e: -v[e])[:sh.group_top]
        if at:
            err = sum(((0.0 if sh.score == "sigmoid" else top - row[e]) + 4) * U * s[e] + U * abs(v[e]) for e in at)
            total = sum(v[e] for e in at)
            groups.append((total, err + U * abs(total), sum(s[e] for e in at), sorted((row[e], b[e]) for e in at)))
    groups.sort(key=lambda x: x[0])
    return [(q[0] - p[0], 2 * (p[1] + q[1] + 31 * U * abs(q[2] - p[2])))
            for p, q in zip(groups, groups[1:]) if p[3] != q[3]]


def assert_groups_apart(sh, logits, bias):
    """Groups that hold different values have scores that both sides order alike (those that hold the same ones tie)."""
    if sh.top_groups < sh.n_groups:
        for row in np.asarray(logits, dtype=np.float64):
            for gap, need in group_gaps(sh, [float(x) for x in row], bias):
                assert gap > need, f"group scores {gap:.3g} apart, {need:.3g} needed"
