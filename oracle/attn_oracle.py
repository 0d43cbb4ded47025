"""Plain, slow CPU oracle for the norms and rotation of query and key heads, the append to a paged cache, and attention over it,
in float64 from the formulas in include/attention.h.

TEST INFRASTRUCTURE, NOT PRODUCT CODE.  It shares no code with the HIP path.
"""

from __future__ import annotations

import numpy as np


def head_norm(x, w, eps, offset):
    """x / sqrt(mean x^2 + eps) * (offset + w) over the last axis."""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (offset + np.asarray(w, dtype=np.float64))


def pair_indices(R, style):
    """First and second members of the rotated pairs."""
    i = np.arange(R // 2)
    return (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)


def rotate(x, positions, inv_freq, R, style):
    """Rotation of [tokens, heads, D] by positions[token] * inv_freq[pair]."""
    y = np.array(x, dtype=np.float64, copy=True)
    a, b = pair_indices(R, style)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def place_of(table_row, t, page_size, n_pages):
    """(page, place) of token number t, or None where it has none."""
    if t < 0 or t // page_size >= len(table_row):
        return None
    page = int(table_row[t // page_size])
    return (page, t % page_size) if 0 <= page < n_pages else None


def attend(q, pages, cu, lens, table, scale, new_max, len_max, tree=None):
    """Attention of the new tokens.  q: [N, n_q, D]; pages: [n_pages, 2, n_kv, page, D].  Returns (out, mag, spread): the result,
    sum_j w_j |v_j| and, a row, the largest over the seen keys of scale sum |q k_j| (both for bounds); rows of no sequence NaN."""
    q, pages = np.asarray(q, dtype=np.float64), np.asarray(pages, dtype=np.float64)
    N, nq, D = q.shape
    nkv, page_size = pages.shape[2], pages.shape[3]
    out, mag, spread = np.full((N, nq, D), np.nan), np.zeros((N, nq, D)), np.zeros((N, nq))
    for b in range(len(lens)):
        n = int(cu[b + 1]) - int(cu[b])
        for i in range(min(n, new_max)):
            row = int(cu[b]) + i
            before = int(lens[b]) - n
            seen = []
            for t in range(min(int(lens[b]), len_max)):
                j = t - before
                if j >= 0 and not (j <= i if tree is None else j < 64 and (int(tree[row]) >> j) & 1):
                    continue
                at = place_of(table[b], t, page_size, pages.shape[0])
                if at is not None:
                    seen.append(at)
            for h in range(nq):
                if not seen:
                    out[row, h] = 0
                    continue
                k = np.stack([pages[p, 0, h // (nq // nkv), o] for p, o in seen])
                v = np.stack([pages[p, 1, h // (nq // nkv), o] for p, o in seen])
                with np.errstate(all="ignore"):
                    s = scale * (k @ q[row, h])
                    if np.all(np.isneginf(s)):
                        out[row, h] = 0
                        continue
                    e = np.exp(s - np.max(s))
                    w = e / e.sum()
                    keep = ~np.isneginf(s)
                    out[row, h] = (w[keep, None] * v[keep]).sum(0)
                    mag[row, h] = (w[keep, None] * np.abs(v[keep])).sum(0)
                    spread[row, h] = np.max(abs(scale) * (np.abs(k) @ np.abs(q[row, h])))
    return out, mag, spread
