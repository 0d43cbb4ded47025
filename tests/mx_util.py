"""Helpers of the microscaled 4-bit GPU tests: seeded matrices, the calls, and bounds on their rounding.

Bound of a product.  Every 4-bit product, scaled by powers of two, is exact in fp32; only the additions round.  In any
order the K of them leave at most g(K) sum |a w|, g(n) = n u / (1 - n u), u = 2^-24; the matrix unit's adder is not
specified as round-to-nearest, and a truncation is off by at most a whole step, so twice that, with 16 more
additions for joining parts: e = 2 g(K + 16) sum |a w|.  The output's rounding adds half a step: eps / 2 |y|.
Gated: |silu'| <= 1.1, and silu and the product are formed with an expf of at most 1 ulp (2 u), a sum, a division
and two products, each within u: |err| <= 1.1 e_g (|u| + e_u) + |silu(g)| e_u + 8 u |y|.
Weighted sum: sum |w_i| e_i, plus 2 g(k' + 32) sum |w_i| |terms| for its own additions, whose order mixes parts of
the products (hence the terms' magnitudes)."""

import numpy as np
import torch

import int4_quantized_expert_amd as M
from oracle import mx_oracle as X

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def g(n):
    return n * U / (1 - n * U)


def rows(rng, n, k, dtype="f32"):
    """Values with rows of several sizes and outliers, exactly representable in dtype."""
    x = rng.normal(size=(n, k)) * np.exp(rng.normal(size=(n, 1)))
    x[rng.random((n, k)) < 0.02] *= 30
    t = torch.from_numpy(x).float()
    return (t.to(torch.bfloat16) if dtype == "bf16" else t).double().numpy()


def to_gpu(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[dtype]).to(DEV)


def matrix(rng, n, k):
    """Random codes and scales of an MX matrix and its values."""
    kp = X.padded(k)
    codes = rng.integers(0, 256, size=(n, kp // 2), dtype=np.uint8)
    scales = rng.integers(118, 128, size=(n, kp // 32)).astype(np.uint8)
    codes[:, (k + 1) // 2:] = 0
    if k % 2:
        codes[:, k // 2] &= 15
    scales[:, -(-k // 32):] = 0
    return codes, scales, X.values(codes, scales, k)


def held(x):
    """What rows stand for once quantised (by the oracle), and their codes and scales."""
    c, s = X.quantize(x)
    return X.values(c, s, x.shape[1]), c, s


def plain_bound(y, mag, k):
    return 2 * g(k + 16) * mag


def gated_bound(a, w, k):
    n = w.shape[0] // 2
    y = a @ w.T
    e = 2 * g(k + 16) * (np.abs(a) @ np.abs(w).T)
    gate, up, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
    out = X.silu(gate) * up
    return out, 1.1 * eg * (np.abs(up) + eu) + np.abs(X.silu(gate)) * eu + 8 * U * np.abs(out)


def expected(a, w, act, k):
    """(y, bound) of a product of held values, before the output's rounding."""
    if act == "swiglu":
        return gated_bound(a, w, k)
    y, mag = X.product(a, w)
    return y, plain_bound(y, mag, k)


def close(out, y, bound, dtype, what=""):
    o = out.double().cpu().numpy()
    assert np.all(np.isfinite(o)), what
    lim = bound + HALF[dtype] * (np.abs(y) + bound) + 2.0 ** -133
    worst = np.max(np.abs(o - y) / np.maximum(lim, 1e-300))
    assert np.all(np.abs(o - y) <= lim), f"{what}: worst err/bound {worst:.3g}"


def workspace(d, T):
    ws = torch.zeros(M.mx_workspace_bytes(d, T), dtype=torch.uint8, device=DEV)
    M.workspace_init(ws)
    return ws
