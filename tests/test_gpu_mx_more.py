"""Products of microscaled matrices on the GPU at the sides of their rules that test_gpu_mx_product does not reach: gated
tiles of 128 rows, every way of grouping for every type of A, and blocks that are not finite on every tile."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
from mx_util import DEV, TYPES, matrix, rows, to_gpu, workspace
from test_gpu_mx_product import Experts, dev, routing, run_experts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("a", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("T", [43, 44, 172, 173])
def test_gated_experts_at_the_tiles_rule(T, a):
    """5 of 9 experts a token: 23 and 24 pairs an expert (tiles of 32 and 64 rows), 95 and 96 (64 and 128)."""
    x = Experts(np.random.default_rng(21), 9, 70, 300, "swiglu")
    run_experts(x, T, 5, a=a)
    run_experts(x, T, 5, a=a, out="bf16", pair_rows=True, combine=True)


@pytest.mark.parametrize("a", ["f32", "mx"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("T,k", [(900, 7), (2500, 9), (3100, 9)])
def test_every_way_of_grouping(T, k, act, a):
    """Pairs kept in registers two and six at a time and more than that, A of other types than bf16; some ids unusable."""
    x = Experts(np.random.default_rng(22), 40, 20, 40, act)
    ids, _ = routing(np.random.default_rng(T), T, 40, k)
    ids[::17, 0] = -1
    ids[5, :] = 40
    ws, _ = run_experts(x, T, k, a=a, ids=ids)
    with pytest.raises(M.MoeError):
        M.status_check(ws)
    run_experts(x, T, k, a=a, combine=True, pair_rows=a == "mx")     # the oracle quantises value by value


def poison_a(x, at, value, dtype):
    """The rows of x as a left operand of the given type, and the same with a value that is not finite in some places."""
    bad = x.copy()
    for r, c in at:
        bad[r, c] = value
    if dtype != "mx":
        return (to_gpu(x, dtype), None), (to_gpu(bad, dtype), None)
    out = []
    for v in (x, bad):
        (n, c), (_, s) = M.mx_shapes(*v.shape)
        codes, scales = torch.zeros(n, c, dtype=torch.uint8, device=DEV), torch.zeros(n, s, dtype=torch.uint8, device=DEV)
        M.mx_quantize(to_gpu(v, "f32"), codes, scales)
        out.append((codes, scales))
    return out


@pytest.mark.parametrize("shape", [(70, 130, 300), (100, 150, 4200), (1800, 1700, 300), (3600, 3500, 300)],
                         ids=["64 rows", "two groups of waves", "128 rows", "256 rows"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("a,value", [("bf16", np.nan), ("f32", np.inf), ("mx", -np.inf)])
def test_dense_tiles_keep_what_is_not_finite_in_its_row_and_column(shape, act, a, value):
    m, n, k = shape
    n = n // 2 if act == "swiglu" else n
    rng = np.random.default_rng(23)
    wc, ws, _ = matrix(rng, n * (2 if act == "swiglu" else 1), k)
    at = [(0, 0), (m // 2 + 1, k - 1), (m - 1, k // 2)]
    cols = [1, n - 1]
    bad_ws = ws.copy()
    bad_ws[1, 0] = 255                                         # a block of the first chunk, one of the last
    bad_ws[(n if act == "swiglu" else 0) + n - 1, -(-k // 32) - 1] = 255      # with a gate the up row
    good, bad = poison_a(rows(rng, m, k), at, value, a)
    d = M.mx_product_desc(n, k, a=a, out="f32", act=act)
    w = workspace(d, m)
    want, got = (torch.full((m, n), 3.0, device=DEV) for _ in range(2))
    M.mx_linear(d, m, *good, dev(wc), dev(ws), want, w)
    M.mx_linear(d, m, *bad, dev(wc), dev(bad_ws), got, w)
    torch.cuda.synchronize()
    hit = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    hit[[r for r, _ in at]] = True
    hit[:, cols] = True
    assert torch.isfinite(want).all()
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])


@pytest.mark.parametrize("T,k,E", [(60, 3, 16), (80, 3, 8), (100, 2, 2)], ids=["32 rows", "64 rows", "128 rows"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("a,value", [("bf16", np.nan), ("f32", np.inf), ("mx", -np.inf)])
def test_expert_tiles_keep_what_is_not_finite_in_its_row_and_column(T, k, E, act, a, value):
    """A row of A that is not finite reaches its own pairs, a block of an expert's matrix that expert's pairs in one column;
    their sums over experts are NaN, the other tokens' as without."""
    N, K = 70, 300
    x = Experts(np.random.default_rng(24), E, N, K, act)
    rng = np.random.default_rng(25)
    ids, w = routing(rng, T, E, k)
    good, bad = poison_a(rows(rng, T, K), [(T // 3, 299), (T - 1, 5)], value, a)
    d = x.desc(k, a)
    wst, it, wt = workspace(d, T), dev(ids), dev(w.astype(np.float32))
    clean = x.pool
    dirty = clean.clone()
    e, col = int(ids[0, 0]), 69
    row = col + (N if act == "swiglu" else 0)
    dirty[int(x.slots[e]) + x.scales_off + row * 16 + 9] = 255             # values 288 to 299 of that row
    hit = torch.zeros(T, k, N, dtype=torch.bool, device=DEV)
    hit[[T // 3, T - 1]] = True
    hit[:, :, col] |= dev(ids == e)
    for weights in (None, wt):
        want, got = (torch.full((T * k if weights is None else T, N), 3.0, device=DEV) for _ in range(2))
        M.mx_experts(d, T, *good, it, weights, x.slots, clean, want, wst)
        M.mx_experts(d, T, *bad, it, weights, x.slots, dirty, got, wst)
        torch.cuda.synchronize()
        here = hit.view(T * k, N) if weights is None else hit.any(1)
        assert torch.isfinite(want).all()
        assert torch.isnan(got[here]).all() and torch.equal(got[~here], want[~here])
    M.status_check(wst)
