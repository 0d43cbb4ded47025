"""Routing from scores on the GPU against the float64 oracle: ids exactly, weights to their one rounding.

Ids.  With a bias or groups the kernel compares double-precision scores, without them the logits themselves; the
tests require every pair of neighbouring oracle keys (and group scores) to be equal or 1e-11 apart, far above the
error of either side's double-precision exp and sums (a few 2^-52).

Weights.  The kernel forms them in double precision and rounds once: |err| <= u |w|, u = 2^-24, plus 2^-45 |w| for the
double-precision steps.  Only the denominator of a softmax that is not divided out again, without bias and groups, is
summed in fp32: each term e_j = exp(d_j), d_j = l_j - max l, has a relative error of at most u |d_j| (the rounded
difference) + 2 u (expf), a lane adds at most 16 of them (15 u), so its relative error is at most
u (sum e_j |d_j| / sum e_j + 17)."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
from oracle import route_oracle as R

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
NINF = float("-inf")


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).double().numpy()


def inputs(T, E, seed, dtype, masked=False, std=1.5):
    rng = np.random.default_rng(seed)
    l = (rng.normal(size=(T, E)) * std).astype(np.float32).astype(np.float64)
    if masked:
        l[rng.random((T, E)) < 0.3] = NINF
        l[rng.random(T) < 0.2] = NINF
    return bf16(l) if dtype == "bf16" else l, (rng.normal(size=E) * 0.1).astype(np.float32).astype(np.float64)


def gpu(sh, logits, bias, dtype, stride=None, stream=None):
    T, E = logits.shape
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x = torch.from_numpy(logits).to(dt).to(DEV)
    if stride:
        wide = torch.full((T, stride), float("nan"), dtype=dt, device=DEV)
        wide[:, :E] = x
        x = wide[:, :E]
    b = None if bias is None else torch.from_numpy(bias).float().to(DEV)
    ids = torch.full((T + 1, sh.top_k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, sh.top_k), 77.0, device=DEV)
    r = M.route_desc(sh.n_experts, sh.top_k, sh.score, sh.n_groups, sh.top_groups, sh.group_top, sh.renormalize, sh.scale, dtype)
    M.route(r, T, x, b, ids[:T], w[:T], stream=stream)
    torch.cuda.synchronize()
    assert (ids[T] == -7).all() and (w[T] == 77.0).all()      # the rows behind the last token
    return ids[:T].cpu().numpy(), w[:T].double().cpu().numpy()


def keys_apart(sh, logits, bias):
    for row in logits:
        s = R.scores(row, sh.score)
        v = np.array([a + (0 if bias is None else b) for a, b in zip(s, bias if bias is not None else s)])
        key = np.array(row, dtype=np.float64) if bias is None else v
        key = key[np.array(row) != NINF]
        if bias is not None:
            gap = np.diff(np.sort(key[np.isfinite(key)]))
            assert np.all((gap == 0) | (gap > 1e-11))


def check(sh, logits, bias, dtype, **kw):
    keys_apart(sh, logits, bias)
    ids, w = gpu(sh, logits, bias, dtype, **kw)
    ids_ref, w_ref = R.route(sh, logits, bias)
    assert np.array_equal(ids, ids_ref)
    rel = U + 2.0 ** -45
    if sh.score == "softmax" and not sh.renormalize and bias is None and sh.top_groups == sh.n_groups:
        with np.errstate(all="ignore"):
            d = np.where(np.isneginf(logits), 0, logits - logits.max(1, keepdims=True))
            e = np.where(np.isneginf(logits), 0, np.exp(d))
            rel = rel + U * (np.nan_to_num((e * np.abs(d)).sum(1) / e.sum(1)) + 17)[:, None]
    assert np.all(np.isfinite(w))
    assert np.all(np.abs(w - w_ref) <= rel * np.abs(w_ref) + 2.0 ** -149)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_plain(score, renorm, dtype):
    for T, E, k, seed in [(1, 1, 1, 1), (1, 5, 5, 2), (3, 64, 8, 3), (5, 65, 64, 4), (9, 512, 10, 5), (2, 1000, 33, 6), (4, 1024, 1, 7)]:
        l, _ = inputs(T, E, seed, dtype)
        check(R.RouteShape(E, k, score, renormalize=renorm, scale=2.5), l, None, dtype)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bias(score, dtype):
    for T, E, k, seed in [(1, 3, 2, 11), (7, 100, 6, 12), (4, 512, 10, 13), (3, 1024, 64, 14)]:
        l, b = inputs(T, E, seed, dtype)
        check(R.RouteShape(E, k, score), l, b, dtype)
        check(R.RouteShape(E, k, score, renormalize=False), l, b, dtype)


@pytest.mark.parametrize("E,k,G,tg,gt", [(256, 8, 8, 4, 2), (512, 10, 8, 3, 2), (64, 4, 64, 9, 2), (63, 5, 7, 2, 1), (96, 32, 3, 1, 2),
                                         (1000, 20, 5, 4, 1), (6, 2, 3, 1, 2), (8, 2, 8, 8, 1), (1024, 64, 2, 1, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, k, G, tg, gt, score):
    for bias in (True, False):
        for masked in (True, False):
            l, b = inputs(13, E, 20 + E + gt, "f32", masked)
            check(R.RouteShape(E, k, score, G, tg, gt, True, 2.5), l, b if bias else None, "f32")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_empty_rows(score):
    for E, k in [(4, 4), (70, 12), (512, 10)]:
        l, b = inputs(8, E, 31, "f32", masked=True)
        l[0] = NINF
        l[1] = NINF
        l[1, E - 1] = 0.5
        for renorm in (True, False):
            check(R.RouteShape(E, k, score, renormalize=renorm), l, None, "f32")
            check(R.RouteShape(E, k, score, renormalize=renorm), l, b, "f32")


def test_many_equal_keys_take_the_lowest_ids():
    for E in (64, 65, 512, 1024):
        for k in (1, 10, 64):
            l = np.zeros((3, E))
            l[1] = -2.0
            l[2, ::3] = 1.0
            check(R.RouteShape(E, k, "sigmoid"), l, None, "f32")
            check(R.RouteShape(E, k, "sigmoid"), l, np.zeros(E), "f32")
            if E % 2 == 0 and k <= E // 2:
                check(R.RouteShape(E, k, "softmax", 2, 1, 2), l, None, "f32")


@pytest.mark.parametrize("E,k,G,tg,gt", [(40, 10, 1, 1, 1), (64, 16, 1, 1, 1), (512, 10, 1, 1, 1), (512, 17, 8, 3, 2), (512, 10, 8, 3, 2),
                                         (1000, 8, 5, 2, 1)])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_closer_than_single_precision(E, k, G, tg, gt, spread, score):
    """Thirty neighbours of a row, in one group or spread over all, have logits one fp32 step apart, in a shuffled order:
    their scores differ by less than single precision tells apart.  Rows of padding between them."""
    rng = np.random.default_rng(71 + E + k)
    T, n, each = 11, 30, E // G
    l, b = inputs(T, E, 72, "f32")
    l = np.minimum(l, 1.5)
    for t in range(T):
        at = rng.permutation(E if spread else each)[:n] + (0 if spread else (t % G) * each)
        l[t, at] = 2.0 + rng.permutation(n) * 2.0 ** -22
    l[4] = NINF
    check(R.RouteShape(E, k, score, G, tg, gt, True, 2.0), l, np.full(E, 0.125), "f32")
    check(R.RouteShape(E, k, score, G, tg, gt, True, 2.0), l, np.zeros(E), "f32")


@pytest.mark.parametrize("size", [1e-3, 0.5, 3.0, 100.0, 1e6])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_biases_of_any_size(size, score, renorm):
    """The larger the bias, the more scores single precision loses in the sum; equal biases leave the order to the scores."""
    l, b = inputs(9, 256, 81, "f32", masked=True)
    b = np.float32(size * (1 + (np.arange(256) % 3) * 0.25)).astype(np.float64) * (1 if size < 50 else -1)
    if size == 1e6:
        l = np.where(np.isneginf(l), l, np.round(l * 4096) / 4096)   # keeps scores apart beyond a double's sum with 1e6
    check(R.RouteShape(256, 9, score, 1, 1, 1, renorm, 1.5), l, b, "f32")
    check(R.RouteShape(256, 9, score, 8, 3, 2, renorm, 1.5), l, b, "f32")


def test_values_that_cancel_to_zero_are_no_empty_row():
    l = np.full((5, 64), NINF)
    l[0, [40, 7, 63]] = 0.0          # score 1/2, value 0
    l[1, [9, 8]] = 0.0
    l[3] = 0.0
    check(R.RouteShape(64, 4, "sigmoid"), l, np.full(64, -0.5), "f32")
    check(R.RouteShape(64, 4, "sigmoid", 4, 2, 2), l, np.full(64, -0.5), "f32")


def test_zeros_of_either_sign_and_far_logits():
    l = np.array([[0.0, -0.0, 0.0, -0.0, -3e38, 3e38], [-500.0, -600.0, -700.0, -1e30, -501.0, -650.0],
                  [80.0, 90.0, -90.0, 100.0, -100.0, 20.0]])
    check(R.RouteShape(6, 6, "softmax"), l, None, "f32")
    ids, w = gpu(R.RouteShape(6, 3, "sigmoid"), l, None, "f32")
    ids_ref, w_ref = R.route(R.RouteShape(6, 3, "sigmoid"), l)
    assert np.array_equal(ids, ids_ref) and np.all(np.abs(w - w_ref) <= (U + 2.0 ** -45) * w_ref + 2.0 ** -149)


def test_nan_orders_last_and_shows_in_the_weights():
    l = np.array([[1.0, np.nan, 3.0, 2.0], [np.nan, np.nan, np.nan, 0.0], [np.nan] * 4])
    for bias in (None, np.array([0.0, 5.0, 0.0, 0.0])):
        ids, w = gpu(R.RouteShape(4, 2, "sigmoid"), l, bias, "f32")
        assert ids.tolist() == [[2, 3], [3, 0], [0, 1]]
        assert np.isfinite(w[0]).all() and np.isnan(w[1:]).all()
    ids, w = gpu(R.RouteShape(4, 2, "softmax", renormalize=False), l, None, "f32")
    assert ids.tolist() == [[2, 3], [3, 0], [0, 1]] and np.isnan(w).all()
    ids, w = gpu(R.RouteShape(4, 2, "softmax"), np.array([[1.0, np.inf, 3.0, 2.0]]), None, "f32")
    assert ids.tolist() == [[1, 2]] and np.isnan(w).all()


def test_strided_rows_and_unaligned_start():
    l, b = inputs(6, 130, 41, "bf16")
    check(R.RouteShape(130, 7, "sigmoid"), l, b, "bf16", stride=133)
    check(R.RouteShape(130, 7, "softmax"), l, None, "bf16", stride=1001)


def test_zero_tokens_and_other_stream():
    r = M.route_desc(16, 2)
    ids = torch.full((1, 2), -7, dtype=torch.int32, device=DEV)
    w = torch.full((1, 2), 7.0, device=DEV)
    M.route(r, 0, torch.zeros(0, 16, device=DEV), None, ids, w)
    torch.cuda.synchronize()
    assert (ids == -7).all() and (w == 7.0).all()
    s = torch.cuda.Stream()
    l, b = inputs(5, 64, 51, "f32")
    s.wait_stream(torch.cuda.current_stream())
    ids, w = gpu(R.RouteShape(64, 3, "sigmoid"), l, b, "f32", stream=s)
    assert np.array_equal(ids, R.route(R.RouteShape(64, 3, "sigmoid"), l, b)[0])


def test_captured_and_replayed():
    """A graph of the call, replayed with new logits between eager calls, gives the eager result every time."""
    r = M.route_desc(256, 8, "sigmoid", 8, 4, 2, scale=2.5)
    T = 33
    x = torch.zeros(T, 256, device=DEV)
    b = torch.randn(256, device=DEV) * 0.1
    out = [(torch.empty(T, 8, dtype=torch.int32, device=DEV), torch.empty(T, 8, device=DEV)) for _ in range(2)]
    M.route(r, T, x, b, *out[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.route(r, T, x, b, *out[0])
    for i in range(4):
        x.copy_(torch.randn(T, 256, device=DEV) * (1 + i))
        g.replay()
        M.route(r, T, x, b, *out[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
