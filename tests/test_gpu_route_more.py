"""Routing from scores on the GPU, against the float64 oracle: more tokens than a wave's share of a block's weights takes
turns over, rows that are not finite, and the router's own logits on the matrix units.  Tolerances as in
test_gpu_route."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
import synth
from gpu_util import DEV, make_layer, oracle_shape, upload
from oracle import moe_oracle as O
from oracle import route_oracle as R
from route_util import assert_groups_apart
from test_gpu_route import NINF, U, check, gpu, inputs, keys_apart

pytestmark = pytest.mark.gpu


def same(got, want, rel):
    """Weights within rel of the oracle's, NaN where it has NaN."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.all(np.abs(got - want)[ok] <= rel * np.abs(want)[ok] + 2.0 ** -149)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bias", [None, 0.1])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("E", [16, 256])
@pytest.mark.parametrize("k", [2, 20])
def test_a_softmax_over_a_nan_or_an_infinity_is_nan(E, k, groups, bias, renorm):
    """Every score of such a row is NaN by the formula, and so is every weight, chosen or not where it stands; without
    groups or a bias the order is that of the logits.  Rows beside them are as ever."""
    k = min(k, 6) if E == 16 else k
    l, b = inputs(9, E, 90 + E, "f32", masked=True)
    for t in (0, 2, 3, 5, 6, 8):        # no row of these is empty
        l[t, t] = 0.25
    l[2, E - 1] = np.nan
    l[3, 5] = np.inf
    l[5, [1, E // 2, E - 2]] = np.nan
    l[6, [3, E - 2]] = np.inf, np.nan
    l[8] = np.nan
    sh = R.RouteShape(E, k, "softmax", groups, max(1, groups // 2), 2, renorm, 1.5)
    b = None if bias is None else b
    keys_apart(sh, l, b)
    assert_groups_apart(sh, l, b)
    ids, w = gpu(sh, l, b, "f32")
    ids_ref, w_ref = R.route(sh, l, b)
    assert np.array_equal(ids, ids_ref)
    assert np.isnan(w_ref[[2, 3, 5, 6, 8]]).all() and not np.isnan(w_ref[[0, 1, 4, 7]]).any()
    same(w, w_ref, U * 26 + 2.0 ** -45)     # 17 u and the mean |d| <= 8 of the fp32 denominator at most


@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("bias", [None, 0.1])
@pytest.mark.parametrize("renorm", [True, False])
def test_a_sigmoid_of_a_nan_or_an_infinity(groups, bias, renorm):
    """A NaN is ordered like a masked expert and touches only its own weight (and the sum that it is part of); infinite
    logits have score 1."""
    l, b = inputs(8, 64, 95, "f32", masked=True)
    l[1] = NINF
    l[2, 5] = np.inf
    l[3, [7, 60]] = np.inf, np.nan
    l[4] = NINF
    l[4, [2, 3]] = np.nan, 1.0
    l[5] = np.nan
    sh = R.RouteShape(64, 6, "sigmoid", groups, max(1, groups // 2), 2, renorm, 1.5)
    b = None if bias is None else b
    keys_apart(sh, l, b)
    assert_groups_apart(sh, l, b)
    ids, w = gpu(sh, l, b, "f32")
    ids_ref, w_ref = R.route(sh, l, b)
    assert np.array_equal(ids, ids_ref)
    same(w, w_ref, U + 2.0 ** -45)


@pytest.mark.parametrize("score,E,k,G,tg,bias,renorm,dtype", [
    ("softmax", 512, 10, 1, 1, False, True, "f32"), ("softmax", 512, 10, 1, 1, False, False, "bf16"),
    ("sigmoid", 256, 16, 8, 3, True, True, "bf16"), ("softmax", 256, 16, 8, 3, True, False, "f32"),
    ("sigmoid", 100, 17, 5, 2, True, False, "f32"), ("softmax", 100, 64, 1, 1, True, True, "f32"),
    ("sigmoid", 33, 1, 3, 1, False, True, "bf16")])
def test_more_tokens_than_the_waves_of_a_block_take_turns_over(score, E, k, G, tg, bias, renorm, dtype):
    """A block's weights are one wave's work, another one every eight blocks of four tokens: 130 tokens have all four
    waves at it, and a last block that is half empty."""
    sh = R.RouteShape(E, k, score, G, tg, 2, renorm, 2.5)
    l, b = inputs(130, E, 101 + E + k, dtype, masked=True)
    b = b if bias else None
    assert_groups_apart(sh, l, b)
    check(sh, l, b, dtype)


def logit_margins(sh, logits, bound, bias):
    """Rows whose choice stays the same while every logit moves by up to its bound: gaps between groups and between the
    first k + 1 keys of those that stay, against twice what the scores can move (|d sigmoid| <= 1/4 |d logit|)."""
    size, ok = sh.n_experts // sh.n_groups, []
    for row, e in zip(logits, bound):
        s = np.array(R.scores([float(x) for x in row], sh.score))
        v, move = s + bias, e.max() / 4 + 2.0 ** -50
        total = np.sort(v.reshape(sh.n_groups, size), 1)[:, -sh.group_top:].sum(1)
        order = np.argsort(-total, kind="stable")
        apart = total[order[sh.top_groups - 1]] - total[order[sh.top_groups]] > 4 * move if sh.top_groups < sh.n_groups else True
        key = np.sort(np.concatenate([v[g * size:(g + 1) * size] for g in order[:sh.top_groups]]))[::-1][:sh.top_k + 1]
        ok.append(bool(apart and np.all(-np.diff(key) > 2 * move)))
    return np.array(ok)


@pytest.mark.parametrize("T", [16, 40, 131])
def test_router_route_on_the_matrix_units(T):
    """bf16 activations and 16 tokens or more: the logits come from the prefill's router kernel.  With the plain rule the same
    routing as router_topk, with a biased sigmoid in groups the oracle's, and the layer of that routing."""
    geo = synth.Geometry(256, 32, 4, 128, 128, 4, "bf16", "bf16")
    data = make_layer(geo, 31, 0, 4 * T, n_cand=16 * T, margin_scale=2.0)
    sh = R.RouteShape(32, 4, "sigmoid", 4, 2, 2, True, 1.25)
    bias = (np.random.default_rng(32).normal(size=32) * 0.3).astype(np.float32).astype(np.float64)
    osh = oracle_shape(geo)
    xs, rw, _ = O.load_inputs(osh, 4 * T, data.x, data.R, data.shared)
    logits = O.router_logits(xs, rw)
    bound = 2 * O.summation_bound(xs, rw, exact_products=True)
    good = np.nonzero(logit_margins(sh, logits, bound, bias))[0][:T]
    assert good.size == T
    data.x, logits, bound = np.ascontiguousarray(data.x[good]), logits[good], bound[good]
    dl = upload(data)
    ws = torch.zeros(M.workspace_bytes(dl.desc, T), dtype=torch.uint8, device=DEV)
    M.workspace_init(ws)

    def call(f):
        ids = torch.full((T + 1, 4), -7, dtype=torch.int32, device=DEV)
        w = torch.full((T + 1, 4), 7.0, device=DEV)
        f(ids[:T], w[:T])
        torch.cuda.synchronize()
        assert (ids[T] == -7).all() and (w[T] == 7.0).all()
        return ids[:T].contiguous(), w[:T].contiguous()
    ids0, w0 = call(lambda i, w: M.router_topk(dl.desc, T, dl.x, dl.R, i, w, ws))
    ids1, w1 = call(lambda i, w: M.router_route(dl.desc, M.route_desc(32, 4), T, dl.x, dl.R, None, i, w, ws))
    assert torch.equal(ids0, ids1) and torch.allclose(w0, w1, rtol=2.0 ** -20, atol=0)   # expf of rounded differences
    r = M.route_desc(32, 4, "sigmoid", 4, 2, 2, True, 1.25)
    b = torch.from_numpy(bias).float().to(DEV)
    ids, w = call(lambda i, w: M.router_route(dl.desc, r, T, dl.x, dl.R, b, i, w, ws))
    ids_ref, w_ref = R.route(sh, logits, bias)
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    # a sigmoid moves by at most the logit's error of itself, the sum of the chosen as much again
    assert np.all(np.abs(w.double().cpu().numpy() - w_ref) <= (2 * bound.max(1, keepdims=True) + U + 2.0 ** -45) * w_ref)
    y = torch.zeros(T, 256, device=DEV)
    M.experts_forward(dl.desc, T, dl.x, ids, w, dl.slots, dl.pool, dl.shared, y, ws)
    M.status_check(ws)
    out = layer_of(osh, data, T, ids_ref, w_ref)
    tol = 2e-3 * np.abs(out).max()                       # the prefill path's tolerance
    assert np.all(np.abs(y.double().cpu().numpy() - out) <= tol)


def layer_of(sh, data, T, ids, w):
    """The oracle's layer with a routing of its caller."""
    xs, _, gv = O.load_inputs(sh, T, data.x, data.R, data.shared)
    blob = np.ascontiguousarray(data.shared).view(np.uint8)[:O.blob_bytes(sh.hidden, sh.shared_inter, sh.bits, sh.sb_dtype)]
    shared = O.parse_blob(blob, sh.hidden, sh.shared_inter, sh.bits, sh.sb_dtype)
    parsed = {int(e): O.parse_blob(O.expert_blob(sh, data.pool, data.slots, int(e)), sh.hidden, sh.inter, sh.bits, sh.sb_dtype)
              for e in np.unique(ids)}
    out = np.zeros((T, sh.hidden))
    for t in range(T):
        for i, e in enumerate(ids[t]):
            out[t] += w[t, i] * O.expert_forward(*parsed[int(e)], xs[t])
        out[t] += O.sigmoid(float(gv @ xs[t])) * O.expert_forward(*shared, xs[t])
    return out
