"""Routing from scores on the GPU, against the float64 oracle: rows that are not finite.  Tolerances as in
test_gpu_route."""

import numpy as np
import pytest

from oracle import route_oracle as R
from route_util import assert_groups_apart
from test_gpu_route import NINF, U, gpu, inputs, keys_apart

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
