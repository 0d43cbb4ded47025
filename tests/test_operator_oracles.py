"""Pins of the routing and microscaled-4-bit oracles: worked examples, closed forms and invariants; mistakes planted
in them are caught."""

import math

import numpy as np
import pytest

from oracle import mx_oracle as X
from oracle import route_oracle as R

NINF = float("-inf")


def test_route_worked_softmax():
    sh = R.RouteShape(4, 2, renormalize=False)
    ids, w = R.route_row(sh, [0.0, math.log(2), math.log(4), math.log(3)])
    assert ids == [2, 3] and np.allclose(w, [0.4, 0.3], atol=1e-15)
    ids, w = R.route_row(R.RouteShape(4, 2, scale=7.0), [0.0, math.log(2), math.log(4), math.log(3)])
    assert np.allclose(w, [4.0, 3.0], atol=1e-14)


def test_route_worked_bias_chooses_but_does_not_weigh():
    # sigmoids 1/2, 3/4, 1/4; the bias lifts the third above the others
    sh = R.RouteShape(3, 2, "sigmoid", renormalize=False)
    ids, w = R.route_row(sh, [0.0, math.log(3), -math.log(3)], [0.0, 0.0, 1.0])
    assert ids == [2, 1] and np.allclose(w, [0.25, 0.75], atol=1e-15)
    ids, w = R.route_row(R.RouteShape(3, 2, "sigmoid"), [0.0, math.log(3), -math.log(3)], [0.0, 0.0, 1.0])
    assert np.allclose(w, [0.25, 0.75], atol=1e-15)


def test_route_worked_groups():
    # groups (0,1) (2,3) (4,5) of sigmoid scores: largest single score in the first, largest pair in the second
    s = [0.9, 0.1, 0.6, 0.55, 0.5, 0.2]
    l = [math.log(p / (1 - p)) for p in s]
    assert R.route_row(R.RouteShape(6, 2, "sigmoid", 3, 1, 1), l)[0] == [0, 1]
    assert R.route_row(R.RouteShape(6, 2, "sigmoid", 3, 1, 2), l)[0] == [2, 3]
    assert R.route_row(R.RouteShape(6, 3, "sigmoid", 3, 2, 2), l)[0] == [0, 2, 3]


def test_route_ties_masks_and_empty_rows():
    sh = R.RouteShape(4, 3)
    assert R.route_row(sh, [1.0, 2.0, 2.0, 1.0])[0] == [1, 2, 0]
    ids, w = R.route_row(sh, [NINF, 2.0, NINF, NINF])
    assert ids == [1, 0, 2] and w == [1.0, 0.0, 0.0]
    ids, w = R.route_row(sh, [NINF] * 4)
    assert ids == [0, 1, 2] and w == [0.0] * 3
    # a masked expert with a large bias stays behind
    ids, _ = R.route_row(R.RouteShape(3, 2, "sigmoid"), [NINF, -5.0, -6.0], [9.0, 0.0, 0.0])
    assert ids == [1, 2]
    # a group with one expert left still counts it
    ids, _ = R.route_row(R.RouteShape(4, 1, "sigmoid", 2, 1, 2), [3.0, NINF, -9.0, -9.0])
    assert ids == [0]


def test_route_invariants():
    rng = np.random.default_rng(0)
    l = rng.normal(size=(20, 24))
    ids, w = R.route(R.RouteShape(24, 5), l)
    assert np.allclose(w.sum(1), 1)
    assert np.array_equal(ids, np.argsort(-l, axis=1, kind="stable")[:, :5])
    shifted, w2 = R.route(R.RouteShape(24, 5), l + 3.0)
    assert np.array_equal(ids, shifted) and np.allclose(w, w2)
    same, _ = R.route(R.RouteShape(24, 5, "sigmoid", 6, 6, 2), l, np.zeros(24))
    assert np.array_equal(ids, same)   # all groups stay, the sigmoid keeps the order


@pytest.mark.parametrize("y,place", [(0.0, 0), (0.25, 0), (0.26, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (2.6, 5),
                                     (3.5, 6), (5.0, 6), (5.01, 7), (7.9, 7)])
def test_mx_nearest_ties_to_even(y, place):
    assert X.nearest(y) == place


def test_mx_worked_block():
    x = np.zeros(32)
    x[:4] = [6.0, -7.9, 0.24, 5.0]            # largest 7.9: e = 0
    codes, scale = X.quantize_block(x)
    assert scale == 127 and codes[:5] == [7, 15, 0, 6, 0]
    x[1] = 8.0                                # largest 8: e = 1, the values halve
    codes, scale = X.quantize_block(x)
    assert scale == 128 and codes[:4] == [5, 6, 0, 4]
    assert X.quantize_block([0.0] * 32) == ([0] * 32, 0)
    assert X.quantize_block([math.inf] + [1.0] * 31) == ([0] * 32, 255)
    assert X.quantize_block([2.0 ** -149] * 32)[1] == 0


def test_mx_round_trip_and_padding():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 300)) * np.exp(rng.normal(size=(3, 1)) * 5)
    codes, scales = X.quantize(x)
    assert codes.shape == (3, 256) and scales.shape == (3, 16)
    assert not codes[:, 150:].any() and not scales[:, 10:].any()
    v = X.values(codes, scales, 300)
    again = X.quantize(v)
    assert np.array_equal(X.values(*again, 300), v)          # what is held is held again
    block = np.abs(x[0, :32]).max()
    assert np.abs(v[0, :32] - x[0, :32]).max() <= block / 4  # half the widest step, or 8 - 6 of the block's 4 .. 8


@pytest.mark.parametrize("mistake", ["ties up", "scale by ceil", "high half first", "no saturation", "odd even"])
def test_mx_planted_mistakes_are_caught(monkeypatch, mistake):
    if mistake == "ties up":
        monkeypatch.setattr(X, "nearest", lambda y: min(range(8), key=lambda i: (abs(min(y, 6.0) - X.LEVELS[i]), -i)))
    elif mistake == "odd even":
        monkeypatch.setattr(X, "nearest", lambda y: min(range(8), key=lambda i: (abs(min(y, 6.0) - X.LEVELS[i]), (i + 1) % 2)))
    elif mistake == "no saturation":
        monkeypatch.setattr(X, "nearest", lambda y: 0 if y > 7 else min(range(8), key=lambda i: (abs(y - X.LEVELS[i]), i % 2)))
    elif mistake == "scale by ceil":
        real = X.quantize_block
        monkeypatch.setattr(X, "quantize_block", lambda x: (real(x)[0], min(real(x)[1] + 1, 254)))
    else:
        real_v = X.values
        monkeypatch.setattr(X, "values", lambda c, s, n: real_v((c >> 4) | (c << 4), s, n))
    with pytest.raises(AssertionError):
        for y, place in [(0.25, 0), (0.75, 2), (5.0, 6), (7.9, 7)]:
            test_mx_nearest_ties_to_even(y, place)
        test_mx_worked_block()
        v = X.values(*X.quantize(np.array([[6.0, 1.0, -3.0]])), 3)
        assert v.tolist() == [[6.0, 1.0, -3.0]]


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_a_softmax_that_is_not_a_number(bad, renormalize):
    """exp(inf - inf) or exp(nan) in the denominator: every score of the row is NaN, whichever experts are chosen."""
    sh = R.RouteShape(4, 2, renormalize=renormalize)
    ids, w = R.route_row(sh, [1.0, bad, 3.0, NINF])
    assert ids == ([1, 2] if bad == math.inf else [2, 0]) and all(x != x for x in w)
    ids, w = R.route_row(sh, [NINF, NINF, 3.0, bad], [0.0] * 4)      # NaN keys: by id, none of the finite ones first
    assert ids == [0, 1] and all(x != x for x in w)
