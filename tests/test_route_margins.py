"""The routing tests on the GPU compare ids with the oracle's exactly.  Here their inputs are looked over without a GPU:
wherever they choose groups, groups that hold different values have scores far enough apart for double precision to order
them alike on both sides (route_util derives how far that is)."""

import itertools

import pytest

import test_gpu_route as G
from oracle import route_oracle as R
from route_util import assert_groups_apart, group_gaps

GROUPED = [G.test_groups, G.test_many_equal_keys_take_the_lowest_ids, G.test_scores_closer_than_single_precision,
           G.test_biases_of_any_size, G.test_values_that_cancel_to_zero_are_no_empty_row]


def arguments(f):
    """Every combination of a test's parametrize marks, as keyword arguments."""
    sets = []
    for m in getattr(f, "pytestmark", []):
        if m.name == "parametrize":
            names = [n.strip() for n in m.args[0].split(",")]
            sets.append([dict(zip(names, v if len(names) > 1 else (v,))) for v in m.args[1]])
    for combination in itertools.product(*sets):
        yield {k: v for part in combination for k, v in part.items()}


@pytest.mark.parametrize("test", GROUPED, ids=lambda f: f.__name__)
def test_group_scores_of_the_gpu_tests_are_apart(test, monkeypatch):
    looked = []

    def oracle_instead(sh, logits, bias, dtype, **kw):
        assert_groups_apart(sh, logits, bias)
        looked.append(sh.top_groups < sh.n_groups)
        return R.route(sh, logits, bias)
    monkeypatch.setattr(G, "gpu", oracle_instead)
    monkeypatch.setattr(G, "keys_apart", lambda *a: None)      # not what this looks at
    for kw in arguments(test):
        test(**kw)
    assert any(looked)


def test_groups_too_close_are_noticed():
    sh = R.RouteShape(4, 1, "sigmoid", 2, 1, 2)
    assert_groups_apart(sh, [[1.0, 2.0, 2.0, 1.0]], None)                        # the same values: they tie on both sides
    assert_groups_apart(sh, [[1.0, 2.0, 2.0, 1.0 + 2.0 ** -40]], None)
    assert group_gaps(sh, [1.0, 2.0, 2.0, 1.0 + 2.0 ** -40], None)[0][0] < 2.0 ** -41
    with pytest.raises(AssertionError):
        assert_groups_apart(sh, [[1.0, 2.0, 2.0, 1.0 + 2.0 ** -51]], None)
    with pytest.raises(AssertionError):      # 1/2 - 1/4 + 1/4: the same score from other values
        assert_groups_apart(sh, [[0.0, 0.0, 0.0, 0.0]], [-0.25, 0.25, 0.0, 0.0])
