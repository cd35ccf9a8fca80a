"""CPU pins of the fp64 distillation where the teacher's logits are not finite."""
import numpy as np
import pytest

from oracle import head_oracle as H


def _case():
    r = np.random.default_rng(7)
    idx = np.array([[0, 3, 6], [2, 4, 5], [1, 0, 2], [4, 5, 1]])
    return r.standard_normal((4, 3)), r.standard_normal((7, 3)), idx, r.standard_normal((4, 3))


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("where", [1, slice(None)], ids=["one", "all"])
@pytest.mark.filterwarnings("ignore:invalid value")
def test_a_row_without_a_distribution_is_not_a_number(value, where):
    x, W, idx, u = _case()
    good = H.head_distill(x, W, idx, u, np.ones(4))
    u[2, where] = value
    o = H.head_distill(x, W, idx, u, np.ones(4))
    assert np.isnan(o["loss"][2]) and np.isnan(o["dx"][2]).all()
    for k in ("loss", "dx"):
        np.testing.assert_array_equal(o[k][[0, 1, 3]], good[k][[0, 1, 3]])


def test_absent_and_impossible_entries_do_not_count():
    x, W, idx, u = _case()
    idx[1, 2], u[1, 2] = -1, np.nan  # absent: not read
    u[2, 0] = -np.inf                # weight 0
    o = H.head_distill(x, W, idx, u, np.ones(4))
    two = H.head_distill(x[1:2], W, idx[1:2, :2], u[1:2, :2], np.ones(1))
    assert o["loss"][1] == pytest.approx(two["loss"][0], rel=1e-12)
    two = H.head_distill(x[2:3], W, idx[2:3, 1:], u[2:3, 1:], np.ones(1))
    assert o["loss"][2] == pytest.approx(two["loss"][0], rel=1e-12)
