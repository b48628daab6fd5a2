"""The exact reference of the selection at hand-worked values."""
import math

from tests import _routedef as ref

inf = math.inf


def test_a_group_with_one_expert_left_has_its_bias_once():
    # sigmoids 0.269, 0.269 | 0.993: with 1 each 2.54 and 1.99, with none 0.54 and 0.99, with -1 -1.46 and -0.01
    l = [-1, -1, 5, -inf]
    for b, want in ((1, 0), (0, 2), (-1, 2), (0.5, 0), (0.4, 2)):  # even at 0.993 - 0.538 = 0.455
        assert ref.select(l, 1, "sigmoid", [b] * 4, 2, 1) == [want], b
    # sigmoids 0.982 | 0.401, 0.401: with 1 each 1.98 and 2.80
    assert ref.select([4, -inf, -0.4, -0.4], 1, "sigmoid", [1] * 4, 2, 1) == [2]
    assert ref.select([4, -inf, -0.4, -0.4], 1, "sigmoid", None, 2, 1) == [0]
    # logits: -2 and 0.5, with 2 each 2 and 2.5, with 4 each 6 and 4.5
    for b, want in ((0, 2), (2, 2), (4, 0)):
        assert ref.select([-1, -1, 0.5, -inf], 1, "softmax", [b] * 4, 2, 1) == [want], b
    # softmax of 1, 1, 4 parts: 1/3 and 2/3, with 1/2 each 4/3 and 7/6
    for b, want in ((0, 2), (0.5, 0)):
        assert ref.select([0, 0, math.log(4), -inf], 1, "softmax_all", [b] * 4, 2, 1) == [want], b


def test_who_is_left():
    assert ref.select([1, 3, 2, 3], 3, "softmax") == [1, 3, 2]
    assert ref.select([-inf] * 3, 2, "sigmoid") == []
    assert ref.select([0, 0, 0, 0], 3, "sigmoid", [0, 0.1, -inf, 0.1]) == [1, 3, 0]
    assert ref.select([0, 5, 3, 3, 4, -inf], 2, "softmax", None, 3, 1) == [2, 3]
    assert ref.select([0, 5, 3, 3, 4, -inf], 2, "softmax", None, 3, 1, "max") == [1, 0]
    assert ref.select([-inf, -inf, 1, -inf], 2, "softmax", None, 2, 2) == [2]
