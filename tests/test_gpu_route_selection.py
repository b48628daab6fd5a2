"""Selections at the edges of their definition, against exact sums of keys."""
import math

import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests import _routedef as ref
from tests._util import require_gpu

pytestmark = pytest.mark.gpu
inf, nan = math.inf, math.nan


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def select(l, k, bias=None, **kw):
    bias = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).cuda()
    return mx.moe_route(torch.as_tensor(l, dtype=torch.float32).cuda(), k, bias=bias, **kw)[0].tolist()


def check(l, k, bias, **kw):
    b = None if bias is None else bias.tolist()
    got = select(l, k, bias, **kw)
    for t, row in enumerate(l.tolist()):
        want = ref.select(row, k, bias=b, **kw)
        assert got[t] == want + [-1] * (k - len(want)), f"token {t}"


# ---------------------------------------------------------------- one bias for all, and groups with one expert left
def test_a_common_bias_counts_for_each_expert_of_a_group():
    for b, want in ((1, 0), (0, 2), (-1, 2), (0.5, 0), (0.4, 2)):
        assert select([[-1, -1, 5, -inf]], 1, [b] * 4, score="sigmoid", groups=2, top_groups=1) == [[want]], b
    assert select([[4, -inf, -0.4, -0.4]], 1, [1] * 4, score="sigmoid", groups=2, top_groups=1) == [[2]]
    for b, want in ((0, 2), (2, 2), (4, 0)):
        assert select([[-1, -1, 0.5, -inf]], 1, [b] * 4, score="softmax", groups=2, top_groups=1) == [[want]], b
    for b, want in ((0, 2), (0.5, 0)):
        assert select([[0, 0, math.log(4), -inf]], 1, [b] * 4, score="softmax_all", groups=2, top_groups=1) == [[want]], b


@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 4, 2, 2), (64, 8, 3, 8), (48, 16, 5, 4), (100, 5, 2, 7), (256, 8, 4, 8),
                                                   (1024, 32, 5, 16)])
@pytest.mark.parametrize("bias", [None, 0.0, 0.375, -0.25, 1.0, -5.0, 1e4])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_a_common_bias_with_masked_experts(score, E, groups, top_groups, k, bias, group_score):
    """Groups that masks leave none, one, two or all of their experts."""
    T, size = 16, E // groups
    l = randn((T, E), E + k)
    left = torch.randint(0, 4, (T, groups), generator=torch.Generator().manual_seed(E))  # 3: all
    place = torch.rand((T, groups, size), generator=torch.Generator().manual_seed(1)).argsort(2).argsort(2)
    l = l.masked_fill(((place >= left[..., None]) & (left[..., None] < 3)).flatten(1), -inf)
    check(l, k, None if bias is None else torch.full((E,), bias), score=score, groups=groups, top_groups=top_groups,
          group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(8, 2), (256, 8), (100, 5)])
def test_a_common_bias_that_32_bits_leave_open(score, E, groups):
    """A group with one expert left against one with two, with the bias that makes them equal to 32 bits."""
    size = E // groups
    for t in range(12):
        row = randn(E, t).fill_(-inf)
        a, c = (t % groups) * size, ((t + 1) % groups) * size + size - 2
        row[a], row[c:c + 2] = randn(1, 50 + t), randn(2, 90 + t)
        if groups > 2:
            row[((t + 2) % groups) * size] = -3.0
        s = ref.scores(row.tolist(), score)
        check(row[None], 1, torch.full((E,), s[a] - s[c] - s[c + 1]), score=score, groups=groups, top_groups=1)


# ---------------------------------------------------------------- a bias of -inf, whatever the logit
def test_a_masked_expert_is_out_whatever_its_logit():
    bias = [-inf, 0, 0, 0.1]
    for junk in (nan, inf, 5.0):
        for score in ("softmax", "sigmoid"):
            e, w = mx.moe_route(torch.tensor([[junk, 1, 2, 0]], device="cuda"), 4, score=score,
                                bias=torch.tensor(bias, device="cuda"))
            assert e.tolist() == [[2, 1, 3, -1]] and torch.isfinite(w).all() and w[0, 3] == 0
    # every score of a softmax over all is NaN then: who is left ties
    for l in ([nan, 1, 2, 0], [inf, 1, 2, 0], [0, 1, nan, 2], [0, 1, inf, 2]):
        assert select([l], 4, bias, score="softmax_all") == [[1, 2, 3, -1]]
    # a group of which only masked experts are NaN is worth what is left in it: 2 keys of -1 against -3 and -4
    l, bias = [nan, -1, -1, 0, -3, -4, -9, -9], [-inf, 0, 0, -inf, 0, 0, 0, 0.1]
    assert select([l], 3, bias, groups=2, top_groups=1) == [[1, 2, -1]]
    l = l[4:] + l[:4]
    assert select([l], 3, bias[4:] + bias[:4], groups=2, top_groups=1) == [[5, 6, -1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(12, 1, 1, 9), (64, 8, 3, 8), (100, 5, 2, 7), (256, 8, 4, 8), (256, 1, 1, 8),
                                                   (1024, 32, 5, 16)])
@pytest.mark.parametrize("most", [0.0, inf])
def test_what_masked_experts_have_for_logits_changes_nothing(score, E, groups, top_groups, k, most):
    """A quarter of the experts is masked.  most: one bias of +inf has every order told in 64 bits."""
    l, bias = randn((20, E), E), 0.1 * randn(E, 1)
    out = torch.randperm(E, generator=torch.Generator().manual_seed(2))[:E // 4]
    bias[out] = -inf
    bias[[e for e in range(E) if e not in out.tolist()][0]] += most
    kw = dict(score=score, groups=groups, top_groups=top_groups)
    l[:, out] = 0.0
    plain, bias = l.clone().cuda(), bias.cuda()
    want = mx.moe_route(plain, k, bias=bias, **kw)
    assert not torch.isin(want[0], out.cuda()).any()
    l[:, out] = torch.tensor([nan, inf, -inf, 3e38])[torch.arange(E // 4) % 4]
    for got, w in zip(mx.moe_route(l.cuda(), k, bias=bias, **kw), want):
        assert torch.equal(got, w)


# ---------------------------------------------------------------- sums below fp32's range
@pytest.mark.parametrize("E,groups", [(12, 1), (12, 4), (60, 1), (100, 5), (256, 1), (256, 8)])
def test_keys_below_fp32s_lowest_rank_as_exact_sums(E, groups):
    """Finite logits and biases, whose sums have no fp32: their experts are there to be selected."""
    low = -3e38 - torch.arange(E) * 1e33
    check(torch.stack((low, low.flip(0))), 3, low, score="softmax", groups=groups, top_groups=max(1, groups // 2))
    # two experts in fp32's range: they come first, and the places left go to the others
    l = low.clone()
    l[[E // 2, E - 1]] = torch.tensor([1.0, 2.0])
    bias = low.clone()
    bias[[E // 2, E - 1]] = torch.tensor([0.5, 0.25])
    check(l[None], 4, bias, score="softmax", groups=groups, top_groups=groups)
    check(l[None], 3, bias, score="softmax", groups=groups, top_groups=groups, group_score="max")
    # masked ones stay out
    bias[0] = -inf
    l[1] = -inf
    check(l[None], E if E <= 16 else 16, bias, score="softmax", groups=groups, top_groups=groups)
