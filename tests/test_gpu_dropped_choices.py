"""Choices dropped between the routing and the plan, in training."""
import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests._util import require_gpu

pytestmark = pytest.mark.gpu
U, BF16 = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def test_dropped_choices_and_their_gradients():
    """Experts over their capacity lose their last choices, in a copy: rows, sums and all gradients without them."""
    T, E, k, D, room = 300, 8, 2, 64, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn((T, E), generator=g, device="cuda").requires_grad_(True)
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16().requires_grad_(True)
    dout = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    experts, weights = mx.moe_route(logits, k, score="sigmoid", renormalize=True)
    before = experts.clone()
    one = torch.nn.functional.one_hot(experts.long().flatten(), E)
    keep = ((one.cumsum(0) * one).sum(1) <= room).view(T, k)
    assert 0 < int((~keep).sum()) < T
    plan = mx.moe_plan(torch.where(keep, experts, -1), E, 32)
    assert torch.equal(experts, before) and int(plan.counts.max()) == room
    rows = mx.moe_gather(x, plan)
    out = mx.moe_combine(rows, plan, weights)
    dx, dl = torch.autograd.grad(out, (x, logits), dout)

    x64, l64, d64 = x.detach().double(), logits.detach().double().requires_grad_(True), dout.double()
    s = torch.sigmoid(l64).gather(1, before.long())
    w = s / s.sum(1, keepdim=True)
    kept = torch.where(keep, w, 0.0).sum(1, keepdim=True)
    (want,) = torch.autograd.grad(kept * x64, l64, d64)
    kept = kept.detach()
    # weights: 24 U and a little (an exponential, sums, a quotient), k products; one rounding to bf16
    assert ((out.double() - kept * x64).abs() <= (BF16 + 40 * U) * (kept * x64).abs()).all()
    # each row's gradient w dout is rounded, then the sum is
    assert ((dx.double() - kept * d64).abs() <= (2 * BF16 + BF16 ** 2 + 40 * U) * (kept * d64).abs()).all()
    # dw = <dout, row> over D terms in fp32: D U of the terms' magnitudes at most; then w (dw - sum w dw)(1 - s), two terms, whose
    # factors each are off by 40 U at most
    mass = (d64 * x64).abs().sum(1, keepdim=True)
    assert ((dl.double() - want).abs() <= (2 * D + 160) * U * mass).all()
    assert ((dl != 0).sum(1) <= k).all() and dl.any()


def test_choices_dropped_in_place_are_noticed():
    """The gradient needs the experts that were selected: overwritten, they are refused, not used."""
    logits = torch.randn((20, 8), device="cuda").requires_grad_(True)
    experts, weights = mx.moe_route(logits, 2)
    experts[3, 1] = -1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        weights.sum().backward()
