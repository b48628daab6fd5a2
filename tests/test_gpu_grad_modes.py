"""The differentiable calls where no gradient will be asked for, and where a second derivative is."""
import pytest
import torch

from mxfp8_precision_moe_gb300 import synth
from tests._util import require_gpu

pytestmark = pytest.mark.gpu

SIZES = (17, 33)  # no multiples of 32: fine wherever W needs no gradient


@pytest.fixture(scope="module")
def mx():
    require_gpu()
    import mxfp8_precision_moe_gb300 as m

    m.load()
    return m


def offs_of(*sizes):
    return torch.tensor(sizes, device="cuda").cumsum(0).to(torch.int32)


def tensors(M, *shapes):
    return [synth.randn_bf16((M, 64), 1.0, seed=3).cuda()] + \
        [synth.randn_bf16(s, 0.1, seed=4 + i).cuda() for i, s in enumerate(shapes)]


class Recorder:
    """The library, with the names of the calls made through it."""

    def __init__(self, lib, names):
        self._lib, self._names = lib, names

    def __getattr__(self, name):
        self._names.append(name)
        return getattr(self._lib, name)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("a_needs", [False, True])
def test_mxfp4_evaluation_with_trainable_weights(mx, monkeypatch, mode, a_needs):
    """Parameters under no_grad: any group sizes, the same result as with detached weights, no copies for a backward."""
    from mxfp8_precision_moe_gb300 import mxfp4

    A, W = tensors(50, (2, 64, 64))
    offs = offs_of(*SIZES)
    want = mx.to_mxfp4_then_scaled_grouped_mm(A, W, offs)
    names, lib = [], mx.load()
    monkeypatch.setattr(mxfp4, "load", lambda: Recorder(lib, names))
    with mode():
        got = mx.to_mxfp4_then_scaled_grouped_mm(A.clone().requires_grad_(a_needs), torch.nn.Parameter(W.clone()), offs)
    assert torch.equal(got, want) and not got.requires_grad
    assert "mxfp4_grouped_mm_fwd" in names and not [n for n in names if n.endswith("_mxfp8_cols")]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("a_needs", [False, True])
def test_mxfp8_evaluation_with_trainable_weights(mx, monkeypatch, mode, a_needs):
    A, W = tensors(50, (2, 64, 64))
    offs = offs_of(*SIZES)
    want = mx.to_mxfp8_then_scaled_grouped_mm(A, W, offs)
    dirs = []
    for name in ("mxfp8_quantize_2d", "mxfp8_quantize_3d_experts"):
        f = getattr(mx, name)
        monkeypatch.setattr(mx, name, lambda x, d, *args, _f=f, **kw: (dirs.append(d), _f(x, d, *args, **kw))[1])
    with mode():
        got = mx.to_mxfp8_then_scaled_grouped_mm(A.clone().requires_grad_(a_needs), torch.nn.Parameter(W.clone()), offs)
    assert torch.equal(got, want) and not got.requires_grad
    assert dirs == [mx.ROW, mx.ROW]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_mxfp8_expert_evaluation_with_trainable_weights(mx, monkeypatch, mode):
    from mxfp8_precision_moe_gb300 import swiglu

    x, *ws = tensors(50, (2, 96, 64), (2, 96, 64), (2, 64, 96))
    offs = offs_of(*SIZES)
    want = mx.mxfp8_swiglu_expert(x, *ws, offs)
    dirs, wise = [], []
    quantize, gateup = swiglu.mxfp8_quantize_2d, swiglu.mxfp8_grouped_mm_swiglu_fwd
    monkeypatch.setattr(swiglu, "mxfp8_quantize_2d", lambda x, d, *args: (dirs.append(d), quantize(x, d, *args))[1])
    monkeypatch.setattr(swiglu, "mxfp8_grouped_mm_swiglu_fwd",
                        lambda *args, token_wise, **kw: (wise.append(token_wise), gateup(*args, token_wise=token_wise, **kw))[1])
    with mode():
        got = mx.mxfp8_swiglu_expert(x, *(torch.nn.Parameter(w.clone()) for w in ws), offs)
    assert torch.equal(got, want) and not got.requires_grad
    assert dirs == [mx.ROW] and wise == [False]


def expert(mx, x, w, offs):
    return mx.mxfp8_swiglu_expert(x, w, w, w, offs)


@pytest.mark.parametrize("call", [
    lambda mx, a, w, o: mx.to_mxfp4_then_scaled_grouped_mm(a, w, o),
    lambda mx, a, w, o: mx.to_mxfp8_then_scaled_grouped_mm(a, w, o),
    expert,
], ids=["mxfp4", "mxfp8", "expert"])
def test_a_second_derivative_is_refused(mx, call):
    """The gradients are kernels' outputs, without a graph: one that is differentiated again raises, and does not count as
    a constant.  Their values do not depend on create_graph."""
    A, W = tensors(96, (2, 64, 64))
    offs = offs_of(32, 64)
    a, w = A.requires_grad_(True), W.requires_grad_(True)
    first = torch.autograd.grad(call(mx, a, w, offs).float().sum(), (a, w))
    assert not any(g.requires_grad for g in first)
    again = torch.autograd.grad(call(mx, a, w, offs).float().sum(), (a, w), create_graph=True)
    assert all(torch.equal(g, f) for g, f in zip(again, first))
    for g in again:
        with pytest.raises(RuntimeError, match="second derivative"):
            (g.float().square().sum() + w.float().sum()).backward(retain_graph=True)
    only, = torch.autograd.grad(call(mx, a, W.detach(), offs).float().sum(), a, create_graph=True)
    assert torch.equal(only, first[0])
