"""The path around the experts without a GPU: the reference at hand-worked values, refusals of the binding and of the C
ABI before any launch, tensors of another device, every declared symbol exported."""
import ctypes
import math
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import mxfp8_precision_moe_gb300 as mx
from tests import _routeref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def plan(T=4, k=2, rows=64, E=2, multiple=32):
    return mx.MoePlan(i32(E), i32(E), i32(rows), i32(T, k), multiple)


def test_reference_selection():
    inf, nan = math.inf, math.nan
    assert ref.select([1, 3, 2, 3], 3, "softmax") == [1, 3, 2]
    assert ref.select([1, nan, -inf, 5], 4, "softmax") == [1, 3, 0]
    assert ref.select([-inf] * 3, 2, "sigmoid") == []
    assert ref.select([0, 0, 0, 0], 2, "sigmoid", bias=[0, 0.1, -inf, 0.1]) == [1, 3]
    # groups of two: worth 0 + 5, 3 + 3, 4 - inf
    assert ref.select([0, 5, 3, 3, 4, -inf], 2, "softmax", groups=3, top_groups=1) == [2, 3]
    assert ref.select([0, 5, 3, 3, 4, -inf], 2, "softmax", groups=3, top_groups=1, group_score="max") == [1, 0]
    assert ref.weights([0, math.log(3)], [1, 0], "softmax") == pytest.approx([0.75, 0.25])
    assert ref.weights([0, 0, math.log(2)], [2], "softmax_all", scale=2.0) == pytest.approx([1.0])
    assert ref.weights([-900, -901], [0, 1], "sigmoid", True) == pytest.approx([1 / (1 + math.exp(-1)), 1 / (1 + math.e)])


@pytest.mark.parametrize("score,renormalize", [("softmax", False), ("softmax_all", False), ("softmax_all", True),
                                               ("sigmoid", False), ("sigmoid", True)])
def test_reference_gradient_against_differences(score, renormalize):
    """Central differences of step h = 1e-5 are off by h^2 / 6 times a third derivative (here under 2) and 1e-16 / h."""
    l, chosen, dw = [0.3, -1.2, 2.0, 0.7, -0.4], [2, 3, 0], [0.7, -1.1, 0.4]
    got = ref.gradient(l, chosen, dw, score, renormalize, 1.5)
    h = 1e-5
    for i in range(5):
        up, down = list(l), list(l)
        up[i] += h
        down[i] -= h
        f = [sum(a * b for a, b in zip(ref.weights(v, chosen, score, renormalize, 1.5), dw)) for v in (up, down)]
        assert abs((f[0] - f[1]) / (2 * h) - got[i]) < 1e-9


def test_reference_plan():
    offs, counts, slot, place = ref.plan([[1, 0], [1, -1], [2, 1]], 4, 2)
    assert offs == [2, 6, 8, 8] and counts == [1, 3, 1, 0]
    assert slot == [1, -1, 0, 2, 5, -1, 4, -1]
    assert place.tolist() == [[2, 0], [3, -1], [6, 4]]


def test_every_declared_symbol_is_exported():
    mx.load()
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxrouting.h")).read(), flags=re.S)
    names = re.findall(r"^\w[\w\s\*]*?\b(mx\w+)\s*\(", src, flags=re.M)
    assert len(names) == 12
    raw = ctypes.CDLL(os.path.join(ROOT, "mxfp8_precision_moe_gb300", "libmxfp8moe.so"))
    assert not [n for n in names if not hasattr(raw, n)]


def test_plan_rows():
    rows = mx.load().mx_moe_plan_rows
    assert rows(0, 2, 8, 32) == 0 and rows(5, 2, 6, 1) == 10
    assert rows(1, 1, 8, 32) == 32       # one row, one group
    assert rows(5, 2, 6, 32) == 192      # at most 6 groups are short, each by 31
    assert rows(100, 2, 3, 32) == 288    # 200 + 93, down to a multiple
    assert rows(1 << 31, 1, 8, 1) == -1 and rows(1 << 30, 2, 8, 1) == -1 and rows(4, 17, 32, 1) == -1
    assert rows(4, 1, 1025, 1) == -1 and rows(4, 1, 8, 0) == -1 and rows(4, 1, 8, 1025) == -1
    size = mx.load().mx_moe_plan_workspace
    assert size(64, 4, 16) == 0 and size(32768, 8, 256) % (256 * 4) == 0 < size(32768, 8, 256) and size(4, 17, 32) == 0


ROUTE = lambda l=None, k=2, **kw: mx.moe_route(torch.zeros(4, 8) if l is None else l, k, **kw)  # noqa: E731
BACK = lambda dh=bf(64, 64), h1=(u8(64, 64), u8(64, 2)), h3=(u8(64, 64), u8(64, 2)), offs=i32(2): (  # noqa: E731
    mx.mxfp8_swiglu_bwd_quantize_mxfp8(dh, h1, h3, offs))
LAYER = lambda x=bf(4, 64), l=torch.zeros(4, 2), g=bf(2, 32, 64), u=bf(2, 32, 64), d=bf(2, 64, 32), k=1, **kw: (  # noqa: E731
    mx.mxfp8_moe_swiglu(x, l, g, u, d, k, **kw))


@pytest.mark.parametrize("call,match", [
    (lambda: ROUTE(), "CUDA"),
    (lambda: ROUTE(torch.zeros(4, 8).double()), "logits"),
    (lambda: ROUTE(torch.zeros(8)), "logits"),
    (lambda: ROUTE(torch.zeros(4, 1025)), "experts"),
    (lambda: ROUTE(torch.zeros(4, 0)), "experts"),
    (lambda: ROUTE(k=0), "top_k"),
    (lambda: ROUTE(k=9), "top_k"),
    (lambda: ROUTE(torch.zeros(4, 32), 17), "top_k"),
    (lambda: ROUTE(score="tanh"), "score"),
    (lambda: ROUTE(groups=3), "groups"),
    (lambda: ROUTE(groups=0), "groups"),
    (lambda: ROUTE(torch.zeros(4, 64), groups=64), "groups"),
    (lambda: ROUTE(groups=4, top_groups=5), "top_groups"),
    (lambda: ROUTE(k=3, groups=4, top_groups=1), "top_groups"),
    (lambda: ROUTE(groups=4, top_groups=2, group_score="sum"), "group_score"),
    (lambda: ROUTE(bias=torch.zeros(7)), "bias"),
    (lambda: ROUTE(bias=torch.zeros(8).double()), "bias"),
    (lambda: mx.moe_plan(i32(4, 2), 8), "CUDA"),
    (lambda: mx.moe_plan(torch.zeros(4, 2), 8), "experts"),
    (lambda: mx.moe_plan(i32(4), 8), "experts"),
    (lambda: mx.moe_plan(i32(4, 17), 32), "top_k"),
    (lambda: mx.moe_plan(i32(4, 0), 32), "top_k"),
    (lambda: mx.moe_plan(i32(4, 2), 0), "num_experts"),
    (lambda: mx.moe_plan(i32(4, 2), 1025), "num_experts"),
    (lambda: mx.moe_plan(i32(4, 2), 8, 0), "multiple"),
    (lambda: mx.moe_plan(i32(4, 2), 8, 1025), "multiple"),
    (lambda: mx.MoePlan(i32(2), i32(3), i32(64), i32(4, 2)), "counts"),
    (lambda: mx.MoePlan(i32(2).long(), i32(2), i32(64), i32(4, 2)), "offs"),
    (lambda: mx.MoePlan(i32(2), i32(2), i32(64).long(), i32(4, 2)), "slot"),
    (lambda: mx.MoePlan(i32(2), i32(2), i32(64), i32(4)), "place"),
    (lambda: mx.MoePlan(i32(2), i32(2), i32(64), i32(2, 4).T), "contiguous"),
    (lambda: mx.moe_gather(bf(4, 64), plan()), "CUDA"),
    (lambda: mx.moe_gather(bf(4, 64), (1, 2)), "plan"),
    (lambda: mx.moe_gather(bf(4, 64).float(), plan()), "x"),
    (lambda: mx.moe_gather(bf(5, 64), plan()), "tokens"),
    (lambda: mx.moe_gather(bf(4, 60), plan()), "multiple of 8"),
    (lambda: mx.moe_gather(bf(4, 0), plan()), "multiple of 8"),
    (lambda: mx.moe_combine(bf(64, 64), plan()), "CUDA"),
    (lambda: mx.moe_combine(bf(63, 64), plan()), "rows"),
    (lambda: mx.moe_combine(bf(64, 64), plan(), torch.zeros(4, 1)), "weights"),
    (lambda: mx.moe_combine(bf(64, 64), plan(), torch.zeros(4, 2).bfloat16()), "weights"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 64), plan()), "CUDA"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 40), plan()), "multiple of 32"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 64), plan(), 4), "dirs"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 64), plan(), 0), "dirs"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 64), plan(multiple=16), mx.COL), "COL"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 64), plan(rows=40), mx.COL), "COL"),
    (lambda: mx.mxfp8_gather_quantize(bf(4, 64), plan(), weights=torch.zeros(8)), "weights"),
    (lambda: mx.mxfp4_gather_quantize(bf(4, 64), plan()), "CUDA"),
    (lambda: mx.mxfp4_gather_quantize(bf(3, 64), plan()), "tokens"),
    (lambda: mx.mxfp4_gather_quantize(bf(4, 48), plan()), "multiple of 32"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 64), u8(512)), "CUDA"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 64), u8(511)), "s:"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 64), u8(1535), offs=i32(2)), "s:"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 64), u8(127), scale_layout=mx.SCALES_COMPACT), "s:"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 48), u8(512)), "multiples of 32"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 48), u8(512), mx.COL), "multiples of 32"),
    (lambda: mx.mxfp8_dequantize_2d(u8(64, 64), u8(512), mx.ROW | mx.COL), "direction"),
    (lambda: mx.mxfp8_dequantize_2d(bf(64, 64), u8(512)), "q:"),
    (lambda: BACK(), "CUDA"),
    (lambda: BACK(dh=bf(64, 48)), "multiples of 32"),
    (lambda: BACK(dh=bf(48, 64)), "multiples of 32"),
    (lambda: BACK(dh=bf(64, 64).float()), "dh"),
    (lambda: BACK(h1=u8(64, 64)), "h1"),
    (lambda: BACK(h1=(u8(64, 32), u8(64, 2))), "h1 codes"),
    (lambda: BACK(h3=(u8(64, 64), u8(127))), "h3 scales"),
    (lambda: BACK(offs=i32(2).long()), "offs"),
    (lambda: LAYER(), "CUDA"),
    (lambda: LAYER(l=torch.zeros(4, 3)), "router_logits"),
    (lambda: LAYER(x=bf(4, 32)), "shapes"),
    (lambda: LAYER(d=bf(2, 32, 64)), "shapes"),
    (lambda: LAYER(g=bf(2, 40, 64), u=bf(2, 40, 64), d=bf(2, 64, 40)), "multiples of 32"),
    (lambda: LAYER(x=torch.zeros(4, 64)), "x"),
    (lambda: LAYER(k=3), "top_k"),
    (lambda: LAYER(w_mxfp8=(1,)), "CUDA|w_mxfp8"),
    (lambda: LAYER(w_mxfp8=(1,), weight_cache=2), "not both"),
])
def test_refusals_of_the_binding(call, match):
    with pytest.raises(ValueError, match=match):
        call()


@pytest.mark.parametrize("kw,match", [
    (dict(groups=3), "groups"), (dict(groups=2, top_groups=3), "top_groups"), (dict(groups=2, group_score="sum"), "group_score"),
    (dict(bias=torch.zeros(3)), "bias"), (dict(bias=torch.zeros(2).double()), "bias"), (dict(bias=torch.zeros(2)), "CUDA"),
    (dict(renormalize=True, score="tanh"), "score"), (dict(top_groups=0), "top_groups"), (dict(scale=2.0), "CUDA")])
def test_refusals_of_the_few_token_layers_routing(kw, match):
    w = (u8(2, 64, 128), u8(2, 512)), (u8(2, 64, 128), u8(2, 512)), (u8(2, 128, 64), u8(2, 512))
    with pytest.raises(ValueError, match=match):
        mx.MxMoeTokens(*w, 1, **kw)


def fake(shape, dtype, index):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=f"cuda:{index}")


def fplan(index):
    f = lambda *s: fake(s, torch.int32, index)  # noqa: E731
    return mx.MoePlan(f(2), f(2), f(64), f(4, 2), 32)


DEVICE_CALLS = {
    "moe_route": lambda i, j: mx.moe_route(fake((4, 8), torch.float32, i), 2, bias=fake((8,), torch.float32, j)),
    "moe_gather": lambda i, j: mx.moe_gather(fake((4, 64), torch.bfloat16, i), fplan(j)),
    "moe_combine": lambda i, j: mx.moe_combine(fake((64, 64), torch.bfloat16, i), fplan(j)),
    "moe_combine weights": lambda i, j: mx.moe_combine(fake((64, 64), torch.bfloat16, i), fplan(i),
                                                       fake((4, 2), torch.float32, j)),
    "mxfp8_gather_quantize": lambda i, j: mx.mxfp8_gather_quantize(fake((4, 64), torch.bfloat16, i), fplan(j)),
    "mxfp8_gather_quantize weights": lambda i, j: mx.mxfp8_gather_quantize(
        fake((4, 64), torch.bfloat16, i), fplan(i), weights=fake((4, 2), torch.float32, j)),
    "mxfp4_gather_quantize": lambda i, j: mx.mxfp4_gather_quantize(fake((4, 64), torch.bfloat16, i), fplan(j)),
    "mxfp8_dequantize_2d": lambda i, j: mx.mxfp8_dequantize_2d(fake((64, 64), torch.uint8, i), fake((512,), torch.uint8, j)),
    "mxfp8_swiglu_bwd_quantize_mxfp8": lambda i, j: mx.mxfp8_swiglu_bwd_quantize_mxfp8(
        fake((64, 64), torch.bfloat16, i), (fake((64, 64), torch.uint8, i), fake((64, 2), torch.uint8, i)),
        (fake((64, 64), torch.uint8, i), fake((64, 2), torch.uint8, j)), fake((2,), torch.int32, i)),
    "mxfp8_moe_swiglu": lambda i, j: mx.mxfp8_moe_swiglu(
        fake((4, 64), torch.bfloat16, i), fake((4, 2), torch.float32, i), fake((2, 32, 64), torch.bfloat16, i),
        fake((2, 32, 64), torch.bfloat16, j), fake((2, 64, 32), torch.bfloat16, i), 1),
}


@pytest.mark.parametrize("name", DEVICE_CALLS)
@pytest.mark.parametrize("i,j", [(0, 1), (1, 0), (1, 1)])
def test_another_device_is_refused(name, i, j, monkeypatch):
    from mxfp8_precision_moe_gb300 import routing

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

    def launch(*args):
        raise AssertionError("a launch was prepared")

    monkeypatch.setattr(routing, "_raw_stream", launch)
    with pytest.raises(ValueError, match="cuda:1"):
        DEVICE_CALLS[name](i, j)


def test_plan_on_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1"):
        mx.moe_plan(fake((4, 2), torch.int32, 1), 8)
    with pytest.raises(ValueError, match="one device"):
        mx.MoePlan(fake((2,), torch.int32, 0), fake((2,), torch.int32, 0), fake((64,), torch.int32, 1),
                   fake((4, 2), torch.int32, 0))


def test_refusals_of_the_c_abi():
    L = mx.load()
    P = ctypes.c_void_p
    a = P(1 << 20)          # never dereferenced: validation fails first
    odd, half = P((1 << 20) + 8), P((1 << 20) + 2)
    ok = dict(l=a, type=0, T=4, E=8, k=2, score=0, bias=None, groups=1, top=1, gs=0, renorm=0, scale=1.0, e=a, w=a, dense=None,
              st=None)
    call = lambda **kw: L.mx_moe_route(*{**ok, **kw}.values())  # noqa: E731
    assert call(T=-1) == 2 and call(E=0) == 2 and call(E=1025) == 2 and call(k=0) == 2 and call(k=9) == 2
    assert call(E=64, k=17) == 2 and call(T=1 << 31) == 2 and call(groups=3) == 2 and call(groups=0) == 2
    assert call(E=64, groups=64, top=64) == 2 and call(groups=2, top=3) == 2 and call(groups=2, top=0) == 2
    assert call(k=5, groups=2, top=1) == 2
    assert call(type=3) == 4 and call(score=3) == 4 and call(score=-1) == 4 and call(gs=2) == 4
    assert call(l=None) == 1 and call(e=None) == 1 and call(w=None) == 1 and call(e=None, w=None) == 1
    assert call(e=None, dense=a) == 1 and call(dense=half) == 3
    assert call(l=half) == 3 and call(w=half) == 3 and call(bias=half) == 3
    assert call(T=0, l=None, e=None, w=None) == 0
    ok = dict(l=a, type=0, T=4, E=8, k=2, score=0, renorm=0, scale=1.0, e=a, dw=a, dl=a, st=None)
    call = lambda **kw: L.mx_moe_route_bwd(*{**ok, **kw}.values())  # noqa: E731
    assert call(E=1025) == 2 and call(k=9) == 2 and call(type=-1) == 4 and call(score=4) == 4
    assert call(dl=None) == 1 and call(dw=None) == 1 and call(dl=half) == 3 and call(T=0, dl=None) == 0
    ok = dict(e=a, ib=4, T=4, k=2, E=8, m=1, rows=8, offs=a, counts=a, slot=a, place=a, ws=None, n=0, st=None)
    call = lambda **kw: L.mx_moe_plan(*{**ok, **kw}.values())  # noqa: E731
    assert call(T=-1) == 2 and call(k=17) == 2 and call(E=1025) == 2 and call(m=0) == 2 and call(rows=7) == 2
    assert call(rows=1 << 31) == 2 and call(ib=2) == 4 and call(e=None) == 1 and call(offs=None) == 1
    assert call(slot=None) == 1 and call(place=None) == 1 and call(T=32768, rows=65536) == 1
    assert call(T=32768, rows=65536, ws=a, n=16 * 8 * 4 - 1) == 2
    assert call(place=half) == 3 and call(ib=8, e=P((1 << 20) + 4)) == 3
    g = lambda x=a, slot=a, place=a, rows=8, T=4, k=2, D=64, out=a: L.mx_moe_gather(x, slot, place, rows, T, k, D, out, None)  # noqa: E731
    assert g(rows=-1) == 2 and g(rows=1 << 31) == 2 and g(k=0) == 2 and g(k=17) == 2 and g(D=0) == 2 and g(D=60) == 3
    assert g(x=None) == 1 and g(slot=None) == 1 and g(place=None) == 1 and g(out=None) == 1 and g(x=odd) == 3
    assert g(slot=half) == 3 and g(rows=0, out=None) == 0
    c = lambda y=a, place=a, w=None, rows=8, T=4, k=2, D=64, out=a: L.mx_moe_combine(y, place, w, rows, T, k, D, out, None)  # noqa: E731
    assert c(T=-1) == 2 and c(T=1 << 31) == 2 and c(D=60) == 3 and c(y=None) == 1 and c(out=odd) == 3 and c(w=half) == 3
    assert c(T=0, out=None) == 0
    b = lambda dout=a, y=a, slot=a, place=a, w=a, rows=8, T=4, k=2, D=64, dy=a, dw=a: (  # noqa: E731
        L.mx_moe_combine_bwd(dout, y, slot, place, w, rows, T, k, D, dy, dw, None))
    assert b(D=4) == 3 and b(k=17) == 2 and b(dout=None) == 1 and b(y=None) == 1 and b(slot=None) == 1 and b(dy=odd) == 3
    assert b(dw=half) == 3 and b(dy=None, dw=None) == 0 and b(T=0, rows=0) == 0
    q = lambda x=a, slot=a, place=a, w=None, rows=64, T=4, k=2, D=64, dirs=3, offs=a, G=2, qr=a, sr=a, qc=a, sc=a: (  # noqa: E731
        L.mxfp8_gather_quantize(x, slot, place, w, rows, T, k, D, dirs, offs, G, qr, sr, qc, sc, None, None))
    assert q(rows=-1) == 2 and q(D=0) == 2 and q(G=0) == 2 and q(G=1025) == 2 and q(T=1 << 31) == 2 and q(dirs=0) == 4
    assert q(dirs=4) == 4 and q(dirs=5) == 4 and q(D=48) == 3 and q(rows=40) == 3 and q(x=None) == 1 and q(offs=None) == 1
    assert q(place=None) == 1 and q(place=half) == 3 and q(qc=None) == 1 and q(sr=odd) == 3 and q(w=half) == 3 and q(rows=0, qr=None) == 0
    f = lambda x=a, slot=a, place=a, rows=64, T=4, k=2, D=64, offs=a, G=2, q=a, s=a: (  # noqa: E731
        L.mxfp4_gather_quantize(x, slot, place, rows, T, k, D, offs, G, q, s, None))
    assert f(T=-1) == 2 and f(k=17) == 2 and f(slot=None) == 1 and f(offs=None) == 1 and f(D=48) == 3 and f(G=0) == 2
    assert f(place=None) == 1 and f(q=None) == 1 and f(x=odd) == 3 and f(slot=half) == 3 and f(rows=0, q=None) == 0
    assert q(rows=2 ** 31 - 128) == f(rows=2 ** 31 - 128) == 2  # whose padded rows pass 32 bits
    o = [a] * 8
    w = lambda dh=a, h1=a, s1=a, h3=a, s3=a, M=64, H=64, offs=a, G=2, outs=o: (  # noqa: E731
        L.mxfp8_swiglu_bwd_quantize_mxfp8(dh, h1, s1, h3, s3, M, H, offs, G, *outs, None, None))
    assert w(dh=None) == 1 and w(s1=None) == 1 and w(s3=None) == 1 and w(offs=None) == 1 and w(outs=o[:7] + [None]) == 1
    assert w(M=-1) == 2 and w(H=0) == 2 and w(G=0) == 2 and w(M=40) == 3 and w(H=48) == 3 and w(h1=odd) == 3 and w(s3=odd) == 3
    assert w(outs=o[:7] + [odd]) == 3
    d = lambda q=a, s=a, M=64, K=64, dir=1, layout=1, offs=None, G=0, out=a: (  # noqa: E731
        L.mxfp8_dequantize(q, s, M, K, dir, layout, offs, G, out, None))
    assert d(M=-1) == 2 and d(K=0) == 2 and d(offs=a) == 2 and d(dir=3) == 4 and d(layout=2) == 4 and d(K=48) == 3
    assert d(M=2 ** 31 - 128, offs=a, G=2) == 2
    assert d(M=40, dir=2) == 3 and d(out=None) == 1 and d(q=odd) == 3 and d(M=0, q=None) == 0
