"""Routing and the plan against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests import _routeref as ref
from tests._util import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def logits_of(T, E, dtype, seed, std=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((T, E), generator=g, device="cuda") * std).to(dtype)


def spread(row, chosen):
    """The largest difference of logits that an exponential was taken of, -inf apart."""
    live = [x for x in row if x != -math.inf]
    return max(live) - min(live) if live else 0.0


def check(logits, k, dw=None, bias=None, experts=None, **kw):
    """The call against the reference, token by token.

    Weights: every exponential's argument is a rounded difference (at most d U of it), expf is good to 2 ulp (4 U), and so
    are numerator and denominator each; a sum of n terms in any order rounds at most n - 1 times, but as a tree of 5 + E / 32
    levels here; the quotient and the scale round once each: (2 d + 24 + E / 32) U in all, plus what fp32's subnormals lose.
    Gradients: w (d - sum w d)(1 - s), whose terms each carry the weights' error and at most 8 roundings more; against the
    sum of the terms' magnitudes, as they cancel; then one rounding to the logits' type."""
    need = dw is not None
    l = logits.detach().requires_grad_(need)
    e, w = mx.moe_route(l, k, bias=bias, **kw)
    T, E = logits.shape
    assert e.shape == w.shape == (T, k) and e.dtype == torch.int32 and w.dtype == torch.float32
    rows = logits.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    sel = {x: kw[x] for x in ("groups", "top_groups", "group_score") if x in kw}
    wkw = {x: kw[x] for x in ("renormalize", "scale") if x in kw}
    score = kw.get("score", "softmax")
    scale = kw.get("scale", 1.0)
    ec, wc = e.cpu().numpy(), w.detach().double().cpu().numpy()
    grad = torch.autograd.grad(w, l, dw)[0].double().cpu().numpy() if need else None
    for t in range(T):
        chosen = ref.select(rows[t], k, score, b, **sel)
        assert ec[t].tolist() == chosen + [-1] * (k - len(chosen)), f"token {t}"
        want = np.array(ref.weights(rows[t], chosen, score, **wkw) + [0.0] * (k - len(chosen)))
        tol = (2 * spread(rows[t], chosen) + 24 + E / 32) * U
        assert np.array_equal(np.isnan(want), np.isnan(wc[t])), f"token {t}"
        if np.isnan(want).any():
            continue
        assert (np.abs(wc[t] - want) <= tol * np.abs(want) + 2.0 ** -126 * abs(scale)).all(), f"token {t}: {wc[t]} {want}"
        if need:
            d = dw[t].double().cpu().numpy()
            gw = ref.gradient(rows[t], chosen, d, score, **wkw)
            p = np.abs(want[:len(chosen)] / scale)
            mass = float((p * np.abs(d[:len(chosen)] * scale)).sum())
            each = np.full(E, 0.0)
            if score == "softmax_all" and not kw.get("renormalize"):
                live = [i for i in range(E) if rows[t][i] != -math.inf]
                for i, v in zip(live, ref.weights(rows[t], live, score)):
                    each[i] = v * mass
            for j, x in enumerate(chosen):
                each[x] += p[j] * (abs(d[j] * scale) + mass)
            err = np.abs(grad[t] - gw)
            assert (err <= (tol + 16 * U) * each * 2 + HALF_STEP[logits.dtype] * np.abs(gw) + 2.0 ** -25).all(), f"token {t}"


KINDS = [dict(score="softmax"), dict(score="softmax_all"), dict(score="softmax_all", renormalize=True),
         dict(score="sigmoid"), dict(score="sigmoid", renormalize=True, scale=2.5), dict(score="softmax", scale=0.5)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, torch.float32), (3, 2, 2, torch.bfloat16), (5, 6, 2, torch.float32), (33, 13, 4, torch.float16),
    (17, 32, 16, torch.float32), (9, 33, 3, torch.bfloat16), (12, 64, 8, torch.float16), (7, 100, 8, torch.float32),
    (6, 160, 6, torch.bfloat16), (5, 256, 8, torch.float32), (4, 257, 1, torch.float32), (3, 513, 16, torch.bfloat16),
    (3, 1024, 16, torch.float32)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route(kw, T, E, k, dtype, with_bias):
    g = torch.Generator(device="cuda").manual_seed(7)
    dw = torch.randn((T, k), generator=g, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1 if with_bias else None
    check(logits_of(T, E, dtype, T + E), k, dw, bias, **kw)


@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [
    (4, 4, 2, 2), (6, 2, 1, 3), (16, 16, 3, 3), (64, 8, 3, 6), (100, 5, 2, 7), (160, 8, 3, 6), (256, 8, 4, 8),
    (256, 32, 1, 8), (1024, 32, 5, 16), (96, 3, 3, 4)])
@pytest.mark.parametrize("with_bias,group_score", [(False, "top2"), (True, "top2"), (False, "max"), (True, "max")])
def test_route_in_groups(score, E, groups, top_groups, k, with_bias, group_score):
    bias = logits_of(1, E, torch.float32, 3, 0.1)[0].contiguous() if with_bias else None
    check(logits_of(9, E, torch.float32, E + k), k, None, bias, score=score, groups=groups, top_groups=top_groups,
          group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
def test_equal_logits_go_to_the_lowest_index(score):
    l = torch.zeros(3, 70, device="cuda")
    l[1, ::2] = 1.0
    l[2, 60:] = -0.0
    e, _ = mx.moe_route(l, 4, score=score)
    assert e.tolist() == [[0, 1, 2, 3], [0, 2, 4, 6], [0, 1, 2, 3]]
    e, _ = mx.moe_route(l, 4, score=score, bias=torch.zeros(70, device="cuda"), groups=7, top_groups=2)
    assert e.tolist() == [[0, 1, 2, 3], [0, 2, 4, 6], [0, 1, 2, 3]]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_and_special_logits(kw, groups):
    """-inf is never selected, rows that it leaves (nearly) empty, NaN first, infinities, the type's lowest value."""
    inf, nan, low = math.inf, math.nan, torch.finfo(torch.float32).min
    l = torch.tensor([
        [-inf] * 8, [-inf] * 7 + [2.0], [-inf, 1.0, -inf, 0.5, -inf, -inf, -inf, -inf], [low] * 8, [low] * 7 + [0.0],
        [1.0, nan, 2.0, -inf, 0.0, 0.0, 0.0, 0.0], [nan] * 8, [0.0, inf, 1.0, 2.0, -1.0, -inf, 0.0, 0.0],
        [-200.0, -201.0, -202.0, -300.0, -201.5, -250.0, -240.0, -230.0],
        [90.0, 100.0, 95.0, 20.0, 50.0, 60.0, -90.0, -100.0]], device="cuda")
    top = {} if groups == 1 else dict(groups=groups, top_groups=3)
    finite = torch.isfinite(l).all(1) | (l == -inf).any(1) & ~(l == inf).any(1) & ~l.isnan().any(1)
    dw = torch.linspace(-1, 1, 30, device="cuda").view(10, 3)
    check(l[finite], 3, dw[finite], **kw, **top)
    check(l[~finite & ~(l == inf).any(1)], 3, **kw, **top)
    # an infinite logit (of softmax over all every score is NaN then, and so is every group's sum): no finite weight can be
    # told for it but of a sigmoid
    e, w = mx.moe_route(l[7:8], 3, **kw, **top)
    assert e[0].tolist() == ref.select(l[7].tolist(), 3, kw["score"], groups=groups, top_groups=3)
    assert kw["score"] == "sigmoid" or w[0].isnan().any()


def test_a_bias_of_minus_infinity_masks_an_expert():
    l = logits_of(20, 12, torch.float32, 1)
    bias = torch.zeros(12, device="cuda")
    bias[[0, 3, 11]] = -math.inf
    bias[5] = math.inf
    for score in ("softmax", "softmax_all", "sigmoid"):
        e, _ = mx.moe_route(l, 9, score=score, bias=bias)
        assert (e[:, 0] == 5).all() and not torch.isin(e, torch.tensor([0, 3, 11], device="cuda")).any()
        e, w = mx.moe_route(l, 10, score=score, bias=bias)
        assert (e[:, 9] == -1).all() and (w[:, 9] == 0).all() and (e[:, :9] >= 0).all()


@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 8, 3, 8), (100, 5, 2, 7), (256, 8, 4, 8), (48, 16, 5, 4)])
@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
@pytest.mark.parametrize("bias", [None, 0.0, 0.375])
def test_coarse_logits_tie(E, groups, top_groups, k, score, bias):
    """Logits of few values, as bf16 gives them: experts tie, and groups with the same two best; scores too, which only the
    logits tell apart (a sigmoid of 40 and more is 1 in any precision)."""
    b = None if bias is None else torch.full((E,), bias, device="cuda")
    for seed, l in enumerate((logits_of(40, E, torch.bfloat16, 5, 2.0), logits_of(40, E, torch.float32, 6, 1.0).mul(2).round(),
                              logits_of(40, E, torch.float32, 7, 1.0).round() + 40.0,
                              logits_of(40, E, torch.float32, 8, 1.0).mul(4).round().div(4) - 30.0)):
        check(l, k, bias=b, score=score, groups=groups, top_groups=top_groups)
        check(l, k, bias=b, score=score)


@pytest.mark.parametrize("E", [12, 60, 100, 256, 1024])
@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_many_infinite_keys(E, score, groups):
    """Infinite biases, of few experts and of nearly all, and sums past fp32's largest: they tie or rank as exact sums do."""
    l = logits_of(6, E, torch.float32, E)
    for n in (1, 3, E // 2, E - 1, E):
        bias = torch.zeros(E, device="cuda")
        bias[torch.randperm(E, generator=torch.Generator().manual_seed(n))[:n].cuda()] = math.inf
        check(l, 3, bias=bias, score=score, groups=groups, top_groups=groups)
        check(l, 2, bias=bias, score=score, groups=groups, top_groups=1)
    huge = torch.full((E,), 3e38, device="cuda") + torch.arange(E, device="cuda") * 1e33
    e, _ = mx.moe_route(huge[None] * torch.ones(2, 1, device="cuda"), 3, score=score, bias=huge)
    if score == "softmax":
        assert e.tolist() == [[E - 1, E - 2, E - 3]] * 2


@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
def test_order_that_32_bits_leave_open(score):
    """Pairs of experts whose keys are made equal to 32 bits: their order is that of the exact sums."""
    E = 64
    l = logits_of(40, E, torch.float32, 11, 1.0)
    for t in range(40):
        row = l[t].double()
        s = {"softmax": row, "softmax_all": torch.softmax(row, 0), "sigmoid": torch.sigmoid(row)}[score]
        bias = torch.zeros(E, device="cuda", dtype=torch.float64)
        bias[0::2] = logits_of(1, E // 2, torch.float32, t, 0.2)[0].double()
        bias[1::2] = s[0::2] + bias[0::2] - s[1::2]
        bias = bias.float()
        check(l[t:t + 1], 16, bias=bias, score=score)
        check(l[t:t + 1], 8, bias=bias, score=score, groups=32, top_groups=5)
        check(l[t:t + 1], 8, bias=bias, score=score, groups=16, top_groups=5, group_score="max")


def test_route_repeats_and_takes_any_layout():
    l = logits_of(300, 64, torch.float32, 5)
    wide = torch.zeros(300, 67, device="cuda")
    wide[:, 3:] = l
    a, b = mx.moe_route(l, 6, score="sigmoid"), mx.moe_route(wide[:, 3:], 6, score="sigmoid")
    c = mx.moe_route(l.T.contiguous().T, 6, score="sigmoid")
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])
    # rows that start off a vector's boundary
    odd = torch.zeros(300 * 64 + 1, device="cuda")
    odd[1:] = l.flatten()
    d = mx.moe_route(odd[1:].view(300, 64), 6, score="sigmoid")
    assert torch.equal(a[0], d[0]) and torch.equal(a[1], d[1])


def test_route_many_tokens_against_counted_ranks():
    """A training batch over 256 experts in 8 groups, the ranking by counting in 64 bits."""
    T, E, k = 3000, 256, 8
    l = logits_of(T, E, torch.float32, 2, 1.5)
    bias = logits_of(1, E, torch.float32, 4, 0.05)[0].contiguous()
    e, w = mx.moe_route(l, k, score="sigmoid", bias=bias, groups=8, top_groups=4, renormalize=True)

    def ranks(v):
        i = torch.arange(v.shape[1], device="cuda")
        a, b = v.unsqueeze(2), v.unsqueeze(1)
        return ((b > a) | ((b == a) & (i.unsqueeze(0) < i.unsqueeze(1)))).sum(2)

    key = torch.sigmoid(l.double()) + bias.double()
    per = key.view(T * 8, 32)
    worth = (per * (ranks(per) < 2)).sum(1).view(T, 8)
    key = key.masked_fill((ranks(worth) >= 4).repeat_interleave(32, 1), -math.inf)
    r = torch.cat([ranks(c) for c in key.split(500)])
    want = torch.empty((T, k), dtype=torch.long, device="cuda")
    at, ex = (r < k).nonzero(as_tuple=True)
    want[at, r[at, ex]] = ex
    assert torch.equal(e.long(), want)
    s = torch.sigmoid(l.double()).gather(1, want)
    s = s / s.sum(1, keepdim=True)
    # sigmoid 6 U twice (itself and in the sum), 5 sums, the quotient, the scale
    assert ((w.double() - s).abs() <= 24 * U * s).all()


def test_route_of_no_tokens():
    l = torch.zeros(0, 8, device="cuda", requires_grad=True)
    e, w = mx.moe_route(l, 2)
    assert e.shape == w.shape == (0, 2)
    assert torch.autograd.grad(w.sum(), l)[0].shape == (0, 8)


def test_route_gradient_modes():
    l = logits_of(4, 8, torch.float32, 1).requires_grad_(True)
    with torch.no_grad():
        assert not mx.moe_route(l, 2)[1].requires_grad
    with torch.inference_mode():
        mx.moe_route(l, 2)
    bias = torch.zeros(8, device="cuda", requires_grad=True)
    e, w = mx.moe_route(l, 2, bias=bias)
    assert w.requires_grad and not e.requires_grad
    (g,) = torch.autograd.grad(w.sum(), l, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (g.sum() + l.sum()).backward()


# ---------------------------------------------------------------- the plan
def check_plan(experts, E, multiple, exact=False):
    p = mx.moe_plan(experts, E, multiple, exact=exact)
    ends, counts, slot, place = ref.plan(experts.cpu().numpy(), E, multiple)
    assert p.offs.tolist() == ends and p.counts.tolist() == counts
    assert np.array_equal(p.place.cpu().numpy(), place)
    got = p.slot.tolist()
    assert got[:len(slot)] == slot and all(s == -1 for s in got[len(slot):])
    assert len(got) == len(slot) if exact else len(got) <= experts.numel() + E * (multiple - 1)
    return p


@pytest.mark.parametrize("T,k,E,multiple", [
    (1, 1, 1, 1), (70, 1, 1, 32), (1, 1, 7, 32), (5, 2, 6, 1), (64, 4, 16, 32), (77, 3, 13, 5), (300, 8, 256, 32), (100, 16, 1024, 1),
    (1024, 4, 16, 128), (1025, 4, 16, 32), (4096, 1, 8, 1), (5000, 3, 100, 32), (9000, 8, 256, 1), (3000, 16, 1024, 3)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_plan(T, k, E, multiple, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + k)
    e = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=dtype)
    check_plan(e, E, multiple)
    check_plan(e, E, multiple, exact=True)
    # choices without a row, at the end and in between; and one expert that takes nearly all
    e[T // 2:T // 2 + 3, 0] = -1
    e[T - T // 4:] = E
    e[::5] = E // 2
    check_plan(e, E, multiple)


@pytest.mark.parametrize("fill", [-1, 0, 5, 6])
@pytest.mark.parametrize("T", [40, 5000])
def test_plan_of_one_group_or_none(fill, T):
    check_plan(torch.full((T, 2), fill, device="cuda", dtype=torch.int32), 6, 32)


def test_plan_of_many_tokens():
    """More choices than a short run's kernels take, against torch's stable sort."""
    T, k, E, multiple = 70000, 16, 300, 32
    e = torch.randint(-1, E, (T, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    p = mx.moe_plan(e, E, multiple)
    flat = e.flatten()
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    padded = (counts + multiple - 1) // multiple * multiple
    ends = padded.cumsum(0)
    assert torch.equal(p.counts.long(), counts) and torch.equal(p.offs.long(), ends)
    order = torch.where(flat >= 0, flat, E).sort(stable=True)[1][:int(counts.sum())]
    row = (ends - padded)[flat[order]] + torch.arange(order.numel(), device="cuda") - (counts.cumsum(0) - counts)[flat[order]]
    slot = torch.full((p.rows,), -1, device="cuda").scatter(0, row, order)
    assert torch.equal(p.slot.long(), slot)
    assert torch.equal(p.place.flatten().long(), torch.full_like(flat, -1).scatter(0, order, row))


@pytest.mark.parametrize("T,k,E,multiple", [
    (524288, 1, 37, 1), (524289, 1, 37, 32), (700000, 1, 1024, 3), (262144, 8, 256, 32), (262145, 8, 300, 1), (900001, 5, 33, 32)])
def test_plan_of_very_many_tokens(T, k, E, multiple):
    """Of so many runs that their counts are summed up first, and just below; against torch's stable sort."""
    g = torch.Generator(device="cuda").manual_seed(T)
    e = torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    e[T // 3:T // 2] = E // 2
    p = mx.moe_plan(e, E, multiple)
    flat = e.flatten().long()
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    padded = (counts + multiple - 1) // multiple * multiple
    ends = padded.cumsum(0)
    assert torch.equal(p.counts.long(), counts) and torch.equal(p.offs.long(), ends)
    order = torch.where(flat >= 0, flat, E).sort(stable=True)[1][:int(counts.sum())]
    row = (ends - padded)[flat[order]] + torch.arange(order.numel(), device="cuda") - (counts.cumsum(0) - counts)[flat[order]]
    assert torch.equal(p.slot.long(), torch.full((p.rows,), -1, device="cuda").scatter(0, row, order))
    assert torch.equal(p.place.flatten().long(), torch.full_like(flat, -1).scatter(0, order, row))


def test_plan_of_nearly_2_31_rows():
    """Row numbers up to the last that 32 bits hold: even tokens go to the first expert, odd ones to the second."""
    T = 2 ** 31 - 3
    e = torch.arange(T, dtype=torch.int32, device="cuda").bitwise_and_(1).view(T, 1)
    p = mx.moe_plan(e, 2)
    first = T // 2 + 1
    assert p.rows == T and p.offs.tolist() == [first, T] and p.counts.tolist() == [first, T - first]
    for at in (0, T // 2 - 1000, T - 2 ** 20):
        t = torch.arange(at, min(at + 2 ** 20, T), device="cuda")
        row = t // 2 + (t & 1) * first
        assert torch.equal(p.place[t, 0].long(), row) and torch.equal(p.slot[row].long(), t)


def test_plan_of_values_past_32_bits():
    e = torch.tensor([[2 ** 32, 1], [-2 ** 33 + 1, 2 ** 40 + 2]], device="cuda")
    check_plan(e, 4, 1)


def test_exact_plan_is_refused_in_a_capture():
    e = torch.zeros((4, 2), device="cuda", dtype=torch.int32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            mx.moe_plan(e, 4, exact=True)
        p = mx.moe_plan(e, 4)
    graph.replay()
    assert p.counts.tolist() == [8, 0, 0, 0]


def test_plan_of_no_tokens():
    p = mx.moe_plan(torch.zeros((0, 2), device="cuda", dtype=torch.int32), 4, 32)
    assert p.rows == 0 and p.offs.tolist() == [0] * 4 and p.counts.tolist() == [0] * 4 and p.place.shape == (0, 2)


def test_plan_takes_strided_experts():
    e = torch.randint(0, 8, (50, 6), device="cuda")
    a, b = mx.moe_plan(e[:, ::2], 8, 32), mx.moe_plan(e[:, ::2].contiguous(), 8, 32)
    assert torch.equal(a.slot, b.slot) and torch.equal(a.place, b.place)


def test_route_and_plan_captured_and_replayed_on_another_stream():
    """Two graphs whose calls have memory of their own, replayed at once beside an eager call."""
    T, E, k = 2000, 64, 4
    graphs = []
    for seed in (1, 2):
        l = logits_of(T, E, torch.float32, seed)
        mx.moe_plan(mx.moe_route(l, k)[0], E, 32)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            e, w = mx.moe_route(l, k, score="sigmoid")
            p = mx.moe_plan(e, E, 32)
        graphs.append((graph, l, e, w, p))
    for seed in (3, 4):
        for i, (graph, l, *_) in enumerate(graphs):
            l.copy_(logits_of(T, E, torch.float32, seed + 10 * i))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for s, (graph, *_) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        mx.moe_plan(torch.randint(0, E, (T, k), device="cuda"), E, 32)
        torch.cuda.synchronize()
        for graph, l, e, w, p in graphs:
            e2, w2 = mx.moe_route(l, k, score="sigmoid")
            p2 = mx.moe_plan(e2, E, 32)
            assert torch.equal(e, e2) and torch.equal(w, w2)
            assert all(torch.equal(getattr(p, n), getattr(p2, n)) for n in ("offs", "counts", "slot", "place"))
