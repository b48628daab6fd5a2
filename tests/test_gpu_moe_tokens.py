"""The routed layer for a few tokens against a plain 64-bit implementation.

The tolerance follows the kernel's roundings.  h1 and h3 are 32-bit sums of D exact products (error at most
D 2^-23 of the sum of magnitudes, in any order); silu and the product add a few 2^-24; so h is known within
delta, and its MX value within what mx(h +- delta) spans.  y adds a 32-bit sum over H and the experts and one
bf16 rounding (2^-8).  Selection compares the given logits exactly, so it has no tolerance."""
import numpy as np
import pytest
import torch

from mxfp8_precision_moe_gb300 import synth
from tests import _mx4ref as ref
from tests._util import f64, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    require_gpu()
    import mxfp8_precision_moe_gb300 as m

    m.load()
    return m


class Layer:
    """Quantized random weights, their 64-bit values, and the kernel over them."""

    def __init__(self, mx, E, D, H, k, bits, score="softmax", seed=0, bad=None):
        self.k, self.bits, self.score, self.E, self.D, self.H = k, bits, score, E, D, H
        ws = [synth.randn_bf16((E, H, D), 1.0 / D ** 0.5, seed=seed + 1),
              synth.randn_bf16((E, H, D), 1.0 / D ** 0.5, seed=seed + 2),
              synth.randn_bf16((E, D, H), 1.0 / H ** 0.5, seed=seed + 3)]
        if bad is not None:
            for w in ws:
                w[bad, 3, 5] = float("nan")
        quant = (lambda w: mx.quantize_expert_weights(w)[:2]) if bits == 8 else mx.mxfp4_quantize_3d_experts
        self.quads = [quant(w.cuda()) for w in ws]
        self.gate, self.up, self.down = [ref.mx_value(f64(w), bits) for w in ws]
        self.op = mx.MxMoeTokens(*self.quads, k, score=score)

    def want(self, x, logits):
        """y and how far the kernel's may be from it."""
        x, logits = f64(x), logits.double().cpu().numpy()
        xq = ref.mx_value(x, self.bits)
        y, tol = np.zeros(x.shape), np.zeros(x.shape)
        for t, (pick, w) in enumerate(ref.route(logits, self.k, self.score)):
            for e, p in zip(pick, w):
                g, u, d = self.gate[e], self.up[e], self.down[e]
                h1, h3 = g @ xq[t], u @ xq[t]
                e1, e3 = (self.D * 2.0 ** -23 * (np.abs(m) @ np.abs(xq[t])) for m in (g, u))
                h = ref.silu(h1) * h3
                delta = 1.1 * e1 * np.abs(h3) + np.abs(ref.silu(h1)) * e3 + 1.1 * e1 * e3 + 2.0 ** -20 * np.abs(h)
                hq = ref.mx_value(h, self.bits)
                span = np.zeros_like(h)
                for way in (1, -1):
                    span = np.maximum(span, np.abs(ref.mx_value(h + way * delta * np.sign(h), self.bits) - hq))
                one = d @ hq
                y[t] += p * one
                tol[t] += p * (np.abs(d) @ span + (self.k * self.H + 16) * 2.0 ** -23 * (np.abs(d) @ np.abs(hq)))
        return y, tol + 2.0 ** -8 * np.abs(y)

    def check(self, x, logits, got=None):
        got = f64(self.op(x, logits) if got is None else got)
        y, tol = self.want(x, logits)
        assert np.array_equal(np.isnan(got), np.isnan(y))
        fin = ~np.isnan(y)
        worst = (np.abs(got - y) - tol)[fin]
        assert worst.size == 0 or worst.max() <= 0, worst.max()


def inputs(T, D, E, seed=0):
    x = synth.randn_bf16((T, D), 1.0, seed=seed + 10).cuda()
    g = torch.Generator().manual_seed(seed + 11)
    return x, torch.randn((T, E), generator=g).cuda()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,E,D,H,k", [
    (1, 1, 32, 32, 1), (1, 4, 256, 128, 1), (1, 8, 416, 160, 3), (5, 6, 352, 160, 2), (2, 3, 640, 288, 3),
    (32, 8, 128, 256, 2), (33, 5, 288, 416, 2), (64, 16, 512, 384, 4), (64, 2, 96, 64, 1), (17, 40, 192, 96, 16),
    (3, 256, 64, 64, 8),
])
def test_matches_the_definition(mx, T, E, D, H, k, bits):
    lay = Layer(mx, E, D, H, k, bits, seed=T + D)
    lay.check(*inputs(T, D, E, seed=T))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,E,D,H,k", [
    (1, 2, 256, 256, 1), (1, 8, 512, 1280, 2), (2, 3, 2304, 256, 1), (3, 4, 256, 2304, 3), (7, 5, 768, 512, 2),
    (8, 16, 1024, 512, 4), (8, 3, 4096, 1024, 1), (8, 3, 4352, 512, 2), (9, 3, 512, 512, 2), (5, 130, 256, 256, 16),
])
def test_whole_chunks_of_few_tokens(mx, T, E, D, H, k, bits):
    """Widths of whole 128-byte chunks, with few and many tiles and steps."""
    lay = Layer(mx, E, D, H, k, bits, seed=T + D)
    lay.check(*inputs(T, D, E, seed=T))


@pytest.mark.parametrize("bits", [8, 4])
def test_edges_of_whole_chunks(mx, bits):
    """Non-finite weights and tokens, unrouted tokens and repeats, all in one batch."""
    lay = Layer(mx, 4, 512, 256, 1, bits, bad=2)
    x, logits = inputs(6, 512, 4)
    logits[:] = 0
    for t, e in enumerate((0, 2, 1, 3, 2, 0)):
        logits[t, e] = 5
    logits[3] = -float("inf")
    x[5, 511] = float("nan")
    y = lay.op(x, logits)
    assert torch.isnan(y).any(1).tolist() == [False, True, False, False, True, True]
    assert torch.isnan(y[1]).all() and torch.isnan(y[5]).all() and not y[3].any()
    want, tol = lay.want(x[[0, 2]], logits[[0, 2]])
    assert (np.abs(f64(y[[0, 2]]) - want) <= tol).all()
    for _ in range(10):
        again = lay.op(x, logits)
        assert torch.equal(again.isnan(), y.isnan()) and torch.equal(again.nan_to_num(), y.nan_to_num())
    logits[:] = -float("inf")
    assert not lay.op(x, logits).any()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,E,D,H,k", [
    (8, 8, 256, 2432, 2), (40, 8, 256, 2432, 2), (1, 2, 256, 2432, 1), (3, 2, 19456, 64, 1), (33, 2, 8192, 256, 1),
    (2, 2, 8192, 288, 2), (20, 2, 256, 8192, 1), (1, 3, 352, 8192, 2),
])
def test_cuts(mx, T, E, D, H, k, bits):
    """Both halves cut each way: into whole tiles of 128 and of 64 rows, and into runs that share tiles."""
    lay = Layer(mx, E, D, H, k, bits, seed=H + T)
    lay.check(*inputs(T, D, E, seed=T + 1))


@pytest.mark.parametrize("T,E,k", [(64, 256, 8), (1, 256, 16), (33, 97, 3), (7, 30, 1), (5, 29, 1), (64, 64, 4), (40, 128, 16)])
@pytest.mark.parametrize("score", ["softmax", "softmax_all"])
def test_many_experts(mx, T, E, k, score):
    """Many experts, with equal logits, -inf and a token that has fewer finite logits than it may select."""
    lay = Layer(mx, E, 64, 32, k, 8, score=score)
    x, logits = inputs(T, 64, E, seed=E)
    logits[:, ::3] = 0.25
    logits[T // 2, 1:] = -float("inf")
    logits[:, E - 1] = -float("inf")
    lay.check(x, logits)


@pytest.mark.parametrize("bits", [8, 4])
def test_wide_layer(mx, bits):
    """Many tiles and steps: runs that begin and end inside tiles, several experts a run."""
    lay = Layer(mx, 6, 2080, 1056, 2, bits, seed=9)
    lay.check(*inputs(7, 2080, 6, seed=3))


@pytest.mark.parametrize("score", ["softmax", "softmax_all", "sigmoid"])
def test_scores(mx, score):
    lay = Layer(mx, 9, 256, 128, 3, 8, score=score)
    lay.check(*inputs(12, 256, 9))


def test_routing_edges(mx):
    lay = Layer(mx, 8, 128, 96, 3, 8)
    x, logits = inputs(10, 128, 8)
    inf, nan = float("inf"), float("nan")
    logits[0] = 0.0                                             # all equal: the lowest three
    logits[1] = torch.tensor([0.0, -0.0, 0.0, -0.0, 0, 0, 0, 0])
    logits[2] = -inf                                            # no expert: zeros
    logits[3] = torch.tensor([-inf] * 6 + [1.0, 2.0])           # two experts only
    logits[4, 5] = nan                                          # the row is NaN
    logits[5] = torch.tensor([3.4e38, -3.4e38, 0, 0, 0, 0, 0, 0])  # the lowest finite value is not -inf
    logits[6] = -3.4e38
    logits[7, 2] = inf                                          # inf - inf
    lay.check(x, logits)
    y = lay.op(x, logits)
    assert not y[2].any() and torch.isnan(y[4]).all() and torch.isnan(y[7]).all()
    logits[:] = -inf
    assert not lay.op(x, logits).any()


@pytest.mark.parametrize("bits", [8, 4])
def test_nonfinite_weights_stay_with_their_expert(mx, bits):
    lay = Layer(mx, 4, 128, 128, 1, bits, bad=2)
    x, logits = inputs(6, 128, 4)
    logits[:] = 0
    for t, e in enumerate((0, 2, 1, 3, 2, 0)):
        logits[t, e] = 5
    y = lay.op(x, logits)
    bad = torch.isnan(y).any(1).tolist()
    assert bad == [False, True, False, False, True, False]
    assert torch.isnan(y[1]).all()                               # a NaN in h's block reaches the whole row
    good = [0, 2, 3, 5]
    want, tol = lay.want(x[good], logits[good])
    assert (np.abs(f64(y[good]) - want) <= tol).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_nonfinite_tokens_stay_in_their_row(mx, bits):
    lay = Layer(mx, 4, 160, 96, 2, bits)
    x, logits = inputs(5, 160, 4)
    x[1, 159], x[3, 0] = float("inf"), float("nan")
    lay.check(x, logits)


def test_zero_and_tiny_tokens(mx):
    lay = Layer(mx, 3, 128, 64, 2, 8)
    x, logits = inputs(4, 128, 3)
    x[0] = 0
    x[1] *= 2.0 ** -120
    x[2] = 2.0 ** -130
    lay.check(x, logits)
    assert not lay.op(x, logits)[0].any()


def test_no_tokens(mx):
    lay = Layer(mx, 3, 64, 64, 2, 8)
    assert lay.op(*inputs(0, 64, 3)).shape == (0, 64)


def test_repeats_exactly_and_takes_other_sizes_between(mx):
    """The same bits every time, whatever ran on the workspace before."""
    lay = Layer(mx, 8, 1056, 544, 2, 4)
    a, b, c = (inputs(T, 1056, 8, seed=T) for T in (3, 64, 30))
    first = lay.op(*a)
    for _ in range(20):
        lay.op(*b)
        assert torch.equal(lay.op(*a), first)
        lay.op(*c)
    lay.check(*a)


def test_out_status_and_logit_types(mx):
    lay = Layer(mx, 4, 128, 64, 2, 8)
    x, logits = inputs(3, 128, 4)
    out, st = torch.empty((3, 128), dtype=torch.bfloat16, device="cuda"), mx.new_status()
    assert lay.op(x, logits, out=out, dev_status=st) is out
    mx.read_status(st)
    half = logits.to(torch.bfloat16)
    assert torch.equal(lay.op(x, half), lay.op(x, half.float()))


def test_other_streams_have_their_own_workspace(mx):
    lay = Layer(mx, 8, 512, 512, 2, 8)
    sets = [inputs(T, 512, 8, seed=T) for T in (1, 9, 40)]
    want = [lay.op(*s) for s in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[] for _ in sets]
    for _ in range(10):
        for i, (s, st) in enumerate(zip(sets, streams)):
            with torch.cuda.stream(st):
                got[i].append(lay.op(*s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, w in zip(got, want) for g in gs)


def test_graph(mx):
    lay = Layer(mx, 4, 256, 128, 2, 4)
    x, logits = inputs(5, 256, 4)
    lay.op(x, logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lay.op(x, logits)
    for seed in (5, 6):
        nx, nl = inputs(5, 256, 4, seed=seed)
        x.copy_(nx)
        logits.copy_(nl)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, lay.op(nx, nl))


def test_graph_beside_eager_calls_of_its_stream(mx):
    """A graph captured on a stream that has run the layer eagerly shares no workspace with those calls."""
    lay = Layer(mx, 4, 256, 128, 2, 8)
    a, b = inputs(5, 256, 4, seed=5), inputs(7, 256, 4, seed=6)
    want = lay.op(*a), lay.op(*b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lay.op(*a)
    torch.cuda.synchronize()
    held = {k: v.data_ptr() for k, v in lay.op._workspaces.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = [lay.op(*a) for _ in range(3)]
    assert {k: v.data_ptr() for k, v in lay.op._workspaces.items()} == held
    for _ in range(20):
        graph.replay()
        with torch.cuda.stream(side):
            z = lay.op(*b)
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[0]) for v in y) and torch.equal(z, want[1])


def test_refusals(mx):
    lay = Layer(mx, 4, 128, 64, 2, 8)
    x, logits = inputs(3, 128, 4)
    op, (g, u, d) = lay.op, lay.quads
    for bad, match in [
        (lambda: op(x.float(), logits), "x:"), (lambda: op(x[:, :64].contiguous(), logits), "x:"),
        (lambda: op(x, logits[:2]), "router_logits"), (lambda: op(x, logits.long()), "router_logits"),
        (lambda: op(x.t().contiguous().t(), logits), "contiguous"), (lambda: op(x.cpu(), logits), "CUDA"),
        (lambda: op(x.clone().requires_grad_(True), logits), "no gradients"),
        (lambda: op(x, logits, out=torch.empty((3, 128), device="cuda")), "out"),
        (lambda: op(*inputs(65, 128, 4)), "at most 64"),
        (lambda: mx.MxMoeTokens(g, u, d, 5), "top_k"), (lambda: mx.MxMoeTokens(g, u, d, 2, score="tanh"), "score"),
        (lambda: mx.MxMoeTokens(g, u, (d[0][:, :, :32].contiguous(), d[1]), 2), "down codes"),
        (lambda: mx.MxMoeTokens((g[0], g[1][:, :100].contiguous()), u, d, 2), "gate scales"),
        (lambda: mx.MxMoeTokens(g, u, d, 2, max_tokens=65), "max_tokens"),
    ]:
        with pytest.raises(ValueError, match=match):
            bad()
    with torch.no_grad():
        op(x.clone().requires_grad_(True), logits)
