"""The few-token layer divides each half of its work among the CTAs in one of three ways.  Every pair of ways, in both
formats, and with one and with several whole tiles a CTA: that the sizes below go those ways, and that the layer is right.

The weights have about 64 elements in a row that are not zero, wherever in the row, so that 32-bit sums stay close to the
64-bit ones at any width: of n terms that are not zero at most n - 1 additions round, by 2^-23 of the sum of magnitudes each
(tensor cores may truncate), in whatever order.  Beyond that the bound is that of test_gpu_moe_tokens."""
import numpy as np
import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests import _mx4ref as ref
from tests._util import f64, require_gpu

# cuts of the two halves ("+": more tiles than CTAs), bits, tokens, experts, D, H
CASES = [
    ("128", "128", 4, 2, 6, 9792, 1568), ("128", "128", 8, 32, 6, 9792, 1696),
    ("128", "128+", 4, 33, 5, 29280, 2080), ("128", "128+", 8, 1, 8, 29344, 1312),
    ("128", "64", 4, 29, 2, 5792, 4896), ("128", "64", 8, 33, 8, 8128, 1184), ("128", "64+", 4, 3, 2, 17472, 5184),
    ("128", "64+", 8, 20, 8, 29120, 1344), ("128", "shared", 4, 33, 6, 64, 1568),
    ("128", "shared", 8, 11, 6, 64, 1568), ("128+", "128", 4, 20, 1, 10048, 29216),
    ("128+", "128", 8, 64, 8, 10784, 3744), ("128+", "64", 4, 8, 1, 6176, 29280),
    ("128+", "64", 8, 32, 8, 9504, 3744), ("128+", "shared", 4, 50, 8, 64, 3616),
    ("128+", "shared", 8, 1, 8, 64, 3616), ("64", "128", 4, 20, 8, 10048, 928), ("64", "128", 8, 33, 8, 9824, 1056),
    ("64", "128+", 4, 16, 8, 29216, 800), ("64", "128+", 8, 1, 6, 29216, 1184), ("64", "64", 4, 40, 1, 64, 64),
    ("64", "64", 8, 2, 1, 64, 64), ("64", "64+", 4, 20, 5, 26464, 1856), ("64", "64+", 8, 1, 4, 19104, 1696),
    ("64", "shared", 4, 16, 8, 64, 544), ("64", "shared", 8, 17, 6, 64, 288), ("64+", "128", 4, 64, 5, 10144, 5664),
    ("64+", "128", 8, 16, 1, 10272, 17472), ("64+", "64", 4, 29, 8, 8640, 3488), ("64+", "64", 8, 5, 5, 6944, 3744),
    ("64+", "64+", 4, 8, 1, 17440, 18624), ("64+", "64+", 8, 16, 1, 18656, 17504),
    ("64+", "shared", 4, 64, 3, 64, 6432), ("64+", "shared", 8, 3, 3, 64, 6432),
    ("shared", "128", 4, 32, 1, 9760, 64), ("shared", "128", 8, 64, 1, 9760, 64),
    ("shared", "128+", 4, 1, 1, 29216, 64), ("shared", "128+", 8, 29, 1, 29216, 64),
    ("shared", "64", 4, 50, 1, 2848, 64), ("shared", "64", 8, 3, 1, 1824, 64),
    ("shared", "64+", 4, 20, 1, 19488, 64), ("shared", "64+", 8, 50, 1, 19488, 64),
    ("shared", "shared", 4, 2, 1, 2848, 19488), ("shared", "shared", 8, 17, 6, 1440, 288),
]
CTAS = 152


def cut(half, bits, T, E, D, H, ctas):
    rows = mx.load().mx_debug_moe_tokens_cut(half, T, E, D, H, bits, ctas)
    assert rows in (1, 64, 128)
    if rows == 1:
        return "shared"
    tiles = (-(-D // 128) if half else E * -(-H // 128)) * 128 // rows
    return f"{rows}{'+' if tiles > ctas else ''}"


def test_cases_cover_every_pair_of_cuts():
    for one, two, *size in CASES:
        assert (cut(0, *size, CTAS), cut(1, *size, CTAS)) == (one, two)
    ways = ("64", "64+", "128", "128+", "shared")
    rare = {("64+", "128+"), ("128+", "64+"), ("128+", "128+")}  # half a billion weights and more
    have = {(one, two, bits) for one, two, bits, *_ in CASES}
    assert have == {(one, two, bits) for one in ways for two in ways for bits in (4, 8) if (one, two) not in rare}
    assert {(T > 16) + (T > 32) for _, _, _, T, *_ in CASES} == {0, 1, 2}


def test_refused_cuts():
    f = mx.load().mx_debug_moe_tokens_cut
    assert f(0, 1, 1, 64, 64, 8, 152) > 0
    assert not any((f(2, 1, 1, 64, 64, 8, 152), f(0, 0, 1, 64, 64, 8, 152), f(0, 1, 0, 64, 64, 8, 152),
                    f(0, 1, 1, 60, 64, 8, 152), f(0, 1, 1, 64, 64, 6, 152), f(0, 1, 1, 64, 64, 8, 0)))


def values(q, s, R, C, bits):
    """64-bit values of one expert's codes [R, ...] and blocked scales, on the GPU."""
    if bits == 8:
        v = q.view(torch.float8_e4m3fn).double()
    else:
        t = torch.tensor(np.concatenate([ref.E2M1, -ref.E2M1]), device="cuda")
        v = t[torch.stack((q & 15, q >> 4), -1).flatten(-2).long()]
    rb, cb = -(-R // 128), -(-C // 128)
    s = s[:rb * cb * 512].reshape(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)[:R, :C // 32]
    scale = torch.ldexp(torch.ones_like(s, dtype=torch.float64), s.int() - 127)
    return (v.unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)


def quantized(E, R, C, bits, g):
    parts = []
    for _ in range(E):
        w = torch.randn((1, R, C), generator=g, device="cuda") / 8
        w = torch.where(torch.rand((1, R, C), generator=g, device="cuda") < 64 / C, w, 0).bfloat16()
        parts.append(mx.quantize_expert_weights(w)[:2] if bits == 8 else mx.mxfp4_quantize_3d_experts(w))
    return tuple(torch.cat(p) for p in zip(*parts))


@pytest.mark.gpu
@pytest.mark.parametrize("one,two,bits,T,E,D,H", CASES)
def test_cuts_are_right(one, two, bits, T, E, D, H):
    require_gpu()
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    assert (cut(0, bits, T, E, D, H, ctas), cut(1, bits, T, E, D, H, ctas)) == (one, two)
    g = torch.Generator("cuda").manual_seed(D + H)
    k = max(-(-E // T), min(2, E))
    gate, up, down = quantized(E, H, D, bits, g), quantized(E, H, D, bits, g), quantized(E, D, H, bits, g)
    x = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    logits = torch.randn((T, E), generator=g, device="cuda")
    for t in range(T):  # every expert is selected
        for i in range(k):
            logits[t, (t * k + i) % E] += 10
    op = mx.MxMoeTokens(gate, up, down, k)
    y = op(x, logits)
    assert torch.equal(op(x, logits), y)
    op.check_status()

    xq = torch.from_numpy(ref.mx_value(f64(x), bits)).cuda()
    picks = ref.route(logits.double().cpu().numpy(), k, "softmax")
    want, tol = (torch.zeros((T, D), dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        who = [t for t in range(T) if e in picks[t][0]]
        assert who
        p = torch.tensor([picks[t][1][picks[t][0].index(e)] for t in who], device="cuda").unsqueeze(1)
        h, err = [], []
        for w in (gate, up):
            v = values(w[0][e], w[1][e], H, D, bits)
            n = int((v != 0).sum(1).max())
            h.append(f64_of(xq[who] @ v.T))
            err.append(f64_of(n * 2.0 ** -23 * (xq[who].abs() @ v.abs().T)))
            del v
        (h1, h3), (e1, e3) = h, err
        h = ref.silu(h1) * h3
        delta = 1.1 * e1 * np.abs(h3) + np.abs(ref.silu(h1)) * e3 + 1.1 * e1 * e3 + 2.0 ** -20 * np.abs(h)
        hq = ref.mx_value(h, bits)
        span = np.zeros_like(h)
        for way in (1, -1):
            span = np.maximum(span, np.abs(ref.mx_value(h + way * delta * np.sign(h), bits) - hq))
        v = values(down[0][e], down[1][e], D, H, bits)
        n = int((v != 0).sum(1).max())
        hq, span = torch.from_numpy(hq).cuda(), torch.from_numpy(span).cuda()
        want[who] += p * (hq @ v.T)
        tol[who] += p * (span @ v.abs().T + (k * n + 16) * 2.0 ** -23 * (hq.abs() @ v.abs().T))
        del v
    tol += 2.0 ** -8 * want.abs()
    worst = ((y.double() - want).abs() - tol).max()
    assert worst <= 0, float(worst)
    assert tol.mean() < 0.1 * want.abs().mean()  # the bound means something


def f64_of(t):
    return t.cpu().numpy()
