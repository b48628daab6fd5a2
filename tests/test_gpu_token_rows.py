"""Token rows into a plan's order and back, as they are and quantized on the way, and the layer made of it all."""
import numpy as np
import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests._util import require_gpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24          # half a step of fp32, relative
BF16 = 2.0 ** -8        # half a step of bf16, relative


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).bfloat16()


def make_plan(T, k, E, multiple, seed=0, idle=True, exact=False):
    e = torch.rand((T, E), generator=gen(seed), device="cuda").topk(k, 1)[1]
    if idle and T > 2:
        e[T // 2, 0] = -1     # a choice without a row, and a token without any
        e[T - 1] = -1
    return mx.moe_plan(e, E, multiple, exact=exact)


def rows_ref(x, plan):
    s = plan.slot.long()
    return torch.where((s >= 0)[:, None], x[s.clamp_min(0) // plan.top_k], torch.zeros((), dtype=x.dtype, device=x.device))


SHAPES = [(1, 1, 1, 1, 8), (1, 1, 5, 32, 32), (3, 2, 4, 1, 40), (5, 2, 6, 32, 352), (77, 3, 13, 5, 264), (64, 16, 40, 32, 1024),
          (300, 8, 256, 32, 96), (1000, 4, 16, 128, 2056), (129, 6, 8, 1, 7168), (513, 1, 3, 32, 128), (40, 5, 9, 1, 16)]


@pytest.mark.parametrize("T,k,E,multiple,D", SHAPES)
def test_gather_and_its_gradient(T, k, E, multiple, D):
    plan = make_plan(T, k, E, multiple, T)
    x = randn((T, D), 1).requires_grad_(True)
    rows = mx.moe_gather(x, plan)
    assert torch.equal(rows, rows_ref(x.detach(), plan))
    d = randn((plan.rows, D), 2)
    (dx,) = torch.autograd.grad(rows, x, d)
    want, mass = choices(d, plan)
    # k - 1 fp32 sums, one rounding to bf16
    assert ((dx.double() - want).abs() <= BF16 * want.abs() + k * U * mass).all()


def choices(y, plan, w=None):
    """sum over j of w y[place] in 64 bits, and the sum of the terms' magnitudes."""
    y = y.double()
    out = torch.zeros((plan.tokens, y.shape[1]), dtype=torch.float64, device="cuda")
    mass = out.clone()
    for j in range(plan.top_k):
        at = plan.place[:, j].long()
        part = torch.where((at >= 0)[:, None], y[at.clamp_min(0)] if y.shape[0] else torch.zeros_like(out), 0.0)
        if w is not None:
            part = part * w[:, j:j + 1].double()
        out += part
        mass += part.abs()
    return out, mass


@pytest.mark.parametrize("T,k,E,multiple,D", SHAPES)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_its_gradients(T, k, E, multiple, D, weighted):
    plan = make_plan(T, k, E, multiple, T)
    y = randn((plan.rows, D), 1).requires_grad_(True)
    w = torch.randn((T, k), generator=gen(3), device="cuda").requires_grad_(True) if weighted else None
    out = mx.moe_combine(y, plan, w)
    want, mass = choices(y.detach(), plan, None if w is None else w.detach())
    assert ((out.double() - want).abs() <= BF16 * want.abs() + k * U * mass).all()
    d = randn((T, D), 2)
    grads = torch.autograd.grad(out, (y, w) if weighted else (y,), d)
    s = plan.slot.long()
    row_w = torch.ones(plan.rows, device="cuda") if w is None else w.detach().flatten()[s.clamp_min(0)]
    dy = torch.where((s >= 0)[:, None], rows_ref(d, plan).double() * row_w.double()[:, None], 0.0)
    # one product in fp32, one rounding to bf16
    assert ((grads[0].double() - dy).abs() <= (BF16 + 2 * U) * dy.abs()).all()
    if weighted:
        at = plan.place.long()
        terms = torch.where((at >= 0)[:, :, None], y.detach().double()[at.clamp_min(0)], 0.0) * d.double()[:, None]
        # products and sums of D terms, each sum by a thread, then a warp, then the CTA: fewer than D / 256 * 8 + 24 roundings
        bound = (D / 32 + 24) * U * terms.abs().sum(2)
        assert ((grads[1].double() - terms.sum(2)).abs() <= bound).all()
        # each gradient by itself
        (dw,) = torch.autograd.grad(mx.moe_combine(y.detach(), plan, w), w, d)
        assert torch.equal(dw, grads[1])
        (dy1,) = torch.autograd.grad(mx.moe_combine(y, plan, w.detach()), y, d)
        assert torch.equal(dy1, grads[0])


def test_combine_gradient_against_differences():
    """<out, d> is linear in w up to out's rounding: a difference over w +- 1 is off by at most two half steps of bf16 of
    the outputs, summed with |d|."""
    plan = make_plan(6, 2, 4, 1, 1, idle=False)
    y, d = randn((plan.rows, 64), 1), randn((6, 64), 2)
    w = torch.rand((6, 2), generator=gen(3), device="cuda").requires_grad_(True)
    (dw,) = torch.autograd.grad(mx.moe_combine(y, plan, w), w, d)
    for t in range(6):
        for j in range(2):
            step = torch.zeros_like(w)
            step[t, j] = 1.0
            up, down = (mx.moe_combine(y, plan, w.detach() + f * step).double() for f in (1, -1))
            got = ((up - down)[t] * d[t].double()).sum() / 2
            tol = BF16 * ((up.abs() + down.abs())[t] * d[t].double().abs()).sum() / 2
            assert (got - dw[t, j].double()).abs() <= 1.01 * tol + 1e-4


def test_rows_without_a_token_do_not_count():
    """NaN and infinities in padding rows, and in rows past the last group, reach no output."""
    plan = make_plan(50, 2, 6, 32, 1)
    y = randn((plan.rows, 64), 1)
    clean = mx.moe_combine(y, plan)
    y[plan.slot < 0] = float("nan")
    assert torch.equal(mx.moe_combine(y, plan), clean)
    w = torch.rand((50, 2), device="cuda").requires_grad_(True)
    (dw,) = torch.autograd.grad(mx.moe_combine(y, plan, w), w, randn((50, 64), 2))
    assert torch.isfinite(dw).all() and (dw[plan.place < 0] == 0).all()


def test_entries_out_of_range_are_none():
    """A plan made by hand whose entries leave the tensors: they count as -1, nothing is read or written there."""
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = mx.MoePlan(i([32]), i([2]), i([0, 1, 99, -7] + [-1] * 28), i([[0], [1], [5000], [-2]]), 32)
    x = randn((4, 64), 1)
    rows = mx.moe_gather(x, plan)
    assert torch.equal(rows[:2], x[:2]) and not rows[2:].any()
    out = mx.moe_combine(rows, plan)
    assert torch.equal(out[:2], x[:2]) and not out[2:].any()
    q = mx.mxfp8_gather_quantize(x, plan, mx.ROW | mx.COL)
    same_copies(q, mx.mxfp8_quantize_2d(rows, mx.ROW | mx.COL, mx.SCALES_BLOCKED, plan.offs), plan, 64)
    q = mx.mxfp4_gather_quantize(x, plan)
    assert torch.equal(q[0], mx.mxfp4_quantize_2d(rows, offs=plan.offs)[0])


def test_gradients_at_any_offset():
    """Autograd hands over views: those of a concatenation start at whatever lies before."""
    T, k, E, D = 40, 2, 4, 32
    plan = make_plan(T, k, E, 1, 1)
    x, w, head = randn((T, D), 1), torch.rand((T, k), device="cuda", generator=gen(2)), randn((3,), 3)
    ws = weights_of(E, D, 32, 4)
    logits = torch.randn((T, E), device="cuda", generator=gen(5))
    for leaves, f in (([x], lambda x: mx.moe_gather(x, plan)),
                      ([randn((plan.rows, D), 6), w], lambda y, w: mx.moe_combine(y, plan, w)),
                      ([x, logits, *ws], lambda x, l, *ws: mx.mxfp8_moe_swiglu(x, l, *ws, k))):
        leaves = [t.detach().requires_grad_(True) for t in leaves]
        out = f(*leaves)
        d = randn(out.shape, 7)
        want = torch.autograd.grad(out, leaves, d)
        whole = torch.cat([head, f(*leaves).flatten()])
        got = torch.autograd.grad(whole, leaves, torch.cat([head, d.flatten()]))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_a_plan_overwritten_before_the_backward_is_noticed():
    x = randn((20, 32), 1).requires_grad_(True)
    for f in (lambda plan: mx.moe_gather(x, plan), lambda plan: mx.moe_combine(mx.moe_gather(x.detach(), plan).requires_grad_(True), plan)):
        plan = make_plan(20, 2, 4, 1, 1)
        out = f(plan)
        plan.place.copy_(make_plan(20, 2, 4, 1, 2).place)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_of_no_tokens():
    plan = mx.moe_plan(torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 4, 32)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    rows = mx.moe_gather(x, plan)
    assert rows.shape == (0, 64) and torch.autograd.grad(rows.sum(), x)[0].shape == (0, 64)
    w = torch.zeros((0, 2), device="cuda", requires_grad=True)
    out = mx.moe_combine(rows, plan, w)
    assert out.shape == (0, 64) and torch.autograd.grad(out.sum(), w)[0].shape == (0, 2)
    assert mx.mxfp8_gather_quantize(x.detach(), plan, mx.ROW | mx.COL)[0].shape == (0, 64)
    assert mx.mxfp4_gather_quantize(x.detach(), plan)[0].shape == (0, 32)
    # tokens that all go nowhere: room for 6 rows of 4 groups, 6 + 4 * 31, down to a multiple of 32
    plan = mx.moe_plan(torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), 4, 32)
    x = randn((3, 64), 1).requires_grad_(True)
    rows = mx.moe_gather(x, plan)
    assert rows.shape == (128, 64) and not rows.any() and not torch.autograd.grad(rows.sum(), x)[0].any()
    assert not mx.moe_combine(rows.detach(), plan).any()
    plan = mx.moe_plan(torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), 4, 32, exact=True)
    rows = mx.moe_gather(x, plan)
    assert rows.shape == (0, 64) and not torch.autograd.grad(rows.sum(), x)[0].any()
    w = torch.ones((3, 2), device="cuda", requires_grad=True)
    out = mx.moe_combine(rows.detach(), plan, w)
    assert out.shape == (3, 64) and not out.any() and not torch.autograd.grad(out.sum(), w)[0].any()


def test_any_layout_is_taken_and_modes():
    plan = make_plan(40, 2, 6, 32, 1)
    x = randn((40, 128), 1)
    assert torch.equal(mx.moe_gather(x.T.contiguous().T, plan), mx.moe_gather(x, plan))
    y, w = randn((plan.rows, 128), 2), torch.rand((2, 40), device="cuda").T
    assert torch.equal(mx.moe_combine(y, plan, w), mx.moe_combine(y, plan, w.contiguous()))
    xg = x.clone().requires_grad_(True)
    rows = mx.moe_gather(xg, plan)
    a = torch.autograd.grad(rows, xg, torch.ones(128, device="cuda", dtype=torch.bfloat16).expand(plan.rows, 128),
                            create_graph=True)[0]
    with pytest.raises(RuntimeError, match="second derivative"):
        (a.sum() + xg.sum()).backward()
    with torch.inference_mode():
        assert not mx.moe_gather(xg, plan).requires_grad
    with pytest.raises(ValueError, match="contiguous"):
        mx.mxfp8_gather_quantize(x.T.contiguous().T, plan)


def test_offsets_past_32_bits():
    """2.2 thousand million elements a matrix, its last rows among what is checked."""
    T, D = 270016, 8192
    x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 4096):
        x[i:i + 4096] = randn((min(4096, T - i), D), i)
    e = torch.randint(0, 4, (T, 1), generator=gen(5), device="cuda")
    plan = mx.moe_plan(e, 4, 32, exact=True)
    rows = mx.moe_gather(x, plan)
    token = plan.slot.long()
    for at in (slice(0, 500), slice(plan.rows // 2, plan.rows // 2 + 500), slice(plan.rows - 500, plan.rows)):
        t = token[at]
        assert torch.equal(rows[at], torch.where((t >= 0)[:, None], x[t.clamp_min(0)], 0.0))
    assert torch.equal(mx.moe_combine(rows, plan), x)
    both = mx.ROW | mx.COL
    got = mx.mxfp8_gather_quantize(x, plan, both)
    same_copies(got, mx.mxfp8_quantize_2d(rows, both, mx.SCALES_BLOCKED, plan.offs), plan, D)
    q, s, *_ = mx.mxfp8_gather_quantize(x, plan)
    same_copies((q, s, None, None), (got[0], got[1], None, None), plan, D)
    values = mx.mxfp8_dequantize_2d(q, s, offs=plan.offs)
    # half a step is 2^-4 of a value, saturation of a block's largest (512 to 448) 2^-3
    assert ((values[-500:].float() - rows[-500:].float()).abs() <= 2.0 ** -3 * rows[-500:].float().abs() + 2.0 ** -9).all()
    del got, q, s, values
    q, s = mx.mxfp4_gather_quantize(x, plan)
    want = mx.mxfp4_quantize_2d(rows, offs=plan.offs)
    assert torch.equal(q, want[0])
    del q, s, want
    w = torch.rand((T, 1), generator=gen(6), device="cuda").requires_grad_(True)
    y = rows.detach().requires_grad_(True)
    dy, dw = torch.autograd.grad(mx.moe_combine(y, plan, w), (y, w), x)
    t = token[-500:]
    assert ((dy[-500:].float() - rows[-500:].float() * torch.where(t >= 0, w.detach().flatten()[t.clamp_min(0)], 0.0)[:, None]).abs()
            <= 2 * BF16 * dy[-500:].float().abs()).all()
    assert ((dw[-500:, 0] - x[-500:].float().square().sum(1)).abs() <= 1e-3 * dw[-500:, 0]).all()


# ---------------------------------------------------------------- quantized on the way
Q_SHAPES = [(1, 1, 1, 32, 32), (5, 2, 6, 32, 352), (77, 3, 13, 32, 160), (300, 8, 256, 32, 96), (1000, 4, 16, 128, 2080),
            (129, 6, 8, 32, 7168), (2000, 1, 3, 32, 128), (64, 16, 40, 64, 1024)]


def blocked_scales(s, plan, cols, K):
    """The bytes of a blocked buffer that the layout uses (the buffer's bound is longer)."""
    offs = plan.offs.tolist()
    sizes = np.diff([0] + offs)
    if len(sizes) == 1:  # one group: the whole matrix
        sizes = np.array([plan.rows])
    padded = int(((sizes + 127) // 128 * 128).sum())
    n = -(-K // 128) * padded * 4 if not cols else -(-K // 128) * 128 * padded // 32
    return s.flatten()[:n]


def same_copies(got, want, plan, D):
    for i, (a, b) in enumerate(zip(got, want)):
        assert (a is None) == (b is None)
        if a is None:
            continue
        if i % 2:
            a, b = blocked_scales(a, plan, i == 3, D), blocked_scales(b, plan, i == 3, D)
        assert torch.equal(a, b), i


@pytest.mark.parametrize("T,k,E,multiple,D", Q_SHAPES)
@pytest.mark.parametrize("dirs", [mx.ROW, mx.COL, mx.ROW | mx.COL])
@pytest.mark.parametrize("weighted", [False, True])
def test_mxfp8_gather_quantize_is_the_two_steps(T, k, E, multiple, D, dirs, weighted):
    plan = make_plan(T, k, E, multiple, T)
    x = randn((T, D), 1)
    x[T // 3] *= 1e4
    rows, w = mx.moe_gather(x, plan), None
    if weighted:
        w = torch.randn((T, k), generator=gen(3), device="cuda")
        y = torch.zeros_like(rows).requires_grad_(True)
        (rows,) = torch.autograd.grad(mx.moe_combine(y, plan, w), y, x)
    got = mx.mxfp8_gather_quantize(x, plan, dirs, w)
    want = mx.mxfp8_quantize_2d(rows, dirs, mx.SCALES_BLOCKED, plan.offs)
    same_copies(got, want, plan, D)


@pytest.mark.parametrize("T,k,E,multiple,D", Q_SHAPES + [(77, 3, 13, 5, 160), (40, 5, 9, 1, 288), (3, 2, 4, 1, 32)])
def test_mxfp4_gather_quantize_is_the_two_steps(T, k, E, multiple, D):
    plan = make_plan(T, k, E, multiple, T, exact=True)
    x = randn((T, D), 1)
    x[T // 3] *= 1e4
    got = mx.mxfp4_gather_quantize(x, plan)
    want = mx.mxfp4_quantize_2d(mx.moe_gather(x, plan), offs=plan.offs)
    assert torch.equal(got[0], want[0])
    assert torch.equal(blocked_scales(got[1], plan, False, D), blocked_scales(want[1], plan, False, D))


def test_gather_quantize_of_special_values():
    plan = make_plan(40, 2, 5, 32, 1, exact=True)
    x = randn((40, 256), 1)
    x[3, 5], x[7, 200], x[9] = float("inf"), float("nan"), 0.0
    x[11] = torch.finfo(torch.bfloat16).max
    x[12] = 2.0 ** -133
    rows = mx.moe_gather(x, plan)
    same_copies(mx.mxfp8_gather_quantize(x, plan, mx.ROW | mx.COL),
                mx.mxfp8_quantize_2d(rows, mx.ROW | mx.COL, mx.SCALES_BLOCKED, plan.offs), plan, 256)
    assert torch.equal(mx.mxfp4_gather_quantize(x, plan)[0], mx.mxfp4_quantize_2d(rows, offs=plan.offs)[0])


E4M3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)],
                    dtype=torch.float64)


def test_dequantize_every_code_and_scale():
    """Every code with every scale byte, against the table of E4M3; compact scales.  Values are exact in bf16 but below its
    smallest subnormal's half steps, where the nearest is wanted: torch's own conversion from 64 bits through 32 (exact)."""
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()          # [256, 256]: a row a scale
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 8).cuda()
    got = mx.mxfp8_dequantize_2d(q, s, scale_layout=mx.SCALES_COMPACT).cpu()
    t = E4M3.clone()
    t[127] = float("nan")
    v = torch.cat([t, -t])[None] * torch.ldexp(torch.ones(256, dtype=torch.float64), torch.arange(256) - 127)[:, None]
    v[255] = float("nan")
    want = v.float().bfloat16()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
    assert torch.equal(torch.signbit(got) & ~got.isnan(), torch.signbit(want) & ~want.isnan())


@pytest.mark.parametrize("sizes,K", [([64], 96), ([32, 0, 96], 160), ([128, 256, 32], 128), ([0, 0, 64], 32),
                                     ([1056, 32, 160, 64], 1056)])
@pytest.mark.parametrize("direction", [mx.ROW, mx.COL])
@pytest.mark.parametrize("extra", [0, 64])
def test_dequantize_reads_what_quantize_writes(sizes, K, direction, extra):
    """Blocked scales with groups against compact ones (whose blocks are the same: sizes are multiples of 32), and rows
    past the last group, which are zeros."""
    M = sum(sizes) + (extra if len(sizes) > 1 else 0)
    x = randn((M, K), 1) * torch.pow(10.0, torch.rand((M, 1), device="cuda") * 4 - 2).bfloat16()
    offs = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    i = 0 if direction == mx.ROW else 2
    c = mx.mxfp8_quantize_2d(x, direction, mx.SCALES_COMPACT)
    want = mx.mxfp8_dequantize_2d(c[i], c[i + 1], direction, mx.SCALES_COMPACT)
    b = mx.mxfp8_quantize_2d(x, direction, mx.SCALES_BLOCKED, offs)
    got = mx.mxfp8_dequantize_2d(b[i], b[i + 1], direction, offs=offs)
    inside = (got if direction == mx.ROW else got.T)[:sum(sizes)]
    assert torch.equal(inside, (want if direction == mx.ROW else want.T)[:sum(sizes)])
    assert not (got if direction == mx.ROW else got.T)[sum(sizes):].any()
    # an element is off by half a step of E4M3 of its block's largest at most
    xs = x.double() if direction == mx.ROW else x.double().T
    top = xs.reshape(xs.shape[0], -1, 32).abs().amax(2).repeat_interleave(32, 1)
    err = (want.double() - xs).abs()
    assert (err <= torch.maximum(2.0 ** -4 * xs.abs(), 2.0 ** -17 * top) + (xs.abs() - 448 / 512 * top).clamp_min(0)).all()
    if len(sizes) == 1:
        g = mx.mxfp8_quantize_2d(x, direction, mx.SCALES_BLOCKED)
        assert torch.equal(mx.mxfp8_dequantize_2d(g[i], g[i + 1], direction), want)


# ---------------------------------------------------------------- activations kept in 8 bits
def kept(x):
    return mx.mxfp8_quantize_2d(x, mx.ROW, mx.SCALES_COMPACT)[:2]


def back(k):
    return mx.mxfp8_dequantize_2d(*k, mx.ROW, mx.SCALES_COMPACT)


@pytest.mark.parametrize("sizes,H", [([32], 32), ([64, 0, 96], 160), ([1056, 32, 160, 64], 1056), ([0, 512, 128], 4096)])
@pytest.mark.parametrize("extra", [0, 64])
@pytest.mark.parametrize("special", [False, True])
def test_swiglu_backward_from_8_bits_is_that_of_their_values(sizes, H, extra, special):
    M = sum(sizes) + (extra if len(sizes) > 1 else 0)
    offs = torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    dh, h1, h3 = randn((M, H), 1, 1e-2), randn((M, H), 2, 2.0), randn((M, H), 3)
    if special:
        h1[3, 5], h3[7, 9], h1[8] = float("inf"), float("nan"), 0.0
        h3[9], h1[10], dh[11] = 2.0 ** -133, torch.finfo(torch.bfloat16).max, 0.0
    k1, k3 = kept(h1), kept(h3)
    got = mx.mxfp8_swiglu_bwd_quantize_mxfp8(dh, k1, k3, offs)
    want = mx.mxfp8_swiglu_bwd_quantize(dh, back(k1), back(k3), offs)
    groups = mx.MoePlan(offs, offs, torch.zeros(M, dtype=torch.int32, device="cuda"),
                        torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
    for a, b in zip(got, want):
        same_copies(a, b, groups, H)


def expert_by_hand(x, ws, offs, d):
    """The expert's outputs and gradients over the public calls, its backward from the values that 8 bits of h1 and h3
    stand for."""
    both = mx.ROW | mx.COL
    xq, xs, xT, xTs = mx.mxfp8_quantize_2d(x, both, mx.SCALES_BLOCKED, offs)
    g, u, o = (mx.quantize_expert_weights(w) for w in ws)
    h1, h3, hq, hs, hT, hTs = mx.mxfp8_grouped_mm_swiglu_fwd(xq, xs, *g[:2], *u[:2], offs)
    y = mx.mxfp8_grouped_mm_fwd(hq, hs, *o[:2], offs)
    dq, ds, dT, dTs = mx.mxfp8_quantize_2d(d, both, mx.SCALES_BLOCKED, offs)
    dh = mx.mxfp8_grouped_mm_dgrad(dq, ds, o[2], o[3], offs)
    a, b = mx.mxfp8_swiglu_bwd_quantize(dh, back(kept(h1)), back(kept(h3)), offs)
    return (y, mx.mxfp8_grouped_mm_dgrad2(a[0], a[1], g[2], g[3], b[0], b[1], u[2], u[3], offs),
            mx.mxfp8_grouped_mm_wgrad(a[2], a[3], xT, xTs, offs), mx.mxfp8_grouped_mm_wgrad(b[2], b[3], xT, xTs, offs),
            mx.mxfp8_grouped_mm_wgrad(dT, dTs, hT, hTs, offs))


@pytest.mark.parametrize("sizes,D,H", [([64, 0, 96], 160, 352), ([512, 256], 256, 512)])
def test_expert_that_keeps_8_bits(sizes, D, H):
    M, offs = sum(sizes), torch.tensor(np.cumsum(sizes), dtype=torch.int32, device="cuda")
    x, ws, d = randn((M, D), 1), weights_of(len(sizes), D, H, 3), randn((M, D), 8, 1e-2)
    leaves = [t.clone().requires_grad_(True) for t in (x, *ws)]
    y = mx.mxfp8_swiglu_expert(*leaves, offs, checkpoint_mxfp8=True)
    for a, b in zip((y,) + torch.autograd.grad(y, leaves, d), expert_by_hand(x, ws, offs, d)):
        assert torch.equal(a, b)
    # the gradients that need none of h1 and h3 are those without the option
    w = ws[2].clone().requires_grad_(True)
    pair = [torch.autograd.grad(mx.mxfp8_swiglu_expert(x, *ws[:2], w, offs, checkpoint_mxfp8=k), w, d)[0] for k in (True, False)]
    assert torch.equal(*pair)


@pytest.mark.parametrize("T,E,D,H,k,route", [(70, 5, 352, 160, 3, dict(score="sigmoid", renormalize=True, scale=2.5)),
                                             (600, 8, 256, 512, 2, dict(score="softmax_all")), (1, 4, 32, 32, 2, {})])
def test_layer_that_keeps_8_bits(T, E, D, H, k, route):
    x, logits, ws = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda"), weights_of(E, D, H, 3)
    d = randn((T, D), 8, 1e-2)
    leaves = [t.clone().requires_grad_(True) for t in (x, logits, *ws)]
    out = mx.mxfp8_moe_swiglu(*leaves, k, checkpoint_mxfp8=True, **route)
    got = torch.autograd.grad(out, leaves, d)
    assert torch.equal(out, mx.mxfp8_moe_swiglu(x, logits, *ws, k, **route))
    # by hand: the steps, with the rows' gradients and the weights' from the kept values
    l = logits.clone().requires_grad_(True)
    e, w = mx.moe_route(l, k, **route)
    plan = mx.moe_plan(e, E, 32, exact=True)
    rows = mx.moe_gather(x, plan)
    dy = torch.autograd.grad(mx.moe_combine(y0 := torch.zeros_like(rows, requires_grad=True), plan, w.detach()), y0, d)[0]
    y, drows, *dws = expert_by_hand(rows, ws, plan.offs, dy)
    xg = x.clone().requires_grad_(True)
    dx = torch.autograd.grad(mx.moe_gather(xg, plan), xg, drows)[0]
    dl = torch.autograd.grad(mx.moe_combine(back(kept(y)), plan, w), l, d)[0]
    for a, b in zip(got, (dx, dl, *dws)):
        assert torch.equal(a, b)


def test_layer_that_keeps_8_bits_holds_less():
    """What lives between forward and backward is less by about 0.97 bytes a value of h1, h3 and the rows."""
    T, E, D, H, k = 4096, 4, 512, 1024, 2
    x, logits, ws = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda"), weights_of(E, D, H, 3)
    leaves = [t.requires_grad_(True) for t in (x, logits, *ws)]
    quads = [mx.quantize_expert_weights(w) for w in ws]
    held = []
    for keep in (False, True, False, True):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = mx.mxfp8_moe_swiglu(*leaves, k, w_mxfp8=quads, checkpoint_mxfp8=keep)
        held.append(torch.cuda.memory_allocated() - before)
        del out
    assert held[:2] == held[2:] and held[0] - held[1] >= 0.9 * T * k * (2 * H + D)


# ---------------------------------------------------------------- the layer
def weights_of(E, D, H, seed):
    return [randn((E, H, D), seed, D ** -0.5), randn((E, H, D), seed + 1, D ** -0.5), randn((E, D, H), seed + 2, H ** -0.5)]


def by_steps(x, logits, ws, k, route, exact=False):
    e, w = mx.moe_route(logits, k, **route)
    plan = mx.moe_plan(e, ws[0].shape[0], 32, exact=exact)
    y = mx.mxfp8_swiglu_expert(mx.moe_gather(x, plan), *ws, plan.offs, check_offsets=exact)
    return mx.moe_combine(y, plan, w)


LAYERS = [(1, 4, 32, 32, 2, {}), (50, 1, 64, 96, 1, dict(score="sigmoid")), (70, 5, 352, 160, 3, dict(score="sigmoid", renormalize=True, scale=2.5)),
          (600, 8, 256, 512, 2, dict(score="softmax_all")),
          (257, 64, 128, 64, 8, dict(score="sigmoid", groups=8, top_groups=3, renormalize=True))]


@pytest.mark.parametrize("T,E,D,H,k,route", LAYERS)
@pytest.mark.parametrize("masked", [False, True])
def test_layer_is_its_steps(T, E, D, H, k, route, masked):
    """Outputs and all five gradients of mxfp8_moe_swiglu, bit for bit those of its steps, also over a plan without rows past
    the last group, whose offsets are checked."""
    x, logits, ws = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda"), weights_of(E, D, H, 3)
    bias = None
    if masked:
        logits[T // 2:] = float("-inf")      # the end of a padded batch
        bias = torch.randn(E, generator=gen(9), device="cuda") * 0.1
        bias[0] = float("-inf") if E > 1 else 0.0   # an expert that takes nothing
        route = dict(route, bias=bias)
    d = randn((T, D), 8, 1e-2)
    results = []
    for f in (lambda a, b, c: mx.mxfp8_moe_swiglu(a, b, *c, k, **route), lambda a, b, c: by_steps(a, b, c, k, route),
              lambda a, b, c: by_steps(a, b, c, k, route, exact=T > 1 or not masked)):  # (no rows at all: not for the expert)
        leaves = [t.clone().requires_grad_(True) for t in (x, logits, *ws)]
        out = f(leaves[0], leaves[1], leaves[2:])
        results.append((out.detach(),) + torch.autograd.grad(out, leaves, d))
    for a, b, c in zip(*results):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b) and torch.equal(a, c)
    if T // 2 and not masked:
        assert all(r.any() for r in results[0][:2])


def test_layer_gradients_by_themselves():
    """Each gradient alone is the one that all of them together give; none where gradients are disabled."""
    T, E, D, H, k, route = LAYERS[2]
    x, logits, ws = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda"), weights_of(E, D, H, 3)
    d = randn((T, D), 8, 1e-2)

    def grads(which):
        leaves = [t.clone().requires_grad_(i in which) for i, t in enumerate((x, logits, *ws))]
        out = mx.mxfp8_moe_swiglu(*leaves, k, **route)
        return out.detach(), dict(zip(which, torch.autograd.grad(out, [leaves[i] for i in which], d)))

    out, every = grads(range(5))
    for i in range(5):
        o, g = grads([i])
        assert torch.equal(o, out) and torch.equal(g[i], every[i])
    with torch.no_grad():
        leaves = [t.clone().requires_grad_(True) for t in (x, logits, *ws)]
        o = mx.mxfp8_moe_swiglu(*leaves, k, **route)
        assert torch.equal(o, out) and not o.requires_grad
    status = mx.new_status()
    quads = [mx.quantize_expert_weights(w) for w in ws]
    assert torch.equal(mx.mxfp8_moe_swiglu(x, logits, *ws, k, w_mxfp8=quads, dev_status=status, **route), out)
    mx.read_status(status)
    cache = mx.Mxfp8WeightCache()
    for _ in range(2):
        assert torch.equal(mx.mxfp8_moe_swiglu(x, logits, *ws, k, weight_cache=cache, **route), out)
    assert cache.hits == 3


def test_layer_agrees_with_the_few_token_layer():
    """The same tokens through both serving paths.  They differ where h rounds to bf16 before it is quantized (2^-8
    relative) and in the order of sums: an element of h then lands on another E4M3 code (steps of 1/8 of it at most, 1/12
    on average) with probability 2^-8 / (1/12), so h and y move by sqrt(2^-8 / 12) = 0.018 in the mean square; twice that."""
    T, E, D, H, k = 33, 8, 256, 512, 2
    x, logits, ws = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda"), weights_of(E, D, H, 3)
    quads = [mx.quantize_expert_weights(w) for w in ws]
    few = mx.MxMoeTokens(*quads, k)(x, logits).double()
    many = mx.mxfp8_moe_swiglu(x, logits, *ws, k).double()
    assert (few - many).norm() <= 2 * (2.0 ** -8 / 12) ** 0.5 * few.norm()


def few_layers(E, D, H, bits, seed, top_k, **route):
    ws = weights_of(E, D, H, seed)
    quads = [mx.quantize_expert_weights(w) if bits == 8 else mx.mxfp4_quantize_3d_experts(w) for w in ws]
    return ws, quads, mx.MxMoeTokens(*quads, top_k, **route)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,E", [(1, 4), (5, 40), (64, 8)])
def test_few_token_layer_routed_by_moe_route(bits, T, E):
    """A bias of zeros changes nothing: the same experts, and with two of them the same sums in the same order, so the
    same bits, whichever kernel routes."""
    _, quads, routed = few_layers(E, 128, 64, bits, 3, 2, bias=torch.zeros(E, device="cuda"))
    x, logits = randn((T, 128), 1), torch.randn((T, E), generator=gen(2), device="cuda")
    want = mx.MxMoeTokens(*quads, 2)(x, logits)
    got = routed(x, logits)
    routed.check_status()
    assert torch.equal(got, want)
    assert torch.equal(routed(x, logits.bfloat16()), mx.MxMoeTokens(*quads, 2)(x, logits.bfloat16()))
    logits[0] = float("-inf")
    assert not routed(x, logits)[0].any()


@pytest.mark.parametrize("E,k,route", [
    (64, 8, dict(score="sigmoid", groups=8, top_groups=3, renormalize=True, scale=2.5)),
    (6, 2, dict(score="softmax_all", renormalize=True)), (12, 3, dict(score="softmax", groups=4, top_groups=2, group_score="max")),
    (8, 1, dict(score="sigmoid", scale=0.5))])
@pytest.mark.parametrize("with_bias", [True, False])
def test_few_token_layer_with_options_agrees_with_the_layer(E, k, route, with_bias):
    """Both serving paths with the same routing; they differ as in test_layer_agrees_with_the_few_token_layer."""
    D, H, T = 256, 512, 20
    bias = torch.randn(E, generator=gen(9), device="cuda") * 0.2 if with_bias else None
    ws, quads, few = few_layers(E, D, H, 8, 3, k, bias=bias, **route)
    x, logits = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda")
    logits[3] = float("-inf")
    a = few(x, logits).double()
    b = mx.mxfp8_moe_swiglu(x, logits, *ws, k, bias=bias, **route).double()
    assert (a - b).norm() <= 2 * (2.0 ** -8 / 12) ** 0.5 * b.norm() and not a[3].any()
    if with_bias:  # the layer reads the bias at each call, captured ones too
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = few(x, logits)
        bias.copy_(-bias)
        graph.replay()
        assert torch.equal(held, few(x, logits)) and not torch.equal(held.double(), a)
        few.check_status()


def test_layer_of_no_tokens():
    ws = [w.requires_grad_(True) for w in weights_of(4, 64, 32, 3)]
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    l = torch.zeros((0, 4), device="cuda", requires_grad=True)
    out = mx.mxfp8_moe_swiglu(x, l, *ws, 2)
    g = torch.autograd.grad(out.sum(), [x, l, *ws])
    assert out.shape == (0, 64) and [t.shape for t in g] == [t.shape for t in (x, l, *ws)]
    assert not any(t.any() for t in g[2:])


def test_layer_captured_forward_and_backward():
    """Two captured training steps replayed on streams of their own, beside an eager one."""
    T, E, D, H, k, route = LAYERS[2]
    ws = weights_of(E, D, H, 3)
    steps = []
    for seed in (1, 2):
        x, logits, d = randn((T, D), seed), torch.randn((T, E), generator=gen(seed), device="cuda"), randn((T, D), 8)

        def step(x=x, logits=logits, d=d):
            leaves = [t.detach().requires_grad_(True) for t in (x, logits, *ws)]
            out = mx.mxfp8_moe_swiglu(*leaves, k, **route)
            return (out.detach(),) + torch.autograd.grad(out, leaves, d)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        steps.append((graph, step, held, x, logits))
    for seed in (5, 6):
        for i, (_, _, _, x, logits) in enumerate(steps):
            x.copy_(randn((T, D), seed + i))
            logits.copy_(torch.randn((T, E), generator=gen(seed + i), device="cuda"))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in steps]
        for s, (graph, *_) in zip(streams, steps):
            with torch.cuda.stream(s):
                graph.replay()
        eager = steps[0][1]()
        torch.cuda.synchronize()
        for got, want in zip(steps[0][2], eager):
            assert torch.equal(got, want)
        for got, want in zip(steps[1][2], steps[1][1]()):
            assert torch.equal(got, want)


def test_on_another_stream():
    s = torch.cuda.Stream()
    T, E, D, H, k, route = LAYERS[3]
    x, logits, ws = randn((T, D), 1), torch.randn((T, E), generator=gen(2), device="cuda"), weights_of(E, D, H, 3)
    want = mx.mxfp8_moe_swiglu(x, logits, *ws, k, **route)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(3):
            got = mx.mxfp8_moe_swiglu(x, logits, *ws, k, **route)
    s.synchronize()
    assert torch.equal(got, want)
