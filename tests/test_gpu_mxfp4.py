"""MXFP4 quantization, its inverse, the 4-bit grouped product and its gradients against a plain 64-bit
implementation.

Codes and scales of a bf16 input are exact (the scale is a power of two, the rounding is on exact values),
so they are compared byte for byte, padding included.  For silu(h1) * h3 the fp32 value is within a few
2^-24 of the exact one (expf 2 ulp, one division, two products, one sum: under 8 half-steps), so a code may differ only where
the exact value is that close to a rounding border, and a scale only where the amax is that close to a power of two."""
import numpy as np
import pytest
import torch

from mxfp8_precision_moe_gb300 import synth
from tests import _mx4ref as ref
from tests._util import f64, require_gpu, sizes_to_ends, u8

pytestmark = pytest.mark.gpu

SIZES = [([1], 32), ([127], 160), ([128], 256), ([129], 288), ([0, 3, 0, 250, 1], 416), ([300, 5], 1056)]


@pytest.fixture(scope="module")
def mx():
    require_gpu()
    import mxfp8_precision_moe_gb300 as m

    m.load()
    return m


def offs_of(sizes):
    return torch.tensor(sizes_to_ends(sizes).astype(np.int32), device="cuda")


def hard_rows(M, K, seed):
    """Rows of very different magnitude, exact ties, zeros, the smallest and the largest bf16 values."""
    x = synth.log_uniform_rows(M, K, seed).float()
    g = torch.Generator().manual_seed(seed + 1)
    for r in range(0, M, 5):
        kind = (r // 5) % 6
        if kind == 0:
            x[r] = 0
        elif kind == 1:   # ties: halves of a step at every magnitude of the grid
            x[r] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])[torch.randint(0, 8, (K,), generator=g)]
        elif kind == 2:
            x[r] = torch.randn(K, generator=g) * 2.0 ** -126
        elif kind == 3:   # bf16 subnormals
            x[r] = torch.randint(-127, 128, (K,), generator=g).float() * 2.0 ** -133
        elif kind == 4:
            x[r] = torch.randn(K, generator=g).sign() * 3.3e38
        else:
            x[r, ::2] *= -1e-20
    return x.to(torch.bfloat16)


def check_codes(q, s, x64, ends, blocked=True):
    code, sc = ref.encode(x64, 4)
    assert np.array_equal(u8(q), ref.pack(code))
    if blocked:
        t = ref.tiles(sc, ends)
        assert np.array_equal(u8(s).reshape(-1)[:t.size], t)
    else:
        assert np.array_equal(u8(s), sc)


@pytest.mark.parametrize("sizes,K", SIZES)
def test_quantize_2d_blocked_groups(mx, sizes, K):
    x = hard_rows(sum(sizes), K, seed=K + len(sizes))
    q, s = mx.mxfp4_quantize_2d(x.cuda(), offs=offs_of(sizes))
    check_codes(q, s, f64(x), sizes_to_ends(sizes))
    back = mx.mxfp4_dequantize_2d(q, s, offs=offs_of(sizes))
    assert np.array_equal(f64(back), ref.mx_value(f64(x), 4))


@pytest.mark.parametrize("M,K", [(1, 32), (33, 96), (130, 384)])
@pytest.mark.parametrize("layout", [0, 1])
def test_quantize_2d_one_group(mx, M, K, layout):
    x = hard_rows(M, K, seed=M)
    q, s = mx.mxfp4_quantize_2d(x.cuda(), layout)
    check_codes(q, s, f64(x), None, blocked=layout == 1)
    assert np.array_equal(f64(mx.mxfp4_dequantize_2d(q, s, layout)), ref.mx_value(f64(x), 4))


@pytest.mark.parametrize("G,N,K", [(1, 32, 32), (3, 130, 160), (2, 256, 288)])
@pytest.mark.parametrize("layout", [0, 1])
def test_quantize_experts(mx, G, N, K, layout):
    w = hard_rows(G * N, K, seed=N).reshape(G, N, K)
    q, s = mx.mxfp4_quantize_3d_experts(w.cuda(), layout)
    for g in range(G):
        check_codes(q[g], s[g], f64(w[g]), None, blocked=layout == 1)
    assert np.array_equal(f64(mx.mxfp4_dequantize_3d_experts(q, s, layout)), ref.mx_value(f64(w), 4))


def test_nonfinite_blocks(mx):
    x = synth.randn_bf16((40, 128), 1.0, seed=3)
    x[0, 5], x[1, 40], x[2, 70], x[39, 127] = float("nan"), float("inf"), -float("inf"), float("nan")
    q, s = mx.mxfp4_quantize_2d(x.cuda())
    check_codes(q, s, f64(x), None)
    back = f64(mx.mxfp4_dequantize_2d(q, s))
    want = ref.mx_value(f64(x), 4)
    assert np.array_equal(np.isnan(back), np.isnan(want)) and np.isnan(back).sum() == 4 * 32
    assert np.array_equal(back[~np.isnan(back)], want[~np.isnan(want)])


@pytest.mark.parametrize("sizes,K", [([32], 32), ([96, 0, 160, 32], 288), ([128], 160), ([256, 64, 32], 416), ([544], 1056)])
def test_quantize_2d_with_mxfp8_columns(mx, sizes, K):
    """Row-wise MXFP4 and column-wise MXFP8 copies of one read: exact, the blocked layouts' padding included."""
    M, ends = sum(sizes), sizes_to_ends(sizes)
    x = hard_rows(M, K, seed=K)
    x[3, 7], x[M - 1, K - 1], x[M - 9, 0] = float("nan"), float("inf"), -float("inf")
    q, s, qT, sT = mx.mxfp4_quantize_2d_mxfp8_cols(x.cuda(), offs_of(sizes))
    check_codes(q, s, f64(x), ends)
    code, sc = ref.encode(f64(x).T, 8)
    assert np.array_equal(u8(qT), code)
    # a group's block columns start on a fresh tile of four
    pad, start = [], 0
    for n in sizes:
        block = np.zeros((K, (n + 127) // 128 * 4), np.uint8)
        block[:, :n // 32] = sc[:, start // 32:(start + n) // 32]
        pad.append(block)
        start += n
    t = ref.tiles(np.concatenate(pad, 1))
    assert np.array_equal(u8(sT).reshape(-1)[:t.size], t)
    if len(sizes) == 1:
        for a, b in zip(mx.mxfp4_quantize_2d_mxfp8_cols(x.cuda()), (q, s, qT, sT)):
            assert a.shape == b.shape and torch.equal(a.flatten()[:512], b.flatten()[:512])


@pytest.mark.parametrize("G,N,K", [(1, 32, 32), (3, 160, 288), (2, 256, 160)])
def test_quantize_experts_with_mxfp8_columns(mx, G, N, K):
    w = hard_rows(G * N, K, seed=N + 1).reshape(G, N, K)
    w[G - 1, 3, 7], w[0, N - 1, K - 1] = float("nan"), -float("inf")
    q, s, qT, sT = mx.mxfp4_quantize_3d_experts_mxfp8_cols(w.cuda())
    for g in range(G):
        check_codes(q[g], s[g], f64(w[g]), None)
        code, sc = ref.encode(f64(w[g]).T, 8)
        assert np.array_equal(u8(qT[g]), code)
        assert np.array_equal(u8(sT[g]), ref.tiles(sc))


def test_gradient_with_weights_kept_quantized(mx):
    """The same gradients whether W's MXFP4 copy is passed in or made on the way."""
    A, W = synth.randn_bf16((160, 96), 1.0, seed=3).cuda(), synth.randn_bf16((2, 64, 96), 0.1, seed=4).cuda()
    got = []
    for q in (None, mx.mxfp4_quantize_3d_experts(W)):
        a, w = A.clone().requires_grad_(True), W.clone().requires_grad_(True)
        mx.to_mxfp4_then_scaled_grouped_mm(a, w, offs_of([32, 128]), w_mxfp4=q).float().square().sum().backward()
        got.append((a.grad, w.grad))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_empty(mx):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    q, s = mx.mxfp4_quantize_2d(x)
    assert q.shape == (0, 32) and mx.mxfp4_dequantize_2d(q, s).shape == (0, 64)
    w = torch.zeros((1, 64, 32), dtype=torch.uint8, device="cuda")
    ws = torch.zeros((1, 512), dtype=torch.uint8, device="cuda")
    assert mx.mxfp4_grouped_mm_fwd(q, s, w, ws, offs_of([0])).shape == (0, 64)
    h, o = mx.mxfp4_swiglu_quantize(x, x, offs=offs_of([0, 0]))
    assert h.shape == (0, 32)
    a = x.clone().requires_grad_(True)
    W = torch.ones((2, 64, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    mx.to_mxfp4_then_scaled_grouped_mm(a, W, offs_of([0, 0])).sum().backward()
    assert a.grad.shape == (0, 64) and not W.grad.any()


@pytest.mark.parametrize("sizes,K", SIZES)
def test_swiglu_quantize(mx, sizes, K):
    M = sum(sizes)
    h1, h3 = synth.randn_bf16((M, K), 2.0, seed=K), synth.randn_bf16((M, K), 1.0, seed=K + 1)
    if M > 2:
        h1[1, :32] = -200.0  # silu underflows to a tiny number
        h1[2, :40], h3[2, :40] = 0.0, 0.0
    q, s = mx.mxfp4_swiglu_quantize(h1.cuda(), h3.cuda(), offs=offs_of(sizes))
    h = ref.silu(f64(h1)) * f64(h3)
    err = 2.0 ** -21 * np.abs(h)
    lo, hi = np.abs(h) - err, np.abs(h) + err
    code, sc = ref.encode(h, 4)
    b = lambda v: v.reshape(M, -1, 32)
    # blocks whose amax is clear of a power of two have the reference's scale
    clear = np.floor(np.log2(np.maximum(b(lo).max(-1), 1e-300))) == np.floor(np.log2(np.maximum(b(hi).max(-1), 1e-300)))
    t = ref.tiles(sc, sizes_to_ends(sizes))
    same = u8(s)[:t.size] == ref.tiles(np.where(clear, sc, 0), sizes_to_ends(sizes))
    loose = ref.tiles((~clear).astype(np.uint8), sizes_to_ends(sizes)).astype(bool)
    assert (same | loose).all() and clear.mean() > 0.99
    # and codes, wherever rounding the two ends of the error interval agrees
    f = np.ldexp(1.0, 127 - sc.astype(np.int64))[..., None]
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    firm = np.searchsorted(mids, b(lo) * f) == np.searchsorted(mids, b(hi) * f)
    firm &= clear[..., None]
    # values this small may flush or round to zero on either side of a code: the sign of zero is not compared
    got = b(ref.unpack(u8(q)))
    want = b(code)
    agree = (got == want) | (((got & 7) == 0) & ((want & 7) == 0))
    assert agree[firm].all() and firm.mean() > 0.99


def test_swiglu_extremes(mx):
    """Blocks of one pair each: exponentials that overflow or vanish, subnormals, the largest values, infinities, NaN."""
    one = [0.0, -0.0, 1e-40, 2.0 ** -126, 0.3, 20.0, 87.0, 90.0, 1e30, 3.3e38]
    gate = torch.tensor([s * v for v in one for s in (1, -1)] + [-86.5, -87.5, -88.5, -100.0, -1000.0]).bfloat16()
    up = torch.tensor([1.0, -3.0, 1e-30, 7e29, 0.0]).bfloat16()
    h1 = gate.repeat_interleave(len(up)).repeat_interleave(32).reshape(-1, 32).cuda()
    h3 = up.repeat(len(gate)).repeat_interleave(32).reshape(-1, 32).cuda()
    q, s = mx.mxfp4_swiglu_quantize(h1, h3, mx.SCALES_COMPACT)
    # the formula in 32 bits: e^-a overflows above 88.73, as it is meant to
    a = f64(h1).astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore", under="ignore", divide="ignore"):
        silu = (a / (1 + np.exp(-a).astype(np.float32))).astype(np.float64)
        v = silu * f64(h3)
        big = np.abs(v) > 3.4e38
        v[big] = np.copysign(np.inf, v[big])
        code, sc = ref.encode(v, 4)
        firm = np.ones(len(v), bool)
        for d in (1 - 8 * 2.0 ** -24, 1 + 8 * 2.0 ** -24):
            c, x = ref.encode(v * d, 4)
            firm &= (c == code).all(1) & (x == sc).all(1)
    firm &= (np.abs(v) > 2.0 ** -125).all(1) | (v == 0).all(1)   # below, the 32-bit product is rounded to a subnormal
    got = ref.unpack(u8(q))
    same = (got == code) | (((got & 7) == 0) & ((code & 7) == 0))
    assert firm.sum() > 60 and same[firm].all() and np.array_equal(u8(s)[firm], sc[firm])
    bad = torch.tensor([float("inf"), -float("inf"), float("nan"), 2.0]).bfloat16().repeat_interleave(32).reshape(-1, 32)
    other = torch.tensor([2.0, 2.0, 2.0, -float("inf")]).bfloat16().repeat_interleave(32).reshape(-1, 32)
    q, s = mx.mxfp4_swiglu_quantize(bad.cuda(), other.cuda(), mx.SCALES_COMPACT)
    assert (u8(s) == 255).all() and ((ref.unpack(u8(q)) & 7) == 7).all()
    assert (ref.unpack(u8(q))[0] == 7).all() and (ref.unpack(u8(q))[3] == 15).all()


def product_bound(a, w, K):
    """bf16 rounding of the result, and a 32-bit sum of K exact products in any order."""
    return lambda o: 2.0 ** -8 * np.abs(o) + K * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)


@pytest.mark.parametrize("sizes,N,K", [
    ([1], 32, 32), ([5, 0, 130], 96, 64), ([128, 128], 128, 256), ([257], 288, 160), ([0, 0, 1, 300, 0], 512, 416),
    ([600, 40], 800, 1312), ([33] * 20, 256, 96),
])
def test_product(mx, sizes, N, K):
    M, G = sum(sizes), len(sizes)
    x = synth.log_uniform_rows(M, K, seed=N)
    w = synth.randn_bf16((G, N, K), 0.3, seed=K)
    offs = offs_of(sizes)
    aq, as_ = mx.mxfp4_quantize_2d(x.cuda(), offs=offs)
    wq, ws = mx.mxfp4_quantize_3d_experts(w.cuda())
    st = mx.new_status()
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_grouped_mm_fwd(aq, as_, wq, ws, offs, out=out, dev_status=st)
    mx.read_status(st)
    a, o, start = ref.mx_value(f64(x), 4), f64(out), 0
    for g, n in enumerate(sizes):
        wv = ref.mx_value(f64(w[g]), 4)
        av = a[start:start + n]
        want = av @ wv.T
        assert (np.abs(o[start:start + n] - want) <= product_bound(av, wv, K)(want)).all()
        start += n


@pytest.mark.parametrize("sizes,N,K", [
    ([300] + [0] * 7, 96, 288), ([200, 1, 31, 32, 33, 0, 2], 288, 160), ([64, 64], 512, 544), ([97, 2, 3], 256, 1056),
    ([1, 0] * 150, 32, 64), ([128, 0], 64, 96), ([129] + [1] * 6, 64, 96),
])
def test_product_of_short_groups(mx, sizes, N, K):
    """64 rows a group and less on average, though single groups may be long (and more than 256 groups)."""
    test_product(mx, sizes, N, K)


def test_product_keeps_nonfinite_blocks_to_their_rows(mx):
    """A NaN in one token or one expert reaches that token's rows and that expert's columns only."""
    sizes, N, K = [40, 50, 60], 64, 320
    x, w = synth.randn_bf16((150, K), 1.0, seed=1), synth.randn_bf16((3, N, K), 1.0, seed=2)
    x[45, 300], w[2, 7, 0] = float("nan"), float("inf")
    offs = offs_of(sizes)
    out = f64(mx.mxfp4_grouped_mm_fwd(*mx.mxfp4_quantize_2d(x.cuda(), offs=offs),
                                      *mx.mxfp4_quantize_3d_experts(w.cuda()), offs))
    want = np.zeros((150, N), bool)
    want[45] = True
    want[90:, 7] = True
    assert np.array_equal(np.isnan(out), want)


def test_product_repeats_and_runs_on_another_stream(mx):
    sizes, N, K = [200, 313], 384, 512
    x, w = synth.randn_bf16((513, K), 1.0, seed=1).cuda(), synth.randn_bf16((2, N, K), 1.0, seed=2).cuda()
    offs = offs_of(sizes)
    one = mx.mxfp4_grouped_mm_fwd(*mx.mxfp4_quantize_2d(x, offs=offs), *mx.mxfp4_quantize_3d_experts(w), offs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two = mx.mxfp4_grouped_mm_fwd(*mx.mxfp4_quantize_2d(x, offs=offs), *mx.mxfp4_quantize_3d_experts(w), offs)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(one, two)


@pytest.mark.parametrize("sizes,N,K", [([32], 32, 32), ([96, 0, 160, 32], 160, 288), ([256, 64], 512, 256)])
def test_differentiable_product(mx, sizes, N, K):
    M, G = sum(sizes), len(sizes)
    A, W = synth.randn_bf16((M, K), 1.0, seed=3), synth.randn_bf16((G, N, K), 0.1, seed=4)
    dOut = synth.randn_bf16((M, N), 1e-3, seed=5)
    a, w = A.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    out = mx.to_mxfp4_then_scaled_grouped_mm(a, w, offs_of(sizes))
    out.backward(dOut.cuda())
    o, dA, dW, start = f64(out), f64(a.grad), f64(w.grad), 0
    for g, n in enumerate(sizes):
        Ag, Wg, Dg = f64(A[start:start + n]), f64(W[g]), f64(dOut[start:start + n])
        pairs = [(o[start:start + n], ref.mx_value(Ag, 4), ref.mx_value(Wg, 4), K),
                 (dA[start:start + n], ref.mx_value(Dg, 8), ref.mx_value(Wg.T.copy(), 8), N)]
        if n:
            pairs.append((dW[g], ref.mx_value(Dg.T.copy(), 8), ref.mx_value(Ag.T.copy(), 8), n))
        else:
            assert not dW[g].any()
        for got, l, r, length in pairs:
            want = l @ r.T
            assert (np.abs(got - want) <= product_bound(l, r, length)(want)).all()
        start += n


def test_gradients_follow_differences(mx):
    """The gradient is that of the unquantized product (quantization counts as the identity): along the
    direction d of steepest ascent the exact product changes by |d|^2, measured by a central difference,
    and the gradient's inner product with d is off by at most its relative error, 2^-4 for each of the two
    MXFP8 operands of a product."""
    sizes, N, K = [64, 96], 128, 192
    A, W = synth.randn_bf16((160, K), 1.0, seed=6), synth.randn_bf16((2, N, K), 0.1, seed=7)
    dOut = synth.randn_bf16((160, N), 1.0, seed=8)
    a, w = A.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    mx.to_mxfp4_then_scaled_grouped_mm(a, w, offs_of(sizes)).backward(dOut.cuda())
    groups = [slice(0, 64), slice(64, 160)]
    A64, W64, D64 = f64(A), f64(W), f64(dOut)

    def loss(x, y):
        return sum(float((D64[s] * (x[s] @ y[g].T)).sum()) for g, s in enumerate(groups))

    dA = np.concatenate([D64[s] @ W64[g] for g, s in enumerate(groups)])
    dW = np.stack([D64[s].T @ A64[s] for s in groups])
    h = 1e-3
    for got, d, step in ((f64(a.grad), dA, lambda k: loss(A64 + k * dA, W64)),
                         (f64(w.grad), dW, lambda k: loss(A64, W64 + k * dW))):
        diff = (step(h) - step(-h)) / (2 * h)
        assert abs(diff - float((got * d).sum())) <= 2 * 2.0 ** -4 * np.linalg.norm(d) ** 2


def test_only_what_needs_a_gradient(mx):
    A, W = synth.randn_bf16((50, 64), 1.0, seed=3).cuda(), synth.randn_bf16((2, 64, 64), 0.1, seed=4).cuda()
    offs = offs_of([17, 33])
    a = A.clone().requires_grad_(True)
    mx.to_mxfp4_then_scaled_grouped_mm(a, W, offs).sum().backward()   # any group sizes without dW
    assert a.grad is not None
    q = mx.mxfp4_quantize_3d_experts(W)
    assert torch.equal(mx.to_mxfp4_then_scaled_grouped_mm(A, W, offs, w_mxfp4=q),
                       mx.to_mxfp4_then_scaled_grouped_mm(A, W, offs))
    with pytest.raises(mx.Mxfp8Error):
        mx.to_mxfp4_then_scaled_grouped_mm(A, W, offs_of([17, 30]))  # does not end at M
