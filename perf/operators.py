"""Cases of the 4-bit routed-expert operators and of the routed layer for a few tokens.

Five kinds of case:

* ``quantize``  MXFP4 quantization of a token matrix [M, K] in ragged groups, or of expert weights
  [G, N, K], and the values its codes and scales stand for (quantize, then dequantize).
* ``swiglu``    the same for h = silu(h1) * h3 of two bf16 matrices, between the up and the down product.
* ``product``   the grouped product of MXFP4 tokens and MXFP4 expert weights, bf16 out.
* ``train``     the differentiable product: quantization and product in 4 bits forward, the gradients of the
  tokens and of the weights through MXFP8.
* ``tokens``    the routed SwiGLU layer for 1 .. 64 tokens: top-k over the router's logits, gate and up,
  SwiGLU, down, weighted sum; the expert weights in MXFP8 or MXFP4.

MX blocks hold 32 elements along the contraction with one power of two 2^e, e = floor(log2 amax) - emax,
clamped at -127; elements are E2M1 (emax 2, largest 6) or E4M3 (emax 8, largest 448), rounded to nearest
even and saturated.
"""
import math

import torch

own = False

BLOCK = 32
EMAX = {4: 2, 8: 8}
LARGEST = {4: 6.0, 8: 448.0}
LEAST_EXP = {4: 0, 8: -6}      # exponent of the smallest normal element
MANTISSA = {4: 1, 8: 3}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a short ragged batch on its way into the 4-bit product: launch latency counts
        dict(name="quantize_small", kind="quantize", form="tokens", M=250, K=256, G=3),
        # the expert weights of a layer, quantized once for serving
        dict(name="quantize_experts", kind="quantize", form="experts", G=16, N=8192, K=5120),
        # SwiGLU between the products of a few dozen tokens
        dict(name="swiglu_small", kind="swiglu", M=77, K=1056, G=4),
        # SwiGLU of a whole training-size token list, Zipf groups
        dict(name="swiglu_scout", kind="swiglu", M=16384, K=8192, G=8),
        # the smallest product
        dict(name="product_tiny", kind="product", M=256, N=128, K=256, G=2, skew=0.0),
        # a prompt's tokens through one projection of 8 experts, Zipf groups
        dict(name="product_scout", kind="product", M=16384, N=8192, K=5120, G=8, skew=1.1),
        # a fine-tuning step's product with its gradients at a small size
        dict(name="train_small", kind="train", M=1024, N=512, K=768, G=4, skew=1.1),
        # forward and backward over imbalanced fine-grained experts
        dict(name="train_imbalanced", kind="train", M=32768, N=2048, K=7168, G=16, skew=1.1),
        # one token of one request: the weights of its expert are all there is to read
        dict(name="tokens1_fp8", kind="tokens", T=1, E=16, D=5120, H=8192, top_k=1, bits=8, score="sigmoid"),
        dict(name="tokens1_fp4", kind="tokens", T=1, E=16, D=5120, H=8192, top_k=1, bits=4, score="sigmoid"),
        # odd widths and a few tokens of a small layer
        dict(name="tokens5_odd", kind="tokens", T=5, E=6, D=352, H=160, top_k=2, bits=8, score="softmax"),
        # a decoding batch over fine-grained experts: nearly all of them are read
        dict(name="tokens64_fp4", kind="tokens", T=64, E=16, D=7168, H=2048, top_k=4, bits=4, score="softmax"),
    ]


def _spread(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // multiple * multiple))


def draw(rng):
    kind = rng.choice(("quantize", "quantize", "swiglu", "product", "product", "train", "tokens", "tokens", "tokens"))
    if kind == "quantize" and rng.random() < 0.4:
        return dict(kind=kind, form="experts", G=rng.randint(1, 16), N=_spread(rng, 32, 8192),
                    K=_spread(rng, 32, 5120, 32))
    if kind in ("quantize", "swiglu"):
        c = dict(kind=kind, M=_spread(rng, 1, 16384), K=_spread(rng, 32, 8192, 32), G=rng.randint(1, 16))
        if kind == "quantize":
            c["form"] = "tokens"
        return c
    if kind in ("product", "train"):
        m = 32 if kind == "train" else 1
        return dict(kind=kind, M=_spread(rng, m, 16384, m), N=_spread(rng, 32, 2048, 32), K=_spread(rng, 32, 7168, 32),
                    G=rng.randint(1, 16), skew=round(rng.uniform(0, 1.5), 2))
    E = rng.choice((4, 6, 8, 13, 16))
    return dict(kind=kind, T=_spread(rng, 1, 64), E=E, D=_spread(rng, 64, 7168, 32), H=_spread(rng, 32, 2048, 32),
                top_k=rng.randint(1, min(4, E)), bits=rng.choice((4, 8)), score=rng.choice(("softmax", "sigmoid")))


def _sizes(M, G, skew, seed, multiple):
    """Group sizes that sum to M, drawn with p_i ~ i^-skew (empty groups occur)."""
    g = torch.Generator().manual_seed(seed)
    p = torch.arange(1, G + 1, dtype=torch.float64) ** -skew
    pick = torch.multinomial(p, M // multiple, replacement=True, generator=g) if M else torch.zeros(0, dtype=torch.long)
    return [int(c) * multiple for c in torch.bincount(pick, minlength=G)]


# ---------------------------------------------------------------- layouts
def _padded_rows(sizes, device):
    """For each row, its place in the layout whose groups start at multiples of 128."""
    t = torch.tensor(sizes, device=device)
    pads = (t + 127) // 128 * 128
    return torch.arange(int(sum(sizes)), device=device) + torch.repeat_interleave(
        (torch.cumsum(pads, 0) - pads) - (torch.cumsum(t, 0) - t), t, output_size=int(sum(sizes)))


def _to_tiles(s):
    """Scale bytes [..., R, C] -> 128 x 4 tiles, flat per matrix; what is past the matrix is 0."""
    R, C = s.shape[-2:]
    rb, cb = -(-R // 128), -(-C // 4)
    full = torch.zeros(s.shape[:-2] + (rb * 128, cb * 4), dtype=torch.uint8, device=s.device)
    full[..., :R, :C] = s
    t = full.reshape(s.shape[:-2] + (rb, 4, 32, cb, 4))
    n = t.dim()
    return t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).reshape(s.shape[:-2] + (-1,)).contiguous()


def _from_tiles(flat, R, C):
    """The scale bytes [..., R, C] out of their tiles."""
    rb, cb = -(-R // 128), -(-C // 4)
    t = flat[..., :rb * cb * 512].reshape(flat.shape[:-1] + (rb, cb, 32, 4, 4))
    n = t.dim()
    return t.permute(*range(n - 5), n - 5, n - 2, n - 3, n - 4, n - 1).reshape(
        flat.shape[:-1] + (rb * 128, cb * 4))[..., :R, :C]


# ---------------------------------------------------------------- the plain form's arithmetic (32 bits)
def _pow2(e):
    """2^e, exactly, for -127 <= e <= 127."""
    return torch.where(e < -126, 1 << 22, (e + 127).to(torch.int32) << 23).to(torch.int32).view(torch.float32)


def _exponent(amax, bits):
    """floor(log2 amax) - emax, at least -127."""
    return torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - EMAX[bits]).clamp_min(-127), -127)


def _round(v, bits):
    """v to the nearest element, ties to even, saturated; v in 32 bits."""
    a = v.abs().clamp_max(LARGEST[bits])
    step = _pow2((torch.frexp(a)[1] - 1).clamp_min(LEAST_EXP[bits]) - MANTISSA[bits])
    return torch.copysign(torch.round(a / step) * step, v)


def _mx(x, bits):
    """x [..., C] in 32 bits -> (elements [..., C], exponents [..., C / 32])."""
    b = x.unflatten(-1, (-1, BLOCK))
    e = _exponent(b.abs().amax(-1), bits)
    return _round(b * _pow2(-e).unsqueeze(-1), bits).flatten(-2), e


def _value(v, e):
    return (v.unflatten(-1, (-1, BLOCK)) * _pow2(e).unsqueeze(-1)).flatten(-2)


def _mx_value(x, bits):
    return _value(*_mx(x, bits))


def _codes(v, bits):
    """Elements -> their codes, as the tensor cores take them: E4M3 a byte each, E2M1 two a byte, even ones low."""
    if bits == 8:
        return v.to(torch.float8_e4m3fn).view(torch.uint8)
    a = v.abs()
    m = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = m | (torch.signbit(v).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _elements(q, bits):
    if bits == 8:
        return q.view(torch.float8_e4m3fn).float()
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    m = (c & 7).float()
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    return torch.where(c >= 8, -a, a)


def _decode(q, s_flat, bits, rows=None):
    """Codes [..., R, C] and tiled scales -> 32-bit values; rows: places of grouped rows in the layout."""
    v = _elements(q, bits)
    R, C = v.shape[-2:]
    if rows is None:
        s = _from_tiles(s_flat, R, C // BLOCK)
    else:
        total = s_flat.numel() // (-(-C // 128) * 4)
        s = _from_tiles(s_flat, total, C // BLOCK)[rows]
    return _value(v, s.int() - 127)


# ---------------------------------------------------------------- inputs
def _randn(shape, std, g):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _weights(shape, std, bits, g):
    """Quantized expert weights as a serving program holds them: codes and tiled scales, expert by expert."""
    q = torch.empty(shape[:2] + (shape[2] * bits // 8,), dtype=torch.uint8, device="cuda")
    s = []
    for i in range(shape[0]):
        v, e = _mx(_randn(shape[1:], std, g).float(), bits)
        q[i] = _codes(v, bits)
        s.append(_to_tiles((e + 127).to(torch.uint8)))
    return q, torch.stack(s)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    st = dict(case=case)
    if kind == "tokens":
        T, E, D, H = case["T"], case["E"], case["D"], case["H"]
        st["x"] = _randn((T, D), 1.0, g)
        st["logits"] = torch.randn((T, E), generator=g, device="cuda")
        st["gate"] = _weights((E, H, D), 0.02, case["bits"], g)
        st["up"] = _weights((E, H, D), 0.02, case["bits"], g)
        st["down"] = _weights((E, D, H), 0.02, case["bits"], g)
        if own:
            import mxfp8_precision_moe_gb300 as mx

            st["layer"] = mx.MxMoeTokens(st["gate"], st["up"], st["down"], case["top_k"], score=case["score"])
        return st
    if kind == "quantize" and case["form"] == "experts":
        st["x"] = _randn((case["G"], case["N"], case["K"]), 0.02, g)
        return st
    M, K, G = case["M"], case["K"], case["G"]
    sizes = _sizes(M, G, case.get("skew", 1.1), seed, 32 if kind == "train" else 1)
    st["sizes"] = sizes
    st["offs"] = torch.tensor(sizes).cumsum(0).to(torch.int32).cuda()
    if kind == "quantize":
        # activations whose rows differ in magnitude
        st["x"] = (torch.randn((M, K), generator=g, device="cuda")
                   * torch.pow(10.0, torch.rand((M, 1), generator=g, device="cuda") * 4 - 2)).to(torch.bfloat16)
    elif kind == "swiglu":
        st["h1"], st["h3"] = _randn((M, K), 1.5, g), _randn((M, K), 1.0, g)
    elif kind == "train":
        st["A"], st["W"] = _randn((M, K), 1.0, g), _randn((G, case["N"], K), 0.02, g)
        st["dOut"] = _randn((M, case["N"]), 1e-3, g)
    else:
        v, e = _mx(_randn((M, K), 1.0, g).float(), 4)
        st["rows"] = _padded_rows(sizes, "cuda")
        s = torch.zeros(((-(-M // 128) + G) * 128, K // BLOCK), dtype=torch.uint8, device="cuda")
        s[st["rows"]] = (e + 127).to(torch.uint8)
        st["a_q"], st["a_s"] = _codes(v, 4), _to_tiles(s)
        st["w_q"], st["w_s"] = _weights((G, case["N"], K), 0.02, 4, g)
    return st


# ---------------------------------------------------------------- one pass
def _grouped(a, w, sizes):
    """a [M, K] by groups with w [G, N, K] -> [M, N], in the inputs' precision."""
    parts = torch.split(a, sizes)
    return torch.cat([p @ w[i].T for i, p in enumerate(parts)])


def _train_plain(st):
    A, W, dOut, sizes = st["A"].float(), st["W"].float(), st["dOut"].float(), st["sizes"]
    out = _grouped(_mx_value(A, 4), _mx_value(W, 4), sizes).to(torch.bfloat16)
    # gradients: every operand in MXFP8 along its product's contraction (groups start at multiples of 32 tokens)
    dA = _grouped(_mx_value(dOut, 8), _mx_value(W.transpose(1, 2), 8), sizes).to(torch.bfloat16)
    at, dt = _mx_value(A.T, 8), _mx_value(dOut.T, 8)
    dW = torch.stack([d @ a.T for d, a in zip(torch.split(dt, sizes, 1), torch.split(at, sizes, 1))])
    return out, dA, dW.to(torch.bfloat16)


def _tokens_plain(st):
    c = st["case"]
    bits, T, E = c["bits"], c["T"], c["E"]
    x = _mx_value(st["x"].float(), bits)
    l = st["logits"]
    order = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    top = l.gather(1, order)
    w = torch.softmax(top, 1) if c["score"] == "softmax" else 1 / (1 + torch.exp(-top))
    p = torch.zeros((T, E), device="cuda").scatter(1, order, w).T.unsqueeze(-1)
    h1 = x @ _decode(*st["gate"], bits).transpose(1, 2)          # [E, T, H]
    h3 = x @ _decode(*st["up"], bits).transpose(1, 2)
    h = _mx_value(h1 / (1 + torch.exp(-h1)) * h3, bits)
    y = h @ _decode(*st["down"], bits).transpose(1, 2)           # [E, T, D]
    return (p * y).sum(0).to(torch.bfloat16)


def run(st):
    kind = st["case"]["kind"]
    if own:
        import mxfp8_precision_moe_gb300 as mx

        if kind == "quantize":
            if st["case"]["form"] == "experts":
                return mx.mxfp4_dequantize_3d_experts(*mx.mxfp4_quantize_3d_experts(st["x"]))
            q, s = mx.mxfp4_quantize_2d(st["x"], offs=st["offs"])
            return mx.mxfp4_dequantize_2d(q, s, offs=st["offs"])
        if kind == "swiglu":
            q, s = mx.mxfp4_swiglu_quantize(st["h1"], st["h3"], offs=st["offs"])
            return mx.mxfp4_dequantize_2d(q, s, offs=st["offs"])
        if kind == "product":
            return mx.mxfp4_grouped_mm_fwd(st["a_q"], st["a_s"], st["w_q"], st["w_s"], st["offs"])
        if kind == "train":
            A, W = st["A"].detach().requires_grad_(True), st["W"].detach().requires_grad_(True)
            out = mx.to_mxfp4_then_scaled_grouped_mm(A, W, st["offs"], check_offsets=False)
            return (out.detach(),) + torch.autograd.grad(out, (A, W), st["dOut"])
        return st["layer"](st["x"], st["logits"])
    if kind == "quantize":
        return _mx_value(st["x"].float(), 4).to(torch.bfloat16)
    if kind == "swiglu":
        h1, h3 = st["h1"].float(), st["h3"].float()
        return _mx_value(h1 / (1 + torch.exp(-h1)) * h3, 4).to(torch.bfloat16)
    if kind == "product":
        a = _decode(st["a_q"], st["a_s"], 4, st["rows"])
        return _grouped(a, _decode(st["w_q"], st["w_s"], 4), st["sizes"]).to(torch.bfloat16)
    if kind == "train":
        return _train_plain(st)
    return _tokens_plain(st)


def work(case):
    kind = case["kind"]
    mx4 = 0.5 + 1 / BLOCK
    if kind == "tokens":
        T, E, D, H = case["T"], case["E"], case["D"], case["H"]
        read = E * (1 - (1 - case["top_k"] / E) ** T)  # distinct experts that T tokens select, on average
        per = case["bits"] / 8 + 1 / BLOCK
        return dict(bytes=read * 3 * D * H * per + 4 * T * D + 4 * T * E, flops=6.0 * T * case["top_k"] * D * H)
    if kind in ("quantize", "swiglu"):
        n = case["K"] * (case["G"] * case["N"] if case.get("form") == "experts" else case["M"])
        # codes and scales are written, read back and written as values
        return dict(bytes=n * ((4 if kind == "swiglu" else 2) + 2 * mx4 + 2), flops=(12 if kind == "swiglu" else 4) * n)
    M, N, K, G = case["M"], case["N"], case["K"], case["G"]
    if kind == "product":
        return dict(bytes=mx4 * (M * K + G * N * K) + 2 * M * N, flops=2.0 * M * N * K)
    return dict(bytes=2 * (2 * M * K + 2 * G * N * K + 2 * M * N), flops=6.0 * M * N * K)


# ---------------------------------------------------------------- the definition in 64 bits
def _two_to(e):
    """2.0 ** e in 64 bits for whole e, -400 <= e <= 400 (a power function may be one step off)."""
    return torch.tensor([2.0 ** k for k in range(-400, 401)], dtype=torch.float64, device="cuda")[e.long() + 400]


def _table(bits):
    """The non-negative elements in the order of their codes."""
    if bits == 4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        v += [(8 + m) * 2.0 ** (e - 10) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")  # the last pattern is no number


def _exact_mx(x, bits):
    """Nearest elements by search among all of them, block by block of the last axis."""
    t = _table(bits)
    shape = x.shape
    b = x.double().reshape(-1, BLOCK)
    out = torch.empty_like(b)
    for lo in range(0, b.shape[0], 1 << 20):
        c = b[lo:lo + (1 << 20)]
        top = c.abs().max(1, keepdim=True)[0]
        e = torch.where(top > 0, torch.floor(torch.log2(top)), torch.full_like(top, -200.0))
        # log2 rounds: at a power of two, or just below one, it can land on the other side
        e = torch.where(_two_to(e) > top, e - 1, e)
        e = torch.where(_two_to(e + 1) <= top, e + 1, e)
        scale = _two_to((e - EMAX[bits]).clamp(min=-127))
        a = c.abs() / scale
        i = torch.bucketize(a, (t[1:] + t[:-1]) / 2)  # a tie falls to the lower code
        j = (i + 1).clamp(max=t.numel() - 1)
        tie = (t[i] + t[j]) / 2 == a
        i = torch.where(tie & (i % 2 == 1), j, i)
        out[lo:lo + (1 << 20)] = torch.sign(c) * t[i] * scale
    return out.reshape(shape)


def _exact_decode(q, s, bits, R, C):
    """Codes and tiled scales of one matrix -> 64-bit values, byte by byte from the layout's formula."""
    r = torch.arange(R, device="cuda").unsqueeze(1)
    k = torch.arange(C // BLOCK, device="cuda").unsqueeze(0)
    at = ((r // 128) * (-(-C // 128)) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
    scale = _two_to(s[at].int() - 127)
    t = _table(bits)
    if bits == 4:
        every = torch.cat((t, -t))
        v = torch.stack((every[(q % 16).long()], every[(q // 16).long()]), -1).reshape(R, C)
    else:
        every = torch.cat((t, t.new_zeros(1), -t, t.new_zeros(1)))
        v = every[q.long()]
    return (v.reshape(R, -1, BLOCK) * scale.unsqueeze(-1)).reshape(R, C)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        return _exact_mx(st["x"], 4)
    if kind == "swiglu":
        h1 = st["h1"].double()
        return _exact_mx(h1 * torch.sigmoid(h1) * st["h3"].double(), 4)
    if kind == "tokens":
        bits, T, D, H = case["bits"], case["T"], case["D"], case["H"]
        x = _exact_mx(st["x"], bits)
        y = torch.zeros((T, D), dtype=torch.float64, device="cuda")
        l = st["logits"].double().cpu()
        chosen = [sorted(range(case["E"]), key=lambda e: (-float(l[t, e]), e))[:case["top_k"]] for t in range(T)]
        for e in range(case["E"]):
            who = [t for t in range(T) if e in chosen[t]]
            if not who:
                continue
            wt = []
            for t in who:
                if case["score"] == "softmax":
                    wt.append(math.exp(l[t, e]) / math.fsum(math.exp(l[t, i]) for i in chosen[t]))
                else:
                    wt.append(1 / (1 + math.exp(-l[t, e])))
            h1 = x[who] @ _exact_decode(st["gate"][0][e], st["gate"][1][e], bits, H, D).T
            h3 = x[who] @ _exact_decode(st["up"][0][e], st["up"][1][e], bits, H, D).T
            h = _exact_mx(h1 * torch.sigmoid(h1) * h3, bits)
            o = h @ _exact_decode(st["down"][0][e], st["down"][1][e], bits, D, H).T
            y[who] += torch.tensor(wt, dtype=torch.float64, device="cuda").unsqueeze(1) * o
        return y
    M, N, K, sizes = case["M"], case["N"], case["K"], st["sizes"]
    if kind == "product":
        out, at, tiles = torch.empty((M, N), dtype=torch.float64, device="cuda"), 0, 0
        for i, n in enumerate(sizes):
            if n:
                a = _exact_decode(st["a_q"][at:at + n], st["a_s"][tiles:], 4, n, K)
                out[at:at + n] = a @ _exact_decode(st["w_q"][i], st["w_s"][i], 4, N, K).T
            at, tiles = at + n, tiles + -(-n // 128) * -(-K // 128) * 512
        return out
    out, dA = (torch.empty((M, n), dtype=torch.float64, device="cuda") for n in (N, K))
    dW, at = torch.zeros((case["G"], N, K), dtype=torch.float64, device="cuda"), 0
    for i, n in enumerate(sizes):
        a, d, w = st["A"][at:at + n], st["dOut"][at:at + n], st["W"][i]
        if n:
            out[at:at + n] = _exact_mx(a, 4) @ _exact_mx(w, 4).T
            dA[at:at + n] = _exact_mx(d, 8) @ _exact_mx(w.T.contiguous(), 8).T
            dW[i] = _exact_mx(d.T.contiguous(), 8) @ _exact_mx(a.T.contiguous(), 8).T
        at += n
    return out, dA, dW
