"""Cases of the path around the routed experts: routing, the plan of the token rows, their dispatch and their combination.

Four kinds of case:

* ``route``     router logits [T, E] -> the top_k experts of each token and their weights; scores by softmax over the
  selected, softmax over all or sigmoid, with a bias that only the selection sees, with experts in groups, with
  renormalised and scaled weights; ``train``: the gradient of the logits too.
* ``plan``      the experts [T, k] of each token -> rows grouped by expert: group ends, group counts, the source of each row
  (t * k + j; -1 for padding) and the row of each choice (-1: the choice names no expert).  Groups are padded to a multiple.
* ``dispatch``  token rows into the plan's order: in bf16 with the gradient of x (``bf16``), or quantized on the way, to
  MXFP4 along the row (``fp4``) or to MXFP8 along the row and down the columns (``fp8``); codes come back as values.
* ``combine``   out[t] = sum over j of w[t, j] y[row of (t, j)]; ``train``: the gradients of y and w too.

MX blocks hold 32 elements with one power of two 2^e, e = floor(log2 amax) - emax, clamped at -127; elements are E2M1
(emax 2, largest 6) or E4M3 (emax 8, largest 448), rounded to nearest even and saturated.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
EMAX = {4: 2, 8: 8}
LARGEST = {4: 6.0, 8: 448.0}
LEAST_EXP = {4: 0, 8: -6}      # exponent of the smallest normal element
MANTISSA = {4: 1, 8: 3}
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a few decoding tokens of a layer that sends each to one of 16 experts: launch latency counts
        dict(name="route_few", kind="route", T=5, E=16, k=1, score="sigmoid", dtype="fp32", train=False),
        # a training batch of the same layer, logits as a bf16 projection gives them
        dict(name="route_top1", kind="route", T=16384, E=16, k=1, score="sigmoid", dtype="bf16", train=True),
        # a training batch over 256 fine-grained experts: 4 of 8 groups, a bias for balance, renormalised weights
        dict(name="route_grouped", kind="route", T=32768, E=256, k=8, score="sigmoid", dtype="fp32", groups=8, top_groups=4,
             bias=True, renormalize=True, scale=2.5, train=True),
        # a decoding batch
        dict(name="plan_few", kind="plan", T=64, E=16, k=4, multiple=1, idle=3),
        # a training batch over fine-grained experts, groups padded for the token-wise quantization
        dict(name="plan_fine", kind="plan", T=32768, E=256, k=8, multiple=32, idle=0),
        # a short prompt on its way into the 4-bit product
        dict(name="dispatch_few", kind="dispatch", form="fp4", T=77, E=4, k=2, D=1056, multiple=1, idle=0),
        # a training batch, one expert a token: MXFP8 rows for the product, columns for the weights' gradient
        dict(name="dispatch_train8", kind="dispatch", form="fp8", T=16384, E=8, k=1, D=5120, multiple=32, idle=0),
        # a long prompt over fine-grained experts, each token to eight of them
        dict(name="dispatch_fine4", kind="dispatch", form="fp4", T=8192, E=256, k=8, D=7168, multiple=1, idle=0),
        # a training batch whose rows stay in bf16, and the gradient of its tokens
        dict(name="dispatch_train16", kind="dispatch", form="bf16", T=16384, E=16, k=4, D=5120, multiple=32, idle=100),
        # a few tokens of a small layer
        dict(name="combine_few", kind="combine", T=5, E=6, k=2, D=352, multiple=1, idle=0, train=False),
        # the prompt over fine-grained experts again, behind the down product
        dict(name="combine_fine", kind="combine", T=8192, E=256, k=8, D=7168, multiple=1, idle=0, train=False),
        # a training batch, with the gradients of the experts' rows and of the weights
        dict(name="combine_train", kind="combine", T=16384, E=16, k=4, D=5120, multiple=32, idle=100, train=True),
    ]


def _spread(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // multiple * multiple))


def draw(rng):
    kind = rng.choice(("route", "route", "plan", "dispatch", "dispatch", "combine", "combine"))
    E = rng.choice((4, 6, 8, 13, 16, 64, 100, 160, 256))
    k = rng.randint(1, min(8, E))
    T = _spread(rng, 1, 32768 if kind in ("route", "plan") else 65536 // k)
    c = dict(kind=kind, T=T, E=E, k=k)
    if kind == "route":
        c["score"] = rng.choice(("softmax", "softmax_all", "sigmoid"))
        c["dtype"] = rng.choice(("fp32", "fp32", "bf16", "fp16"))
        c["train"] = rng.random() < 0.6
        if rng.random() < 0.5:
            c["bias"] = True
        if c["score"] != "softmax" and rng.random() < 0.5:
            c["renormalize"] = True
        if rng.random() < 0.5:
            c["scale"] = round(rng.uniform(0.5, 4), 2)
        fit = [g for g in (2, 4, 5, 8, 16) if E % g == 0]
        if fit and rng.random() < 0.5:
            g = rng.choice(fit)
            c["groups"], c["top_groups"] = g, rng.randint(max(1, -(-k * g // E)), g)
        return c
    if kind == "dispatch":
        c["form"] = rng.choice(("fp4", "fp8", "bf16"))
    c["multiple"] = 32 if kind == "dispatch" and c["form"] == "fp8" else rng.choice((1, 32, 128))
    if kind != "plan":
        c["D"] = _spread(rng, 32, 7168, 32)
    if kind == "combine":
        c["train"] = rng.random() < 0.5
    idle = rng.choice((0, 0, rng.randint(0, 50)))
    c["idle"] = min(idle, c["T"] - 1)
    while work(c)["bytes"] > 1.6e9:
        c["T"] = c["T"] * 2 // 3
        c["idle"] = min(idle, c["T"] - 1)
    return c


# ---------------------------------------------------------------- the plan, plainly
def _bound(T, E, k, multiple):
    """Rows that always suffice: every group can be short of a multiple by multiple - 1."""
    return (T * k + min(E, T * k) * (multiple - 1)) // multiple * multiple


def _plan(experts, E, multiple):
    """-> group ends [E], counts [E], source of each row [bound], row of each choice [T, k]; choices in the order of
    their tokens within a group."""
    T, k = experts.shape
    e = experts.long().flatten()
    live = (e >= 0) & (e < E)
    counts = torch.bincount(e[live], minlength=E)
    padded = (counts + multiple - 1) // multiple * multiple
    ends = padded.cumsum(0)
    key = torch.where(live, e, E)
    order = torch.sort(key, stable=True)[1][:int(live.sum())]
    group = e[order]
    row = (ends - padded)[group] + torch.arange(order.numel(), device=e.device) - (counts.cumsum(0) - counts)[group]
    slot = torch.full((_bound(T, E, k, multiple),), -1, dtype=torch.int32, device=e.device)
    slot[row] = order.int()
    place = torch.full((T * k,), -1, dtype=torch.int32, device=e.device)
    place[order] = row.int()
    return ends.int(), counts.int(), slot, place.view(T, k)


# ---------------------------------------------------------------- inputs
def _randn(shape, std, g):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _popularity(E, g):
    """How much likelier some experts are than others, as logits: Zipf's law with exponent 0.7 over a random order."""
    return -0.7 * torch.log(1 + torch.randperm(E, generator=g, device="cuda").float())


def _experts(case, g):
    """k different experts for each token, some much likelier.  The group sizes are the case's, so that the rows of the
    plan are as many for every seed; which token goes where, and which expert has which size, is the seed's."""
    T, E, k, idle = case["T"], case["E"], case["k"], case["idle"]
    fixed = torch.Generator(device="cuda").manual_seed(1000 * T + 10 * E + k)
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=fixed, device="cuda").clamp(1e-20, 1 - 1e-7)))
    experts = (noise + _popularity(E, fixed)).topk(k, dim=1)[1]
    experts = torch.randperm(E, generator=g, device="cuda")[experts]
    live = T - idle
    experts[:live] = experts[:live][torch.randperm(live, generator=g, device="cuda")]
    experts[live:] = -1  # the end of a padded batch takes no expert
    return experts.int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, E, k = case["T"], case["E"], case["k"]
    st = dict(case=case)
    if case["kind"] == "route":
        # scores that differ from token to token, with some experts in favour; the bias leans against those
        fav = _popularity(E, g)
        st["logits"] = (torch.randn((T, E), generator=g, device="cuda") * 1.5 + 0.5 * fav).to(TYPES[case["dtype"]])
        st["bias"] = (0.02 * torch.randn(E, generator=g, device="cuda") - 0.05 * fav) if case.get("bias") else None
        st["dw"] = torch.randn((T, k), generator=g, device="cuda") * 1e-3
        return st
    experts = _experts(case, g)
    st["experts"] = experts
    if case["kind"] == "plan":
        return st
    ends, counts, slot, place = _plan(experts, E, case["multiple"])
    M, D = int(ends[-1]), case["D"]
    st["slot"], st["place"] = slot[:M].long(), place.long()
    if own:
        import mxfp8_precision_moe_gb300 as mx

        st["plan"] = mx.moe_plan(experts, E, case["multiple"], exact=True)
    if case["kind"] == "dispatch":
        st["x"] = _randn((T, D), 1.0, g)
        if case["form"] == "bf16":
            st["dy"] = _randn((M, D), 1e-3, g)
        return st
    st["y"] = _randn((M, D), 1.0, g)
    st["w"] = torch.rand((T, k), generator=g, device="cuda") + 0.05
    st["w"] /= st["w"].sum(1, keepdim=True)
    if case["train"]:
        st["dout"] = _randn((T, D), 1e-3, g)
    return st


# ---------------------------------------------------------------- one pass, plainly
def _keys(l, bias, case):
    """What the selection ranks, in 64 bits (neighbours at the border may be closer than 32 tell): the score plus the
    bias, or, without bias and groups, the logit, which orders as its score does."""
    l = l.double()
    if bias is None and case.get("groups", 1) == 1:
        return l
    if case["score"] == "sigmoid":
        l = 1 / (1 + torch.exp(-l))
    elif case["score"] == "softmax_all":
        p = torch.exp(l - l.max(1, keepdim=True)[0])
        l = p / p.sum(1, keepdim=True)
    return l if bias is None else l + bias.double()


def _route_plain(st):
    c = st["case"]
    T, E, k, score, scale = c["T"], c["E"], c["k"], c["score"], c.get("scale", 1.0)
    keys = _keys(st["logits"], st["bias"], c)
    if c.get("groups", 1) > 1:
        # a group is worth the sum of its two best
        per = keys.view(T, c["groups"], -1)
        worth = torch.sort(per, dim=2, descending=True)[0][:, :, :2].sum(2)
        best = torch.sort(worth, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        stay = torch.zeros(worth.shape, dtype=torch.bool, device="cuda").scatter(1, best, True)
        keys = torch.where(stay.unsqueeze(2), per, -math.inf).flatten(1)
    experts = torch.sort(keys, dim=1, descending=True, stable=True)[1][:, :k]
    l = st["logits"].float()
    chosen = l.gather(1, experts)
    if score == "softmax_all" and not c.get("renormalize"):
        p = torch.exp(l - l.max(1, keepdim=True)[0])
        p = p / p.sum(1, keepdim=True)
        w = p.gather(1, experts)
    elif score == "sigmoid":
        w = 1 / (1 + torch.exp(-chosen))
        if c.get("renormalize"):
            total = w.sum(1, keepdim=True)
            w = w / total
    else:
        w = torch.exp(chosen - chosen.max(1, keepdim=True)[0])
        w = w / w.sum(1, keepdim=True)
    if not c["train"]:
        return experts.int(), w * scale
    d = st["dw"] * scale
    if score == "softmax_all" and not c.get("renormalize"):
        dl = torch.zeros_like(p).scatter(1, experts, d)
        dl = p * (dl - (d * w).sum(1, keepdim=True))
    else:
        if score == "sigmoid":
            s = 1 / (1 + torch.exp(-chosen))
            if c.get("renormalize"):
                d = (d - (d * w).sum(1, keepdim=True)) / total
            d = d * s * (1 / (1 + torch.exp(chosen)))
        else:
            d = w * (d - (d * w).sum(1, keepdim=True))
        dl = torch.zeros_like(l).scatter(1, experts, d)
    return experts.int(), w * scale, dl.to(st["logits"].dtype)


def _pow2(e):
    """2^e, exactly, for -127 <= e <= 127."""
    return torch.where(e < -126, 1 << 22, (e + 127).to(torch.int32) << 23).to(torch.int32).view(torch.float32)


def _mx_value(x, bits):
    """The values that x [..., C], quantized along its last axis, is held as."""
    b = x.unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax)[1] - 1 - EMAX[bits]).clamp_min(-127), -127).unsqueeze(-1)
    v = b * _pow2(-e)
    a = v.abs().clamp_max(LARGEST[bits])
    step = _pow2((torch.frexp(a)[1] - 1).clamp_min(LEAST_EXP[bits]) - MANTISSA[bits])
    return (torch.copysign(torch.round(a / step) * step, v) * _pow2(e)).flatten(-2)


def _rows(x, slot, k):
    """x's rows in the plan's order; zeros where a row is padding."""
    return torch.where((slot >= 0).unsqueeze(1), x[slot.clamp_min(0) // k], 0.0)


def _sum_choices(y, place, w=None):
    """sum over j of w[t, j] y[place[t, j]], in 32 bits."""
    out = torch.zeros((place.shape[0], y.shape[1]), device="cuda")
    for j in range(place.shape[1]):
        at = place[:, j]
        part = y[at.clamp_min(0)].float()
        if w is not None:
            part = part * w[:, j:j + 1]
        out += torch.where((at >= 0).unsqueeze(1), part, 0.0)
    return out


def run(st):
    c = st["case"]
    kind = c["kind"]
    if own:
        import mxfp8_precision_moe_gb300 as mx

        if kind == "route":
            l = st["logits"]
            if c["train"]:
                l = l.detach().requires_grad_(True)
            experts, w = mx.moe_route(l, c["k"], score=c["score"], bias=st["bias"], groups=c.get("groups", 1),
                                      top_groups=c.get("top_groups"), renormalize=c.get("renormalize", False),
                                      scale=c.get("scale", 1.0))
            if not c["train"]:
                return experts, w
            return experts, w.detach(), torch.autograd.grad(w, l, st["dw"])[0]
        if kind == "plan":
            p = mx.moe_plan(st["experts"], c["E"], c["multiple"])
            return p.offs, p.counts, p.slot, p.place
        plan = st["plan"]
        if kind == "dispatch":
            if c["form"] == "fp4":
                q, s = mx.mxfp4_gather_quantize(st["x"], plan)
                return mx.mxfp4_dequantize_2d(q, s, offs=plan.offs)
            if c["form"] == "fp8":
                q, s, qT, sT = mx.mxfp8_gather_quantize(st["x"], plan, mx.ROW | mx.COL)
                return (mx.mxfp8_dequantize_2d(q, s, offs=plan.offs),
                        mx.mxfp8_dequantize_2d(qT, sT, mx.COL, offs=plan.offs))
            x = st["x"].detach().requires_grad_(True)
            rows = mx.moe_gather(x, plan)
            return rows.detach(), torch.autograd.grad(rows, x, st["dy"])[0]
        if not c["train"]:
            return mx.moe_combine(st["y"], plan, st["w"])
        y, w = st["y"].detach().requires_grad_(True), st["w"].detach().requires_grad_(True)
        out = mx.moe_combine(y, plan, w)
        return (out.detach(),) + torch.autograd.grad(out, (y, w), st["dout"])
    if kind == "route":
        return _route_plain(st)
    if kind == "plan":
        return _plan(st["experts"], c["E"], c["multiple"])
    slot, place, k = st["slot"], st["place"], c["k"]
    if kind == "dispatch":
        rows = _rows(st["x"].float(), slot, k)
        if c["form"] == "fp4":
            return _mx_value(rows, 4).to(torch.bfloat16)
        if c["form"] == "fp8":
            return (_mx_value(rows, 8).to(torch.bfloat16),
                    _mx_value(rows.T.contiguous(), 8).to(torch.bfloat16))
        return rows.to(torch.bfloat16), _sum_choices(st["dy"], place).to(torch.bfloat16)
    out = _sum_choices(st["y"], place, st["w"]).to(torch.bfloat16)
    if not c["train"]:
        return out
    dout = st["dout"].float()
    wr = torch.where(slot >= 0, st["w"].flatten()[slot.clamp_min(0)], 0.0)
    dy = _rows(dout, slot, k) * wr.unsqueeze(1)
    dw = torch.zeros_like(st["w"])
    for j in range(k):
        at = place[:, j]
        dw[:, j] = torch.where(at >= 0, (st["y"][at.clamp_min(0)].float() * dout).sum(1), 0.0)
    return out, dy.to(torch.bfloat16), dw


def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    kind = case["kind"]
    if kind == "route":
        size = 4 if case["dtype"] == "fp32" else 2
        passes = 2 if case["train"] else 1  # the logits in; their gradient out
        return dict(bytes=T * E * size * passes + T * k * (8 + 4 * (passes - 1)), flops=10.0 * T * E * passes)
    live = (T - case["idle"]) * k
    M = live + min(E, live) * (case["multiple"] - 1) / 2  # on average
    if kind == "plan":
        return dict(bytes=4 * (2 * T * k + _bound(T, E, k, case["multiple"]) + 2 * E), flops=4.0 * T * k)
    D = case["D"]
    if kind == "dispatch":
        if case["form"] == "bf16":
            return dict(bytes=2 * D * (2 * T + 2 * M), flops=1.0 * live * D)
        mx = (0.5 if case["form"] == "fp4" else 1) + 1 / BLOCK
        copies = 1 if case["form"] == "fp4" else 2
        # x is read; codes and scales are written, read back and written as values
        return dict(bytes=D * (2 * T + M * copies * (2 * mx + 2)), flops=4.0 * M * D * copies)
    if not case["train"]:
        return dict(bytes=2 * D * (live + T) + 8 * T * k, flops=2.0 * live * D)
    return dict(bytes=2 * D * (live + M + 2 * T) + 12 * T * k, flops=5.0 * live * D)


# ---------------------------------------------------------------- the definition in 64 bits
def _rank(v):
    """Of each value its place when a row is ordered, the largest first, equal ones by their index: by counting."""
    n = v.shape[1]
    i = torch.arange(n, device="cuda")
    out = torch.empty(v.shape, dtype=torch.long, device="cuda")
    step = max(1, (1 << 26) // (n * n))
    for lo in range(0, v.shape[0], step):
        a, b = v[lo:lo + step].unsqueeze(2), v[lo:lo + step].unsqueeze(1)
        out[lo:lo + step] = ((b > a) | ((b == a) & (i.unsqueeze(0) < i.unsqueeze(1)))).sum(2)
    return out


def _exact_route(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    l = st["logits"].double().requires_grad_(True)
    with torch.no_grad():
        key = {"softmax": lambda: l, "softmax_all": lambda: torch.softmax(l, 1), "sigmoid": lambda: torch.sigmoid(l)}[
            c["score"] if st["bias"] is not None or c.get("groups", 1) > 1 else "softmax"]()
        if st["bias"] is not None:
            key = key + st["bias"].double()
        if c.get("groups", 1) > 1:
            per = key.reshape(T * c["groups"], -1)
            worth = (per * (_rank(per) < 2)).sum(1).reshape(T, -1)
            gone = (_rank(worth) >= c["top_groups"]).repeat_interleave(E // c["groups"], 1)
            key = key.masked_fill(gone, -math.inf)
        rank = _rank(key)
        at, e = (rank < k).nonzero(as_tuple=True)
        experts = torch.empty((T, k), dtype=torch.long, device="cuda")
        experts[at, rank[at, e]] = e
    if c["score"] == "softmax_all":
        w = torch.softmax(l, 1).gather(1, experts)
    elif c["score"] == "sigmoid":
        w = torch.sigmoid(l).gather(1, experts)
    else:
        w = torch.softmax(l.gather(1, experts), 1)
    if c.get("renormalize"):
        w = w / w.sum(1, keepdim=True)
    w = w * c.get("scale", 1.0)
    if not c["train"]:
        return experts.int(), w.detach()
    return experts.int(), w.detach(), torch.autograd.grad(w, l, st["dw"].double())[0]


def _exact_plan(experts, E, multiple):
    T, k = experts.shape
    e = experts.cpu().numpy().reshape(-1)
    slot = np.full(_bound(T, E, k, multiple), -1, np.int32)
    place = np.full(T * k, -1, np.int32)
    counts, ends, at = np.zeros(E, np.int32), np.zeros(E, np.int32), 0
    for i in range(E):
        who = np.flatnonzero(e == i)
        counts[i] = who.size
        slot[at:at + who.size] = who
        place[who] = np.arange(at, at + who.size)
        at += -(-who.size // multiple) * multiple
        ends[i] = at
    return tuple(torch.from_numpy(v).cuda() for v in (ends, counts, slot, place.reshape(T, k)))


def _two_to(e):
    """2.0 ** e in 64 bits for whole e, -400 <= e <= 400 (a power function may be one step off)."""
    return torch.tensor([2.0 ** i for i in range(-400, 401)], dtype=torch.float64, device="cuda")[e.long() + 400]


def _table(bits):
    """The non-negative elements in the order of their codes."""
    if bits == 4:
        return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        v += [(8 + m) * 2.0 ** (e - 10) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")  # the last pattern is no number


def _exact_mx(x, bits):
    """Nearest elements by search among all of them, block by block of the last axis; as bf16 (every value is one)."""
    t = _table(bits)
    b = x.reshape(-1, BLOCK)
    out = torch.empty_like(b)
    for lo in range(0, b.shape[0], 1 << 20):
        c = b[lo:lo + (1 << 20)].double()
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
        out[lo:lo + (1 << 20)] = (torch.sign(c) * t[i] * scale).to(torch.bfloat16)
    return out.reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    kind, k = case["kind"], case["k"]
    if kind == "route":
        return _exact_route(st)
    if kind == "plan":
        return _exact_plan(st["experts"], case["E"], case["multiple"])
    ends, _, slot, place = _exact_plan(st["experts"], case["E"], case["multiple"])
    M, T, D = int(ends[-1]), case["T"], case["D"]
    real = (slot[:M] >= 0).nonzero().flatten()      # the rows that hold a token, their tokens and their choices
    source = slot[real].long()
    token = torch.div(source, k, rounding_mode="floor")
    if kind == "dispatch":
        rows = torch.zeros((M, D), dtype=torch.bfloat16, device="cuda")
        rows[real] = st["x"][token]
        if case["form"] == "fp4":
            return _exact_mx(rows, 4)
        if case["form"] == "fp8":
            return _exact_mx(rows, 8), _exact_mx(rows.T.contiguous(), 8)
        dx = torch.zeros((T, D), dtype=torch.float64, device="cuda")
        dx.index_add_(0, token, st["dy"][real].double())
        return rows, dx
    w = st["w"].double().flatten()[source].unsqueeze(1)
    out = torch.zeros((T, D), dtype=torch.float64, device="cuda")
    out.index_add_(0, token, st["y"][real].double() * w)
    if not case["train"]:
        return out
    dy = torch.zeros((M, D), dtype=torch.float64, device="cuda")
    dy[real] = st["dout"][token].double() * w
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    for lo in range(0, real.numel(), 8192):
        at = slice(lo, lo + 8192)
        dw[source[at]] = (st["y"][real[at]].double() * st["dout"][token[at]].double()).sum(1)
    return out, dy, dw.view(T, k)
