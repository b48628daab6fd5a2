"""The path around the routed experts: routing, the plan of the token rows, their dispatch (in bf16, or quantized
on the way to MXFP8 or MXFP4) and their combination, and the routed SwiGLU layer made of them (C ABI:
``include/mxrouting.h``).

    experts, weights = mx.moe_route(logits, top_k, score="sigmoid", bias=balance, renormalize=True)
    plan = mx.moe_plan(experts, E, multiple=32)
    rows = mx.moe_gather(x, plan)                       # [plan.rows, D], grouped by expert
    y = mx.mxfp8_swiglu_expert(rows, gate, up, down, plan.offs, check_offsets=False)
    out = mx.moe_combine(y, plan, weights)              # [T, D]

or all of it, with the gather inside the quantizations, as ``mxfp8_moe_swiglu``.  Nothing here waits for the device
(but ``moe_plan(..., exact=True)``), and a sum's order is fixed: equal inputs give equal bits.

Every call can be captured into a CUDA graph, backward passes too: with the usual warm-up on a side stream, and while no
graph of an eager forward of the same leaves is alive (torch ties a leaf's accumulation to the stream it first saw).
"""
from __future__ import annotations

import torch

from . import (COL, MAX_GROUPS, ROW, SCALES_BLOCKED, SCALES_COMPACT, _bytes_at_least, _check_quad, _cuda,
               _expert_blocked_bytes, _first_order, _offsets, _status_word, _tensor, _u8, check, load,
               mxfp8_grouped_mm_dgrad, mxfp8_grouped_mm_dgrad2, mxfp8_grouped_mm_fwd, mxfp8_grouped_mm_swiglu_fwd,
               mxfp8_grouped_mm_wgrad, mxfp8_quantize_2d, mxfp8_scale_bytes, mxfp8_scale_bytes_colgroups,
               mxfp8_swiglu_bwd_quantize, quantize_expert_weights)
from .moe_tokens import MAX_TOP_K, SCORES
from .mxfp4 import _good, _group_bytes

_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without building an object

LOGITS_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
GROUP_SCORES = {"top2": 0, "max": 1}
MAX_EXPERT_GROUPS, MAX_MULTIPLE = 32, 1024


def _on_device(*ts):
    """As _cuda, for tensors that a call makes contiguous itself."""
    here = torch._C._cuda_getDevice() if ts[0].is_cuda else -1
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("mxfp8: every tensor must live on a CUDA device")
        if t.get_device() != here:
            raise ValueError(f"mxfp8: a tensor lives on {t.device}, and the current device, on which the kernels "
                             f"launch, is cuda:{here}")


# ---------------------------------------------------------------- routing
def _route_args(T, E, top_k, score, bias, groups, top_groups, group_score, renormalize, scale):
    """The checked options, as the C ABI takes them."""
    if not 1 <= E <= MAX_GROUPS:
        raise ValueError(f"logits: 1 .. {MAX_GROUPS} experts, got {E}")
    if not 1 <= top_k <= min(E, MAX_TOP_K):
        raise ValueError(f"top_k: 1 .. {min(E, MAX_TOP_K)}, got {top_k}")
    if score not in SCORES:
        raise ValueError(f"score: one of {sorted(SCORES)}, got {score!r}")
    if group_score not in GROUP_SCORES:
        raise ValueError(f"group_score: one of {sorted(GROUP_SCORES)}, got {group_score!r}")
    if not 1 <= groups <= MAX_EXPERT_GROUPS or E % groups:
        raise ValueError(f"groups: 1 .. {MAX_EXPERT_GROUPS}, a divisor of {E}, got {groups}")
    if top_groups is None:
        top_groups = groups
    if not 1 <= top_groups <= groups or top_k > top_groups * (E // groups):
        raise ValueError(f"top_groups: 1 .. {groups} with at least {top_k} experts in them, got {top_groups}")
    if bias is not None:
        _tensor(bias, "bias", torch.float32, shape=(E,))
    if T * top_k >= 2 ** 31:
        raise ValueError(f"logits: at most 2^31 - 1 choices, got {T} tokens of {top_k}")
    return int(top_k), SCORES[score], int(groups), int(top_groups), GROUP_SCORES[group_score], bool(renormalize), float(scale)


def _route_into(logits, bias, args, experts, weights, dense):
    T, E = logits.shape
    top_k, score, groups, top_groups, group_score, renormalize, scale = args
    check(load().mx_moe_route(logits.data_ptr(), LOGITS_TYPES[logits.dtype], T, E, top_k, score,
                              None if bias is None else bias.data_ptr(), groups, top_groups, group_score, renormalize,
                              scale, experts, weights, dense, _raw_stream(logits.device.index)), "mx_moe_route")


def _route(logits, bias, args):
    T, top_k, dev = logits.shape[0], args[0], logits.device
    experts = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    _route_into(logits, bias, args, experts.data_ptr(), weights.data_ptr(), None)
    return experts, weights


def _route_dense(logits, bias, args):
    """The weights [T, E] fp32, -inf for what is not selected: what the layer for a few tokens takes."""
    dense = torch.empty(logits.shape, dtype=torch.float32, device=logits.device)
    _route_into(logits, bias, args, None, None, dense.data_ptr())
    return dense


def _route_bwd(logits, experts, dweights, args):
    T, E = logits.shape
    top_k, score, _, _, _, renormalize, scale = args
    dlogits = torch.empty_like(logits)
    check(load().mx_moe_route_bwd(logits.data_ptr(), LOGITS_TYPES[logits.dtype], T, E, top_k, score, renormalize, scale,
                                  experts.data_ptr(), dweights.data_ptr(), dlogits.data_ptr(),
                                  _raw_stream(logits.device.index)), "mx_moe_route_bwd")
    return dlogits


class _MoeRoute(torch.autograd.Function):

    @staticmethod
    def forward(ctx, logits, bias, args):
        experts, weights = _route(logits, bias, args)
        ctx.mark_non_differentiable(experts)
        ctx.set_materialize_grads(False)  # no zeros for the experts' place
        ctx.save_for_backward(logits, experts)
        ctx.args = args
        return experts, weights

    @staticmethod
    @_first_order
    def backward(ctx, _, dweights):
        if dweights is None:
            return None, None, None
        logits, experts = ctx.saved_tensors
        return _route_bwd(logits, experts, dweights.contiguous(), ctx.args), None, None


def moe_route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
              groups: int = 1, top_groups: int | None = None, group_score: str = "top2", renormalize: bool = False,
              scale: float = 1.0):
    """The experts of each token and their weights: logits [T, E] (fp32, bf16 or fp16) -> (experts [T, top_k] int32,
    weights [T, top_k] fp32), the weights differentiable in the logits.  E <= 1024, top_k <= 16.

    Experts are ranked by score(logit) + bias (without a bias, or with the same one for all, by the logits, which order as
    their scores do), largest first; equal ones by their index, NaN above everything; an expert whose logit or bias is -inf is
    never selected.  A token that has fewer than top_k experts to select gets
    -1 with weight 0 in the places left.  (The gradient reads the experts: change a copy, not this tensor.)

    score: "softmax" (the ranking takes the logits, the weights are a softmax over the selected), "softmax_all" (over all
    experts) or "sigmoid".  bias [E] fp32: for balance; it moves the ranking, not the weights, and has no gradient.
    renormalize: the selected scores divided by their sum.  scale: a factor of all weights.
    groups: the experts lie in so many groups of neighbours (a divisor of E, 32 at most), each worth the sum of its two
    largest keys (group_score "top2"; of the one, where one of its experts can be selected), bias included, or its largest
    ("max"); only the top_groups best groups are selected from.

    Where 32 bits leave the order of two sums open, they are compared in 64."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.dtype not in LOGITS_TYPES:
        raise ValueError("logits: expected [T, E] in fp32, bf16 or fp16")
    args = _route_args(logits.shape[0], logits.shape[1], top_k, score, bias, groups, top_groups, group_score, renormalize,
                       scale)
    _on_device(logits, bias)
    logits = logits.contiguous()
    if bias is not None:
        bias = bias.detach().contiguous()
    if logits.requires_grad and torch.is_grad_enabled():
        return _MoeRoute.apply(logits, bias, args)
    return _route(logits, bias, args)


# ---------------------------------------------------------------- the plan
class MoePlan:
    """Rows of tokens grouped by expert (``moe_plan``); int32 tensors of one device:

    offs [E]      end row of each expert's group, for the grouped products (of one expert: all rows)
    counts [E]    rows of the group that hold a token
    slot [rows]   t * top_k + j, the choice that the row holds; -1: none (padding, and rows past offs[E - 1])
    place [T, top_k]  the row that holds the choice; -1: none

    rows, tokens (T), top_k and ``multiple`` are numbers.  Group sizes are multiples of ``multiple``.

    slot and place say the same: place[t, j] = r where slot[r] = t * top_k + j, and a choice that is dropped is -1 in both
    (some kernels read the one, some the other).  To drop choices, give ``moe_plan`` a copy of the experts with -1 in their
    places, as ``torch.where(keep, experts, -1)`` does: ``moe_route``'s own tensor is what its gradient reads, and changed in
    place it is refused there."""

    __slots__ = ("offs", "counts", "slot", "place", "multiple", "rows", "tokens", "top_k")

    def __init__(self, offs, counts, slot, place, multiple: int = 1):
        _offsets(offs)
        _tensor(counts, "counts", torch.int32, shape=offs.shape)
        _tensor(slot, "slot", torch.int32, 1)
        _tensor(place, "place", torch.int32, 2)
        if not 1 <= place.shape[1] <= MAX_TOP_K:
            raise ValueError(f"place: [T, top_k] with top_k 1 .. {MAX_TOP_K} expected, got {tuple(place.shape)}")
        if not 1 <= multiple <= MAX_MULTIPLE:
            raise ValueError(f"multiple: 1 .. {MAX_MULTIPLE}, got {multiple}")
        for t in (offs, counts, slot, place):
            if not t.is_contiguous() or t.device != offs.device:
                raise ValueError("MoePlan: contiguous tensors of one device expected")
        self._fill(offs, counts, slot, place, int(multiple))

    def _fill(self, offs, counts, slot, place, multiple):
        self.offs, self.counts, self.slot, self.place, self.multiple = offs, counts, slot, place, multiple
        self.rows = slot.shape[0]
        self.tokens, self.top_k = place.shape
        return self


def moe_plan(experts: torch.Tensor, num_experts: int, multiple: int = 1, *, exact: bool = False) -> MoePlan:
    """Group the rows of T tokens by expert: experts [T, top_k] (int32 or int64; a value outside 0 .. num_experts - 1
    takes no row).  Rows lie by expert and, within an expert, in the order of the tokens; group sizes are padded to
    multiples of ``multiple`` (32 where the weights need gradients).

    The rows' number depends on the experts, which are on the device.  By default the plan has as many as can be
    needed, T * top_k + E * (multiple - 1) at most, and those past offs[E - 1] are in no group (the grouped products do
    not touch them; ``check_offsets`` would refuse them); ``exact`` reads the number back, which waits for the device (and so
    cannot be captured into a graph), and has only those."""
    if not isinstance(experts, torch.Tensor) or experts.dtype not in (torch.int32, torch.int64) or experts.dim() != 2:
        raise ValueError("experts: expected [T, top_k] in int32 or int64")
    T, k = experts.shape
    E = int(num_experts)
    if not 1 <= E <= MAX_GROUPS:
        raise ValueError(f"num_experts: 1 .. {MAX_GROUPS}, got {E}")
    if not 1 <= k <= MAX_TOP_K:
        raise ValueError(f"experts: top_k 1 .. {MAX_TOP_K}, got {k}")
    if not 1 <= multiple <= MAX_MULTIPLE:
        raise ValueError(f"multiple: 1 .. {MAX_MULTIPLE}, got {multiple}")
    _on_device(experts)
    if exact and torch.cuda.is_current_stream_capturing():
        raise ValueError("exact: the rows' number cannot be read back in a captured call")
    n = T * k
    if n + E * multiple >= 2 ** 31:
        raise ValueError(f"experts: too many rows for 32-bit row numbers ({T} tokens of {k})")
    rows = (n + min(E, n) * (multiple - 1)) // multiple * multiple  # mx_moe_plan_rows
    experts = experts.contiguous()
    dev = experts.device
    L = load()
    nbytes = L.mx_moe_plan_workspace(T, k, E)
    # (tensors of their own: views of one allocation take the host longer than allocations do)
    offs, counts = (torch.empty(E, dtype=torch.int32, device=dev) for _ in range(2))
    slot, place = torch.empty(rows, dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.int32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    check(L.mx_moe_plan(experts.data_ptr(), experts.element_size(), T, k, E, multiple, rows, offs.data_ptr(),
                        counts.data_ptr(), slot.data_ptr(), place.data_ptr(), None if ws is None else ws.data_ptr(), nbytes,
                        _raw_stream(dev.index)), "mx_moe_plan")
    if exact:
        slot = slot[:int(offs[-1])]
    return MoePlan.__new__(MoePlan)._fill(offs, counts, slot, place, multiple)


# ---------------------------------------------------------------- rows
# A small call's time is the host's: what a correct call looks like is asked first, in a few expressions, and the named
# checks, which say what is wrong, follow where the answer is no.
def _good_rows(x, n: int, multiple: int, plan, weights=None) -> bool:
    here = torch._C._cuda_getDevice() if isinstance(x, torch.Tensor) and x.is_cuda else -2
    return (_good(x, torch.bfloat16, 2, here) and x.shape[0] == n and x.shape[1] % multiple == 0 and x.shape[1] >= multiple
            and plan.offs.get_device() == here
            and (weights is None or (_good(weights, torch.float32, 2, here) and weights.shape == plan.place.shape)))


def _rows_matrix(x, name: str, n: int, what: str, multiple: int = 8):
    _tensor(x, name, torch.bfloat16, 2)
    if x.shape[0] != n:
        raise ValueError(f"{name}: one row for each of the plan's {n} {what} expected, got {tuple(x.shape)}")
    if x.shape[1] < multiple or x.shape[1] % multiple:
        raise ValueError(f"{name}: the last dimension must be a positive multiple of {multiple}, got {x.shape[1]}")


def _choice_weights(weights, plan):
    if weights is not None:
        _tensor(weights, "weights", torch.float32, shape=plan.place.shape)


def _plan_of(plan):
    if not isinstance(plan, MoePlan):
        raise ValueError("plan: expected a MoePlan")
    return plan


def _incoming(grad):
    """A gradient as the kernels read it: autograd may hand over a view of any strides and at any offset."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def _gather(x, slot, place):
    (T, D), rows = x.shape, slot.shape[0]
    out = torch.empty((rows, D), dtype=torch.bfloat16, device=x.device)
    check(load().mx_moe_gather(x.data_ptr(), slot.data_ptr(), place.data_ptr(), rows, T, place.shape[1], D, out.data_ptr(),
                               _raw_stream(x.device.index)), "mx_moe_gather")
    return out


def _combine(y, place, weights):
    (rows, D), (T, k) = y.shape, place.shape
    out = torch.empty((T, D), dtype=torch.bfloat16, device=y.device)
    check(load().mx_moe_combine(y.data_ptr(), place.data_ptr(), None if weights is None else weights.data_ptr(), rows, T, k,
                                D, out.data_ptr(), _raw_stream(y.device.index)), "mx_moe_combine")
    return out


def _combine_bwd(dout, y, slot, place, weights, need_dy: bool, need_dw: bool):
    (T, D), rows, k = dout.shape, slot.shape[0], place.shape[1]
    dev = dout.device
    dy = torch.empty((rows, D), dtype=torch.bfloat16, device=dev) if need_dy else None
    dw = torch.empty((T, k), dtype=torch.float32, device=dev) if need_dw else None
    check(load().mx_moe_combine_bwd(dout.data_ptr(), y.data_ptr() if need_dw else None, slot.data_ptr(), place.data_ptr(),
                                    None if weights is None else weights.data_ptr(), rows, T, k, D,
                                    None if dy is None else dy.data_ptr(), None if dw is None else dw.data_ptr(),
                                    _raw_stream(dev.index)), "mx_moe_combine_bwd")
    return dy, dw


class _MoeGather(torch.autograd.Function):

    @staticmethod
    def forward(ctx, x, plan):
        ctx.save_for_backward(plan.place)  # (so that a plan overwritten in between is noticed)
        return _gather(x, plan.slot, plan.place)

    @staticmethod
    @_first_order
    def backward(ctx, drows):
        return _combine(_incoming(drows), ctx.saved_tensors[0], None), None


def moe_gather(x: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """Token rows in the plan's order: x [T, D] bf16 -> [plan.rows, D], zeros in rows without a token.  D a multiple of 8.
    Differentiable: a token's gradient is the sum of its rows' in fp32, rounded once."""
    if not _good_rows(x, _plan_of(plan).tokens, 8, plan):
        _rows_matrix(x, "x", plan.tokens, "tokens")
        _on_device(x, plan.offs)
        x = x.contiguous()
    if x.requires_grad and torch.is_grad_enabled():
        return _MoeGather.apply(x, plan)
    return _gather(x, plan.slot, plan.place)


class _MoeCombine(torch.autograd.Function):

    @staticmethod
    def forward(ctx, y, weights, plan):
        ctx.save_for_backward(y if ctx.needs_input_grad[1] else None, weights, plan.slot, plan.place)
        return _combine(y, plan.place, weights)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        y, weights, slot, place = ctx.saved_tensors
        need_dy, need_dw = ctx.needs_input_grad[:2]
        return _combine_bwd(_incoming(dout), y, slot, place, weights, need_dy, need_dw) + (None,)


def moe_combine(y: torch.Tensor, plan: MoePlan, weights: torch.Tensor | None = None) -> torch.Tensor:
    """The tokens' sums of their rows: out[t] = sum over j of weights[t, j] * y[plan.place[t, j]]; y [plan.rows, D] bf16,
    weights [T, top_k] fp32 (none: ones) -> [T, D] bf16.  fp32 sums in the order of j, rounded once; a choice without a row
    counts nothing, a token without any gets zeros.  D a multiple of 8.  Differentiable in y (rows without a token get
    zeros) and in the weights."""
    if not _good_rows(y, _plan_of(plan).rows, 8, plan, weights):
        _rows_matrix(y, "y", plan.rows, "rows")
        _choice_weights(weights, plan)
        _on_device(y, plan.offs, weights)
        y = y.contiguous()
        if weights is not None:
            weights = weights.contiguous()
    if (y.requires_grad or (weights is not None and weights.requires_grad)) and torch.is_grad_enabled():
        return _MoeCombine.apply(y, weights, plan)
    return _combine(y, plan.place, weights)


# ---------------------------------------------------------------- rows, quantized on the way
def mxfp8_gather_quantize(x: torch.Tensor, plan: MoePlan, dirs: int = ROW, weights: torch.Tensor | None = None,
                          dev_status: torch.Tensor | None = None):
    """``mxfp8_quantize_2d(moe_gather(x, plan), dirs, SCALES_BLOCKED, plan.offs)`` without the rows in between:
    (q_row [rows, D], s_row, q_col [D, rows], s_col), None for a direction not asked for (ROW, COL or both).  With
    weights [T, top_k] the rows are bf16(weight * row), which is what ``moe_combine`` hands back to its rows' gradient.
    D a multiple of 32; the plan's multiple one of 32 for COL."""
    if dirs not in (ROW, COL, ROW | COL):
        raise ValueError("dirs: ROW, COL or both expected")
    if not _good_rows(x, _plan_of(plan).tokens, 32, plan, weights) or dev_status is not None \
            or (dirs & COL and (plan.multiple % 32 or plan.rows % 32)):
        _rows_matrix(x, "x", plan.tokens, "tokens", 32)
        if dirs & COL and (plan.multiple % 32 or plan.rows % 32):
            raise ValueError(f"plan: COL needs groups of multiples of 32 rows, got multiples of {plan.multiple}")
        _choice_weights(weights, plan)
        _status_word(dev_status)
        _cuda(x, plan.offs, weights, dev_status)
    (T, D), M, G, dev = x.shape, plan.rows, plan.offs.shape[0], x.device
    q_row = s_row = q_col = s_col = None
    if dirs & ROW:
        q_row, s_row = _u8((M, D), dev), _u8(mxfp8_scale_bytes(M, D, G, SCALES_BLOCKED), dev)
    if dirs & COL:
        q_col, s_col = _u8((D, M), dev), _u8(mxfp8_scale_bytes_colgroups(D, M, G), dev)
    at = [None if t is None else t.data_ptr() for t in (weights, q_row, s_row, q_col, s_col, dev_status)]
    check(load().mxfp8_gather_quantize(x.data_ptr(), plan.slot.data_ptr(), plan.place.data_ptr(), at[0], M, T, plan.top_k, D,
                                       dirs, plan.offs.data_ptr(), G, *at[1:], _raw_stream(dev.index)), "mxfp8_gather_quantize")
    return q_row, s_row, q_col, s_col


def mxfp4_gather_quantize(x: torch.Tensor, plan: MoePlan):
    """``mxfp4_quantize_2d(moe_gather(x, plan), offs=plan.offs)`` without the rows in between: (q [rows, D/2], s).  D a
    multiple of 32.  Rows past the last group are not written."""
    if not _good_rows(x, _plan_of(plan).tokens, 32, plan):
        _rows_matrix(x, "x", plan.tokens, "tokens", 32)
        _cuda(x, plan.offs)
    (T, D), M, G, dev = x.shape, plan.rows, plan.offs.shape[0], x.device
    q, s = _u8((M, D // 2), dev), _u8(_group_bytes(M, D, G), dev)
    check(load().mxfp4_gather_quantize(x.data_ptr(), plan.slot.data_ptr(), plan.place.data_ptr(), M, T, plan.top_k, D,
                                       plan.offs.data_ptr(), G, q.data_ptr(), s.data_ptr(), _raw_stream(dev.index)),
          "mxfp4_gather_quantize")
    return q, s


def mxfp8_dequantize_2d(q: torch.Tensor, s: torch.Tensor, direction: int = ROW, scale_layout: int = SCALES_BLOCKED,
                        offs: torch.Tensor | None = None) -> torch.Tensor:
    """The values that one copy of ``mxfp8_quantize_2d`` (with the same layout and offs) stands for, in bf16: of the
    row-wise copy q [M, K] (ROW) or of the column-wise one q [K, M] (COL), in q's shape.  Exact, but for values below
    bf16's smallest subnormal.  What lies in no group is 0."""
    _tensor(q, "q", torch.uint8, 2)
    if direction not in (ROW, COL):
        raise ValueError("direction: ROW or COL expected")
    if scale_layout not in (SCALES_COMPACT, SCALES_BLOCKED):
        raise ValueError("scale_layout: SCALES_COMPACT or SCALES_BLOCKED expected")
    M, K = q.shape if direction == ROW else q.shape[::-1]
    if K < 32 or K % 32 or (direction == COL and M % 32):
        raise ValueError(f"q: multiples of 32 expected, got {tuple(q.shape)}")
    G = 1
    if offs is not None:
        _offsets(offs)
        G = offs.shape[0]
    if scale_layout == SCALES_COMPACT:
        need = q.numel() // 32
    elif direction == ROW:
        need = mxfp8_scale_bytes(M, K, G, SCALES_BLOCKED) if G > 1 else _expert_blocked_bytes(M, K)
    else:
        need = mxfp8_scale_bytes_colgroups(K, M, G) if G > 1 else _expert_blocked_bytes(K, M)
    _bytes_at_least(s, "s", need)
    _cuda(q, s, offs)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    check(load().mxfp8_dequantize(q.data_ptr(), s.data_ptr(), M, K, direction, scale_layout,
                                  None if offs is None else offs.data_ptr(), G, out.data_ptr(),
                                  _raw_stream(q.device.index)), "mxfp8_dequantize")
    return out


# ---------------------------------------------------------------- activations kept in 8 bits
def mxfp8_swiglu_bwd_quantize_mxfp8(dh: torch.Tensor, h1, h3, offs: torch.Tensor, dev_status: torch.Tensor | None = None):
    """``mxfp8_swiglu_bwd_quantize`` with h1 and h3 kept in 8 bits: each (q [M, H], s [M, H/32]) as
    ``mxfp8_quantize_2d(h, ROW, SCALES_COMPACT)`` gives them.  Returns what that call does for the values they stand for."""
    _tensor(dh, "dh", torch.bfloat16, 2)
    M, H = dh.shape
    if H < 32 or H % 32 or M % 32:
        raise ValueError(f"dh: multiples of 32 expected, got {tuple(dh.shape)}")
    for name, h in (("h1", h1), ("h3", h3)):
        if not isinstance(h, (tuple, list)) or len(h) != 2:
            raise ValueError(f"{name}: expected (codes, scales)")
        _tensor(h[0], f"{name} codes", torch.uint8, shape=(M, H))
        _bytes_at_least(h[1], f"{name} scales", M * (H // 32))
    _offsets(offs)
    _status_word(dev_status)
    _cuda(dh, *h1, *h3, offs, dev_status)
    G, dev = offs.shape[0], dh.device

    def outs():
        return (_u8((M, H), dev), _u8(mxfp8_scale_bytes(M, H, G, SCALES_BLOCKED), dev), _u8((H, M), dev),
                _u8(mxfp8_scale_bytes_colgroups(H, M, G), dev))

    o1, o3 = outs(), outs()
    check(load().mxfp8_swiglu_bwd_quantize_mxfp8(dh.data_ptr(), *(t.data_ptr() for t in (*h1, *h3)), M, H, offs.data_ptr(), G,
                                                 *(t.data_ptr() for t in (*o1, *o3)),
                                                 None if dev_status is None else dev_status.data_ptr(),
                                                 _raw_stream(dev.index)), "mxfp8_swiglu_bwd_quantize_mxfp8")
    return o1, o3


def _keep_mxfp8(x):
    """An activation for the backward, in 8 bits: (codes, compact scales)."""
    return mxfp8_quantize_2d(x, ROW, SCALES_COMPACT)[:2]


# ---------------------------------------------------------------- the layer
class _Mxfp8MoeSwiGLU(torch.autograd.Function):
    """Route, plan, gather + quantize, gate and up with SwiGLU, down, combine.  The backward's rows are quantized the
    same way, straight from dout, and the tokens' gradients are added up from the experts'."""

    @staticmethod
    def forward(ctx, x, logits, Wg, Wu, Wd, bias, route, quads, keep8, dev_status):
        need_dx, need_dl, need_dWg, need_dWu, need_dWd = ctx.needs_input_grad[:5]
        front = need_dx or need_dWg or need_dWu
        st = ctx.dev_status = dev_status
        ctx.empty = None
        if x.shape[0] == 0:
            ctx.empty = [(t.shape, t.dtype) for t in (x, logits, Wg, Wu, Wd)]
            return torch.empty_like(x)
        qg, qu, qd = quads
        qg = _check_quad(qg, Wg, need_dx) if qg is not None else quantize_expert_weights(Wg)
        qu = _check_quad(qu, Wu, need_dx) if qu is not None else quantize_expert_weights(Wu)
        qd = _check_quad(qd, Wd, front) if qd is not None else quantize_expert_weights(Wd)
        experts, weights = _route(logits, bias, route)
        # the backward's quantizations run along the tokens too, in blocks of 32
        plan = moe_plan(experts, Wg.shape[0], 32 if front or need_dWd else 1)
        dirs = ROW | (COL if need_dWg or need_dWu else 0)
        xq, xs, xTq, xTs = mxfp8_gather_quantize(x, plan, dirs, dev_status=st)
        h1, h3, hq, hs, hTq, hTs = mxfp8_grouped_mm_swiglu_fwd(xq, xs, *qg[:2], *qu[:2], plan.offs, token_wise=need_dWd,
                                                               dev_status=st)
        y = mxfp8_grouped_mm_fwd(hq, hs, *qd[:2], plan.offs, dev_status=st)
        ctx.plan, ctx.route = plan, route
        # what the backward reads of h1, h3 and y: themselves, or 8 bits of each
        kept = []
        for t, needed in ((h1, front), (h3, front), (y, need_dl)):
            kept += (None, None) if not needed else _keep_mxfp8(t) if keep8 else (t, None)
        ctx.save_for_backward(logits if need_dl else None, experts, weights, *kept, xTq, xTs, hTq, hTs, qg[2], qg[3], qu[2],
                              qu[3], qd[2], qd[3])
        return _combine(y, plan.place, weights)

    @staticmethod
    @_first_order
    def backward(ctx, dout):
        if ctx.empty is not None:  # no tokens: no gradients
            return tuple(dout.new_zeros(s, dtype=d) if n else None
                         for (s, d), n in zip(ctx.empty, ctx.needs_input_grad)) + (None,) * 5
        (logits, experts, weights, h1, h1_s, h3, h3_s, y, y_s, xTq, xTs, hTq, hTs, gTq, gTs, uTq, uTs, dTq,
         dTs) = ctx.saved_tensors
        need_dx, need_dl, need_dWg, need_dWu, need_dWd = ctx.needs_input_grad[:5]
        plan, st = ctx.plan, ctx.dev_status
        offs = plan.offs
        dout = _incoming(dout)
        front = need_dx or need_dWg or need_dWu
        dlogits = dx = dWg = dWu = dWd = None
        if need_dl:
            if y_s is not None:
                y = mxfp8_dequantize_2d(y, y_s, ROW, SCALES_COMPACT)
            _, dw = _combine_bwd(dout, y, plan.slot, plan.place, weights, False, True)
            dlogits = _route_bwd(logits, experts, dw, ctx.route)
        if front or need_dWd:
            dirs = (ROW if front else 0) | (COL if need_dWd else 0)
            dq, ds, dqT, dsT = mxfp8_gather_quantize(dout, plan, dirs, weights, dev_status=st)
            if need_dWd:
                dWd = mxfp8_grouped_mm_wgrad(dqT, dsT, hTq, hTs, offs, dev_status=st)
        if front:
            dh = mxfp8_grouped_mm_dgrad(dq, ds, dTq, dTs, offs, dev_status=st)
            if h1_s is not None:
                a1, a3 = mxfp8_swiglu_bwd_quantize_mxfp8(dh, (h1, h1_s), (h3, h3_s), offs, dev_status=st)
            else:
                a1, a3 = mxfp8_swiglu_bwd_quantize(dh, h1, h3, offs, dev_status=st)
            if need_dx:
                rows = mxfp8_grouped_mm_dgrad2(a1[0], a1[1], gTq, gTs, a3[0], a3[1], uTq, uTs, offs, dev_status=st)
                dx = _combine(rows, plan.place, None)
            if need_dWg:
                dWg = mxfp8_grouped_mm_wgrad(a1[2], a1[3], xTq, xTs, offs, dev_status=st)
            if need_dWu:
                dWu = mxfp8_grouped_mm_wgrad(a3[2], a3[3], xTq, xTs, offs, dev_status=st)
        return dx, dlogits, dWg, dWu, dWd, None, None, None, None, None


def mxfp8_moe_swiglu(x: torch.Tensor, router_logits: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
                     top_k: int, *, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
                     top_groups: int | None = None, group_score: str = "top2", renormalize: bool = False,
                     scale: float = 1.0, w_mxfp8=None, weight_cache=None, checkpoint_mxfp8: bool = False,
                     dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """A routed SwiGLU layer for any number of tokens, differentiable in x, the logits and the weights:

        out[t] = sum over the selected e of w[t, e] (silu(x[t] Wg[e]^T) * (x[t] Wu[e]^T)) Wd[e]^T

    x [T, D], Wg and Wu [E, H, D], Wd [E, D, H] bf16, D and H multiples of 32; router_logits [T, E] fp32, bf16 or fp16;
    out [T, D] bf16.  Routing as ``moe_route``, the experts as ``mxfp8_swiglu_expert`` (and the same numbers as
    ``moe_route``, ``moe_plan``, ``moe_gather``, ``mxfp8_swiglu_expert`` and ``moe_combine`` in turn); token rows are
    gathered inside the quantizations, forward and backward.  It does not wait for the device.

    w_mxfp8, weight_cache: as for ``mxfp8_swiglu_expert``.  checkpoint_mxfp8: what the backward reads of h1, h3 and the
    experts' rows is kept in MXFP8 (1.03 bytes a value instead of 2; x and h are in 8 bits either way); outputs stay as they
    are, gradients are those at the rounded values.  dev_status: an int32 word (``new_status``) that the kernels
    report errors into, to be read with ``read_status``."""
    for name, t, dim in (("x", x, 2), ("Wg", Wg, 3), ("Wu", Wu, 3), ("Wd", Wd, 3)):
        _tensor(t, name, torch.bfloat16, dim)
    E, H, D = Wg.shape
    if tuple(Wu.shape) != (E, H, D) or tuple(Wd.shape) != (E, D, H) or x.shape[1] != D:
        raise ValueError("shapes: x [T, D], Wg and Wu [E, H, D], Wd [E, D, H]")
    if D < 32 or D % 32 or H < 32 or H % 32:
        raise ValueError(f"D and H must be positive multiples of 32, got {D} and {H}")
    T = x.shape[0]
    if not isinstance(router_logits, torch.Tensor) or router_logits.dtype not in LOGITS_TYPES \
            or tuple(router_logits.shape) != (T, E):
        raise ValueError(f"router_logits: expected [{T}, {E}] in fp32, bf16 or fp16")
    route = _route_args(T, E, top_k, score, bias, groups, top_groups, group_score, renormalize, scale)
    _status_word(dev_status)
    if w_mxfp8 is not None and weight_cache is not None:
        raise ValueError("pass w_mxfp8 or weight_cache, not both")
    _on_device(x, router_logits, Wg, Wu, Wd, bias, dev_status)
    if weight_cache is not None:
        w_mxfp8 = tuple(weight_cache.get(W) for W in (Wg, Wu, Wd))
    quads = tuple(w_mxfp8) if w_mxfp8 is not None else (None, None, None)
    if len(quads) != 3:
        raise ValueError("w_mxfp8 must be (gate, up, down) quadruples")
    x, router_logits = x.contiguous(), router_logits.contiguous()
    if bias is not None:
        bias = bias.detach().contiguous()
    if not torch.is_grad_enabled():  # ctx.needs_input_grad asks requires_grad alone, and is set in evaluation too
        x, router_logits, Wg, Wu, Wd = (t.detach() for t in (x, router_logits, Wg, Wu, Wd))
    return _Mxfp8MoeSwiGLU.apply(x, router_logits, Wg, Wu, Wd, bias, route, quads, bool(checkpoint_mxfp8),
                                 dev_status)
