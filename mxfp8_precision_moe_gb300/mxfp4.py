"""The 4-bit side of the routed experts: MXFP4 quantization, its inverse, the grouped product and
a differentiable product (C ABI: ``include/mxfp4moe.h``).

MXFP4 is E2M1 elements with one E8M0 scale per 32 elements along the contraction (OCP
Microscaling v1.0): e = floor(log2 amax) - 2 clamped at -127, elements x 2^-e rounded to nearest
even and saturated at 6, scale byte e + 127.  Codes are ``torch.uint8``, two to a byte along the
last dimension (element 2i in the low half of byte i); scales are ``torch.uint8`` in the same
compact or blocked layouts as the MXFP8 ones.
"""
from __future__ import annotations

import torch

from . import (COL, ROW, SCALES_BLOCKED, SCALES_COMPACT, _bytes_at_least, _cuda, _expert_blocked_bytes, _offsets, _p,
               _status_word, _stream, _tensor, _u8, check, load, mxfp8_check_offsets, mxfp8_grouped_mm_dgrad,
               mxfp8_grouped_mm_wgrad, mxfp8_quantize_2d, mxfp8_quantize_3d_experts, mxfp8_scale_bytes, new_status,
               read_status)


def _width(K: int, name: str):
    if K < 32 or K % 32:
        raise ValueError(f"{name}: the last dimension must be a positive multiple of 32, got {K}")


def _row_scales(M: int, K: int, G: int, layout: int, device):
    if layout == SCALES_COMPACT:
        return _u8((M, K // 32), device)
    if layout != SCALES_BLOCKED:
        raise ValueError("scale_layout: SCALES_COMPACT or SCALES_BLOCKED expected")
    return _u8((mxfp8_scale_bytes(M, K, G, SCALES_BLOCKED),), device)


def mxfp4_quantize_2d(x: torch.Tensor, scale_layout: int = SCALES_BLOCKED, offs: torch.Tensor | None = None):
    """Quantize x[M, K] (bf16) along K.  Returns (q [M, K/2], s): s [M, K/32] compact, or a flat
    blocked buffer whose row groups come from offs (none: one group), padding bytes zero.  offs must
    end at M: rows outside every group are not written."""
    _tensor(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _width(K, "x")
    if offs is not None:
        _offsets(offs)
    _cuda(x, offs)
    G = int(offs.numel()) if offs is not None else 1
    q, s = _u8((M, K // 2), x.device), _row_scales(M, K, G, scale_layout, x.device)
    check(load().mxfp4_quantize_2d(_p(x), M, K, scale_layout, _p(offs), G, _p(q), _p(s), _stream(x.device)),
          "mxfp4_quantize_2d")
    return q, s


def mxfp4_swiglu_quantize(h1: torch.Tensor, h3: torch.Tensor, scale_layout: int = SCALES_BLOCKED,
                          offs: torch.Tensor | None = None):
    """h = silu(h1) * h3 of two bf16 matrices [M, K], computed in fp32 and quantized as
    mxfp4_quantize_2d does (h is not rounded to bf16 on the way).  Returns (q, s)."""
    _tensor(h1, "h1", torch.bfloat16, 2)
    M, K = h1.shape
    _tensor(h3, "h3", torch.bfloat16, shape=(M, K))
    _width(K, "h1")
    if offs is not None:
        _offsets(offs)
    _cuda(h1, h3, offs)
    G = int(offs.numel()) if offs is not None else 1
    q, s = _u8((M, K // 2), h1.device), _row_scales(M, K, G, scale_layout, h1.device)
    check(load().mxfp4_swiglu_quantize(_p(h1), _p(h3), M, K, scale_layout, _p(offs), G, _p(q), _p(s),
                                       _stream(h1.device)), "mxfp4_swiglu_quantize")
    return q, s


def mxfp4_quantize_3d_experts(w: torch.Tensor, scale_layout: int = SCALES_BLOCKED):
    """Quantize expert weights w[G, N, K] (bf16) along K.  Returns (q [G, N, K/2], s): s
    [G, N, K/32] compact, or [G, bytes] with one blocked buffer per expert."""
    _tensor(w, "w", torch.bfloat16, 3)
    G, N, K = w.shape
    _width(K, "w")
    _cuda(w)
    q = _u8((G, N, K // 2), w.device)
    if scale_layout == SCALES_COMPACT:
        s = _u8((G, N, K // 32), w.device)
    else:
        s = _u8((G, _expert_blocked_bytes(N, K)), w.device)
    check(load().mxfp4_quantize_3d_experts(_p(w), G, N, K, scale_layout, _p(q), _p(s), _stream(w.device)),
          "mxfp4_quantize_3d_experts")
    return q, s


def mxfp4_dequantize_2d(q: torch.Tensor, s: torch.Tensor, scale_layout: int = SCALES_BLOCKED,
                        offs: torch.Tensor | None = None) -> torch.Tensor:
    """The values [M, K] that q [M, K/2] and s (as mxfp4_quantize_2d returns them, with the same
    layout and offs) stand for, in bf16: every E2M1 value times a power of two is a bf16."""
    _tensor(q, "q", torch.uint8, 2)
    M, K = q.shape[0], 2 * q.shape[1]
    _width(K, "q")
    if offs is not None:
        _offsets(offs)
    G = int(offs.numel()) if offs is not None else 1
    need = M * (K // 32) if scale_layout == SCALES_COMPACT else \
        (mxfp8_scale_bytes(M, K, G, SCALES_BLOCKED) if offs is not None else _expert_blocked_bytes(M, K))
    _bytes_at_least(s, "s", need)
    _cuda(q, s, offs)
    out = torch.empty((M, K), dtype=torch.bfloat16, device=q.device)
    check(load().mxfp4_dequantize(_p(q), _p(s), 1, M, K, scale_layout, _p(offs), G, _p(out), _stream(q.device)),
          "mxfp4_dequantize")
    return out


def mxfp4_dequantize_3d_experts(q: torch.Tensor, s: torch.Tensor,
                                scale_layout: int = SCALES_BLOCKED) -> torch.Tensor:
    """The values [G, N, K] of expert weights quantized by mxfp4_quantize_3d_experts, in bf16."""
    _tensor(q, "q", torch.uint8, 3)
    G, N, K = q.shape[0], q.shape[1], 2 * q.shape[2]
    _width(K, "q")
    _bytes_at_least(s, "s", G * (N * (K // 32) if scale_layout == SCALES_COMPACT else _expert_blocked_bytes(N, K)))
    _cuda(q, s)
    out = torch.empty((G, N, K), dtype=torch.bfloat16, device=q.device)
    check(load().mxfp4_dequantize(_p(q), _p(s), G, N, K, scale_layout, None, 0, _p(out), _stream(q.device)),
          "mxfp4_dequantize")
    return out


def mxfp4_grouped_mm_fwd(a_q, a_s, w_q, w_s, offs, out=None, dev_status=None):
    """out[m, n] = sum_k A[m,k] W[g][n,k] for rows m of group g; a_q [M, K/2] with blocked row-group
    scales, w_q [G, N, K/2] with blocked per-expert scales; bf16 [M, N]."""
    _tensor(a_q, "a_q", torch.uint8, 2)
    _tensor(w_q, "w_q", torch.uint8, 3)
    M, K = a_q.shape[0], 2 * a_q.shape[1]
    G, N, _ = w_q.shape
    _tensor(w_q, "w_q", torch.uint8, shape=(G, N, K // 2))
    _width(K, "a_q")
    _offsets(offs, G)
    _bytes_at_least(a_s, "a_s", mxfp8_scale_bytes(M, K, G, SCALES_BLOCKED))
    _bytes_at_least(w_s, "w_s", G * _expert_blocked_bytes(N, K))
    if out is not None:
        _tensor(out, "out", torch.bfloat16, shape=(M, N))
    _status_word(dev_status)
    _cuda(a_q, a_s, w_q, w_s, offs, out, dev_status)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    check(load().mxfp4_grouped_mm_fwd(_p(a_q), _p(a_s), _p(w_q), _p(w_s), _p(offs), G, M, N, K, _p(out),
                                      _p(dev_status), _stream(a_q.device)), "mxfp4_grouped_mm_fwd")
    return out


class _ToMxfp4ThenScaledGroupedMM(torch.autograd.Function):
    """Forward: A and W quantized to MXFP4 along K, one grouped product.  Backward: both gradients
    on the MXFP8 path, dA = dOut W and dW = dOut^T A with every operand in MXFP8 along its own
    contraction.  Gradients keep 8 bits because E2M1's single mantissa bit rounds away most of what
    small gradients carry; the forward, which tolerates it best, takes the 4-bit rate."""

    @staticmethod
    def forward(ctx, A, W, offs, w_mxfp4, check_offsets):
        need_dA, need_dW = ctx.needs_input_grad[:2]
        st = None
        if check_offsets:
            st = new_status(A.device)
            mxfp8_check_offsets(offs, A.shape[0], 32 if need_dW else 1, st)
        A = A.contiguous()
        aq, as_ = mxfp4_quantize_2d(A, SCALES_BLOCKED, offs)
        wq, ws = w_mxfp4 if w_mxfp4 is not None else mxfp4_quantize_3d_experts(W.contiguous())
        out = mxfp4_grouped_mm_fwd(aq, as_, wq, ws, offs, dev_status=st)
        aTq = aTs = None
        if need_dW and A.shape[0]:  # the token-wise MXFP8 copy for dW: half the bytes of A itself
            _, _, aTq, aTs = mxfp8_quantize_2d(A, COL, SCALES_BLOCKED, offs, st)
        if st is not None:
            read_status(st, "to_mxfp4_then_scaled_grouped_mm (group offsets)")
        ctx.save_for_backward(aTq, aTs, W if need_dA else None, offs)
        ctx.shape_W = W.shape
        return out

    @staticmethod
    def backward(ctx, dOut):
        aTq, aTs, W, offs = ctx.saved_tensors
        need_dA, need_dW = ctx.needs_input_grad[:2]
        dirs = (ROW if need_dA else 0) | (COL if need_dW else 0)
        dA = dW = None
        if dOut.shape[0] == 0:
            return (dOut.new_empty((0, ctx.shape_W[2])) if need_dA else None,
                    dOut.new_zeros(ctx.shape_W) if need_dW else None, None, None, None)
        dq, ds, dTq, dTs = mxfp8_quantize_2d(dOut.contiguous().to(torch.bfloat16), dirs, SCALES_BLOCKED, offs)
        if need_dA:
            _, _, wTq, wTs = mxfp8_quantize_3d_experts(W.detach().contiguous(), COL)
            dA = mxfp8_grouped_mm_dgrad(dq, ds, wTq, wTs, offs)
        if need_dW:
            dW = mxfp8_grouped_mm_wgrad(dTq, dTs, aTq, aTs, offs)
        return dA, dW, None, None, None


def to_mxfp4_then_scaled_grouped_mm(A: torch.Tensor, W: torch.Tensor, offs: torch.Tensor, *, w_mxfp4=None,
                                    check_offsets: bool = True) -> torch.Tensor:
    """Differentiable grouped GEMM with an MXFP4 forward: out[m] = A[m] @ W[g]^T for rows m of group
    g (offs = int32 cumulative end rows).  A [M, K] bf16, W [G, N, K] bf16, out [M, N] bf16; K and N
    multiples of 32.  Quantization is the identity for gradients, which are computed from MXFP8
    operands (group sizes must then be multiples of 32 where W needs a gradient).

    w_mxfp4: (q, s) from ``mxfp4_quantize_3d_experts(W)``, when the weights are kept quantized.
    check_offsets: as for ``to_mxfp8_then_scaled_grouped_mm`` (a device check, one stream
    synchronization per forward)."""
    if A.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise ValueError("to_mxfp4_then_scaled_grouped_mm expects bf16 A and W")
    if offs.dtype != torch.int32:
        raise ValueError("offs must be int32")
    if A.dim() != 2 or W.dim() != 3 or A.shape[1] != W.shape[2]:
        raise ValueError("to_mxfp4_then_scaled_grouped_mm: A [M, K] and W [G, N, K] expected")
    G, N, K = W.shape
    _width(K, "A")
    _width(N, "W^T")
    _offsets(offs, G)
    if w_mxfp4 is not None:
        if len(w_mxfp4) != 2:
            raise ValueError("w_mxfp4 must be (codes, scales)")
        _tensor(w_mxfp4[0], "w_mxfp4 codes", torch.uint8, shape=(G, N, K // 2))
        _bytes_at_least(w_mxfp4[1], "w_mxfp4 scales", G * _expert_blocked_bytes(N, K))
    return _ToMxfp4ThenScaledGroupedMM.apply(A, W, offs, w_mxfp4, bool(check_offsets))
