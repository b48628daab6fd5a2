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

from . import (COL, MAX_GROUPS, ROW, SCALES_BLOCKED, SCALES_COMPACT, _bytes_at_least, _cuda, _expert_blocked_bytes,
               _first_order, _here, _offsets, _status_word, _tensor, _u8, check, load, mxfp8_check_offsets, new_status, read_status)

# torch's handle of a device's current stream as an integer: a few tenths of a microsecond, where
# torch.cuda.current_stream() builds an object in several
_raw_stream = torch._C._cuda_getCurrentRawStream


def _width(K: int, name: str):
    if K < 32 or K % 32:
        raise ValueError(f"{name}: the last dimension must be a positive multiple of 32, got {K}")


def _group_bytes(M: int, K: int, G: int) -> int:
    """Blocked scale bytes of M rows in G groups (the bound of mxfp8_scale_bytes)."""
    return ((M + 127) // 128 + G) * ((K + 127) // 128) * 512


def _col_bytes(R: int, M: int, G: int) -> int:
    """Blocked scale bytes of R token-wise quantized rows (the bound of mxfp8_scale_bytes_colgroups)."""
    return ((R + 127) // 128) * ((M + 127) // 128 + G) * 512


def _row_scales(dev, M: int, K: int, G: int, layout: int):
    if layout == SCALES_COMPACT:
        return _u8((M, K // 32), dev)
    if layout != SCALES_BLOCKED:
        raise ValueError("scale_layout: SCALES_COMPACT or SCALES_BLOCKED expected")
    return _u8(_group_bytes(M, K, G), dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


# A small call's time is the host's, and the named checks of __init__ are a third of it.  So what a correct call
# looks like is asked in one expression first, and the checks, which say what is wrong, follow where the answer is no.
# here: the device of the call, as _here returns it.
def _good(t, dtype, ndim, here):
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == here and t.dim() == ndim
            and t.is_contiguous())


def _scales(s, nbytes, here):
    return (isinstance(s, torch.Tensor) and s.dtype is torch.uint8 and s.get_device() == here and s.numel() >= nbytes
            and s.is_contiguous())


def _matrix(x, name: str, offs, other=None, other_name: str = ""):
    """Checks a bf16 matrix x [M, K], one more of its shape and its row groups; returns M, K, groups and their
    address."""
    here = _here(x)
    if not (_good(x, torch.bfloat16, 2, here) and (offs is None or _good(offs, torch.int32, 1, here))
            and (other is None or (_good(other, torch.bfloat16, 2, here) and other.shape == x.shape))):
        _tensor(x, name, torch.bfloat16, 2)
        if other is not None:
            _tensor(other, other_name, torch.bfloat16, shape=x.shape)
        _width(x.shape[1], name)
        if offs is not None:
            _offsets(offs)
        _cuda(x, other, offs)
    M, K = x.shape
    if K < 32 or K % 32:
        _width(K, name)
    if offs is None:
        return M, K, 1, None
    G = offs.shape[0]
    if not 1 <= G <= MAX_GROUPS:
        _offsets(offs)
    return M, K, G, offs.data_ptr()


def mxfp4_quantize_2d(x: torch.Tensor, scale_layout: int = SCALES_BLOCKED, offs: torch.Tensor | None = None):
    """Quantize x[M, K] (bf16) along K.  Returns (q [M, K/2], s): s [M, K/32] compact, or a flat
    blocked buffer whose row groups come from offs (none: one group), padding bytes zero.  offs must
    end at M: rows outside every group are not written."""
    M, K, G, off = _matrix(x, "x", offs)
    dev = x.device
    q, s = _u8((M, K // 2), dev), _row_scales(dev, M, K, G, scale_layout)
    check(load().mxfp4_quantize_2d(x.data_ptr(), M, K, scale_layout, off, G, q.data_ptr(), s.data_ptr(),
                                   _raw_stream(dev.index)), "mxfp4_quantize_2d")
    return q, s


def mxfp4_quantize_2d_mxfp8_cols(x: torch.Tensor, offs: torch.Tensor | None = None,
                                 dev_status: torch.Tensor | None = None):
    """Both copies of x[M, K] (bf16) that a product with an MXFP4 forward and an MXFP8 weight gradient needs, from
    one read: (q, s) as mxfp4_quantize_2d returns them and (qT [K, M], sT) as mxfp8_quantize_2d(x, COL) does, with
    blocked scales.  M and the group sizes multiples of 32."""
    M, K, G, off = _matrix(x, "x", offs)
    if M % 32:
        raise ValueError(f"x: a multiple of 32 rows is needed, got {M}")
    _status_word(dev_status)
    _cuda(dev_status)
    dev = x.device
    q, s, qT, sT = (_u8((M, K // 2), dev), _u8(_group_bytes(M, K, G), dev), _u8((K, M), dev),
                    _u8(_col_bytes(K, M, G), dev))
    check(load().mxfp4_quantize_2d_mxfp8_cols(x.data_ptr(), M, K, off, G, q.data_ptr(), s.data_ptr(), qT.data_ptr(),
                                              sT.data_ptr(), _ptr(dev_status), _raw_stream(dev.index)),
          "mxfp4_quantize_2d_mxfp8_cols")
    return q, s, qT, sT


def mxfp4_swiglu_quantize(h1: torch.Tensor, h3: torch.Tensor, scale_layout: int = SCALES_BLOCKED,
                          offs: torch.Tensor | None = None):
    """h = silu(h1) * h3 of two bf16 matrices [M, K], computed in fp32 and quantized as
    mxfp4_quantize_2d does (h is not rounded to bf16 on the way).  Returns (q, s)."""
    if h3 is None:
        _tensor(h3, "h3", torch.bfloat16)
    M, K, G, off = _matrix(h1, "h1", offs, h3, "h3")
    dev = h1.device
    q, s = _u8((M, K // 2), dev), _row_scales(dev, M, K, G, scale_layout)
    check(load().mxfp4_swiglu_quantize(h1.data_ptr(), h3.data_ptr(), M, K, scale_layout, off, G, q.data_ptr(),
                                       s.data_ptr(), _raw_stream(dev.index)), "mxfp4_swiglu_quantize")
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
    check(load().mxfp4_quantize_3d_experts(_ptr(w), G, N, K, scale_layout, _ptr(q), _ptr(s), _raw_stream(w.device.index)),
          "mxfp4_quantize_3d_experts")
    return q, s


def mxfp4_quantize_3d_experts_mxfp8_cols(w: torch.Tensor, dev_status: torch.Tensor | None = None):
    """Expert weights w[G, N, K] (bf16) for a product with an MXFP4 forward and MXFP8 gradients, from one read:
    (q [G, N, K/2], s) as mxfp4_quantize_3d_experts returns them and (qT [G, K, N], sT) as mxfp8_quantize_3d_experts(w,
    COL) does, with blocked scales.  N and K multiples of 32."""
    _tensor(w, "w", torch.bfloat16, 3)
    G, N, K = w.shape
    _width(K, "w")
    _width(N, "w^T")
    _status_word(dev_status)
    _cuda(w, dev_status)
    dev = w.device
    q, s, qT, sT = (_u8((G, N, K // 2), dev), _u8((G, _expert_blocked_bytes(N, K)), dev), _u8((G, K, N), dev),
                    _u8((G, _expert_blocked_bytes(K, N)), dev))
    check(load().mxfp4_quantize_3d_experts_mxfp8_cols(_ptr(w), G, N, K, _ptr(q), _ptr(s), _ptr(qT), _ptr(sT),
                                                      _ptr(dev_status), _raw_stream(dev.index)),
          "mxfp4_quantize_3d_experts_mxfp8_cols")
    return q, s, qT, sT


def mxfp4_dequantize_2d(q: torch.Tensor, s: torch.Tensor, scale_layout: int = SCALES_BLOCKED,
                        offs: torch.Tensor | None = None) -> torch.Tensor:
    """The values [M, K] that q [M, K/2] and s (as mxfp4_quantize_2d returns them, with the same
    layout and offs) stand for, in bf16: every E2M1 value times a power of two is a bf16."""
    here = _here(q)
    good = _good(q, torch.uint8, 2, here) and (offs is None or _good(offs, torch.int32, 1, here))
    if not good:
        _tensor(q, "q", torch.uint8, 2)
    M, K = q.shape
    K *= 2
    if K < 32 or K % 32:
        _width(K, "q")
    if not good and offs is not None:
        _offsets(offs)
    G = offs.numel() if offs is not None else 1
    if not 1 <= G <= MAX_GROUPS:
        _offsets(offs)
    need = M * (K // 32) if scale_layout == SCALES_COMPACT else \
        (_group_bytes(M, K, G) if offs is not None else _expert_blocked_bytes(M, K))
    if not (good and _scales(s, need, here)):
        _bytes_at_least(s, "s", need)
        _cuda(q, s, offs)
    dev = q.device
    out = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    check(load().mxfp4_dequantize(q.data_ptr(), s.data_ptr(), 1, M, K, scale_layout, _ptr(offs), G, out.data_ptr(),
                                  _raw_stream(dev.index)), "mxfp4_dequantize")
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
    check(load().mxfp4_dequantize(_ptr(q), _ptr(s), G, N, K, scale_layout, None, 0, _ptr(out), _raw_stream(q.device.index)),
          "mxfp4_dequantize")
    return out


def mxfp4_grouped_mm_fwd(a_q, a_s, w_q, w_s, offs, out=None, dev_status=None):
    """out[m, n] = sum_k A[m,k] W[g][n,k] for rows m of group g; a_q [M, K/2] with blocked row-group
    scales, w_q [G, N, K/2] with blocked per-expert scales; bf16 [M, N].  dev_status: an int32 word (``new_status``) for
    errors the device finds; without one they are not reported."""
    here = _here(a_q)
    good = _good(a_q, torch.uint8, 2, here) and _good(w_q, torch.uint8, 3, here) and _good(offs, torch.int32, 1, here)
    if not good:
        _tensor(a_q, "a_q", torch.uint8, 2)
        _tensor(w_q, "w_q", torch.uint8, 3)
    (M, Kb), (G, N, Wb) = a_q.shape, w_q.shape
    K = 2 * Kb
    if Wb != Kb:
        _tensor(w_q, "w_q", torch.uint8, shape=(G, N, Kb))
    if K < 32 or K % 32:
        _width(K, "a_q")
    if not good or offs.numel() != G or not 1 <= G <= MAX_GROUPS:
        _offsets(offs, G)
    a_bytes, w_bytes = _group_bytes(M, K, G), G * _expert_blocked_bytes(N, K)
    if not (good and _scales(a_s, a_bytes, here) and _scales(w_s, w_bytes, here)) or out is not None or dev_status is not None:
        _bytes_at_least(a_s, "a_s", a_bytes)
        _bytes_at_least(w_s, "w_s", w_bytes)
        if out is not None:
            _tensor(out, "out", torch.bfloat16, shape=(M, N))
        _status_word(dev_status)
        _cuda(a_q, a_s, w_q, w_s, offs, out, dev_status)
    dev = a_q.device
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    check(load().mxfp4_grouped_mm_fwd(a_q.data_ptr(), a_s.data_ptr(), w_q.data_ptr(), w_s.data_ptr(), offs.data_ptr(), G,
                                      M, N, K, out.data_ptr(), _ptr(dev_status), _raw_stream(dev.index)),
          "mxfp4_grouped_mm_fwd")
    return out


def _on_one_device(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("mxfp4: every tensor must live on a CUDA device")
        if t.device != ts[0].device:
            raise ValueError(f"mxfp4: tensors on {ts[0].device} and {t.device}")
    if _here(ts[0]) < 0:
        raise ValueError(f"mxfp4: the tensors live on {ts[0].device}, which is not the current device, on which the "
                         "kernels launch")


def _carve(like: torch.Tensor, *sizes: int):
    """One allocation for several buffers of a call: the tensor that owns it and their addresses, each on a
    256-byte boundary.  (An allocation costs the host as much as a launch; a step at a small size has few of both.)"""
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += (n + 255) // 256 * 256
    buf = _u8(total, like.device)
    base = buf.data_ptr()
    return (buf,) + tuple(base + at for at in starts)


class _ToMxfp4ThenScaledGroupedMM(torch.autograd.Function):
    """Forward: A and W quantized to MXFP4 along K, one grouped product.  Backward: both gradients
    on the MXFP8 path, dA = dOut W and dW = dOut^T A with every operand in MXFP8 along its own
    contraction.  Gradients keep 8 bits because E2M1's single mantissa bit rounds away most of what
    small gradients carry; the forward, which tolerates it best, takes the 4-bit rate.

    Shapes, types and devices are checked in to_mxfp4_then_scaled_grouped_mm; the calls below go to the
    library directly."""

    @staticmethod
    def forward(ctx, A, W, offs, w_mxfp4, check_offsets, dev_status):
        need_dA, need_dW = ctx.needs_input_grad[:2]
        L, stream = load(), _raw_stream(A.device.index)
        (M, K), (G, N, _) = A.shape, W.shape
        st = ctx.dev_status = dev_status
        if check_offsets:
            if st is None:
                st = new_status(A.device)
            mxfp8_check_offsets(offs, M, 32 if need_dW else 1, st)
        status, off = _ptr(st), offs.data_ptr()
        A = A.contiguous()
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
        aT = wT = None
        if M:
            a_sizes = (M * (K // 2), _group_bytes(M, K, G))
            if w_mxfp4 is None:
                Wc = W.contiguous()
                _hold, aq, as_, wq, ws = _carve(A, *a_sizes, G * N * (K // 2), G * _expert_blocked_bytes(N, K))
                if need_dA:  # W's copy along N for dA, from the same read
                    wT, wTq, wTs = _carve(A, G * K * N, G * _expert_blocked_bytes(K, N))
                    check(L.mxfp4_quantize_3d_experts_mxfp8_cols(Wc.data_ptr(), G, N, K, wq, ws, wTq, wTs, status,
                                                                 stream), "mxfp4_quantize_3d_experts_mxfp8_cols")
                else:
                    check(L.mxfp4_quantize_3d_experts(Wc.data_ptr(), G, N, K, SCALES_BLOCKED, wq, ws, stream),
                          "mxfp4_quantize_3d_experts")
            else:
                _hold, aq, as_ = _carve(A, *a_sizes)
                wq, ws = w_mxfp4[0].data_ptr(), w_mxfp4[1].data_ptr()
            if need_dW:  # the token-wise MXFP8 copy for dW, half the bytes of A itself, from the same read
                aT, aTq, aTs = _carve(A, K * M, _col_bytes(K, M, G))
                check(L.mxfp4_quantize_2d_mxfp8_cols(A.data_ptr(), M, K, off, G, aq, as_, aTq, aTs, status, stream),
                      "mxfp4_quantize_2d_mxfp8_cols")
            else:
                check(L.mxfp4_quantize_2d(A.data_ptr(), M, K, SCALES_BLOCKED, off, G, aq, as_, stream),
                      "mxfp4_quantize_2d")
            check(L.mxfp4_grouped_mm_fwd(aq, as_, wq, ws, off, G, M, N, K, out.data_ptr(), status, stream),
                  "mxfp4_grouped_mm_fwd")
        if check_offsets:
            read_status(st, "to_mxfp4_then_scaled_grouped_mm (group offsets)")
        ctx.save_for_backward(aT, wT, W if need_dA and wT is None else None, offs)
        ctx.sizes = (G, M, N, K)
        return out

    @staticmethod
    @_first_order
    def backward(ctx, dOut):
        aT, wT, W, offs = ctx.saved_tensors
        need_dA, need_dW = ctx.needs_input_grad[:2]
        G, M, N, K = ctx.sizes
        dOut = dOut.contiguous().to(torch.bfloat16)
        dA = torch.empty((M, K), dtype=torch.bfloat16, device=dOut.device) if need_dA else None
        if M == 0:
            return dA, dOut.new_zeros((G, N, K)) if need_dW else None, None, None, None, None
        dW = torch.empty((G, N, K), dtype=torch.bfloat16, device=dOut.device) if need_dW else None
        L, stream, off, status = load(), _raw_stream(dOut.device.index), offs.data_ptr(), _ptr(ctx.dev_status)
        row = (M * N, _group_bytes(M, N, G)) if need_dA else (0, 0)
        w = (G * K * N, G * _expert_blocked_bytes(K, N)) if need_dA and wT is None else (0, 0)
        col = (N * M, _col_bytes(N, M, G)) if need_dW else (0, 0)
        _hold, dq, ds, wq, ws, dTq, dTs = _carve(dOut, *row, *w, *col)
        dirs = (ROW if need_dA else 0) | (COL if need_dW else 0)
        check(L.mxfp8_quantize_2d(dOut.data_ptr(), M, N, dirs, SCALES_BLOCKED, off, G, dq if need_dA else None,
                                  ds if need_dA else None, dTq if need_dW else None, dTs if need_dW else None, status,
                                  stream), "mxfp8_quantize_2d")
        if need_dA:
            if wT is not None:
                wq = wT.data_ptr()
                ws = wq + (G * K * N + 255) // 256 * 256  # as _carve laid them out in the forward
            else:
                W = W.contiguous()
                check(L.mxfp8_quantize_3d_experts(W.data_ptr(), G, N, K, COL, SCALES_BLOCKED, None, None, wq, ws, status,
                                                  stream), "mxfp8_quantize_3d_experts")
            check(L.mxfp8_grouped_mm_dgrad(dq, ds, wq, ws, off, G, M, N, K, dA.data_ptr(), status, stream),
                  "mxfp8_grouped_mm_dgrad")
        if need_dW:
            q = aT.data_ptr()
            s = q + (K * M + 255) // 256 * 256  # as _carve laid them out in the forward
            check(L.mxfp8_grouped_mm_wgrad(dTq, dTs, q, s, off, G, M, N, K, dW.data_ptr(), status, stream),
                  "mxfp8_grouped_mm_wgrad")
        return dA, dW, None, None, None, None


def to_mxfp4_then_scaled_grouped_mm(A: torch.Tensor, W: torch.Tensor, offs: torch.Tensor, *, w_mxfp4=None,
                                    check_offsets: bool = True, dev_status: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable grouped GEMM with an MXFP4 forward: out[m] = A[m] @ W[g]^T for rows m of group
    g (offs = int32 cumulative end rows).  A [M, K] bf16, W [G, N, K] bf16, out [M, N] bf16; K and N
    multiples of 32.  Quantization is the identity for gradients, which are computed from MXFP8
    operands (group sizes must then be multiples of 32 where W needs a gradient).  With gradients
    disabled (no_grad, inference_mode) nothing is prepared for a backward, and any group sizes go.

    w_mxfp4: (q, s) from ``mxfp4_quantize_3d_experts(W)``, when the weights are kept quantized.
    check_offsets: as for ``to_mxfp8_then_scaled_grouped_mm`` (a device check, one stream
    synchronization per forward).
    dev_status: an int32 word (``new_status``) that the kernels of the forward and of the backward report errors into,
    to be read with ``read_status``.  Without one only a forward that checks its offsets reports what its kernels find."""
    if A.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise ValueError("to_mxfp4_then_scaled_grouped_mm expects bf16 A and W")
    if offs.dtype != torch.int32:
        raise ValueError("offs must be int32")
    if A.dim() != 2 or W.dim() != 3 or A.shape[1] != W.shape[2]:
        raise ValueError("to_mxfp4_then_scaled_grouped_mm: A [M, K] and W [G, N, K] expected")
    M, (G, N, K) = A.shape[0], W.shape
    _width(K, "A")
    _width(N, "W^T")
    _offsets(offs, G)
    if w_mxfp4 is not None:
        if len(w_mxfp4) != 2:
            raise ValueError("w_mxfp4 must be (codes, scales)")
        _tensor(w_mxfp4[0], "w_mxfp4 codes", torch.uint8, shape=(G, N, K // 2))
        _bytes_at_least(w_mxfp4[1], "w_mxfp4 scales", G * _expert_blocked_bytes(N, K))
    _status_word(dev_status)
    _on_one_device(A, W, offs, *(w_mxfp4 or ()), *(() if dev_status is None else (dev_status,)))
    if w_mxfp4 is not None and not (w_mxfp4[0].is_contiguous() and w_mxfp4[1].is_contiguous()):
        raise ValueError("w_mxfp4: tensors must be contiguous")
    if not offs.is_contiguous():
        raise ValueError("offs: must be contiguous")
    if M % 32 and W.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"A: a multiple of 32 rows is needed where W needs a gradient, got {M}")
    if not torch.is_grad_enabled():  # ctx.needs_input_grad asks requires_grad alone, and is set in evaluation too
        A, W = A.detach(), W.detach()
    return _ToMxfp4ThenScaledGroupedMM.apply(A, W, offs, w_mxfp4, bool(check_offsets), dev_status)
