"""A routed SwiGLU layer for a few tokens in one launch (C ABI: ``mx_moe_tokens`` in
``include/mxfp4moe.h``): the serving form of the routed experts.

For token t with router logits l_t:

    S_t = the top_k largest of l_t,   w_te = softmax over S_t (or over all experts, or sigmoid)
    h_te = silu(x_t Wg_e^T) * (x_t Wu_e^T),   y_t = sum_{e in S_t} w_te h_te Wd_e^T

The weights are the quantized ones the framework already keeps, in MXFP8 or MXFP4; x and h are
quantized to the same format along each product's contraction, as on the path for long token lists.
"""
from __future__ import annotations

import torch

from . import _bytes_at_least, _cuda, _expert_blocked_bytes, _status_word, _tensor, check, load, new_status

_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without building an object

SCORES = {"softmax": 0, "softmax_all": 1, "sigmoid": 2}
MAX_TOKENS, MAX_EXPERTS, MAX_TOP_K = 64, 256, 16


class MxMoeTokens:
    """The layer over given expert weights.

    gate, up: (codes [E, H, D], blocked scales), down: (codes [E, D, H], blocked scales), as
    ``quantize_expert_weights`` (its first two tensors; a whole quadruple is accepted) or
    ``mxfp4_quantize_3d_experts`` (codes two to a byte) returns them.  The codes' width tells the
    format.  D and H multiples of 32, E <= 256, top_k <= min(E, 16), max_tokens <= 64.

    score: "softmax" (over the selected experts), "softmax_all" (over all experts) or "sigmoid".  The weight multiplies
    an expert's output.  (Where the input is to be scaled instead, which SwiGLU tells apart, and top_k is 1: scale x and
    leave the score at "softmax", whose only weight is 1.)

    The layer holds references to the weights and one workspace for each stream it is called on (a call
    captured into a graph takes one of the graph's memory).  It computes no gradients.

    A call does not wait for the device.  What the device finds (a wait between CTAs that ran out of time: the output is
    then incomplete) goes to the layer's own status word, which ``check_status`` reads, or to the caller's dev_status."""

    def __init__(self, gate, up, down, top_k: int, *, score: str = "softmax", max_tokens: int = MAX_TOKENS):
        pairs = []
        for name, w in (("gate", gate), ("up", up), ("down", down)):
            if not isinstance(w, (tuple, list)) or len(w) < 2:
                raise ValueError(f"{name}: expected (codes, scales)")
            _tensor(w[0], f"{name} codes", torch.uint8, 3)
            pairs.append((w[0], w[1]))
        (gq, gs), (uq, us), (dq, ds) = pairs
        E, H, wide = gq.shape
        D = dq.shape[1]
        if wide == D:
            bits = 8
        elif 2 * wide == D:
            bits = 4
        else:
            raise ValueError(f"gate codes [E, H, {wide}] and down codes [E, {D}, ...]: the gate's width must be D "
                             "(MXFP8) or D / 2 (MXFP4)")
        _tensor(uq, "up codes", torch.uint8, shape=(E, H, wide))
        _tensor(dq, "down codes", torch.uint8, shape=(E, D, H * bits // 8))
        if D < 32 or D % 32 or H < 32 or H % 32:
            raise ValueError(f"D and H must be positive multiples of 32, got {D} and {H}")
        if not 1 <= E <= MAX_EXPERTS:
            raise ValueError(f"1 .. {MAX_EXPERTS} experts, got {E}")
        if not 1 <= top_k <= min(E, MAX_TOP_K):
            raise ValueError(f"top_k: 1 .. {min(E, MAX_TOP_K)}, got {top_k}")
        if score not in SCORES:
            raise ValueError(f"score: one of {sorted(SCORES)}, got {score!r}")
        if not 1 <= max_tokens <= MAX_TOKENS:
            raise ValueError(f"max_tokens: 1 .. {MAX_TOKENS}, got {max_tokens}")
        for name, s, rows, cols in (("gate", gs, H, D), ("up", us, H, D), ("down", ds, D, H)):
            _bytes_at_least(s, f"{name} scales", E * _expert_blocked_bytes(rows, cols))
        _cuda(gq, gs, uq, us, dq, ds)
        if len({t.device for t in (gq, gs, uq, us, dq, ds)}) != 1:
            raise ValueError("the weights must live on one device")
        self.E, self.H, self.D, self.bits, self.top_k = E, H, D, bits, int(top_k)
        self.score, self.max_tokens, self.device = score, int(max_tokens), gq.device
        self._weights = pairs
        self._call = load().mx_moe_tokens
        self._bytes = int(load().mx_moe_tokens_workspace(self.max_tokens, E, D, H, self.top_k, bits))
        if self._bytes == 0:
            raise ValueError("the layer is too large for the kernel's 32-bit tile counts")
        self._fixed = (E, D, H, self.top_k, SCORES[score], bits) + tuple(t.data_ptr() for w in pairs for t in w)
        self._workspaces: dict[int, torch.Tensor] = {}
        with torch.inference_mode(False):  # a tensor made in inference mode could not be zeroed outside of it
            self._status = new_status(self.device)

    def _new_workspace(self) -> torch.Tensor:
        ws = torch.empty(self._bytes, dtype=torch.uint8, device=self.device)
        ws[:256].zero_()  # the grid barrier; every launch leaves it at zero
        return ws

    def _workspace(self, stream: int) -> torch.Tensor:
        # A captured call gets memory of its graph's pool, zeroed by the graph: the graph may run on any stream, beside
        # eager calls on the one that it was captured on.
        if torch.cuda.is_current_stream_capturing():
            return self._new_workspace()
        ws = self._workspaces.get(stream)
        if ws is None:
            ws = self._workspaces[stream] = self._new_workspace()
        return ws

    def check_status(self) -> None:
        """Synchronize, and raise Mxfp8Error if a call since the last check, eager or captured, has reported an error."""
        status = int(self._status.item())
        if status:
            self._status.zero_()
            check(status, "MxMoeTokens")

    def __call__(self, x: torch.Tensor, router_logits: torch.Tensor, out: torch.Tensor | None = None,
                 dev_status: torch.Tensor | None = None) -> torch.Tensor:
        """x [T, D] bf16, router_logits [T, E] (fp32; fp16 and bf16 are widened), T <= max_tokens -> y
        [T, D] bf16.  A token whose logits are all -inf gets zeros; one with a NaN logit gets NaN.
        dev_status: an int32 word for errors the device finds (``new_status``, ``read_status``), in place of the
        layer's own."""
        T = x.shape[0] if x.dim() == 2 else -1
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.D:
            raise ValueError(f"x: expected bf16 [T, {self.D}], got {x.dtype} {tuple(x.shape)}")
        if T > self.max_tokens:
            raise ValueError(f"x: at most {self.max_tokens} tokens, got {T}")
        if tuple(router_logits.shape) != (T, self.E):
            raise ValueError(f"router_logits: expected [{T}, {self.E}], got {tuple(router_logits.shape)}")
        if router_logits.dtype != torch.float32:
            if router_logits.dtype not in (torch.bfloat16, torch.float16):
                raise ValueError(f"router_logits: expected a floating type, got {router_logits.dtype}")
            router_logits = router_logits.float()
        if torch.is_grad_enabled() and (x.requires_grad or router_logits.requires_grad):
            raise ValueError("MxMoeTokens computes no gradients: call it under torch.no_grad()")
        if out is not None:
            _tensor(out, "out", torch.bfloat16, shape=(T, self.D))
        _status_word(dev_status)
        _cuda(x, router_logits, out, dev_status)
        if x.device != self.device or router_logits.device != self.device:
            raise ValueError(f"x and router_logits must live on {self.device}")
        if out is None:
            out = torch.empty((T, self.D), dtype=torch.bfloat16, device=self.device)
        if T == 0:
            return out
        stream = _raw_stream(self.device.index)
        ws = self._workspace(stream)
        E, D, H, k, score, bits, *weights = self._fixed
        check(self._call(x.data_ptr(), router_logits.data_ptr(), T, E, D, H, k, score, bits, *weights, ws.data_ptr(),
                         self._bytes, out.data_ptr(), (self._status if dev_status is None else dev_status).data_ptr(),
                         stream), "mx_moe_tokens")
        return out
