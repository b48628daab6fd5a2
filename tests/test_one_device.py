"""Kernels launch on the calling thread's current device, so every call refuses tensors of another one, before anything
is allocated or launched.  (Fake tensors: no GPU is needed to have them on two.)"""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import mxfp8_precision_moe_gb300 as mx


def t(shape, dtype, index):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=f"cuda:{index}")


def bf(index, *shape):
    return t(shape, torch.bfloat16, index)


def u8(index, *shape):
    return t(shape, torch.uint8, index)


def offs(index):
    return t((2,), torch.int32, index)


def word(index):
    return t((1,), torch.int32, index)


@pytest.fixture(autouse=True)
def current_device_is_zero(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

    def launch(*args):
        raise AssertionError("a launch was prepared")

    from mxfp8_precision_moe_gb300 import moe_tokens, mxfp4

    for m in (mxfp4, moe_tokens):
        monkeypatch.setattr(m, "_raw_stream", launch)
    monkeypatch.setattr(mx, "_stream", launch)


# a call that works on device i, with one tensor or all of them elsewhere
CALLS = {
    "mxfp8_quantize_2d": lambda i, j: mx.mxfp8_quantize_2d(bf(i, 128, 64), mx.ROW, mx.SCALES_BLOCKED, offs(j)),
    "mxfp8_quantize_3d_experts": lambda i, j: mx.mxfp8_quantize_3d_experts(bf(i, 2, 64, 64), dev_status=word(j)),
    "mxfp8_grouped_mm_fwd": lambda i, j: mx.mxfp8_grouped_mm_fwd(u8(i, 128, 64), u8(i, 4096), u8(j, 2, 64, 64),
                                                                 u8(j, 2, 2048), offs(i)),
    "mxfp8_check_offsets": lambda i, j: mx.mxfp8_check_offsets(offs(i), 128, 1, word(j)),
    "mxfp4_quantize_2d": lambda i, j: mx.mxfp4_quantize_2d(bf(i, 128, 64), offs=offs(j)),
    "mxfp4_quantize_2d_mxfp8_cols": lambda i, j: mx.mxfp4_quantize_2d_mxfp8_cols(bf(i, 128, 64), offs(i), word(j)),
    "mxfp4_swiglu_quantize": lambda i, j: mx.mxfp4_swiglu_quantize(bf(i, 128, 64), bf(j, 128, 64)),
    "mxfp4_quantize_3d_experts_mxfp8_cols": lambda i, j: mx.mxfp4_quantize_3d_experts_mxfp8_cols(bf(i, 2, 64, 64), word(j)),
    "mxfp4_dequantize_2d": lambda i, j: mx.mxfp4_dequantize_2d(u8(i, 128, 32), u8(j, 512)),
    "mxfp4_dequantize_2d offs": lambda i, j: mx.mxfp4_dequantize_2d(u8(i, 128, 32), u8(i, 2048), offs=offs(j)),
    "mxfp4_dequantize_3d_experts": lambda i, j: mx.mxfp4_dequantize_3d_experts(u8(i, 2, 64, 32), u8(j, 2, 512)),
    "mxfp4_grouped_mm_fwd": lambda i, j: mx.mxfp4_grouped_mm_fwd(u8(i, 128, 32), u8(i, 2048), u8(j, 2, 64, 32),
                                                                 u8(j, 2, 512), offs(i)),
    "mxfp4_grouped_mm_fwd out": lambda i, j: mx.mxfp4_grouped_mm_fwd(u8(i, 128, 32), u8(i, 2048), u8(i, 2, 64, 32),
                                                                     u8(i, 2, 512), offs(i), out=bf(j, 128, 64)),
    "mxfp4_grouped_mm_fwd offs": lambda i, j: mx.mxfp4_grouped_mm_fwd(u8(i, 128, 32), u8(i, 2048), u8(i, 2, 64, 32),
                                                                      u8(i, 2, 512), offs(j)),
    "to_mxfp4_then_scaled_grouped_mm": lambda i, j: mx.to_mxfp4_then_scaled_grouped_mm(bf(i, 128, 64), bf(j, 2, 64, 64),
                                                                                      offs(i)),
    "MxMoeTokens": lambda i, j: mx.MxMoeTokens((u8(i, 2, 64, 128), u8(i, 2, 512)), (u8(i, 2, 64, 128), u8(j, 2, 512)),
                                               (u8(i, 2, 128, 64), u8(i, 2, 512)), 1),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("i,j", [(0, 1), (1, 0), (1, 1)])
def test_another_device_is_refused(name, i, j):
    with pytest.raises(ValueError, match="cuda:1"):
        CALLS[name](i, j)


@pytest.mark.parametrize("name", ["mxfp4_quantize_2d", "mxfp4_quantize_3d_experts"])
def test_a_matrix_alone_on_another_device_is_refused(name):
    x = bf(1, 128, 64) if name == "mxfp4_quantize_2d" else bf(1, 2, 64, 64)
    with pytest.raises(ValueError, match="cuda:1"):
        getattr(mx, name)(x)


def layer_on(index):
    """A layer of the weights' device, without the constructor's call of the library."""
    op = object.__new__(mx.MxMoeTokens)
    op.E, op.H, op.D, op.bits, op.top_k = 2, 64, 128, 8, 1
    op.score, op.max_tokens, op.device = "softmax", 64, torch.device("cuda", index)
    return op


@pytest.mark.parametrize("layer,x,logits,out,status", [
    (1, 1, 1, None, None), (0, 1, 0, None, None), (0, 0, 1, None, None), (0, 0, 0, 1, None), (0, 0, 0, None, 1),
])
def test_few_token_call_on_another_device_is_refused(layer, x, logits, out, status):
    with pytest.raises(ValueError, match="cuda:1"):
        layer_on(layer)(bf(x, 3, 128), t((3, 2), torch.float32, logits), out=None if out is None else bf(out, 3, 128),
                        dev_status=None if status is None else word(status))
