"""The 4-bit calls without a GPU: the reference's own arithmetic, refusals of the binding and of the C ABI
before any launch, and every declared symbol exported."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests import _mx4ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OFFS = torch.tensor([64, 128], dtype=torch.int32)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_reference_rounding():
    """The reference itself at hand-worked values."""
    x = np.zeros(32)
    x[:10] = [6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.26, 4.9]
    code, s = ref.encode(x, 4)
    assert s[0] == 127                                    # amax 6: 2^0
    assert code[:10].tolist() == [7, 6, 6, 4, 4, 2, 2, 0, 9, 6]
    code, s = ref.encode(np.full(32, 7.99), 4)            # saturates at 6 of its own scale
    assert s[0] == 127 and (code == 7).all()
    assert ref.encode(np.zeros(32), 4)[1][0] == 0
    x[3] = np.inf
    code, s = ref.encode(x, 4)
    assert s[0] == 255 and code[8] == 15 and code[0] == 7
    assert ref.E4M3.size == 127 and ref.E4M3[-1] == 448 and ref.E4M3[8] == 2.0 ** -6
    code, s = ref.encode(np.full(32, 448.0 * 2 ** 5), 8)
    assert s[0] == 132 and (code == 0x7E).all()


def test_every_declared_symbol_is_exported():
    mx.load()
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxfp4moe.h")).read(), flags=re.S)
    names = re.findall(r"^\w[\w\s\*]*?\b(mx\w+)\s*\(", src, flags=re.M)
    assert len(names) >= 5
    raw = ctypes.CDLL(os.path.join(ROOT, "mxfp8_precision_moe_gb300", "libmxfp8moe.so"))
    assert not [n for n in names if not hasattr(raw, n)]


@pytest.mark.parametrize("call,match", [
    (lambda: mx.mxfp4_quantize_2d(bf(128, 64)), "CUDA"),
    (lambda: mx.mxfp4_quantize_2d_mxfp8_cols(bf(128, 64)), "CUDA"),
    (lambda: mx.mxfp4_quantize_2d_mxfp8_cols(bf(128, 48)), "multiple of 32"),
    (lambda: mx.mxfp4_quantize_2d_mxfp8_cols(bf(128, 64), OFFS.long()), "offs"),
    (lambda: mx.mxfp4_quantize_3d_experts(bf(2, 64, 64)), "CUDA"),
    (lambda: mx.mxfp4_quantize_3d_experts_mxfp8_cols(bf(2, 64, 64)), "CUDA"),
    (lambda: mx.mxfp4_quantize_3d_experts_mxfp8_cols(bf(2, 48, 64)), "multiple of 32"),
    (lambda: mx.mxfp4_swiglu_quantize(bf(8, 64), bf(8, 64)), "CUDA"),
    (lambda: mx.mxfp4_dequantize_2d(u8(8, 32), u8(512)), "CUDA"),
    (lambda: mx.mxfp4_dequantize_3d_experts(u8(2, 8, 32), u8(2, 512)), "CUDA"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 32), u8(2048), u8(2, 64, 32), u8(2, 512), OFFS), "CUDA"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64), bf(2, 64, 64), OFFS), "CUDA"),
    (lambda: mx.mxfp4_quantize_2d(bf(128, 64).float()), "x"),
    (lambda: mx.mxfp4_quantize_2d(bf(128)), "x"),
    (lambda: mx.mxfp4_quantize_2d(bf(128, 48)), "multiple of 32"),
    (lambda: mx.mxfp4_quantize_2d(bf(128, 64), offs=OFFS.long()), "offs"),
    (lambda: mx.mxfp4_quantize_2d(bf(128, 64), offs=OFFS[:0]), "offs"),
    (lambda: mx.mxfp4_swiglu_quantize(bf(8, 64), bf(8, 32)), "h3"),
    (lambda: mx.mxfp4_dequantize_2d(u8(8, 32), u8(15), mx.SCALES_COMPACT), "s:"),
    (lambda: mx.mxfp4_dequantize_2d(u8(8, 32), u8(511)), "s:"),
    (lambda: mx.mxfp4_dequantize_3d_experts(u8(2, 8, 32), u8(2, 500)), "s:"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 32), u8(1535), u8(2, 64, 32), u8(2, 512), OFFS), "a_s"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 32), u8(2048), u8(2, 64, 32), u8(1023), OFFS), "w_s"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 32), u8(2048), u8(2, 64, 64), u8(2, 512), OFFS), "w_q"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 32), u8(2048), u8(3, 64, 32), u8(3, 512), OFFS), "offs"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 32), u8(2048), u8(2, 64, 32), u8(2, 512), OFFS, out=bf(128, 32)), "out"),
    (lambda: mx.mxfp4_grouped_mm_fwd(u8(128, 24), u8(2048), u8(2, 64, 24), u8(2, 512), OFFS), "multiple of 32"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64).float(), bf(2, 64, 64), OFFS), "bf16"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64), bf(2, 64, 32), OFFS), "A \\[M, K\\]"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64), bf(2, 48, 64), OFFS), "multiple of 32"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64), bf(2, 64, 64), OFFS.long()), "int32"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64), bf(2, 64, 64), OFFS, w_mxfp4=(u8(2, 64, 32),)),
     "w_mxfp4"),
    (lambda: mx.to_mxfp4_then_scaled_grouped_mm(bf(128, 64), bf(2, 64, 64), OFFS,
                                                w_mxfp4=(u8(2, 64, 64), u8(2, 512))), "w_mxfp4"),
])
def test_refusals_of_the_binding(call, match):
    with pytest.raises(ValueError, match=match):
        call()


@pytest.mark.parametrize("make,match", [
    (lambda: mx.MxMoeTokens(u8(2, 64, 128), u8(2, 512), u8(2, 128, 64), 1), "gate"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 128), u8(2, 512)), (u8(2, 64, 128), u8(2, 512)), (u8(2, 100, 64), u8(2, 512)),
                            1), "gate codes"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 128), u8(2, 512)), (u8(2, 32, 128), u8(2, 512)), (u8(2, 128, 64), u8(2, 512)),
                            1), "up codes"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 128), u8(2, 512)), (u8(2, 64, 128), u8(2, 512)), (u8(2, 128, 32), u8(2, 512)),
                            1), "down codes"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 128), u8(2, 512)), (u8(2, 64, 128), u8(2, 512)), (u8(2, 128, 64), u8(2, 512)),
                            3), "top_k"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 128), u8(2, 511)), (u8(2, 64, 128), u8(2, 512)), (u8(2, 128, 64), u8(2, 512)),
                            1), "gate scales"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 48), u8(2, 512)), (u8(2, 64, 48), u8(2, 512)), (u8(2, 48, 64), u8(2, 512)),
                            1), "multiples of 32"),
    (lambda: mx.MxMoeTokens((u8(300, 32, 32), u8(300, 512)), (u8(300, 32, 32), u8(300, 512)),
                            (u8(300, 32, 32), u8(300, 512)), 1), "experts"),
    (lambda: mx.MxMoeTokens((u8(2, 64, 128), u8(2, 512)), (u8(2, 64, 128), u8(2, 512)), (u8(2, 128, 64), u8(2, 512)),
                            1), "CUDA"),
])
def test_refusals_of_the_few_token_layer(make, match):
    with pytest.raises(ValueError, match=match):
        make()


def test_refusals_of_the_c_abi():
    L = mx.load()
    P = ctypes.c_void_p
    a = P(1 << 20)          # never dereferenced: validation fails first
    odd = P((1 << 20) + 8)
    q2, q3, sw = L.mxfp4_quantize_2d, L.mxfp4_quantize_3d_experts, L.mxfp4_swiglu_quantize
    assert q2(a, 64, 48, 1, None, 0, a, a, None) == 3
    assert q2(a, -1, 64, 1, None, 0, a, a, None) == 2
    assert q2(a, 64, 0, 1, None, 0, a, a, None) == 2
    assert q2(a, 64, 64, 2, None, 0, a, a, None) == 4
    assert q2(None, 64, 64, 1, None, 0, a, a, None) == 1
    assert q2(a, 64, 64, 1, a, 0, a, a, None) == 2      # offsets of no groups
    assert q2(a, 64, 64, 1, a, 1025, a, a, None) == 2
    assert q2(odd, 64, 64, 1, None, 0, a, a, None) == 3
    assert q2(a, 64, 64, 1, None, 0, odd, a, None) == 3
    assert sw(a, None, 64, 64, 1, None, 0, a, a, None) == 1
    assert sw(a, odd, 64, 64, 1, None, 0, a, a, None) == 3
    assert q3(a, 0, 64, 64, 1, a, a, None) == 2
    assert q3(a, 2, 0, 64, 1, a, a, None) == 2
    assert q3(a, 2, 64, 33, 1, a, a, None) == 3
    both = L.mxfp4_quantize_2d_mxfp8_cols
    assert both(a, 33, 64, None, 0, a, a, a, a, None, None) == 3
    assert both(a, 32, 48, None, 0, a, a, a, a, None, None) == 3
    assert both(a, -32, 64, None, 0, a, a, a, a, None, None) == 2
    assert both(a, 32, 64, a, 0, a, a, a, a, None, None) == 2
    assert both(a, 32, 64, None, 0, a, a, None, a, None, None) == 1
    assert both(a, 32, 64, None, 0, a, a, a, odd, None, None) == 3
    assert both(None, 0, 64, None, 0, None, None, None, None, None, None) == 0
    both = L.mxfp4_quantize_3d_experts_mxfp8_cols
    assert both(a, 0, 32, 64, a, a, a, a, None, None) == 2
    assert both(a, 2, 0, 64, a, a, a, a, None, None) == 2
    assert both(a, 2, 33, 64, a, a, a, a, None, None) == 3
    assert both(a, 2, 32, 64, a, None, a, a, None, None) == 1
    assert both(odd, 2, 32, 64, a, a, a, a, None, None) == 3
    dq = L.mxfp4_dequantize
    assert dq(a, a, 2, 64, 64, 1, a, 2, a, None) == 4   # row groups of several matrices
    assert dq(a, None, 1, 64, 64, 1, None, 0, a, None) == 1
    mm = L.mxfp4_grouped_mm_fwd
    assert mm(a, a, a, a, None, 2, 64, 64, 64, a, None, None) == 1
    assert mm(a, a, a, a, a, 0, 64, 64, 64, a, None, None) == 2
    assert mm(a, a, a, a, a, 2, 64, 48, 64, a, None, None) == 3
    assert mm(a, a, a, a, a, 2, 64, 64, 48, a, None, None) == 3
    assert mm(a, a, odd, a, a, 2, 64, 64, 64, a, None, None) == 3
    assert mm(a, a, a, a, a, 2, 1 << 32, 64, 64, a, None, None) == 2
    mt = L.mx_moe_tokens
    ok = dict(x=a, l=a, T=4, E=8, D=64, H=64, k=2, score=0, bits=8, g=a, gs=a, u=a, us=a, d=a, ds=a, ws=a, n=1 << 40,
              y=a, st=None, stream=None)
    call = lambda **kw: mt(*{**ok, **kw}.values())
    assert call(T=65) == 2 and call(T=-1) == 2 and call(E=0) == 2 and call(E=257) == 2 and call(k=0) == 2
    assert call(k=9) == 2 and call(E=32, k=17) == 2 and call(D=0) == 2 and call(D=48) == 3 and call(H=40) == 3
    assert call(bits=6) == 4 and call(score=3) == 4 and call(x=None) == 1 and call(l=None) == 1 and call(ws=None) == 1
    assert call(y=odd) == 3 and call(gs=odd) == 3 and call(l=P((1 << 20) + 2)) == 3 and call(D=1 << 40) == 2
    assert call(T=0, x=None) == 0
    size = L.mx_moe_tokens_workspace
    assert size(65, 8, 64, 64, 2, 8) == 0 and size(4, 8, 64, 64, 9, 8) == 0 and size(4, 8, 60, 64, 2, 8) == 0
    assert size(4, 8, 64, 64, 2, 8) > 0 and size(64, 8, 64, 64, 2, 8) > size(4, 8, 64, 64, 2, 8)
