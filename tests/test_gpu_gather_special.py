"""Special values through the gathering quantizations, each kernel against the quantization of the gathered rows."""
import math

import pytest
import torch

import mxfp8_precision_moe_gb300 as mx
from tests._util import require_gpu
from tests.test_gpu_token_rows import blocked_scales, make_plan, randn, same_copies

pytestmark = pytest.mark.gpu
inf, nan = math.inf, math.nan


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def special_tokens(T, D):
    """Rows of which blocks hold infinities and NaN of both signs, in either half and in both, zeros of both signs, bf16's
    largest, its smallest normal and subnormals, values at a rounding's middle and next to a power of two."""
    x = randn((T, D), 1)
    big, tiny, sub = torch.finfo(torch.bfloat16).max, 2.0 ** -126, 2.0 ** -133
    for i, v in enumerate((inf, -inf, nan, -nan)):
        x[4 * i, 5] = x[4 * i + 1, 32 + 20] = v
        x[4 * i + 2, 64], x[4 * i + 2, 64 + 31] = v, -v
        x[4 * i + 3] = v
    signs = torch.where(torch.arange(D, device="cuda") % 3 == 0, -1.0, 1.0).bfloat16()
    for i, v in enumerate((0.0, big, tiny, sub, 3 * sub, 448.0, 464.0, 6.0, 5.0, 1.0625, 2.0 ** -9, 2.0 ** 119, 255.0)):
        x[16 + i] = v * signs
        x[29 + i, ::2] = v * signs[::2]
        x[42 + i, D - 32 + 7] = v
    # a NaN's sign is a bit that only its pattern shows
    x.view(torch.int16)[55, 3], x.view(torch.int16)[55, 19] = 0x7FFF, -1
    x.view(torch.int16)[56, 16:32] = -64  # 0xFFC0
    return x


@pytest.mark.parametrize("k,E,multiple,D", [(2, 5, 32, 256), (1, 3, 32, 96), (8, 64, 32, 1056), (3, 1, 32, 160)])
def test_special_values(k, E, multiple, D):
    T = 60
    plan = make_plan(T, min(k, E), E, multiple, 1, idle=False)
    x = special_tokens(T, D)
    rows = mx.moe_gather(x, plan)
    assert torch.equal(rows.view(torch.int16)[plan.place[:, 0].long()], x.view(torch.int16))
    both = mx.mxfp8_quantize_2d(rows, mx.ROW | mx.COL, mx.SCALES_BLOCKED, plan.offs)
    same_copies(mx.mxfp8_gather_quantize(x, plan, mx.ROW), (*both[:2], None, None), plan, D)        # by token
    same_copies(mx.mxfp8_gather_quantize(x, plan, mx.ROW | mx.COL), both, plan, D)                   # by tiles
    same_copies(mx.mxfp8_gather_quantize(x, plan, mx.COL), (None, None, *both[2:]), plan, D)


@pytest.mark.parametrize("k,E,multiple,D", [(2, 5, 32, 256), (1, 3, 1, 96), (8, 64, 5, 1056), (3, 1, 1, 160)])
def test_special_values_in_4_bits(k, E, multiple, D):
    plan = make_plan(60, min(k, E), E, multiple, 1, idle=False, exact=True)
    x = special_tokens(60, D)
    got, want = mx.mxfp4_gather_quantize(x, plan), mx.mxfp4_quantize_2d(mx.moe_gather(x, plan), offs=plan.offs)
    assert torch.equal(got[0], want[0])
    assert torch.equal(blocked_scales(got[1], plan, False, D), blocked_scales(want[1], plan, False, D))


@pytest.mark.parametrize("dirs", [mx.ROW, mx.COL, mx.ROW | mx.COL])
def test_special_values_and_weights(dirs):
    """bf16(w x) of special values and special weights."""
    plan = make_plan(60, 2, 5, 32, 1, idle=False)
    x, w = special_tokens(60, 256), torch.rand((60, 2), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    w[::7, 0], w[1::7, 1], w[2::7, 0], w[3::7, 1] = inf, nan, 0.0, 1e-38
    slot = plan.slot.long()
    rows = torch.where((slot >= 0)[:, None], x[slot.clamp_min(0) // 2].float() * w.flatten()[slot.clamp_min(0)][:, None], 0.0)
    want = mx.mxfp8_quantize_2d(rows.bfloat16(), dirs, mx.SCALES_BLOCKED, plan.offs)
    got = mx.mxfp8_gather_quantize(x, plan, dirs, w)
    for i, (a, b) in enumerate(zip(got, want)):
        if a is None:
            assert b is None
        elif i % 2:
            assert torch.equal(blocked_scales(a, plan, i == 3, 256), blocked_scales(b, plan, i == 3, 256))
        else:
            # codes, but for the sign of a NaN, which a product does not define
            assert torch.equal(torch.where(a & 127 == 127, 127, a), torch.where(b & 127 == 127, 127, b))


def test_4_bits_and_their_scales_past_32_bits():
    """4.4 thousand million bytes of rows, codes and scales to the last."""
    T, D = 270016, 8192
    x = torch.empty((T, D), dtype=torch.bfloat16, device="cuda")
    for i in range(0, T, 8192):
        x[i:i + 8192] = randn((min(8192, T - i), D), i, 2.0 ** (i // 8192 % 9 - 4))
    e = torch.randint(0, 4, (T, 1), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    plan = mx.moe_plan(e, 4, 32, exact=True)
    got = mx.mxfp4_gather_quantize(x, plan)
    want = mx.mxfp4_quantize_2d(mx.moe_gather(x, plan), offs=plan.offs)
    assert torch.equal(got[0], want[0])
    assert torch.equal(blocked_scales(got[1], plan, False, D), blocked_scales(want[1], plan, False, D))
