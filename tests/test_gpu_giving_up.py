"""The few-token layer's waits between CTAs when they run out (with a limit of nothing, and nothing else wrong): the launch
ends by itself, reports it, and leaves the workspace ready.  A producer that gives up has copies in flight, which have to
land before the CTA leaves."""
import time

import pytest
import torch

from tests._util import require_gpu
from tests.test_gpu_moe_tokens import Layer, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    require_gpu()
    import mxfp8_precision_moe_gb300 as m

    m.load()
    return m


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,E,D,H,k", [(1, 4, 512, 256, 1), (7, 6, 2080, 1056, 2), (64, 8, 1024, 2432, 2)])
def test_waits_that_run_out(mx, T, E, D, H, k, bits):
    lay = Layer(mx, E, D, H, k, bits, seed=T)
    op, (x, logits) = lay.op, inputs(T, D, E, seed=T)
    call, debug = op._call, mx.load().mx_debug_moe_tokens
    want = op(x, logits)
    lay.check(x, logits, want)
    for _ in range(5):
        op._call = lambda *args: debug(*args[:-1], 0, args[-1])
        torch.cuda.synchronize()
        start = time.monotonic()
        op(x, logits)
        with pytest.raises(mx.Mxfp8Error, match="TIMEOUT"):
            op.check_status()
        assert time.monotonic() - start < 1.0
        op._call = call
        assert torch.equal(op(x, logits), want)
        op.check_status()
    op._call = lambda *args: debug(*args[:-1], 10 ** 9, args[-1])
    assert torch.equal(op(x, logits), want)
    op.check_status()


def test_limit_is_checked(mx):
    lay = Layer(mx, 2, 64, 64, 1, 8)
    debug = mx.load().mx_debug_moe_tokens
    lay.op._call = lambda *args: debug(*args[:-1], 10 ** 10 + 1, args[-1])
    with pytest.raises(mx.Mxfp8Error, match="SHAPE"):
        lay.op(*inputs(1, 64, 2))
