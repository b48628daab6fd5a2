"""Errors that the device finds reach the caller: the few-token layer's own status word, and the one handed to the
differentiable 4-bit product, forward and backward."""
import pytest
import torch

from mxfp8_precision_moe_gb300 import synth
from tests._util import require_gpu

pytestmark = pytest.mark.gpu

TIMEOUT = 8  # MXFP8_ERR_TIMEOUT


@pytest.fixture(scope="module")
def mx():
    require_gpu()
    import mxfp8_precision_moe_gb300 as m

    m.load()
    return m


def layer(mx):
    ws = [synth.randn_bf16(s, 0.1, seed=i).cuda() for i, s in enumerate([(4, 64, 128), (4, 64, 128), (4, 128, 64)])]
    return mx.MxMoeTokens(*(mx.mxfp4_quantize_3d_experts(w) for w in ws), 2)


def test_few_token_layer_keeps_a_status_word(mx):
    op = layer(mx)
    x, logits = synth.randn_bf16((3, 128), 1.0, seed=9).cuda(), torch.randn(3, 4, device="cuda")
    call, passed = op._call, []
    op._call = lambda *args: (passed.append(args[-2]), call(*args))[1]
    y = op(x, logits)
    op.check_status()                          # nothing to report
    own = torch.full((1,), TIMEOUT, dtype=torch.int32, device="cuda")  # what a kernel that gives up writes
    op._status.copy_(own)
    assert torch.equal(op(x, logits), y)       # an unread error stands until it is asked for
    with pytest.raises(mx.Mxfp8Error, match="TIMEOUT"):
        op.check_status()
    op.check_status()                          # reported once
    st = mx.new_status()
    op(x, logits, dev_status=st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op(x, logits)
    graph.replay()
    torch.cuda.synchronize()
    word = op._status.data_ptr()
    assert passed == [word, word, st.data_ptr(), word]


def test_few_token_layer_made_in_inference_mode(mx):
    with torch.inference_mode():
        op = layer(mx)
    op._status.copy_(torch.full((1,), TIMEOUT, dtype=torch.int32, device="cuda"))
    with pytest.raises(mx.Mxfp8Error, match="TIMEOUT"):
        op.check_status()
    with torch.inference_mode():
        op.check_status()


class Recorder:
    """The library, with every argument of the calls made through it."""

    def __init__(self, lib, seen):
        self._lib, self._seen = lib, seen

    def __getattr__(self, name):
        f = getattr(self._lib, name)

        def call(*args):
            self._seen.append((name, args))
            return f(*args)

        return call


@pytest.mark.parametrize("check", [False, True])
def test_differentiable_product_reports_into_a_given_word(mx, monkeypatch, check):
    from mxfp8_precision_moe_gb300 import mxfp4

    A = synth.randn_bf16((96, 64), 1.0, seed=1).cuda().requires_grad_(True)
    W = synth.randn_bf16((2, 64, 64), 0.1, seed=2).cuda().requires_grad_(True)
    offs = torch.tensor([32, 96], dtype=torch.int32, device="cuda")
    seen, lib, st = [], mx.load(), mx.new_status()
    monkeypatch.setattr(mxfp4, "load", lambda: Recorder(lib, seen))
    out = mx.to_mxfp4_then_scaled_grouped_mm(A, W, offs, check_offsets=check, dev_status=st)
    forward = len(seen)
    out.float().square().sum().backward()
    mx.read_status(st)
    reporting = [(n, a) for n, a in seen if n.startswith(("mxfp8_", "mxfp4_grouped", "mxfp4_quantize_2d_", "mxfp4_quantize_3d_experts_"))]
    assert forward == 3 and len(seen) == 6 and len(reporting) == 6
    assert all(a[-2] == st.data_ptr() for _, a in reporting)
    bad = torch.tensor([32, 90], dtype=torch.int32, device="cuda")
    with pytest.raises(mx.Mxfp8Error):
        mx.to_mxfp4_then_scaled_grouped_mm(A, W, bad, dev_status=mx.new_status())


def test_refusals_of_a_status_word(mx):
    A, W = synth.randn_bf16((64, 64), 1.0, seed=1).cuda(), synth.randn_bf16((1, 64, 64), 0.1, seed=2).cuda()
    offs = torch.tensor([64], dtype=torch.int32, device="cuda")
    for bad in (torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                torch.zeros(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="dev_status|CUDA"):
            mx.to_mxfp4_then_scaled_grouped_mm(A, W, offs, dev_status=bad)
