"""Errors that the device finds reach the caller: the few-token layer's own status word."""
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
