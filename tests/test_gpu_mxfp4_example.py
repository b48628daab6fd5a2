"""examples/mxfp4_layer.py: the 4-bit operators as a user runs them together."""
import importlib.util
import os

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_layer.py")


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("mxfp4_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_dispatch_pads_groups(example):
    logits = torch.randn(50, 4, device="cuda")
    logits[:, 3] = -9.0
    token, weight, ends = example.dispatch(logits, 2, multiple=32)
    assert (ends % 32 == 0).all() and ends[2] == ends[3] == token.numel()
    kept = token[token >= 0]
    assert torch.equal(kept.bincount(minlength=50), torch.full((50,), 2, device="cuda"))
    total = torch.zeros(50, device="cuda").index_add(0, kept, weight[token >= 0])
    # two softmax terms, one sum: under four roundings of 2^-24
    assert (total - 1).abs().max() <= 4 * 2.0 ** -24 and not weight[token < 0].any()


@pytest.mark.parametrize("E,D,H,k", [(8, 256, 512, 2), (5, 352, 160, 3)])
def test_paths_agree(example, E, D, H, k):
    """The prompt's path rounds gate and up products to bf16 (2^-9 of each) before SwiGLU, the other does not, so h
    differs by about d = 2^-8 relative, and both quantize it to steps of s = 1/4 of an element on average.  An element
    lands on another code with probability d / s and then moves by s: sqrt(d s) = 0.031 relative in the mean square,
    the same for y, a sum of products with such errors.  Four times that is allowed."""
    grads, many, few, _, _ = example.run(E, D, H, k, prompt=70, follow=6)
    assert all(torch.isfinite(d).all() and d.any() for d in grads)
    assert many.shape == few.shape == (6, D)
    assert (many.float() - few.float()).norm() <= 4 * (2.0 ** -8 / 4) ** 0.5 * few.float().norm()
