"""The prompt's and the few-token path of examples/mxfp4_layer.py, expert by expert: every token goes to one expert, so a
mistake in one of many shows in the rows of its tokens."""
import importlib.util
import os

import pytest
import torch

from tests._util import require_gpu

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_layer.py")


@pytest.mark.parametrize("E,D,H", [(24, 512, 768), (7, 288, 416), (64, 256, 256)])
def test_every_expert_agrees(E, D, H):
    """The paths round h1 and h3 differently, which moves a row by 0.031 relative in the mean square (the estimate of
    test_paths_agree); four times that is allowed here too, but for each row by itself."""
    require_gpu()
    spec = importlib.util.spec_from_file_location("mxfp4_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    g = torch.Generator("cuda").manual_seed(E)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()

    layer = example.ServingLayer(rand(E, H, D, scale=D ** -0.5), rand(E, H, D, scale=D ** -0.5),
                                 rand(E, D, H, scale=H ** -0.5), 1)
    T = min(2 * E, 64)
    x, logits = rand(T, D), torch.zeros((T, E), device="cuda")
    logits[torch.arange(T), torch.arange(T) % E] = 5.0
    many, few = layer.prompt(x, logits).double(), layer.tokens(x, logits).double()
    assert few.norm(dim=1).min() > 0
    apart = (many - few).norm(dim=1) / few.norm(dim=1)
    assert apart.max() <= 4 * (2.0 ** -8 / 4) ** 0.5, apart.max()
