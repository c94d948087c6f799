"""What the example of depthwise residual blocks says of itself: its forward and backward passes are calls of
this library; PyTorch allocates and makes views, no more."""
import importlib.util
import os
import sys

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NO_WORK = {"aten::empty", "aten::empty_strided", "aten::empty_like", "aten::view", "aten::_unsafe_view", "aten::as_strided",
           "aten::detach", "aten::alias"}


class Calls(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.names = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.add(func._schema.name)
        return func(*args, **(kwargs or {}))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_passes_are_calls_of_the_library(dtype):
    spec = importlib.util.spec_from_file_location("residual_blocks_calls", os.path.join(ROOT, "examples", "residual_blocks.py"))
    example = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = example
    spec.loader.exec_module(example)
    params = example.make_params(2, 3, 64, dtype)
    x = torch.randn(2, 8, 8, 64, device="cuda")
    dy = torch.randn(2, 8, 8, 64, device="cuda").to(dtype)
    with Calls() as seen:
        y, saved = example.forward(x, params, 0.1, 3, 0)
        dx, grads = example.backward(dy, saved, params, 0.1, 3, 0)
    assert seen.names <= NO_WORK, seen.names - NO_WORK
    assert dx.dtype == torch.float32 and dx.shape == x.shape
