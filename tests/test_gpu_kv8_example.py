"""The layer of examples/sparse_layer.py runs, for prompts and captured single tokens."""
import importlib.util
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer(dtype):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    spec = importlib.util.spec_from_file_location("sparse_layer", os.path.join(ROOT, "examples", "sparse_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    worst, apart = mod.run(prompts=(300, 33, 1), steps=4, hidden=512, q_heads=8, kv_heads=2, head_dim=128, page=16, keep=6, dtype=dtype)
    # the result and the attention's, which the o projection takes, are rounded to dtype: two
    # half steps; weights (2^-11) and the projection's fp32 sums beside them
    assert worst <= 2 * torch.finfo(dtype).eps / 2 + 2.0 ** -10
    # everything kept is attention over all pages: the steps' distances from both are the same
    # numbers, and the largest error is taken over the prompts' too
    worst, apart = mod.run(prompts=(90, 33, 1), steps=3, hidden=512, q_heads=8, kv_heads=2, head_dim=128, page=16, keep=6, dtype=dtype)
    assert 0 < apart <= worst
