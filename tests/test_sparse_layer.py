"""The example layer (append -> select -> attend -> MoE): decoding through a CUDA graph against one prefill."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefill,steps", [(700, 8), (63, 3)])
def test_decoding_agrees_with_prefill(cuda_dev, prefill, steps):
    """The two take different kernels (one token's heads, tiles of 128 rows; decode and grouped-GEMM experts).
    Where every block is selected in both (63 tokens) only rounding differs: a few BF16 steps (2^-8 each) of the
    layer's output.  With more blocks than the six taken, a rejected block's bounds may also differ: a step
    sees the bounds of a block that is still filling, the prefill those of the filled one; such blocks are
    among the forced last two, so the lists agree as well."""
    import sparse_layer
    step, full = sparse_layer.run(prefill, steps)
    assert step.shape == full.shape == (2, steps, 512)
    assert bool(torch.isfinite(step.float()).all())
    off = (step.float() - full.float()).norm() / full.float().norm()
    assert float(off) <= 4 * 2.0 ** -8
