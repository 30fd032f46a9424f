"""The example layer over trees of drafts (resize -> rotate -> append -> attend -> MoE -> compact -> resize, beams that share a
prompt's pages), stepped through a CUDA graph, against one prefill over every beam's whole text."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompt,steps", [(200, 6), (64, 2), (3, 9)])
def test_drafts_agree_with_prefill(cuda_dev, prompt, steps):
    """Both see the same context, so that only rounding differs: a few BF16 steps (2^-8 each) of every token's output, as for the
    layer that decodes token by token.  The two take other kernels (a token's heads or tiles of the attention; decode and
    grouped-GEMM experts), and the accepted keys and values have been moved.  Where two experts' scores lie within that
    rounding of one another a token may take the other one, whose output has nothing to do with the first's: such
    tokens are few and left out."""
    import draft_tree
    tree, full, same, used = draft_tree.run(prompt, steps)
    assert tree.shape == full.shape and tree.shape[1] == 512 and len(tree) >= 3 * steps
    assert bool(torch.isfinite(tree.float()).all()) and int((~same).sum()) <= len(tree) // 10
    off = (tree.float() - full.float()).norm(dim=1) / full.float().norm(dim=1)
    assert float(off[same].max()) <= 4 * 2.0 ** -8
    assert used[0] == used[1] - 2 * (prompt // 64)   # the prompt's whole blocks are there once
