"""A workspace sized for the most tokens of a call serves every smaller call too."""
import pytest
import torch

import kv_reference as R
from bit_routed_expert_gb300 import KvCache, kv_attend_tree, kv_attend_tree_workspace


@pytest.mark.parametrize("H", [1, 2, 3, 4, 8, 40, 610])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_attention(H, G, D):
    sizes = [kv_attend_tree_workspace(T, H * G, H, D) for T in range(1, 1400)]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
def test_tree_attention_of_fewer_tokens(cuda_dev):
    """One and two tokens of four kv heads once needed more than three."""
    D, H, G, n = 128, 4, 8, 700
    b = R.batch([n], [3])
    pages, _, _ = R.filled(b, [n], H, D)
    c = KvCache(pages.to(cuda_dev), torch.zeros((len(pages), H, 2, D), dtype=torch.int8, device=cuda_dev),
                torch.zeros((len(pages), H), dtype=torch.int8, device=cuda_dev))
    q = R.rows(5, 3, H * G, D).to(cuda_dev)
    seq, pos, table = b.on(cuda_dev)
    ws = torch.full((kv_attend_tree_workspace(3, H * G, H, D),), 255, dtype=torch.uint8, device=cuda_dev)
    for T in (1, 2, 3):
        got = kv_attend_tree(q[:T], c, seq[:T], pos[:T], table, ws=ws)
        want = kv_attend_tree(q[:T], c, seq[:T], pos[:T], table)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
