"""A workspace sized for the most tokens of a call serves every smaller call too."""
import pytest
import torch

import kv_reference as R
from bit_routed_expert_gb300 import (KvCache, kv_attend_tree, kv_attend_tree_workspace, moe_expert_ffn_workspace, moe_route_workspace,
                                     synth)
from helpers import device_layer


@pytest.mark.parametrize("H", [1, 2, 3, 4, 8, 40, 610])
@pytest.mark.parametrize("G", [1, 3, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_attention(H, G, D):
    sizes = [kv_attend_tree_workspace(T, H * G, H, D) for T in range(1, 1400)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (64, 8), (384, 6), (1024, 32)])
def test_moe(E, k):
    """The small-batch router, for up to 32 tokens, needs more than the other for some more."""
    sizes = [moe_route_workspace(T, E) for T in range(1, 700)]
    assert sizes == sorted(sizes)
    sizes = [moe_expert_ffn_workspace(T, k, E, 512, 256, 256) for T in range(1, 700)]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("T_max", [33, 64, 127])
def test_moe_layer_of_fewer_tokens(cuda_dev, T_max):
    layer, full = device_layer(3, 0, synth.TINY, T_max, cuda_dev), device_layer(3, 0, synth.TINY, 256, cuda_dev)
    x = R.rows(4, T_max, synth.TINY.d).to(cuda_dev)
    for T in (T_max, 24, 32, 1, T_max, 9):
        out, info = layer.forward(x[:T])
        want, also = full.forward(x[:T])
        assert torch.equal(out, want) and torch.equal(info["ids"], also["ids"])
    assert int(layer.dev_err) == 0


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
