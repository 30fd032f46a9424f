"""kv_attend where one key's logits are large, token by token and in tiles: from 2^20 on such a token has all of the weight or none, so
that the outputs stay what they are however large its logit becomes."""
import pytest
import torch

import kv_reference as R
import test_kv_tree as base
from bit_routed_expert_gb300 import kv_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [40, 2304])
def test_one_large_key(cuda_dev, T):
    D, G, n, x = 64, 8, 2304, 70
    b = R.batch([n], [T], seed=2)
    pages, _, _ = R.filled(b, [n], 1, D, seed=3)
    kc, vc, ks, vs = R.views(pages, D)
    pg, at = int(b.table[0, x // 64]), x % 64
    kc[pg, 0, at], kc[pg, 0, at, 0] = 0, 0x38   # 1 in channel 0
    g = torch.Generator().manual_seed(1)
    q = R.rows(4, T, G, D, gain=0.5)
    q[:, :, 0] = (torch.rand(T, G, generator=g) + 0.5).to(torch.bfloat16)
    q[::3, :, 0] *= -1
    ids = torch.tensor([1, 5, 9], dtype=torch.int32).expand(T, 1, 3).contiguous().to(cuda_dev)
    seq, pos, table = b.on(cuda_dev)
    v = R.VALUES[vc[pg, 0, at].long()] * 2.0 ** (int(vs[pg, 0, at]) - 127)
    one = (torch.tensor(b.pos) >= x)[:, None] & (q[:, :, 0] > 0)
    first = None
    for e in (20, 24, 25, 26, 27, 28, 29, 30, 31, 40, 64, 100, 119):
        ks[pg, 0, at] = 127 + e
        out, lse = (y.cpu() for y in kv_attend(q.to(cuda_dev), base.on(cuda_dev, pages, 1, D), seq, pos, table, ids, scale=1.0))
        assert bool(((out[one].double() - v).abs() <= (2.0 ** -8 + 2.0 ** -10) * v.abs()).all()), e
        assert bool(((lse[one].double() - q[:, :, 0][one].double() * 2.0 ** e).abs() <= 2.0 ** (e - 16)).all()), e
        if first is None:
            first = out, lse
        assert torch.equal(out[~one], first[0][~one]) and torch.equal(lse[~one], first[1][~one]), e
