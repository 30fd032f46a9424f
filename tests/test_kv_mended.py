"""Cases of the key/value cache calls that answered wrongly once, against the definitions in 64 bits."""
import pytest
import torch

import kv_reference as R
from test_kv_cache import check_select

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sink,local,k", [(0, 1, 7), (1, 2, 16), (0, 3, 40)])
@pytest.mark.parametrize("blocks", [511, 512, 513, 514, 515, 1025])
def test_select_last_piece_holds_only_forced_blocks(cuda_dev, blocks, sink, local, k):
    """The kernels select from pieces of 512 blocks; where the last piece has none but local blocks, which are taken
    anyway, its selection ends at once and the list held so far is passed on as it is."""
    D, H, G, T = 64, 1, 2, 40
    b = R.batch([2560], [1])
    cache = R.filled(b, [2560], H, D)
    g = torch.Generator().manual_seed(blocks)
    n = R.Batch([0] * T, list(range(64 * blocks - T, 64 * blocks)),
                torch.randint(0, b.n_pages, (1, blocks), generator=g).to(torch.int32), b.n_pages)
    check_select(cuda_dev, n, cache, R.rows(blocks, T, G, D), k, sink, local)
