"""What an append to the block-scaled fp8 cache leaves behind after wrong
offsets."""
import numpy as np
import pytest
import torch

from tests import fp8_block_ref as ref
from tests.test_fp8_block_gpu import _Cache, _ints, _rows, _table

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("off", [[0, 700, 10, 700], [0, 300, 200, 700], [5, 3, 650, 700],
                                 [-1, 200, 400, 700], [0, 200, 400, 800], [0, 700, 701, 700]])
def test_wrong_offsets_write_whole_blocks_or_none(lib, off):
    """After wrong offsets each block of the sequences is as it was or as its
    run makes it, codes and scale; nothing else is touched."""
    rng = np.random.default_rng(93)
    H, d, n, B = 2, 64, 700, 3
    table, total = _table(rng, [11] * B)
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    x = _rows(rng, n, H, d, torch.bfloat16)
    lib.kv_append_fp8_block(x.to(DEV), x.to(DEV), *dev, _ints([0] * B), _ints(table),
                            offsets=_ints(off))
    assert lib.last_error() == lib.ERR_BAD_SEQLEN
    made = _Cache(rng, total, H, d)
    made.k, made.ks = cache.k.copy(), cache.ks.copy()
    for b in range(B):
        if 0 <= off[b] <= off[b + 1] <= n:
            ref.append(x.double().numpy(), made.k, made.ks, [0], [off[b], off[b + 1]],
                       table[b:b + 1])
    codes, scales = dev[0].cpu().numpy(), dev[2].cpu().numpy()
    for blk in range(total):
        for h in range(H):
            old = (codes[blk, h] == cache.k[blk, h]).all() and scales[blk, h] == cache.ks[blk, h]
            new = (codes[blk, h] == made.k[blk, h]).all() and scales[blk, h] == made.ks[blk, h]
            assert old or new, (blk, h)
