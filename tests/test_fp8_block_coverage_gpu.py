"""The block-scaled fp8 decode over values that show each block of a long
sequence: what bounds on sums of random values cannot see."""
import numpy as np
import pytest

from tests import fp8_block_ref as ref
from tests.test_fp8_block_gpu import _decode_case
from workloads import BLOCK_SIZE

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctas", [0, 1, 7, 50])
@pytest.mark.parametrize("group,d", [(4, 64), (12, 64), (32, 64), (4, 128), (12, 128), (32, 128),
                                     (4, 256), (12, 256), (32, 256)])
def test_every_block_of_a_long_sequence_counts_once(lib, group, d, ctas):
    """q = 0, and the values of block j are 2^(j / d) in one column and 0 in the
    others: a block that is lost, doubled or given to another head changes its
    column by 1/31 of it or more, where rounding is 2^-8."""
    rng = np.random.default_rng(82)
    lens = [20011, 1, 700, 4096]
    H_kv = 2

    def column(b, j, h):
        return (j + 7 * h + 3 * b) % d

    def tweak(cache, table):
        cache.v[:] = 0
        cache.vs[:] = 2.0 ** -3
        for b, T in enumerate(lens):
            for j in range(-(-T // BLOCK_SIZE)):
                for h in range(H_kv):
                    cache.v[table[b][j], h, :, column(b, j, h)] = ref.encode(
                        np.float64(2.0 ** (j // d)))
    got, _, _ = _decode_case(lib, rng, H_kv * group, H_kv, d, lens, 1, 0, 0, tweak=tweak,
                             scale=0.0, ctas=ctas)
    got = got.double().cpu().numpy()
    for b, T in enumerate(lens):
        want = np.zeros((H_kv, d))
        for j in range(-(-T // BLOCK_SIZE)):
            for h in range(H_kv):
                n = min(BLOCK_SIZE, T - j * BLOCK_SIZE)
                want[h, column(b, j, h)] += n * 2.0 ** (j // d - 3) / T
        err = np.abs(got[b, 0].reshape(H_kv, group, d) - want[:, None])
        assert (err <= (2.0 ** -8 + 2.0 ** -18) * want[:, None]).all(), f"sequence {b}"
