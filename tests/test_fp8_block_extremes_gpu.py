"""The block-scaled fp8 decode with V scales of any size beside one another."""
import numpy as np
import pytest

from tests import fp8_block_ref as ref
from tests.test_fp8_block_gpu import _decode_case
from workloads import BLOCK_SIZE

pytestmark = pytest.mark.gpu

# Exponents of the V scales of blocks that follow one another (two make a
# tile), None for a scale of 0: what the append can leave, 2^-126 to 2^120.
SPREADS = {
    "one_tile": [64, -64],
    "one_tile_small_first": [-64, 64],
    "falling": [64, 64, -64, -64, -64, -64],
    "rising": [-64, -64, -64, -64, 64, 64],
    "zero_beside_large": [None, 64],
    "zeros_then_large": [None, None, 64, 64],
    "large_then_zeros": [64, 64, None, None, None],
    "all_smallest": [-126, -126, -126],
    "whole_range": [-126, 119, None, -7, 119, -126],
    "ordinary_among_smallest": [-126, -7, -126, -126, -126],
    "all_zero": [None, None, None],
}


@pytest.mark.parametrize("ctas,wide", [(0, 0), (1, 100), (4, 100), (0, 100)],
                         ids=["whole", "1_cta", "4_ctas", "all_sms"])
@pytest.mark.parametrize("name", SPREADS)
@pytest.mark.parametrize("group,d", [(4, 64), (12, 128), (32, 128), (4, 256), (32, 256)])
def test_equal_weights_under_any_v_scales(lib, group, d, name, ctas, wide):
    """q = 0: every key weighs 1 / T, whatever its block's scale is; values are
    1 and 2 times the scale, so that nothing but the output is rounded (and the
    sum in fp32, 2^-20)."""
    exponents = SPREADS[name]
    T = BLOCK_SIZE * len(exponents) - 7

    def tweak(cache, table):
        cache.v = ref.encode(np.broadcast_to(1.0 + np.arange(d) % 2, cache.v.shape))
        for j, e in enumerate(exponents):
            cache.vs[table[0][j]] = 0 if e is None else np.float32(2.0) ** e
    rng = np.random.default_rng(80)
    got, cache, (_, _, _, table, _) = _decode_case(
        lib, rng, 2 * group, 2, d, [T], 1, 0, 0, tweak=tweak, scale=0.0, ctas=ctas, wide=wide)
    per_block = [BLOCK_SIZE] * (len(exponents) - 1) + [BLOCK_SIZE - 7]
    mean = sum(n * (0.0 if e is None else 2.0 ** e) for n, e in zip(per_block, exponents)) / T
    want = mean * (1.0 + np.arange(d) % 2)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= (2.0 ** -8 + 2.0 ** -18) * want).all(), (got[0, 0, 0, :2], want[:2])


@pytest.mark.parametrize("ctas,wide", [(0, 0), (5, 100)], ids=["whole", "5_ctas"])
@pytest.mark.parametrize("group,d", [(4, 64), (12, 128), (32, 256)])
def test_unequal_weights_under_spread_v_scales(lib, group, d, ctas, wide):
    """Ordinary scores under V scales from 2^-90 to 2^40, several beside one
    another: judged by the largest scale, as the values themselves are."""
    rng = np.random.default_rng(81)
    lens = [700, 129, 64]

    def tweak(cache, table):
        e = rng.choice([-90.0, -30.0, -7.0, 40.0], cache.vs.shape)
        cache.vs[:] = np.where(rng.random(e.shape) < 0.2, 0.0, np.exp2(e))
    got, cache, (q, k, v, table, scale) = _decode_case(
        lib, rng, 2 * group, 2, d, lens, 2, 0, 0, tweak=tweak, ctas=ctas, wide=wide)
    want, weighted = ref.decode(q.double().numpy(), k, v, lens, table, scale)
    got = got.double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * weighted + 2.0 ** -100
    over = np.abs(got - want) / bound
    assert over.max() <= 1, f"{over.max():.2f} of the bound"
