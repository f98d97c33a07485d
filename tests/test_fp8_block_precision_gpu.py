"""How near the block-scaled fp8 decode comes to 64 bits: the bits of
a single weight, and the bar that the library's other decodes keep to."""
import numpy as np
import pytest

from tests import fp8_block_ref as ref
from tests.parity import BF16_REL_L2, errors
from tests.test_fp8_block_gpu import DECODES, _decode_case
from workloads import BLOCK_SIZE

pytestmark = pytest.mark.gpu


# (query heads of a K/V head: 4, 12 and 32 rows take the three column forms)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [4, 12, 32])
def test_decode_holds_weights_in_eleven_bits(lib, group, d):
    """Sequences of a few keys whose values cancel: what is left shows each
    weight's rounding.  A weight is rounded to f16 (2^-11 of it); scores, their
    exponentials and the sum are fp32, 2^-14 together; the output is bf16."""
    rng = np.random.default_rng(70 + group + d)
    lens = [2 + i % 5 for i in range(40)]

    def tweak(cache, table):
        signs = np.where(np.arange(BLOCK_SIZE) % 2, -1.0, 1.0)[None, None, :, None]
        cache.v = ref.encode(np.broadcast_to(signs * 112.0, cache.v.shape))
        cache.vs[:] = 2.0 ** -6
    got, cache, (q, k, v, table, scale) = _decode_case(
        lib, rng, 2 * group, 2, d, lens, 1, 0, 0, tweak=tweak)
    want, weighted = ref.decode(q.double().numpy(), k, v, lens, table, scale)
    got = got.double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14) * weighted
    over = np.abs(got - want) / bound
    assert over.max() <= 1, f"{over.max():.2f} of the bound"


@pytest.mark.parametrize("case", [c for c in DECODES if max(c[3]) >= 64],
                         ids=[f"q{c[0]}_kv{c[1]}_d{c[2]}_L{c[4]}_w{c[5]}"
                              for c in DECODES if max(c[3]) >= 64])
def test_decode_meets_the_bar_of_the_other_kernels(lib, case):
    """The relative L2 that every decode of the library keeps to."""
    H_q, H_kv, d, lens, q_len, window, sink = case
    rng = np.random.default_rng(71 + H_q + d)
    got, _, (q, k, v, table, scale) = _decode_case(lib, rng, *case)
    want, _ = ref.decode(q.double().numpy(), k, v, lens, table, scale, window=window, sink=sink)
    _, rel = errors(got.float().cpu().numpy(), want)
    assert rel <= BF16_REL_L2, rel
