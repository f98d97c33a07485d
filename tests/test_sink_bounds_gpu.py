"""A kept prefix as long as an int counts shows every key."""
import numpy as np
import pytest
import torch

from tests.test_fp8_block_gpu import _check, _decode_case
from tests.test_vis_gpu import _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
LARGEST = 2 ** 31 - 1


@pytest.mark.parametrize("q_len", [1, 3])
def test_block_scaled_decode(lib, q_len):
    lens = [700, 65, 0]
    got, cache, inputs = _decode_case(lib, np.random.default_rng(97), 8, 2, 128, lens, q_len, 10,
                                      LARGEST)
    _check(got, cache, inputs, lens, 0, 0)


@pytest.mark.parametrize("path", [0, 1, 2])
def test_decode_ext(lib, path):
    lens = torch.tensor([300, 64], dtype=torch.int32)
    q, k, v, table = _inputs(98, 2, 8, 1, 64, 10, 5)
    args = [x.to(DEV) for x in (q, k, v, lens, table)]
    lib.set_gqa_path(path)
    try:
        got = lib.decode_gqa_ext(*args, 0.1, window=10, sink_tokens=LARGEST)
        want = lib.decode_gqa_ext(*args, 0.1)
        assert lib.last_error() == lib.OK
    finally:
        lib.set_gqa_path(-1)
    assert torch.equal(got, want)
