"""The block-scaled fp8 cache where calls reach furthest: many query positions,
scales that are no powers of two, blocks beyond 4 GiB, a million tokens."""
import numpy as np
import pytest
import torch

from tests import fp8_block_ref as ref
from tests.test_fp8_block_gpu import _check, _decode_case, _ints, _offsets, _rows
from workloads import BLOCK_SIZE

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("wide", [0, 100], ids=["narrow", "wide"])
@pytest.mark.parametrize("H_q,H_kv,d,window,sink", [(8, 2, 64, 0, 0), (8, 2, 128, 70, 5),
                                                    (6, 6, 256, 33, 0)])
def test_a_chunk_of_query_positions(lib, H_q, H_kv, d, window, sink, wide):
    """150 positions a sequence: its rows come in chunks of 32, whose tiles may
    hold no key that a row, or a whole chunk, sees."""
    lens = [150, 401, 70]
    got, cache, inputs = _decode_case(lib, np.random.default_rng(100), H_q, H_kv, d, lens, 150,
                                      window, sink, wide=wide)
    _check(got, cache, inputs, lens, window, sink)
    assert (got[2, :80] == 0).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scales_that_are_no_powers_of_two(lib, sign):
    rng = np.random.default_rng(101)
    lens = [700, 65]

    def tweak(cache, table):
        cache.ks[:] = rng.uniform(0.002, 0.02, cache.ks.shape)
        cache.vs[:] = rng.uniform(0.002, 0.02, cache.vs.shape)
    for group, d in ((4, 64), (12, 128), (32, 256)):
        got, cache, inputs = _decode_case(lib, rng, 2 * group, 2, d, lens, 1, 0, 0, tweak=tweak,
                                          scale=sign / np.sqrt(d), wide=50)
        _check(got, cache, inputs, lens, 0, 0)


def test_blocks_beyond_four_gib(lib):
    """The same calls on the first blocks of a small cache and on the last ones
    of a cache of 4.5 GiB for K and as much for V."""
    rng = np.random.default_rng(102)
    H, d, pos, cnt = 4, 256, [0, 30], [200, 170]
    many = (9 << 29) // (H * BLOCK_SIZE * d)
    off = _offsets(cnt)
    k, v = (_rows(rng, off[-1], H, d, torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((2, 8, d))).bfloat16().to(DEV)
    low = np.arange(8, dtype=np.int32).reshape(2, 4)
    results = []
    for blocks in (8, many):
        table = _ints(low + (blocks - 8))
        dev = [torch.zeros((blocks, H, BLOCK_SIZE, d), dtype=torch.uint8, device=DEV)
               for _ in range(2)]
        dev += [torch.zeros((blocks, H), device=DEV) for _ in range(2)]
        lib.kv_append_fp8_block(k, v, *dev, _ints(pos), table, offsets=_ints(off))
        rows = lib.kv_read_fp8_block(*dev, _ints(pos), table, off[-1], offsets=_ints(off))
        out = lib.decode_gqa_fp8_block(q, *dev, _ints([200, 200]), table, 0.06)
        assert lib.last_error() == lib.OK
        results.append([x[-8:].clone() for x in dev] + list(rows) + [out])
        del dev
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_a_million_tokens(lib):
    """q = 0 over equal values but for one late block: every key weighs 2^-20."""
    T, H_q, H_kv, d = 1 << 20, 8, 2, 64
    blocks = T // BLOCK_SIZE
    k = torch.zeros((blocks, H_kv, BLOCK_SIZE, d), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    one = int(ref.encode(np.float64(1.0)))
    v[blocks - 2, 1] = int(ref.encode(np.float64(256.0)))
    v[:, 0] = one
    s = torch.ones((blocks, H_kv), device=DEV)
    table = torch.randperm(blocks, device=DEV).to(torch.int32)
    q = torch.zeros((1, H_q, d), dtype=torch.bfloat16, device=DEV)
    out = lib.decode_gqa_fp8_block(q, k, v, s, s, _ints([T]), table[None], 1.0)
    assert lib.last_error() == lib.OK
    assert (out[0, :4] == 1.0).all()
    assert (out[0, 4:] == 64 * 256 * 2.0 ** -20).all()
