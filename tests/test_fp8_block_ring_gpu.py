"""Append to and read back from a ring table with an explicit global set."""
import numpy as np
import pytest
import torch

from tests import fp8_block_ref as ref
from tests.test_fp8_block_gpu import _Cache, _ints, _offsets, _rows, _table
from workloads import BLOCK_SIZE

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (positions, counts, global rows (-1 ends a row), window, ring)
RUNS = [
    ([0], [900], [[3, 5, 70, 300]], 128, 4),
    ([0, 0], [900, 640], [[0, 5, 300, 301, 700], [64, 639, -1, -1, -1]], 100, 3),
    ([0, 0, 0], [1300, 65, 64], [[5, 700, 1299], [1, 2, 64], [-1, -1, -1]], 190, 4),
]


def _ring_table(pos, counts, rows, ring, spare=3):
    """Global slot k names the block of its position from that block's first
    row on, and the ring slot names the same block while the ring holds it (a
    block that the ring has left has one of its own)."""
    n_g = len(rows[0])
    free = iter(range(1, 10000))
    table = np.full((len(pos), n_g + ring), -1, dtype=np.int32)
    for b, row in enumerate(rows):
        last = (pos[b] + counts[b] - 1) // BLOCK_SIZE
        held = {}
        for blk in range(max(0, last - ring + 1), last + 1):
            held[blk] = table[b, n_g + blk % ring] = next(free)
        prev = -1
        for k, p in enumerate(row):
            if p <= prev:
                break
            prev = p
            if p // BLOCK_SIZE not in held:
                held[p // BLOCK_SIZE] = next(free)
            table[b, k] = held[p // BLOCK_SIZE]
    return table, int(table.max()) + 1 + spare


def _full(rng, pos, counts, H, d, dtype, lib):
    """The run appended to a cache without a ring, on the host: definition."""
    off = _offsets(counts)
    table, total = _table(rng, [-(-(p + n) // BLOCK_SIZE) for p, n in zip(pos, counts)])
    cache = _Cache(rng, total, H, d)
    k, v = (_rows(rng, off[-1], H, d, dtype) for _ in range(2))
    ref.append(k.double().numpy(), cache.k, cache.ks, pos, off, table)
    ref.append(v.double().numpy(), cache.v, cache.vs, pos, off, table)
    return off, table, cache, k, v


@pytest.mark.parametrize("H,d,dtype", [(2, 64, torch.bfloat16), (8, 128, torch.float32),
                                       (1, 256, torch.bfloat16)])
@pytest.mark.parametrize("run", RUNS, ids=["one", "two", "three"])
def test_prompt_through_a_ring_with_a_global_set(lib, run, H, d, dtype):
    """A prompt longer than the ring: the blocks of global positions are kept in
    their global slots, are read back from there, and the decode over the ring
    is the decode over the whole cache, bit for bit."""
    pos, counts, rows, window, ring = run
    rng = np.random.default_rng(90 + H + len(pos))
    off, full_table, full, k, v = _full(rng, pos, counts, H, d, dtype, lib)
    table, total = _ring_table(pos, counts, rows, ring)
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    gp = _ints(rows)
    kw = dict(window=window, ring_blocks=ring, global_pos=gp)
    lib.kv_append_fp8_block(k.to(DEV), v.to(DEV), *dev, _ints(pos), _ints(table),
                            offsets=_ints(off), **kw)
    assert lib.last_error() == lib.OK
    n_g = len(rows[0])
    for b in range(len(pos)):
        last = (counts[b] - 1) // BLOCK_SIZE
        ends = next((i for i, p in enumerate(rows[b]) if p < 0), n_g)
        slots = {p // BLOCK_SIZE: s for s, p in reversed(list(enumerate(rows[b][:ends])))
                 if p < counts[b]}
        for blk in range(max(0, last - ring + 1), last + 1):
            slots.setdefault(blk, n_g + blk % ring)
        for blk, slot in slots.items():
            n = min(BLOCK_SIZE, counts[b] - blk * BLOCK_SIZE)
            mine, theirs = int(table[b][slot]), int(full_table[b][blk])
            assert torch.equal(dev[0][mine, :, :n].cpu(),
                               torch.from_numpy(full.k[theirs, :, :n])), (b, blk)
            assert torch.equal(dev[3][mine].cpu(), torch.from_numpy(full.vs[theirs])), (b, blk)
            # the block's rows one by one, as any run of the reader may ask
            first = blk * BLOCK_SIZE
            got = lib.kv_read_fp8_block(
                *dev, _ints([first] * len(pos)), _ints(table), n,
                offsets=_ints([0] * (b + 1) + [n] * (len(pos) - b)), dtype=torch.float32, **kw)
            assert lib.last_error() == lib.OK
            for x, c, s in zip(got, (full.k, full.v), (full.ks, full.vs)):
                want = ref.dense(c, s)[theirs, :, :n].transpose(1, 0, 2)
                assert np.array_equal(x.double().cpu().numpy(), want), (b, blk)
    q = torch.from_numpy(rng.standard_normal((len(pos), 4 * H, d))).bfloat16().to(DEV)
    # a query that is itself global needs the history that the ring has left
    lens = _ints([n if n - 1 not in r or n <= window else n - 1 for n, r in zip(counts, rows)])
    got = lib.decode_gqa_fp8_block(q, *dev, lens, _ints(table), 0.1, **kw)
    want = lib.decode_gqa_fp8_block(q, *full.device(), lens, _ints(full_table), 0.1,
                                    window=window, global_pos=gp)
    assert lib.last_error() == lib.OK
    # the same blocks in the same order, cut the same way
    assert torch.equal(got, want)


def test_steps_through_a_ring_with_a_global_set(lib):
    """One token a call: rows go through the ring slots, as kv_append_ext's do,
    also where the global slot is not named yet."""
    rng = np.random.default_rng(91)
    H, d, window, ring, rows = 2, 64, 100, 3, [[0, 300]]
    table = np.array([[-1, -1, 1, 2, 3]], dtype=np.int32)
    cache = _Cache(rng, 5, H, d)
    dev = cache.device()
    for t in (0, 63, 64, 300):
        x = _rows(rng, 1, H, d, torch.bfloat16)
        lib.kv_append_fp8_block(x.to(DEV), x.to(DEV), *dev, _ints([t]), _ints(table),
                                window=window, ring_blocks=ring, global_pos=_ints(rows))
        for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
            ref.append(x.double().numpy(), c, s, [t % BLOCK_SIZE], [0, 1],
                       [[1 + t // BLOCK_SIZE % ring]])
    assert lib.last_error() == lib.OK
    cache.check(dev, "steps")


def test_run_goes_on_in_a_global_block_that_the_ring_leaves(lib):
    """Rows 0-5 of block 1 come in one call through the ring, the rest in a run
    that leaves the block behind: it keeps its scale or grows it."""
    rng = np.random.default_rng(94)
    H, d, window, ring, rows = 2, 128, 100, 3, [[3, 66, 300]]
    before = np.array([[1, 2, -1, 1, 2, 3]], dtype=np.int32)
    after = np.array([[1, 2, 9, 6, 7, 5]], dtype=np.int32)
    cache = _Cache(rng, 10, H, d)
    dev = cache.device()
    full_table = np.array([[1, 2, 10, 11, 9, 12, 13, 14, 5, 6, 7]], dtype=np.int32)
    full = _Cache(rng, 15, H, d)
    kw = dict(window=window, ring_blocks=ring, global_pos=_ints(rows))
    for table, pos, n in ((before, 0, 70), (after, 70, 630)):
        k, v = (_rows(rng, n, H, d, torch.bfloat16) for _ in range(2))
        lib.kv_append_fp8_block(k.to(DEV), v.to(DEV), *dev, _ints([pos]), _ints(table),
                                offsets=_ints([0, n]), **kw)
        ref.append(k.double().numpy(), full.k, full.ks, [pos], [0, n], full_table)
        ref.append(v.double().numpy(), full.v, full.vs, [pos], [0, n], full_table)
    assert lib.last_error() == lib.OK
    for phys, held in ((1, 64), (2, 64), (9, 64), (5, 64), (6, 64), (7, 60)):
        assert torch.equal(dev[0][phys, :, :held].cpu(), torch.from_numpy(full.k[phys, :, :held]))
        assert torch.equal(dev[1][phys, :, :held].cpu(), torch.from_numpy(full.v[phys, :, :held]))
        assert torch.equal(dev[2][phys].cpu(), torch.from_numpy(full.ks[phys]))


def test_read_of_an_unnamed_global_block_is_flagged(lib):
    """A global slot that names nothing reads as zeros, not as the ring's block."""
    rng = np.random.default_rng(92)
    H, d = 1, 64
    table = np.array([[-1, 0, 1, 2]], dtype=np.int32)
    cache = _Cache(rng, 3, H, d)
    k, _ = lib.kv_read_fp8_block(*cache.device(), _ints([5]), _ints(table), 1, window=100,
                                 ring_blocks=3, global_pos=_ints([[7]]))
    assert lib.last_error() == lib.ERR_BAD_BLOCK
    assert (k == 0).all()
