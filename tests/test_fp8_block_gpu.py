"""GPU parity of the block-scaled fp8 cache against its fp64 definition:
append and read-back exactly, decode within the rounding of its weights and of
its bf16 output."""
import numpy as np
import pytest
import torch

from tests import fp8_block_ref as ref
from workloads import BLOCK_SIZE

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _offsets(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def _codes(rng, n_blocks, H, d):
    """Any code but the NaNs."""
    c = rng.integers(0, 254, (n_blocks, H, BLOCK_SIZE, d))
    return (c + (c >= 127)).astype(np.uint8)


def _scales(rng, n_blocks, H, lo=-8, hi=-4):
    return np.exp2(rng.integers(lo, hi, (n_blocks, H))).astype(np.float32)


def _rows(rng, n, H, d, dtype):
    """Rows whose magnitude varies from row to row, a tenth of them by 2^6."""
    mag = np.exp2(rng.integers(-3, 3, (n, 1, 1)) + 6 * (rng.random((n, 1, 1)) < 0.1))
    x = torch.from_numpy(rng.standard_normal((n, H, d)) * mag).to(dtype)
    return x


def _table(rng, blocks, extra=2):
    total = sum(blocks) + extra
    perm = rng.permutation(total)
    t = np.full((len(blocks), max(max(blocks), 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(blocks):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, total


class _Cache:
    def __init__(self, rng, n_blocks, H, d, lo=-8, hi=-4):
        self.k, self.v = (_codes(rng, n_blocks, H, d) for _ in range(2))
        self.ks, self.vs = (_scales(rng, n_blocks, H, lo, hi) for _ in range(2))

    def device(self):
        return [torch.from_numpy(x.copy()).to(DEV) for x in (self.k, self.v, self.ks, self.vs)]

    def check(self, dev, what):
        for name, mine, theirs in zip(("k", "v", "ks", "vs"),
                                      (self.k, self.v, self.ks, self.vs), dev):
            got = theirs.cpu().numpy()
            if mine.dtype == np.float32:
                assert np.array_equal(got.view(np.uint32), mine.view(np.uint32)), f"{what} {name}"
            else:
                # the two NaN codes are one value
                same = (got == mine) | (((got & 127) == 127) & ((mine & 127) == 127))
                assert same.all(), f"{what} {name}: {(~same).sum()} codes differ"


# ------------------------------------------------------------------ append

APPENDS = [
    # (H_kv, d, positions, counts, dtype)
    (8, 128, [70, 3, 127, 64], [1, 1, 1, 1], torch.bfloat16),
    (1, 64, [0], [1], torch.float32),
    (2, 64, [0, 63, 5, 64], [64, 2, 59, 0], torch.bfloat16),
    (3, 256, [1, 0, 200], [130, 65, 1], torch.float32),
    (4, 128, [10, 0, 0, 31], [0, 300, 1, 97], torch.bfloat16),
    (2, 128, [i % 70 for i in range(70)], [i % 5 for i in range(70)], torch.bfloat16),
]


@pytest.mark.parametrize("H,d,pos,cnt,dtype", APPENDS,
                         ids=[f"kv{c[0]}_d{c[1]}_B{len(c[2])}" for c in APPENDS])
def test_append_is_exact(lib, H, d, pos, cnt, dtype):
    rng = np.random.default_rng(10 + d + len(pos))
    off = _offsets(cnt)
    table, total = _table(rng, [-(-(p + n) // BLOCK_SIZE) for p, n in zip(pos, cnt)])
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    k, v = (_rows(rng, off[-1], H, d, dtype) for _ in range(2))
    single = all(n == 1 for n in cnt)
    lib.kv_append_fp8_block(k.to(DEV), v.to(DEV), *dev, _ints(pos), _ints(table),
                            offsets=None if single else _ints(off))
    assert lib.last_error() == lib.OK
    ref.append(k.double().numpy(), cache.k, cache.ks, pos, off, table)
    ref.append(v.double().numpy(), cache.v, cache.vs, pos, off, table)
    cache.check(dev, "append")


def test_append_special_values(lib):
    """Zero rows, infinities, NaN, the smallest and the largest numbers, amax on
    and just above a power of two times 448, ties between two codes."""
    rng = np.random.default_rng(11)
    H, d = 2, 64
    rows = np.zeros((9, H, d), dtype=np.float32)
    rows[1, 0, :3] = [np.inf, -np.inf, 3.0]
    rows[1, 1, 5] = np.nan
    rows[2] = 1e-45
    rows[3] = 3.4e38
    rows[4, :, 0] = 448.0
    rows[5, :, 0] = np.nextafter(np.float32(448.0), np.float32(1e9))
    rows[6, :, :] = np.linspace(-448, 448, 2 * d).reshape(H, d)
    rows[6, 0, :4] = [17.0, 19.0, -17.0, 0.0009765625]     # ties (448 keeps the scale at 1)
    rows[7] = 2.0 ** -126
    rows[8, 0, 0] = -0.0
    pos, off = [0] * 9, list(range(10))
    table, total = _table(rng, [1] * 9)
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    new = torch.from_numpy(rows)
    lib.kv_append_fp8_block(new.to(DEV), new.to(DEV), *dev, _ints(pos), _ints(table))
    assert lib.last_error() == lib.OK
    for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
        ref.append(rows.astype(np.float64), c, s, pos, off, table)
    cache.check(dev, "special")


def test_append_grows_a_block_token_by_token(lib):
    """Sixty-six single-token steps with growing and shrinking rows: the block's
    scale never falls, and its earlier rows are rounded as the definition says."""
    rng = np.random.default_rng(12)
    H, d = 2, 128
    table, total = _table(rng, [2, 2])
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    for t in range(66):
        x = torch.from_numpy(rng.standard_normal((2, H, d)) * 2.0 ** rng.integers(-6, 6, (2, H, 1)))
        x = x.bfloat16()
        lib.kv_append_fp8_block(x.to(DEV), x.to(DEV), *dev, _ints([t, t]), _ints(table))
        for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
            ref.append(x.double().numpy(), c, s, [t, t], [0, 1, 2], table)
    assert lib.last_error() == lib.OK
    cache.check(dev, "steps")


def test_append_columns_of_a_projection(lib):
    """K and V as columns of one [tokens][(H_q + 2 H_kv) d] projection, rows
    behind the last sequence unused."""
    rng = np.random.default_rng(13)
    H, d, pos, cnt = 2, 64, [60, 0], [10, 7]
    off = _offsets(cnt)
    fused = torch.from_numpy(rng.standard_normal((off[-1] + 5, 8 * d))).bfloat16().to(DEV)
    k, v = (fused[:, a * d:(a + 2) * d].unflatten(1, (H, d)) for a in (4, 6))
    table, total = _table(rng, [2, 1])
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    lib.kv_append_fp8_block(k, v, *dev, _ints(pos), _ints(table), offsets=_ints(off))
    assert lib.last_error() == lib.OK
    ref.append(k.double().cpu().numpy(), cache.k, cache.ks, pos, off, table)
    ref.append(v.double().cpu().numpy(), cache.v, cache.vs, pos, off, table)
    cache.check(dev, "columns")


@pytest.mark.parametrize("sink", [0, 70])
def test_append_through_a_ring(lib, sink):
    """A run longer than the ring keeps the blocks that stay, and reads back."""
    rng = np.random.default_rng(14)
    H, d, ring = 2, 64, 3
    width = -(-sink // BLOCK_SIZE) + ring
    pos, cnt = [0, 130], [500, 100]
    off = _offsets(cnt)
    table, total = _table(rng, [width, width])
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    k, v = (_rows(rng, off[-1], H, d, torch.bfloat16) for _ in range(2))
    kw = dict(window=100, sink_tokens=sink, ring_blocks=ring)
    lib.kv_append_fp8_block(k.to(DEV), v.to(DEV), *dev, _ints(pos), _ints(table),
                            offsets=_ints(off), **kw)
    assert lib.last_error() == lib.OK
    for x, c, s in ((k, cache.k, cache.ks), (v, cache.v, cache.vs)):
        ref.append(x.double().numpy(), c, s, pos, off, table, sink=sink, ring=ring)
    cache.check(dev, "ring")
    last = [p + n for p, n in zip(pos, cnt)]
    tail = [100, 40]
    got = lib.kv_read_fp8_block(*dev, _ints([t - n for t, n in zip(last, tail)]), _ints(table),
                                sum(tail), offsets=_ints(_offsets(tail)), dtype=torch.float32, **kw)
    assert lib.last_error() == lib.OK
    for x, c, s in zip(got, (cache.k, cache.v), (cache.ks, cache.vs)):
        values, at = ref.dense(c, s), 0
        for b, n in enumerate(tail):
            for t in range(last[b] - n, last[b]):
                phys = table[b][ref.slot_of(t // BLOCK_SIZE, sink, ring)]
                assert np.array_equal(x[at].double().cpu().numpy(), values[phys, :, t % BLOCK_SIZE])
                at += 1


def test_append_skips_and_flags_what_is_out_of_range(lib):
    rng = np.random.default_rng(15)
    H, d = 1, 64
    table = np.array([[0, 99], [1, -1], [2, 3], [4, 5]], dtype=np.int32)
    pos, cnt = [60, 64, -1, 120], [10, 3, 2, 20]      # bad id, bad id, before, behind the table
    off = _offsets(cnt)
    cache = _Cache(rng, 6, H, d)
    dev = cache.device()
    x = _rows(rng, off[-1], H, d, torch.bfloat16)
    lib.kv_append_fp8_block(x.to(DEV), x.to(DEV), *dev, _ints(pos), _ints(table),
                            offsets=_ints(off))
    assert lib.last_error() == lib.ERR_BAD_BLOCK
    rows = x.double().numpy()
    for c, s in ((cache.k, cache.ks), (cache.v, cache.vs)):
        ref.append(rows[0:4], c, s, [60], [0, 4], table[:1])
        ref.append(rows[15:23], c, s, [120], [0, 8], table[3:])
    cache.check(dev, "skipped")


@pytest.mark.parametrize("off", [[0, 5, 3, 6], [0, 2, 4, 700], [-1, 2, 4, 6]])
def test_append_and_read_flag_bad_offsets(lib, off):
    """The runs whose ends are wrong are skipped, the others done."""
    rng = np.random.default_rng(16)
    H, d, n = 1, 64, 6
    table, total = _table(rng, [1, 1, 1])
    cache = _Cache(rng, total, H, d)
    dev = cache.device()
    x = _rows(rng, n, H, d, torch.bfloat16)
    lib.kv_append_fp8_block(x.to(DEV), x.to(DEV), *dev, _ints([0, 0, 0]), _ints(table),
                            offsets=_ints(off))
    assert lib.last_error() == lib.ERR_BAD_SEQLEN
    lib.kv_read_fp8_block(*dev, _ints([0, 0, 0]), _ints(table), n, offsets=_ints(off))
    assert lib.last_error() == lib.ERR_BAD_SEQLEN


# ------------------------------------------------------------------ read

READS = [
    # (H_kv, d, positions, counts, dtype)
    (8, 128, [70, 0, 63], [130, 1, 2], torch.bfloat16),
    (2, 64, [0, 5, 7], [64, 0, 333], torch.float32),
    (3, 256, [31], [90], torch.bfloat16),
]


@pytest.mark.parametrize("H,d,pos,cnt,dtype", READS, ids=[f"kv{c[0]}_d{c[1]}" for c in READS])
def test_read_is_exact(lib, H, d, pos, cnt, dtype):
    rng = np.random.default_rng(20 + d)
    off = _offsets(cnt)
    table, total = _table(rng, [-(-(p + n) // BLOCK_SIZE) for p, n in zip(pos, cnt)])
    cache = _Cache(rng, total, H, d, -20, 20)
    cache.vs[rng.random(cache.vs.shape) < 0.2] = 0
    n = off[-1] + 3                                   # rows behind the last sequence
    out = [torch.full((n, H, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    got = lib.kv_read_fp8_block(*cache.device(), _ints(pos), _ints(table), n, offsets=_ints(off),
                                dtype=dtype, out=out)
    assert lib.last_error() == lib.OK
    assert got[0] is out[0] and got[1] is out[1]
    for x, c, s in zip(got, (cache.k, cache.v), (cache.ks, cache.vs)):
        values = ref.dense(c, s)
        want = np.full((n, H, d), 7.0)
        for b, p in enumerate(pos):
            for t in range(cnt[b]):
                phys = table[b][(p + t) // BLOCK_SIZE]
                want[off[b] + t] = values[phys, :, (p + t) % BLOCK_SIZE]
        assert torch.equal(x.cpu(), torch.from_numpy(want).to(dtype))


def test_read_gives_zeros_for_missing_blocks(lib):
    rng = np.random.default_rng(21)
    H, d = 2, 64
    cache = _Cache(rng, 2, H, d)
    table = np.array([[0, 77], [1, -1]], dtype=np.int32)
    k, _ = lib.kv_read_fp8_block(*cache.device(), _ints([62, -3]), _ints(table), 9,
                                 offsets=_ints([0, 4, 8]), dtype=torch.float32)
    assert lib.last_error() == lib.ERR_BAD_BLOCK
    k = k.cpu().double().numpy()
    assert np.array_equal(k[:2], ref.dense(cache.k, cache.ks)[0, :, 62:].transpose(1, 0, 2))
    assert (k[2:] == 0).all()


# ------------------------------------------------------------------ decode

DECODES = [
    # (H_q, H_kv, d, lens, q_len, window, sink)
    (32, 8, 128, [1000, 65, 1], 1, 0, 0),
    (8, 8, 64, [700, 300, 64], 1, 0, 0),
    (24, 4, 256, [3000, 129], 1, 0, 0),
    (32, 1, 128, [600, 64, 128, 129], 1, 0, 0),
    (12, 1, 64, [200, 0, 63], 1, 0, 0),
    (40, 8, 128, [193], 1, 0, 0),
    (32, 8, 128, [2000, 90, 301, 300], 1, 300, 16),
    (24, 4, 256, [1500, 64], 1, 1, 0),
    (4, 2, 64, [800, 77], 1, 128, 130),
    (32, 8, 128, [500, 5, 3, 130], 5, 0, 0),
    (8, 4, 64, [500, 66, 2], 3, 64, 0),
    (32, 1, 256, [260, 7], 6, 100, 10),
    (32, 32, 128, [300, 1], 2, 70, 5),
    (70, 1, 64, [150], 1, 0, 0),
    (6, 2, 256, [0, 0], 2, 0, 0),
]


def _decode_case(lib, rng, H_q, H_kv, d, lens, q_len, window, sink, ring=0, global_pos=None,
                 lo=-8, hi=-4, table=None, tweak=None, scale=None, ctas=0, wide=0, **call):
    B = len(lens)
    if table is None:
        table, total = _table(rng, [-(-t // BLOCK_SIZE) for t in lens])
        if wide > table.shape[1]:              # room for sequences that are longer yet
            more = np.full((B, wide - table.shape[1]), -1, dtype=np.int32)
            table = np.concatenate([table, more], axis=1)
    else:
        total = int(table.max()) + 1
    cache = _Cache(rng, total, H_kv, d, lo, hi)
    # unit variance in codes of up to 448 / 2^7
    cache.k, cache.v = (ref.encode(rng.standard_normal(cache.k.shape) * 128) for _ in range(2))
    if tweak:
        tweak(cache, table)
    q = torch.from_numpy(rng.standard_normal((B, q_len, H_q, d))).bfloat16()
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    lib.set_num_ctas(ctas)
    try:
        got = lib.decode_gqa_fp8_block(
            q.to(DEV), *cache.device(), _ints(lens), _ints(table), scale, window=window,
            sink_tokens=sink, ring_blocks=ring,
            global_pos=None if global_pos is None else _ints(global_pos), **call)
    finally:
        lib.set_num_ctas(0)
    assert lib.last_error() == lib.OK
    k, v = ref.dense(cache.k, cache.ks), ref.dense(cache.v, cache.vs)
    return got, cache, (q, k, v, table, scale)


def _check(got, cache, inputs, lens, window, sink, ring=0, global_pos=None, what=""):
    q, k, v, table, scale = inputs
    want, weighted = ref.decode(q.double().numpy(), np.nan_to_num(k), np.nan_to_num(v), lens, table,
                                scale, window=window, sink=sink, ring=ring, global_pos=global_pos)
    ref.assert_decode(got.float(), want, weighted, float(cache.vs.max()), what)


@pytest.mark.parametrize("ctas", [0, 7], ids=["all_sms", "7_ctas"])
@pytest.mark.parametrize("case", DECODES, ids=[f"q{c[0]}_kv{c[1]}_d{c[2]}_L{c[4]}_w{c[5]}"
                                               for c in DECODES])
def test_decode_matches_oracle(lib, case, ctas):
    H_q, H_kv, d, lens, q_len, window, sink = case
    rng = np.random.default_rng(30 + H_q + d)
    got, cache, inputs = _decode_case(lib, rng, *case, ctas=ctas)
    _check(got, cache, inputs, lens, window, sink)
    none = [[max(t - q_len + i + 1, 0) == 0 for i in range(q_len)] for t in lens]
    assert (got[torch.tensor(none, device=DEV)] == 0).all()


@pytest.mark.parametrize("ctas", [0, 1, 3], ids=["all_sms", "1_cta", "3_ctas"])
@pytest.mark.parametrize("case", DECODES, ids=[f"q{c[0]}_kv{c[1]}_d{c[2]}_L{c[4]}_w{c[5]}"
                                               for c in DECODES])
def test_decode_split_over_ctas(lib, case, ctas):
    """A table wide enough for long sequences: the same units, cut anywhere."""
    H_q, H_kv, d, lens, q_len, window, sink = case
    rng = np.random.default_rng(60 + H_q + d)
    got, cache, inputs = _decode_case(lib, rng, *case, ctas=ctas, wide=100)
    _check(got, cache, inputs, lens, window, sink)


@pytest.mark.parametrize("q_len,window", [(1, 0), (3, 100)])
def test_decode_many_sequences(lib, q_len, window):
    """More sequences than one warp plans for, some of them empty."""
    rng = np.random.default_rng(61)
    lens = [(37 * i * i) % 700 for i in range(45)]
    for wide in (0, 100):
        got, cache, inputs = _decode_case(lib, rng, 4, 2, 64, lens, q_len, window, 0, wide=wide)
        _check(got, cache, inputs, lens, window, 0)


def test_decode_many_short_units_of_a_cta(lib):
    """Units of one block each, several to a CTA: every ring turns over."""
    rng = np.random.default_rng(62)
    lens = [1 + (11 * i) % 64 for i in range(30)]
    for H_q, H_kv, d in ((32, 32, 64), (32, 8, 256), (64, 2, 128)):
        got, cache, inputs = _decode_case(lib, rng, H_q, H_kv, d, lens, 1, 0, 0, wide=100, ctas=5)
        _check(got, cache, inputs, lens, 0, 0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_long_and_split(lib, d):
    """One sequence over many splits, and a sequence of one key beside it."""
    case = (8, 2, d, [20011, 1], 1, 0, 0)
    rng = np.random.default_rng(31 + d)
    got, cache, inputs = _decode_case(lib, rng, *case)
    _check(got, cache, inputs, case[3], 0, 0)


def test_decode_scales_of_all_sizes(lib):
    """Block scales of V from 2^-30 to 2^-4, some 0."""
    rng = np.random.default_rng(32)

    def tweak(cache, table):
        cache.ks[:] = _scales(rng, *cache.ks.shape, -12, -6)
        cache.vs[rng.random(cache.vs.shape) < 0.2] = 0
    case = (8, 2, 128, [1500, 333], 2, 0, 0)
    got, cache, inputs = _decode_case(lib, rng, *case, lo=-30, hi=-3, tweak=tweak)
    _check(got, cache, inputs, case[3], 0, 0)


def test_decode_one_key_far_ahead(lib):
    """A first key that takes nearly all weight, thousands that share a small
    rest: what they add together is not lost."""
    rng = np.random.default_rng(33)
    H_q, H_kv, d, T = 4, 1, 128, 9000

    def tweak(cache, table):
        cache.k[:] = 0
        cache.k[table[0][0], 0, 0, :] = ref.encode(np.full(d, 128.0))
        cache.ks[:] = 2.0 ** -7
        cache.vs[:] = 2.0 ** -7
        cache.v[:] = ref.encode(np.full(d, 256.0))
        cache.v[table[0][0], 0, 0] = 0
    got, cache, inputs = _decode_case(lib, rng, H_q, H_kv, d, [T], 1, 0, 0, tweak=tweak, scale=0.0)
    q, k, v, table, _ = inputs
    q = torch.ones((1, 1, H_q, d), dtype=torch.bfloat16)
    # the first score is 128, the others 0: weights 1 and 2^-20 at this scale
    scale = 20 * np.log(2.0) / d
    got = lib.decode_gqa_fp8_block(q.to(DEV), *cache.device(), _ints([T]), _ints(table), scale)
    want = 2.0 * (T - 1) * 2.0 ** -20 / (1 + (T - 1) * 2.0 ** -20)
    # half a step of the output and of the weights, and the scale's own rounding to fp32
    err = np.abs(got.double().cpu().numpy() / want - 1)
    assert err.max() <= 2 * 2.0 ** -8 + 2.0 ** -18, err.max()


def test_decode_ignores_what_no_query_sees(lib):
    """NaN codes and NaN scales in rows behind the sequence, before the window
    and in blocks that nobody holds."""
    rng = np.random.default_rng(34)
    lens, window = [500, 70, 129], 100

    def tweak(cache, table):
        seen = np.zeros(cache.k.shape[:1] + (BLOCK_SIZE,), dtype=bool)
        for b, t in enumerate(lens):
            for p in range(max(t - window, 0), t):
                seen[table[b][p // BLOCK_SIZE], p % BLOCK_SIZE] = True
        for c in (cache.k, cache.v):
            c.transpose(0, 2, 1, 3)[~seen] = 127
        for s in (cache.ks, cache.vs):
            s[~seen.any(axis=1)] = np.nan
    for d in (64, 128, 256):
        got, cache, inputs = _decode_case(lib, rng, 8, 2, d, lens, 1, window, 0, tweak=tweak)
        cache.vs = np.nan_to_num(cache.vs)
        _check(got, cache, inputs, lens, window, 0, what=f"d {d}")


def test_decode_nan_stays_with_its_sequence_and_head(lib):
    rng = np.random.default_rng(35)

    def tweak(cache, table):
        cache.k[table[0][1], 1, 3, 5] = 127
    lens = [300, 301]
    got, cache, inputs = _decode_case(lib, rng, 8, 2, 128, lens, 1, 0, 0, tweak=tweak)
    assert got[0, 0, 4:].isnan().all()
    q, k, v, table, scale = inputs
    want, weighted = ref.decode(q.double().numpy(), np.nan_to_num(k), v, lens, table, scale)
    got = got.float().cpu().numpy()
    vs = float(cache.vs.max())
    ref.assert_decode(got[1], want[1], weighted[1], vs)
    ref.assert_decode(got[0, 0, :4], want[0, 0, :4], weighted[0, 0, :4], vs)


@pytest.mark.parametrize("sink,q_len", [(0, 1), (70, 1), (0, 4)])
def test_decode_ring_table(lib, sink, q_len):
    rng = np.random.default_rng(36)
    window, ring, lens = 150, 5, [1000, 149, 400]
    width = -(-sink // BLOCK_SIZE) + ring
    table, _ = _table(rng, [width] * 3, extra=0)
    case = (8, 2, 128, lens, q_len, window, sink)
    got, cache, inputs = _decode_case(lib, rng, *case, ring=ring, table=table)
    _check(got, cache, inputs, lens, window, sink, ring=ring)


@pytest.mark.parametrize("H_q,d,wide", [(8, 64, 0), (8, 256, 50), (64, 128, 50)])
def test_decode_global_set(lib, H_q, d, wide):
    rng = np.random.default_rng(37)
    lens, window = [900, 300, 640], 128
    gp = np.array([[0, 5, 200, 201], [299, -1, -1, -1], [64, 127, 639, -1]], dtype=np.int32)
    got, cache, inputs = _decode_case(lib, rng, H_q, 2, d, lens, 1, window, 0, global_pos=gp,
                                      wide=wide)
    _check(got, cache, inputs, lens, window, 0, global_pos=gp)


def test_decode_global_set_through_a_ring(lib):
    rng = np.random.default_rng(38)
    lens, window, ring = [900, 100], 128, 4
    gp = np.array([[3, 70, 300], [1, 2, 3]], dtype=np.int32)
    table, _ = _table(rng, [3 + ring] * 2, extra=0)
    got, cache, inputs = _decode_case(lib, rng, 8, 2, 128, lens, 1, window, 0, ring=ring,
                                      global_pos=gp, table=table)
    _check(got, cache, inputs, lens, window, 0, ring=ring, global_pos=gp)


def test_decode_strided_queries_and_given_output(lib):
    rng = np.random.default_rng(39)
    H_q, H_kv, d, lens = 8, 2, 64, [200, 91]
    _, cache, (q, k, v, table, scale) = _decode_case(lib, rng, H_q, H_kv, d, lens, 1, 0, 0)
    wide = torch.zeros((2, H_q + 3, d), dtype=torch.bfloat16, device=DEV)
    wide[:, :H_q] = q[:, 0].to(DEV)
    out = torch.empty((2, H_q, d), dtype=torch.bfloat16, device=DEV)
    got = lib.decode_gqa_fp8_block(wide[:, :H_q], *cache.device(), _ints(lens), _ints(table), scale,
                                   out=out)
    assert got is out
    _check(got[:, None], cache, (q, k, v, table, scale), lens, 0, 0)


def test_decode_extreme_queries(lib):
    """Rows of tiny and huge queries beside ordinary ones, a query of zeros, one
    with an infinity (its output is NaN, as softmax over infinities is)."""
    rng = np.random.default_rng(40)
    H_q, H_kv, d, lens = 8, 2, 128, [333]
    _, cache, (q, k, v, table, scale) = _decode_case(lib, rng, H_q, H_kv, d, lens, 1, 0, 0)
    q = q.float()
    q[0, 0, 0] *= 1e-30
    q[0, 0, 1] *= 8.0
    q[0, 0, 2] = 0
    q[0, 0, 3, 1:] *= 2.0 ** -12
    q[0, 0, 4, 7] = float("inf")
    q = q.bfloat16()
    got = lib.decode_gqa_fp8_block(q.to(DEV), *cache.device(), _ints(lens), _ints(table), scale)
    assert lib.last_error() == lib.OK
    assert got[0, 0, 4].isnan().all()
    rest = [0, 1, 2, 3, 5, 6, 7]
    want, weighted = ref.decode(q.double().nan_to_num(posinf=0.0).numpy(), k, v, lens, table, scale)
    # the scores of the row times 8 are 8 times as far off
    extra = np.ones((H_q, 1))
    extra[1] = 2.0
    ref.assert_decode(got[0, 0, rest].float(), want[0, 0, rest], (weighted[0, 0] * extra)[rest],
                      float(cache.vs.max()))


def test_decode_flags_bad_blocks_and_lengths(lib):
    rng = np.random.default_rng(41)
    _, cache, (q, k, v, table, scale) = _decode_case(lib, rng, 8, 2, 128, [200, 91], 1, 0, 0)
    bad = table.copy()
    bad[0, 1] = 1000
    got = lib.decode_gqa_fp8_block(q.to(DEV), *cache.device(), _ints([200, 91]), _ints(bad), scale)
    assert lib.last_error() == lib.ERR_BAD_BLOCK
    want, weighted = ref.decode(q.double().numpy(), k, v, [200, 91], table, scale)
    ref.assert_decode(got[1].float(), want[1], weighted[1], float(cache.vs.max()))
    for lens in ([-1, 91], [64 * table.shape[1] + 1, 91]):
        got = lib.decode_gqa_fp8_block(q.to(DEV), *cache.device(), _ints(lens), _ints(table), scale)
        assert lib.last_error() == lib.ERR_BAD_SEQLEN
        assert (got[0] == 0).all()
        ref.assert_decode(got[1].float(), want[1], weighted[1], float(cache.vs.max()))


# ------------------------------------------------------------------ together

def test_append_decode_read_steps_in_a_graph(lib):
    """A prompt appended, then steps of append and decode replayed from a graph,
    and from a second one with a workspace of its own; then the whole cache read
    back."""
    rng = np.random.default_rng(50)
    B, H_q, H_kv, d, steps = 3, 8, 2, 128, 5
    start = [100, 63, 1]
    table, total = _table(rng, [3, 2, 1])
    cache = _Cache(rng, total, H_kv, d)
    dev = cache.device()
    off = _offsets(start)
    k0, v0 = (_rows(rng, off[-1], H_kv, d, torch.bfloat16) for _ in range(2))
    lib.kv_append_fp8_block(k0.to(DEV), v0.to(DEV), *dev, _ints([0] * B), _ints(table),
                            offsets=_ints(off))
    for x, c, s in ((k0, cache.k, cache.ks), (v0, cache.v, cache.vs)):
        ref.append(x.double().numpy(), c, s, [0] * B, off, table)
    pos, lens = _ints(start), _ints([t + 1 for t in start])
    q = torch.zeros((B, H_q, d), dtype=torch.bfloat16, device=DEV)
    k, v = (torch.zeros((B, H_kv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tab, scale = _ints(table), 1 / np.sqrt(d)
    ws = [lib.fp8_block_workspace(q, dev[0]) for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    stream = torch.cuda.Stream()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0], stream=stream):
        lib.kv_append_fp8_block(k, v, *dev, pos, tab)
        lib.decode_gqa_fp8_block(q, *dev, lens, tab, scale, out=outs[0], workspace=ws[0])
        pos += 1
    with torch.cuda.graph(graphs[1], stream=stream):
        lib.decode_gqa_fp8_block(q, *dev, lens, tab, scale, out=outs[1], workspace=ws[1])
    for step in range(steps):
        qh, kh, vh = (torch.from_numpy(rng.standard_normal((B, h, d)) * m).bfloat16()
                      for h, m in ((H_q, 1.0), (H_kv, 2.0 ** step), (H_kv, 2.0 ** step)))
        q.copy_(qh)
        k.copy_(kh)
        v.copy_(vh)
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        at = [t + step for t in start]
        for x, c, s in ((kh, cache.k, cache.ks), (vh, cache.v, cache.vs)):
            ref.append(x.double().numpy(), c, s, at, list(range(B + 1)), table)
        cache.check(dev, f"step {step}")
        want, weighted = ref.decode(qh.double().numpy()[:, None], ref.dense(cache.k, cache.ks),
                                    ref.dense(cache.v, cache.vs), [t + 1 for t in at], table, scale)
        for out in outs:
            ref.assert_decode(out[:, None].float(), want, weighted, float(cache.vs.max()),
                              f"step {step}")
        lens += 1
    assert lib.last_error() == lib.OK
    n = [t + steps for t in start]
    got = lib.kv_read_fp8_block(*dev, _ints([0] * B), tab, sum(n), offsets=_ints(_offsets(n)),
                                dtype=torch.float32)
    for x, c, s in zip(got, (cache.k, cache.v), (cache.ks, cache.vs)):
        values, at = ref.dense(c, s), 0
        for b in range(B):
            for t in range(n[b]):
                want = values[table[b][t // BLOCK_SIZE], :, t % BLOCK_SIZE]
                assert np.array_equal(x[at].double().cpu().numpy(), want)
                at += 1


def test_calls_on_another_stream(lib):
    rng = np.random.default_rng(51)
    _, cache, (q, k, v, table, scale) = _decode_case(lib, rng, 8, 2, 128, [200, 91], 1, 0, 0)
    dev, qd, lens, tab = cache.device(), q.to(DEV), _ints([200, 91]), _ints(table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [lib.decode_gqa_fp8_block(qd, *dev, lens, tab, scale, stream=s) for s in streams]
    for s in streams:
        s.synchronize()
    assert torch.equal(got[0], got[1])
    _check(got[0], cache, (q, k, v, table, scale), [200, 91], 0, 0)


def test_decode_same_result_every_time(lib):
    rng = np.random.default_rng(52)
    got, cache, (q, k, v, table, scale) = _decode_case(lib, rng, 8, 2, 128, [5000, 91], 1, 0, 0)
    dev = cache.device()
    for _ in range(3):
        again = lib.decode_gqa_fp8_block(q.to(DEV), *dev, _ints([5000, 91]), _ints(table), scale)
        assert torch.equal(got, again)
