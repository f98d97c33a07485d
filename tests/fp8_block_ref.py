"""The block-scaled fp8 cache in fp64 on the host, from its definition, for the
tests: code values come from the oracle's E4M3 table, codes by looking up the
nearest value (ties to the even code), attention from the oracle."""
import math

import numpy as np
import torch

import oracle as orc
from workloads import BLOCK_SIZE

_VALUES = orc.e4m3_table()
_MAGNITUDES = _VALUES[:127]                          # 0 .. 448, ascending


def encode(x):
    """Nearest E4M3 codes of fp64 values, saturated; NaN stays NaN."""
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)), 448.0)
    hi = np.clip(np.searchsorted(_MAGNITUDES, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _MAGNITUDES[hi] - a, a - _MAGNITUDES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_for(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s; 0 for 0."""
    if amax == 0:
        return 0.0
    m, e = math.frexp(amax / 448.0)                  # in [0.5, 1) * 2^e
    return max(math.ldexp(1.0, e - 1 if m == 0.5 else e), 2.0 ** -126)


def slot_of(blk, sink, ring):
    a = -(-sink // BLOCK_SIZE)
    return blk if ring <= 0 or blk < a else a + blk % ring


def append(new, codes, scale, positions, offsets, table, sink=0, ring=0):
    """Host cache (codes uint8, scale fp32; changed in place) after an append
    of rows new [tokens][H][d] (fp64)."""
    for b, pos in enumerate(positions):
        o0, n = offsets[b], offsets[b + 1] - offsets[b]
        if n == 0:
            continue
        last = (pos + n - 1) // BLOCK_SIZE
        for blk in range(pos // BLOCK_SIZE, last + 1):
            a = -(-sink // BLOCK_SIZE)
            if ring > 0 and blk >= a and blk + ring <= last:
                continue                             # a later block takes its slot
            phys = table[b][slot_of(blk, sink, ring)]
            r0 = max(pos - blk * BLOCK_SIZE, 0)
            r1 = min(pos + n - blk * BLOCK_SIZE, BLOCK_SIZE)
            rows = new[o0 + blk * BLOCK_SIZE + r0 - pos:o0 + blk * BLOCK_SIZE + r1 - pos]
            for h in range(codes.shape[1]):
                x = rows[:, h]
                fin = np.abs(x[np.isfinite(x)])
                need = scale_for(fin.max() if fin.size else 0.0)
                old = float(scale[phys, h]) if r0 > 0 else 0.0
                s = max(old, need)
                if r0 > 0 and s != old:
                    codes[phys, h, :r0] = encode(_VALUES[codes[phys, h, :r0]] * (old / s))
                codes[phys, h, r0:r1] = encode(x / s if s > 0 else x)
                scale[phys, h] = s


def dense(codes, scale):
    """fp64 cache values [blocks][H][64][d]; a scale of 0 makes 0 of any number."""
    return _VALUES[codes] * scale.astype(np.float64)[:, :, None, None]


def decode(q, k, v, lens, table, scale, window=0, sink=0, ring=0, global_pos=None):
    """(out, weighted |v|) in fp64 for q [B][L][H_q][d]: the second is the sum of
    weights times |v|, what relative errors of the weights are measured in."""
    L = q.shape[1]
    outs = []
    for values in (v, np.abs(v)):
        o = np.zeros(q.shape)
        for i in range(L):
            at = np.asarray([max(t - L + i + 1, 0) for t in lens], dtype=np.int32)
            o[:, i] = orc.decode_gqa_vis(np.ascontiguousarray(q[:, i]), k, values, at, table,
                                         scale, window=window, sink=sink, ring=ring,
                                         global_pos=global_pos)
        outs.append(o)
    return outs


def assert_decode(got, ref, weighted, v_scale_max, what=""):
    """The output is bf16 (half a step, 2^-8 of the value).  Each weight may be
    held as the sum of two E4M3 numbers, the second the remainder of the first:
    2^-4 of 2^-4, or 2^-8 of the weight, and where the second is subnormal 2^-22
    of the 128-key tile's largest weighted scale; the sum of that over a tile is
    2^-15 of 448 scales at most.  Score and sum rounding in fp32 stays under a
    quarter of 2^-8."""
    got = torch.as_tensor(got).double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(ref) + 1.25 * 2.0 ** -8 * weighted + 2.0 ** -15 * 448 * v_scale_max
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, worst "
                           f"{np.abs(got - ref)[bad][:4]} against {bound[bad][:4]}")
