"""The testing and timing hooks on the block-scaled fp8 decode."""
import ctypes

import numpy as np
import pytest
import torch

from tests.test_fp8_block_gpu import _check, _decode_case, _ints

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("ctas,wide", [(0, 0), (0, 100), (3, 100)],
                         ids=["whole", "all_sms", "3_ctas"])
@pytest.mark.parametrize("group,d", [(4, 64), (12, 128), (32, 256)])
def test_forced_timeout_returns_status_and_context_survives(lib, group, d, ctas, wide):
    """A wait that nothing ends gives up after 5 ms and says so, once; the next
    call is right."""
    rng = np.random.default_rng(95)
    lens = [700, 0, 65]
    case = (2 * group, 2, d, lens, 1, 0, 0)
    _, cache, (q, _, _, table, scale) = _decode_case(lib, rng, *case, wide=wide)
    args = (q.to(DEV), *cache.device(), _ints(lens), _ints(table), scale)
    lib.set_num_ctas(ctas)
    try:
        lib.debug_force_timeout(True, 5_000_000)
        got = lib.decode_gqa_fp8_block(*args)
        assert lib.last_error() == lib.ERR_TIMEOUT
        assert (got[1] == 0).all()                    # no key, no wait
        again = lib.decode_gqa_fp8_block(*args)
        assert lib.last_error() == lib.OK
    finally:
        lib.debug_force_timeout(False)
        lib.set_num_ctas(0)
    want, cache, inputs = _decode_case(lib, np.random.default_rng(95), *case, wide=wide, ctas=ctas)
    assert torch.equal(again, want)
    _check(again, cache, inputs, lens, 0, 0)


@pytest.mark.parametrize("wide", [0, 100], ids=["whole", "split"])
def test_profile_events_are_recorded_around_the_kernel(lib, wide):
    rng = np.random.default_rng(96)
    lens = [3000, 65]
    _, cache, (q, _, _, table, scale) = _decode_case(lib, rng, 8, 2, 128, lens, 1, 0, 0, wide=wide)
    args = (q.to(DEV), *cache.device(), _ints(lens), _ints(table), scale)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    for e in events:                                  # torch makes them when first recorded
        e.record()
    torch.cuda.synchronize()
    first = [e.cuda_event for e in events]
    start, stop = ((ctypes.c_void_p * 2)(*first[i::2]) for i in range(2))
    c = lib.load()
    assert c.attn_set_profile_events(start, stop, 2) == lib.OK
    try:
        for _ in range(2):
            lib.decode_gqa_fp8_block(*args)
            torch.cuda._sleep(2_000_000)              # about a millisecond, not part of it
        torch.cuda.synchronize()
    finally:
        assert c.attn_set_profile_events(None, None, 0) == lib.OK
    between = events[1].elapsed_time(events[2])
    assert between > 0.3
    for i in range(2):
        assert 0 < events[2 * i].elapsed_time(events[2 * i + 1]) < 0.3
