"""A kept prefix of any length: the largest does not wrap around (CPU: the call
is refused before anything is launched)."""
import pytest

import decode_attention_kv_paged_b200 as attn
from tests.test_fp8_block_host import _append, _decode, _read

LARGEST = 2 ** 31 - 1


@pytest.mark.parametrize("sink", [LARGEST, LARGEST - 62])
@pytest.mark.parametrize("call", [_append, _read, _decode])
def test_a_prefix_longer_than_the_table_leaves_no_room_for_a_ring(call, sink):
    vis = attn.Visibility(100, sink, 4, None, 0)
    over = dict(vis=vis, max_blocks=8, num_blocks=8)
    assert call(**over) == attn.ERR_ARG
