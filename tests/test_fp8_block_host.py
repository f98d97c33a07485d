"""CPU-only checks of the block-scaled fp8 cache: the test definition against
the oracle, and the refusals of its entry points (no kernel is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import decode_attention_kv_paged_b200 as attn
import oracle as orc
from tests import fp8_block_ref as ref

P, N = ctypes.c_void_p(256), ctypes.c_void_p(0)     # never dereferenced: refused first


def test_definition_encodes_as_the_oracle_does():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(2000) * np.exp2(rng.integers(-12, 10, 2000)),
                        orc.e4m3_table()[:127], [0.0, -0.0, 1e9, -1e9, 17.0, 19.0, 2.0 ** -10]])
    x = x.astype(np.float32).astype(np.float64)
    assert [orc.e4m3_encode(v) for v in x] == ref.encode(x).tolist()
    t = orc.e4m3_table()
    good = ~np.isnan(t)
    assert np.array_equal(t[ref.encode(t[good])], t[good])


def test_definition_of_the_scale():
    assert ref.scale_for(0.0) == 0.0
    assert ref.scale_for(448.0) == 1.0
    assert ref.scale_for(np.nextafter(np.float32(448), np.float32(500))) == 2.0
    assert ref.scale_for(1e-45) == 2.0 ** -126
    for a in np.exp2(np.random.default_rng(2).uniform(-100, 100, 500)):
        s = ref.scale_for(a)
        assert a <= 448 * s and a > 224 * s


def _append(**over):
    a = dict(k_new=P, v_new=P, k_stride=2 * 128, v_stride=2 * 128, k_cache=P, v_cache=P, k_scale=P,
             v_scale=P, positions=P, offsets=P, block_table=P, B=1, n_tokens=0, H_kv=2, d=128,
             max_blocks=1, num_blocks=1, dtype=attn.BF16, vis=None, stream=N)
    a.update(over)
    return attn.load().kv_append_fp8_block(*a.values())


@pytest.mark.parametrize("over", [
    dict(k_new=N), dict(v_cache=N), dict(k_scale=N), dict(positions=N), dict(block_table=N),
    dict(k_new=ctypes.c_void_p(264)), dict(k_cache=ctypes.c_void_p(264)),
    dict(v_scale=ctypes.c_void_p(258)), dict(offsets=ctypes.c_void_p(258)), dict(B=0),
    dict(n_tokens=-1), dict(H_kv=0), dict(max_blocks=0), dict(num_blocks=0),
    dict(k_stride=2 * 128 - 8), dict(v_stride=2 * 128 + 4), dict(dtype=attn.FP8_E4M3),
    dict(offsets=N, n_tokens=2), dict(vis=attn.Visibility(0, 0, 4, None, 0))])
def test_append_refusals(over):
    assert _append(**over) == attn.ERR_ARG


@pytest.mark.parametrize("over", [dict(d=32, k_stride=64, v_stride=64), dict(H_kv=70000)])
def test_append_unsupported(over):
    assert _append(**over) == attn.ERR_UNSUPPORTED


def test_append_of_nothing_launches_nothing():
    assert _append() == attn.OK


def _read(**over):
    a = dict(k_cache=P, v_cache=P, k_scale=P, v_scale=P, positions=P, offsets=P, block_table=P,
             k_out=P, v_out=P, B=1, n_tokens=0, H_kv=2, d=128, max_blocks=1, num_blocks=1,
             dtype=attn.F32, zero_rest=0, vis=None, stream=N)
    a.update(over)
    return attn.load().kv_read_fp8_block(*a.values())


@pytest.mark.parametrize("over", [
    dict(k_cache=N), dict(v_out=N), dict(v_scale=N), dict(k_out=ctypes.c_void_p(264)),
    dict(positions=ctypes.c_void_p(257)), dict(B=-1), dict(n_tokens=-1), dict(dtype=7),
    dict(offsets=N, n_tokens=3)])
def test_read_refusals(over):
    assert _read(**over) == attn.ERR_ARG


def test_read_unsupported_and_empty():
    assert _read(d=96) == attn.ERR_UNSUPPORTED
    assert _read() == attn.OK


def _decode(**over):
    a = dict(q=P, q_stride=8 * 128, k_cache=P, v_cache=P, k_scale=P, v_scale=P, seq_lens=P,
             block_table=P, out=P, B=1, q_len=1, H_q=8, H_kv=2, d=128, scale=1.0, vis=None,
             workspace=P, workspace_bytes=0, stream=N, max_blocks=4, num_blocks=4)
    a.update(over)
    return attn.load().attn_decode_gqa_fp8_block(*a.values())


@pytest.mark.parametrize("over", [
    dict(q=N), dict(out=N), dict(workspace=N), dict(seq_lens=N), dict(k_scale=N),
    dict(q=ctypes.c_void_p(264)), dict(workspace=ctypes.c_void_p(16)),
    dict(seq_lens=ctypes.c_void_p(258)), dict(B=0), dict(q_len=0), dict(H_q=9), dict(H_kv=0),
    dict(q_stride=8 * 128 - 8), dict(q_stride=8 * 128 + 4), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(max_blocks=0), dict(num_blocks=0), dict(max_blocks=1 << 25),
    # a ring that a window of 100 and the second query's reach do not fit
    dict(vis=attn.Visibility(100, 0, 2, None, 0)),
    dict(q_len=40, vis=attn.Visibility(100, 0, 3, None, 0))])
def test_decode_refusals(over):
    assert _decode(**over) == attn.ERR_ARG


@pytest.mark.parametrize("over", [
    dict(d=96), dict(d=32), dict(B=1 << 28, q_len=16), dict(num_blocks=1 << 30),
    dict(q_len=2, vis=attn.Visibility(64, 0, 0, 256, 1))])
def test_decode_unsupported(over):
    assert _decode(**over) == attn.ERR_UNSUPPORTED


def test_python_refusals():
    cpu = torch.zeros((1, 2, 64, 64), dtype=torch.uint8)
    s = torch.zeros((1, 2))
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        attn.kv_append_fp8_block(x, x, cpu, cpu, s, s, i, i[None])
    with pytest.raises(ValueError):
        attn.kv_read_fp8_block(cpu, cpu, s, s, i, i[None], 1)
    with pytest.raises(ValueError):
        attn.decode_gqa_fp8_block(x, cpu, cpu, s, s, i, i[None], 1.0)
