"""Refusals of the window-with-sinks calls, before any launch (no GPU)."""
import ctypes

import pytest

import gqa_decode_attention_kv_gb300 as gq
from gqa_decode_attention_kv_gb300 import build as gbuild

OK, INVALID = 0, 1


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gq.load()


def _desc():
    return gq.KVCacheDesc(k=0x10000, v=0x20000, k_scale=None, v_scale=None, num_blocks=64, num_kv_heads=8,
                          block_size=16, head_dim=128, dtype=2, stride_block=8 * 16 * 128, stride_head=16 * 128,
                          stride_token=128)


@pytest.mark.parametrize("sinks,batch,expect", [(-1, 4, INVALID), (-1, 0, INVALID), (4, 0, OK), (0, 0, OK)])
def test_negative_sinks_are_refused(lib, sinks, batch, expect):
    d = _desc()
    opts = gq.DecodeOpts(1, 32, 0, 0, 0, 0, None, None)
    assert lib.gqa_decode_sinks(ctypes.byref(d), 0x30000, 2, 32, 0x40000, 8, 0x50000, batch, 0.1, 0x60000, 0, 0x70000,
                                1 << 20, ctypes.byref(opts), sinks, None, None) == expect
    assert lib.gqa_prefill_sinks(ctypes.byref(d), 0x30000, 2, 32, 0x40000, 16, 0x50000, 8, 0x60000, batch, 0.1, 32,
                                 sinks, 0, 0x70000, 0, 0, None, None) == expect


def test_the_calls_keep_the_checks_of_the_plain_ones(lib):
    d = _desc()
    opts = gq.DecodeOpts(1, -3, 0, 0, 0, 0, None, None)
    assert lib.gqa_decode_sinks(ctypes.byref(d), 0x30000, 2, 32, 0x40000, 8, 0x50000, 4, 0.1, 0x60000, 0, 0x70000,
                                1 << 20, ctypes.byref(opts), 4, None, None) == INVALID
    assert lib.gqa_prefill_sinks(ctypes.byref(d), 0x30000, 2, 32, 0x40000, 16, 0x50000, 8, 0x60000, 4, 0.1, -1, 4,
                                 0, 0x70000, 0, 0, None, None) == INVALID
    assert lib.gqa_prefill_sinks(ctypes.byref(d), 0x30000, 2, 32, 0x40000, 16, 0x50000, 8, 0x60000, 4, 0.1, 32, 4,
                                 -1, 0x70000, 0, 0, None, None) == INVALID
