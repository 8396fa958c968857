"""Refusals of the page calls, before any launch (no GPU)."""
import ctypes

import pytest
import torch

import gqa_decode_attention_kv_gb300 as gq
from gqa_decode_attention_kv_gb300 import build as gbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
R, T, L, WS = 0x10000, 0x20000, 0x30000, 0x40000


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gq.load()


def test_workspace_sizes(lib):
    f = lib.gqa_kv_pages_workspace_size
    assert f(0, 4) == f(-1, 4) == f(100, -1) == f(2 ** 31, 4) == f(100, 2 ** 21) == 0
    assert f(100, 4) >= 4 * (100 + 5) and f(10 ** 6, 0) >= 4 * (10 ** 6 + 977)


@pytest.mark.parametrize("kw,expect", [
    (dict(refs=None), INVALID), (dict(refs=R + 4), INVALID), (dict(nb=0), INVALID), (dict(nb=2 ** 31), UNSUPPORTED),
    (dict(table=None), INVALID), (dict(maxb=0), INVALID), (dict(B=-1), INVALID), (dict(B=2 ** 20 + 1), UNSUPPORTED),
    (dict(lens=None), INVALID), (dict(n=-1), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE),
    (dict(ws=WS + 8), INVALID), (dict(B=0, table=None, lens=None, ws=None), OK), (dict(n=0, ws=None), OK),
    (dict(maxb=2 ** 27), INVALID),
])
def test_reserve_refusals(lib, kw, expect):
    a = dict(refs=R, nb=100, table=T, maxb=8, lens=L, B=4, n=1, ws=WS, wsb=1 << 20)
    a.update(kw)
    assert lib.gqa_kv_pages_reserve(a["refs"], a["nb"], a["table"], a["maxb"], a["lens"], None, a["n"], a["B"], a["ws"],
                                    a["wsb"], None, None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), INVALID), (dict(rows=8193), UNSUPPORTED), (dict(n=8193), UNSUPPORTED), (dict(src=None), INVALID),
    (dict(dst=None), INVALID), (dict(pairs=None), INVALID), (dict(count=None), INVALID), (dict(rp=None), INVALID),
    (dict(lens=None), INVALID), (dict(rows=0, table=None), INVALID), (dict(wsb=100), WORKSPACE), (dict(refs=None), INVALID),
])
def test_fork_refusals(lib, kw, expect):
    a = dict(refs=R, nb=100, table=T, rows=4, maxb=8, lens=L, src=0x50000, dst=0x60000, n=2, pairs=0x70000,
             count=0x80000, rp=0x90000, ws=WS, wsb=1 << 20)
    a.update(kw)
    assert lib.gqa_kv_pages_fork(a["refs"], a["nb"], a["table"], a["rows"], a["maxb"], a["lens"], a["src"], a["dst"],
                                 a["n"], a["pairs"], a["count"], a["rp"], a["ws"], a["wsb"], None, None) == expect


def test_free_trim_and_compact_refusals(lib):
    free, trim, compact = lib.gqa_kv_pages_free, lib.gqa_kv_pages_trim, lib.gqa_kv_pages_compact
    assert free(R, 100, T, 4, 8, L, None, 2, None, None) == INVALID
    assert free(R, 100, T, 4, 8, None, 0x50000, 2, None, None) == INVALID
    assert free(R, 100, T, 4, 8, L, 0x50000, -2, None, None) == INVALID
    assert free(R, 100, T, 4, 8, L, None, 0, None, None) == OK
    assert trim(R, 100, T, 8, L, 4, 0, 0, None, None) == INVALID        # no window: nothing ever leaves it
    assert trim(R, 100, T, 8, L, 4, 16, -1, None, None) == INVALID
    assert trim(R, 100, T, 8, None, 4, 16, 0, None, None) == INVALID
    assert trim(R, 100, None, 8, None, 0, 16, 0, None, None) == OK
    assert compact(R, 100, T, 4, 8, None, 3, 0x60000, WS, 1 << 20, None, None) == INVALID
    assert compact(R, 100, T, 4, 8, 0x50000, -1, 0x60000, WS, 1 << 20, None, None) == INVALID
    assert compact(R, 100, T, 4, 8, 0x50000, 3, None, WS, 1 << 20, None, None) == INVALID
    assert compact(R, 100, T, 4, 8, 0x50000, 3, 0x60000, WS, 128, None, None) == WORKSPACE


def _cache(**kw):
    base = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, num_blocks=64, num_kv_heads=8, block_size=16,
                head_dim=128, dtype=2, stride_block=8 * 16 * 128, stride_head=16 * 128, stride_token=128)
    base.update(kw)
    return gq.KVCacheDesc(**base)


@pytest.mark.parametrize("second,expect", [
    (dict(num_blocks=63), INVALID), (dict(dtype=1), INVALID), (dict(stride_block=8 * 16 * 128 + 128), INVALID),
    (dict(num_kv_heads=4), INVALID), (dict(k=None), INVALID), (dict(head_dim=96), UNSUPPORTED),
])
def test_copy_refuses_caches_that_differ(lib, second, expect):
    pair = (gq.KVCacheDesc * 2)(_cache(), _cache(**second))
    assert lib.gqa_kv_copy_pages(pair, 2, 0x50000, 0x60000, 4, None, 0, None, None) == expect


def test_copy_refusals(lib):
    c = _cache()
    f = lib.gqa_kv_copy_pages
    assert f(ctypes.byref(c), -1, 0x50000, 0x60000, 4, None, 0, None, None) == INVALID
    assert f(ctypes.byref(c), 1, None, 0x60000, 4, None, 0, None, None) == INVALID
    assert f(ctypes.byref(c), 1, 0x50000, None, 4, None, 0, None, None) == INVALID
    assert f(ctypes.byref(c), 1, 0x50000, 0x60000, -4, None, 0, None, None) == INVALID
    assert f(None, 0, None, None, 0, None, 0, None, None) == OK
    assert f(ctypes.byref(c), 1, None, None, 0, 0x70000, 3, None, None) == OK     # no KIVI cache: no rows to copy
    kc = _cache(dtype=6, k_scale=0x100, v_scale=0x200, residual_rows=4)
    assert f(ctypes.byref(kc), 1, 0x50000, 0x60000, 4, 0x70000, 3, None, None) == INVALID   # no residual


def test_binding_checks_the_pool():
    i32 = torch.int32
    refs, table, lens = torch.zeros(8, dtype=i32), torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        gq.kv_pages_free(refs, table, lens, lens)
    with pytest.raises(ValueError, match="int32"):
        gq.kv_pages_trim(refs.long(), table, lens, 8)
    with pytest.raises(ValueError, match="1-D"):
        gq._row_list(_OnGpu(table), "rows")


class _OnGpu:
    """A CPU tensor that says it is on the GPU: the shape checks alone run."""
    def __init__(self, t):
        self.t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)
