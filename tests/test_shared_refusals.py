"""Refusals of the shared decode, its plan and the read-back, before any launch (no GPU)."""
import ctypes

import pytest
import torch

import gqa_decode_attention_kv_gb300 as gq
from gqa_decode_attention_kv_gb300 import build as gbuild

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gq.load()


def _desc(**kw):
    base = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, num_blocks=64, num_kv_heads=8, block_size=16,
                head_dim=128, dtype=2, stride_block=8 * 16 * 128, stride_head=16 * 128, stride_token=128)
    base.update(kw)
    return gq.KVCacheDesc(**base)


CODED = dict(k_scale=0x30000, v_scale=0x40000)


@pytest.mark.parametrize("cache,kw,expect", [
    (dict(), dict(B=0), OK),
    (dict(), dict(B=-1), INVALID), (dict(), dict(H=0), INVALID), (dict(), dict(H=12), INVALID),
    (dict(), dict(maxb=0), INVALID), (dict(), dict(maxb=2 ** 27), INVALID), (dict(), dict(T=-1), INVALID),
    (dict(), dict(T=17), UNSUPPORTED), (dict(), dict(H=8 * 65), UNSUPPORTED), (dict(), dict(B=8192), UNSUPPORTED),
    (dict(), dict(B=4000, maxb=2 ** 17), UNSUPPORTED), (dict(), dict(max_group=-1), INVALID),
    (dict(), dict(scale=float("nan")), INVALID), (dict(), dict(scale=float("inf")), INVALID),
    (dict(), dict(q=None), INVALID), (dict(), dict(q=0x30004), INVALID), (dict(), dict(table=None), INVALID),
    (dict(), dict(lens=None), INVALID), (dict(), dict(groups=None), INVALID), (dict(), dict(groups=0x80004), INVALID),
    (dict(), dict(out=None), INVALID), (dict(), dict(out=0x60008), INVALID), (dict(), dict(out_dtype=3), UNSUPPORTED),
    (dict(), dict(q_dtype=1), UNSUPPORTED), (dict(), dict(q_dtype=0), UNSUPPORTED), (dict(), dict(ws=0x70010), INVALID),
    (dict(dtype=0), dict(q_dtype=0), UNSUPPORTED),                                  # fp32 caches
    (dict(dtype=6, **CODED), dict(), UNSUPPORTED),                                  # K scaled by channel
    (dict(dtype=3), dict(), INVALID), (dict(dtype=3, **CODED), dict(q_dtype=0), UNSUPPORTED),
    (dict(head_dim=96), dict(), UNSUPPORTED), (dict(block_size=32), dict(), UNSUPPORTED), (dict(k=None), dict(), INVALID),
    (dict(stride_token=64), dict(), INVALID),
])
def test_decode_refusals(lib, cache, kw, expect):
    a = dict(q=0x30000, q_dtype=2, H=32, table=0x40000, maxb=8, lens=0x50000, B=4, T=1, scale=0.1, groups=0x80000,
             max_group=0, out=0x60000, out_dtype=0, ws=0x70000, wsb=1 << 30)
    a.update(kw)
    d = _desc(**cache)
    assert lib.gqa_decode_shared(ctypes.byref(d), a["q"], a["q_dtype"], a["H"], a["table"], a["maxb"], a["lens"], a["B"],
                                 a["T"], a["scale"], a["groups"], a["max_group"], a["out"], a["out_dtype"], a["ws"],
                                 a["wsb"], None, None) == expect


def test_plan_sizes(lib):
    f = lib.gqa_kv_pages_groups_size
    assert f(-1) == f(8193) == 0
    for B in (0, 1, 7, 8192):
        assert f(B) >= 4 * (3 + 5 * B) and f(B) % 16 == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0, table=None, lens=None, plan=None), OK), (dict(B=-1), INVALID), (dict(B=8193), UNSUPPORTED),
    (dict(maxb=0), INVALID), (dict(maxb=2 ** 27), INVALID), (dict(min_blocks=-1), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(plan=None), INVALID), (dict(plan=0x30004), INVALID), (dict(bytes=100), WORKSPACE),
])
def test_plan_refusals(lib, kw, expect):
    a = dict(table=0x10000, maxb=8, lens=0x20000, B=16, min_blocks=1, plan=0x30000, bytes=1 << 20)
    a.update(kw)
    assert lib.gqa_kv_pages_groups(a["table"], a["maxb"], a["lens"], a["B"], a["min_blocks"], a["plan"], a["bytes"], None,
                                   None) == expect


@pytest.mark.parametrize("cache,kw,expect", [
    (dict(), dict(B=0), OK), (dict(), dict(most=0), OK), (dict(), dict(total=0), OK),
    (dict(), dict(B=-1), INVALID), (dict(), dict(most=-1), INVALID), (dict(), dict(total=-1), INVALID),
    (dict(), dict(maxb=0), INVALID), (dict(), dict(maxb=2 ** 27), INVALID), (dict(), dict(out_dtype=3), UNSUPPORTED),
    (dict(), dict(start=None, total=127), INVALID), (dict(), dict(k=None), INVALID), (dict(), dict(v=None), INVALID),
    (dict(), dict(k=0x50008), INVALID), (dict(), dict(table=None), INVALID), (dict(), dict(pos=None), INVALID),
    (dict(), dict(most=2 ** 30, B=64), UNSUPPORTED), (dict(dtype=5), dict(), INVALID), (dict(dtype=9), dict(), INVALID),
])
def test_read_refusals(lib, cache, kw, expect):
    a = dict(k=0x50000, v=0x60000, out_dtype=0, total=128, start=0x70000, most=32, table=0x80000, maxb=8, pos=0x90000, B=4)
    a.update(kw)
    d = _desc(**cache)
    assert lib.gqa_kv_read(ctypes.byref(d), a["k"], a["v"], a["out_dtype"], a["total"], a["start"], a["most"], a["table"],
                           a["maxb"], a["pos"], a["B"], None, None) == expect


class _OnCuda(torch.Tensor):
    """A CPU tensor that says it is on the GPU: the checks before the device's alone run."""
    is_cuda = True


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32).as_subclass(_OnCuda)


def _cache():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    return gq.PagedKVCache(k, k.clone(), 4, 2, 64, 2 * 16 * 64, 16 * 64, 64)


def test_binding_checks_the_plan():
    plan = gq.PrefixGroups(_i32(gq._groups_size_of(3) // 4), 3)
    assert plan.count.shape == (2,) and plan.start.shape == (4,)
    assert all(getattr(plan, n).shape == (3,) for n in ("blocks", "rows", "slot", "group"))
    with pytest.raises(AttributeError):
        plan.parents
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16).as_subclass(_OnCuda)
    with pytest.raises(ValueError, match="3 rows, q holds 4"):
        gq.gqa_decode_shared(_cache(), q, _i32(4, 9), _i32(4), 0.1, plan)
    with pytest.raises(ValueError, match="groups"):
        gq.gqa_decode_shared(_cache(), q, _i32(4, 9), _i32(4), 0.1, gq.PrefixGroups(_i32(20), 4))
    with pytest.raises(ValueError, match="context_lens"):
        gq.gqa_decode_shared(_cache(), q, _i32(4, 9), _i32(3), 0.1, plan)
    with pytest.raises(ValueError, match="head_dim"):
        gq.gqa_decode_shared(_cache(), q[..., :32].contiguous(), _i32(4, 9), _i32(4), 0.1, plan)
    with pytest.raises(ValueError, match="CUDA"):
        gq.kv_pages_groups(torch.zeros(4, 9, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="at most 4 rows"):
        gq.kv_pages_groups(_i32(4, 9), _i32(5))
    with pytest.raises(ValueError, match="max_blocks"):
        gq.kv_pages_groups(_i32(4), _i32(4))


def test_binding_checks_the_rows_read():
    c, table, pos, start = _cache(), _i32(2, 9), _i32(2), _i32(3)
    rows = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d).as_subclass(_OnCuda)  # noqa: E731
    with pytest.raises(ValueError, match="total_tokens is required"):
        gq.kv_read(c, table, pos, token_start=start, max_tokens=4)
    with pytest.raises(ValueError, match="B \\* max_tokens = 8"):
        gq.kv_read(c, table, pos, max_tokens=4, total_tokens=9)
    with pytest.raises(ValueError, match="must not be negative"):
        gq.kv_read(c, table, pos, max_tokens=-4)
    with pytest.raises(ValueError, match="token_start"):
        gq.kv_read(c, table, pos, token_start=_i32(2), max_tokens=4, total_tokens=8)
    with pytest.raises(ValueError, match="k_out"):
        gq.kv_read(c, table, pos, max_tokens=4, k_out=rows(2, 4, 2, 32))
    with pytest.raises(ValueError, match="v_out"):
        gq.kv_read(c, table, pos, max_tokens=4, k_out=rows(2, 4, 2, 64), v_out=rows(2, 4, 2, 64, d=torch.float32))
    with pytest.raises(ValueError, match="not torch.int8"):
        gq.kv_read(c, table, pos, max_tokens=4, dtype=torch.int8)
    with pytest.raises(ValueError, match="overlaps"):
        x = rows(2, 4, 2, 64)
        gq.kv_read(c, table, pos, max_tokens=4, k_out=x, v_out=x)
    with pytest.raises(ValueError, match="positions"):
        gq.kv_read(c, table, _i32(2, 1), max_tokens=4)
