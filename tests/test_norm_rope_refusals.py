"""Refusals of the norm-and-rotation calls, before any launch (no GPU)."""
import ctypes

import pytest
import torch

import gqa_decode_attention_kv_gb300 as gq
from gqa_decode_attention_kv_gb300 import build as gbuild

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return gq.load()


def _cache(**kw):
    base = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, num_blocks=64, num_kv_heads=8, block_size=16,
                head_dim=128, dtype=2, stride_block=8 * 16 * 128, stride_head=16 * 128, stride_token=128)
    base.update(kw)
    return gq.KVCacheDesc(**base)


def _desc(**kw):
    base = dict(q_weight=0x1000, k_weight=0x2000, rope=0x3000, weight_dtype=2, eps=1e-6, rope_rows=100, rotary_dim=128,
                interleaved=0)
    base.update(kw)
    return gq.NormRopeDesc(**base)


def _append(lib, cache=None, desc=None, q=0x30000, qs=32 * 128, qo=0x40000, H=32, k=0x50000, ks=8 * 128, v=0x60000,
            vs=8 * 128, dtype=2, tokens=4, start=None, T=1, table=0x70000, maxb=8, pos=0x80000, B=4):
    c, d = cache or _cache(), desc or _desc()
    return lib.gqa_qk_norm_rope_append(ctypes.byref(c), ctypes.byref(d), q, qs, qo, H, k, ks, v, vs, dtype, tokens,
                                       start, T, table, maxb, pos, None, B, None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(q=0x30004), INVALID), (dict(qo=None), INVALID), (dict(qo=0x40008), INVALID),
    (dict(qs=31 * 128), INVALID),                    # tokens would overlap
    (dict(ks=8 * 128 + 4), INVALID),                 # 8 bytes: not a multiple of 16
    (dict(v=None), INVALID), (dict(dtype=1), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(tokens=5), INVALID),                       # not batch * T
    (dict(tokens=-1), INVALID), (dict(H=0), INVALID), (dict(table=None), INVALID), (dict(pos=None), INVALID),
    (dict(maxb=0), INVALID), (dict(T=-1), INVALID), (dict(tokens=0, B=0), OK),
    (dict(cache=_cache(dtype=6, k_scale=0x100, v_scale=0x200)), UNSUPPORTED),   # KIVI-style cache
    (dict(cache=_cache(head_dim=96)), UNSUPPORTED),
    (dict(desc=_desc(rotary_dim=24)), UNSUPPORTED), (dict(desc=_desc(rotary_dim=144)), INVALID),
    (dict(desc=_desc(rotary_dim=0)), INVALID), (dict(desc=_desc(rope_rows=0)), INVALID),
    (dict(desc=_desc(rope=0x3004)), INVALID), (dict(desc=_desc(interleaved=2)), INVALID),
    (dict(desc=_desc(eps=-1.0)), INVALID), (dict(desc=_desc(eps=float("nan"))), INVALID),
    (dict(desc=_desc(weight_dtype=3)), UNSUPPORTED), (dict(desc=_desc(q_weight=0x1004)), INVALID),
])
def test_append_refusals(lib, kw, expect):
    assert _append(lib, **kw) == expect


def _dense(lib, desc=None, q=0x30000, qs=32 * 128, qo=0x40000, k=0x50000, ks=8 * 128, ko=0x60000, d=128, dtype=2,
           tokens=4, pos=0x70000):
    r = desc or _desc()
    return lib.gqa_qk_norm_rope(ctypes.byref(r), q, qs, qo, 32, k, ks, ko, 8, d, dtype, tokens, pos, None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(d=80), UNSUPPORTED), (dict(pos=None), INVALID), (dict(ko=None), INVALID), (dict(k=0x50002), INVALID),
    (dict(dtype=4), UNSUPPORTED), (dict(tokens=0, q=None, k=None, qo=None, ko=None, pos=None), OK),
    (dict(ks=100), INVALID),
])
def test_dense_refusals(lib, kw, expect):
    assert _dense(lib, **kw) == expect


def test_table_refusals(lib):
    f = lib.gqa_rope_table
    assert f(0x1000, 10, 63, 1e4, None) == INVALID
    assert f(0x1000, 10, 0, 1e4, None) == INVALID
    assert f(0x1000, -1, 64, 1e4, None) == INVALID
    assert f(0x1000, 10, 64, 0.0, None) == INVALID
    assert f(0x1000, 10, 64, float("inf"), None) == INVALID
    assert f(0x1008, 10, 64, 1e4, None) == INVALID
    assert f(None, 0, 64, 1e4, None) == OK


def test_binding_checks_rows():
    q = torch.zeros(4, 6, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gq._token_rows(q, "q", q)
    with pytest.raises(ValueError, match="contiguous"):
        gq._token_rows(q[:, ::2], "q", q[:, ::2])
    with pytest.raises(ValueError, match="does not go"):
        gq._token_rows(torch.zeros(3, 6, 64, dtype=torch.bfloat16), "k", q)
    with pytest.raises(ValueError, match="heads"):
        gq._token_rows(q, "k", q, 3)
    with pytest.raises(ValueError, match="dtype"):
        gq._token_rows(q.float(), "k", q)
    x = torch.zeros(4, 6, 6, 64, dtype=torch.bfloat16)[:, :3]
    with pytest.raises(ValueError, match="evenly"):
        gq._token_rows(x, "q", x)
    with pytest.raises(ValueError, match="overlap"):
        y = torch.zeros(64 * 20).as_strided((4, 6, 64), (64, 64, 1))
        gq._token_rows(_FakeCuda(y), "q", y)


class _FakeCuda:
    """A CPU tensor that says it is on the GPU: the stride checks alone run."""
    def __init__(self, t):
        self.t = t

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_binding_checks_the_description():
    q = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="q_weight"):
        gq._norm_rope_desc(q, None, torch.zeros(32), None, 1e-6, False)
    with pytest.raises(ValueError, match="dtype"):
        gq._norm_rope_desc(q, None, torch.zeros(64, dtype=torch.float64), None, 1e-6, False)
    with pytest.raises(ValueError, match="rope"):
        gq._norm_rope_desc(q, torch.zeros(5, 32), None, None, 1e-6, False)
    with pytest.raises(ValueError, match="overlaps"):
        base = torch.zeros(5, 4, 64)
        gq._same_or_apart(base[:4], base[1:], "q_out")
    gq._same_or_apart(q, q, "q_out")
    with pytest.raises(ValueError, match="overlaps"):
        gq._same_or_apart(q, q, "q_out", False)             # another input's memory
    gq._same_or_apart(base[:2], base[2:], "q_out", False)
