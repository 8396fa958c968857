"""Decode with sink tokens over caches whose outer axes lie in another order than the
pool's, 16-bit and coded, through the C ABI."""
import pytest
import torch

import gqa_inputs as gi
from helpers import TOL, max_abs_err
from plain import attend_case

pytestmark = pytest.mark.gpu

LENS = [1, 17, 100, 0, 333]


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def _permuted(gq, case, order):
    """The case's pool with its outer axes (block, kv-head, slot) laid out in `order`;
    scales keep their place. Strides count elements, two to a byte for 4-bit codes."""
    def lay(t):
        return t.permute(*order, 3).contiguous()
    k, v = lay(case.k_cache), lay(case.v_cache)
    per = 2 if case.cache_dtype in ("i4", "i4kc") else 1
    stride = [0, 0, 0]
    for axis, at in zip(order, k.stride()):
        stride[axis] = at * per
    code = {"i4": gq.GQA_DTYPE_I4, "i4kc": gq.GQA_DTYPE_I4_KC}.get(case.cache_dtype)
    return gq.PagedKVCache(k, v, case.num_blocks, case.num_kv_heads, case.head_dim, *stride, case.k_scale, case.v_scale,
                           code, getattr(case, "k_residual", None))


@pytest.mark.parametrize("order", [(0, 2, 1), (1, 0, 2), (2, 0, 1), (1, 2, 0), (2, 1, 0)])
@pytest.mark.parametrize("dtype,H,K,T,d", [("bf16", 8, 4, 1, 128), ("f16", 8, 4, 3, 64), ("f32", 8, 4, 1, 64),
                                           ("fp8", 8, 4, 1, 128), ("i8", 8, 1, 2, 128), ("i4", 24, 2, 1, 128),
                                           ("i4kc", 8, 4, 1, 128), ("i8", 8, 4, 1, 64)])
def test_axis_orders(gq, dtype, H, K, T, d, order):
    case = gi.make_case(len(LENS), H, K, d, LENS, dtype, seed=81, device="cuda", queries=T)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for window, sinks in ((40, 20), (7, 3)):
        out = gq.gqa_decode(_permuted(gq, case, order), case.q, case.block_table, case.context_lens, case.scale, err=err,
                            window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert max_abs_err(out, attend_case(case, window, sinks)) <= TOL
