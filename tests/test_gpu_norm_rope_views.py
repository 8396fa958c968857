"""Norm and rotation of views whose token stride means nothing: one token, or none."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens", [0, 1])
@pytest.mark.parametrize("pad", [3, 8])
def test_one_token_of_a_projection_with_odd_rows(gq, dtype, tokens, pad):
    """[H, d], [K, d], [K, d] side by side in rows of any length: the row's start is aligned,
    and there is no second one."""
    H, K, d = 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn((4, (H + 2 * K) * d + pad), generator=g, device="cuda").to(dtype)[:tokens]
    def part(lo, heads):
        return rows.as_strided((tokens, heads, d), (rows.stride(0), d, 1), rows.storage_offset() + lo * d)
    q, k, v = part(0, H), part(H, K), part(H + K, K)
    assert q.stride(0) % 8 or pad == 8
    rope, w = gq.rope_table(32, d), torch.rand(d, generator=g, device="cuda").to(dtype)
    pos = torch.full((tokens,), 17, dtype=torch.int32, device="cuda")
    kw = dict(rope=rope, q_weight=w, k_weight=w)
    want = gq.qk_norm_rope(q.contiguous(), k.contiguous(), pos, **kw)
    got = gq.qk_norm_rope(q, k, pos, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    caches = [gq.PagedKVCache.allocate(4, K, d, dtype) for _ in range(2)]
    table, at = torch.tensor([[2, 1]] * tokens, dtype=torch.int32, device="cuda").reshape(tokens, 2), pos[:tokens]
    outs = [gq.qk_norm_rope_append(c, a, b, e, table, at, **kw)
            for c, (a, b, e) in zip(caches, ((q.contiguous(), k.contiguous(), v.contiguous()), (q, k, v)))]
    assert torch.equal(outs[0], outs[1])
    torch.cuda.synchronize()
    if tokens:
        for x, y in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
            assert torch.equal(x[1, :, 1], y[1, :, 1])
        assert torch.equal(caches[1].v[1, :, 1], v[0])
