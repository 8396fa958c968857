"""Lists of page copies that are used again, by another call than the one that made them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("side", [False, True])
@pytest.mark.parametrize("kind", ["int4kc", torch.bfloat16])
def test_a_compaction_with_a_forks_list_moves_no_residual_rows(gq, kind, side):
    """Fork, the child goes its own way, then a compaction that uses the fork's list: the
    child's open block, unquantised in its residual row, stays what it has become."""
    stream = torch.cuda.Stream() if side else None
    gen = torch.Generator(device="cuda").manual_seed(1)
    rows, blocks, pages, K, d = 4, 4, 32, 2, 64
    cache = gq.PagedKVCache.allocate(pages, K, d, kind, residual_rows=rows if kind == "int4kc" else 0)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).random_(0, 256, generator=gen)
    if kind == "int4kc":
        cache.k_residual.normal_(generator=gen)
    refs, table = torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.full((rows, blocks), -1, dtype=torch.int32,
                                                                                  device="cuda")
    lens, err = _i32([0] * rows), torch.zeros(1, dtype=torch.int32, device="cuda")
    copies = gq.PageCopies(torch.zeros((16, 2), dtype=torch.int32, device="cuda"), _i32([0, 0]),
                           torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    new = _i32([30, 20, 0, 0])
    gq.kv_pages_reserve(refs, table, lens, new, err=err)
    lens += new
    gq.kv_pages_fork(refs, table, lens, _i32([1]), _i32([2]), copies=copies, err=err)
    gq.kv_copy_pages(cache, copies, err=err)
    assert copies.rows.tolist() == [[1, 2]] and copies.count.tolist()[0] == 1
    if kind == "int4kc":
        assert torch.equal(cache.k_residual[2], cache.k_residual[1])
        cache.k_residual[2].normal_(generator=gen)       # what the child's own appends leave there
        mine = cache.k_residual.clone()
    gq.kv_pages_free(refs, table, lens, _i32([0]), err=err)
    held = {(b, j): cache.k[p].clone() for b, r in enumerate(table.tolist()) for j, p in enumerate(r) if p >= 0}
    torch.cuda.synchronize()
    got = gq.kv_pages_compact(refs, table, copies=copies, err=err, stream=stream)
    gq.kv_copy_pages(cache, got, err=err, stream=stream)
    gq.kv_copy_pages(cache, copies, err=err, stream=stream)      # the list itself says the same
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and copies.count.tolist()[0] == 2 and int(copies.count[1]) == 3
    for (b, j), k in held.items():
        assert torch.equal(cache.k[int(table[b, j])].view(torch.uint8), k.view(torch.uint8))
    if kind == "int4kc":
        assert torch.equal(cache.k_residual, mine)
    # and it serves the next fork
    again = gq.kv_pages_fork(refs, table, lens, _i32([2]), _i32([3]), copies=copies, err=err)
    assert again.rows.tolist() == [[2, 3]] and int(err.item()) == 0
