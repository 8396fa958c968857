"""The shared decode with plans that a caller wrote wrong: what is flagged, and what the rows
outside the fault get. Bounds as in test_gpu_shared.py: 2^-11 of the largest |v|."""
import numpy as np
import pytest
import torch

import shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def overlap(plan, B, blocks):
    """Every second group over all rows, the others of none."""
    plan.count.fill_(B)
    plan.start.copy_(torch.tensor([0, B] * B)[:B + 1])
    plan.blocks.fill_(blocks)
    plan.rows.copy_(torch.arange(B))
    plan.slot.copy_(torch.arange(B))
    plan.group.copy_(2 * (torch.arange(B) // 2))


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_overlapping_groups_are_flagged(gq, kind):
    B, blocks = 9, 20
    bt = shared.batch([(blocks, [16 * blocks + 1 + i for i in range(B)])], [], 26)
    cache, values = shared.pool(kind, bt.pages, 2, 64, 27, gq)
    q = torch.randn(B, 1, 8, 64, generator=torch.Generator().manual_seed(28)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    dq = q[:, 0].contiguous().cuda()
    plan = gq.kv_pages_groups(table, lens)
    overlap(plan, B, blocks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.gqa_decode_shared(cache, dq, table, lens, 0.1, plan, err=err)
    assert int(err) == gq.GQA_DEVERR_ROW
    assert torch.isfinite(got).all()
    # the next call on the same workspace, with the plan made again
    err.zero_()
    got = gq.gqa_decode_shared(cache, dq, table, lens, 0.1, gq.kv_pages_groups(table, lens), err=err)
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    assert int(err) == 0
    assert np.abs(got.view(q.shape).double().cpu().numpy() - want).max() <= np.abs(values[1]).max() * 2.0 ** -11


def test_overlapping_groups_whose_steps_pass_32_bits(gq):
    """4096 groups of 8191 rows of 64 queries over 1100 pages: 4096 * 2048 * 275 steps of the
    two-tile form are more than 2^31."""
    B, G, blocks = 8191, 64, 1100
    assert 4096 * -(-B * G // 256) * (blocks // 4) > 2 ** 31
    cache, _ = shared.pool("bf16", blocks + 1, 1, 64, 30, gq)
    table = torch.arange(blocks + 1, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    lens = torch.full((B,), 16 * blocks + 5, dtype=torch.int32, device="cuda")
    q = torch.randn(B, G, 64, generator=torch.Generator().manual_seed(31)).bfloat16().cuda()
    plan = gq.kv_pages_groups(table, lens)
    assert plan.count.tolist() == [1, B]
    overlap(plan, B, blocks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan, err=err)
    assert int(err) == gq.GQA_DEVERR_ROW
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("kind", ["f16", "int4"])
@pytest.mark.parametrize("bad", [-9, 7, 2 ** 31 - 1])
def test_a_first_row_outside_the_batch_is_flagged(gq, kind, bad):
    """The shared pages are read through it: the group's other rows do not get another row's. Rows
    of the other group and alone, and the first row itself (in no slot now), are as they were."""
    bt = shared.batch([(9, [150, 160, 170]), (12, [200, 210, 220])], [60], 40)
    cache, values = shared.pool(kind, bt.pages, 2, 128, 41, gq)
    B = len(bt.lens)
    assert B == 7
    q = torch.randn(B, 1, 8, 128, generator=torch.Generator().manual_seed(42)).to(shared.DTYPES.get(kind, torch.bfloat16))
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    for slot in (0, 3):                                          # the first rows of both groups
        fresh = gq.kv_pages_groups(table, lens)
        rows = fresh.rows.tolist()
        fresh.rows[slot] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, 0.1, fresh, err=err)
        assert int(err) == gq.GQA_DEVERR_ROW
        assert torch.isfinite(got).all()
        want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
        rest = [b for b in range(B) if b not in rows[slot + 1:slot + 3]]
        assert np.abs((got.view(q.shape).double().cpu().numpy() - want)[rest]).max() <= np.abs(values[1]).max() * 2.0 ** -11
    assert plan.count.tolist() == [2, 6]


@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 1])
def test_bounds_past_32_bits(gq, bound):
    """No row shares so many pages; so large a group is one of more than 128 query rows."""
    bt = shared.batch([(9, [150, 160, 170])], [60], 60)
    cache, values = shared.pool("bf16", bt.pages, 2, 64, 61, gq)
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    assert gq.kv_pages_groups(table, lens, bound).count.tolist() == [0, 0]
    q = torch.randn(4, 1, 8, 64, generator=torch.Generator().manual_seed(62)).bfloat16()
    got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, 0.1, gq.kv_pages_groups(table, lens),
                               max_group=bound)
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    assert np.abs(got.view(q.shape).double().cpu().numpy() - want).max() <= np.abs(values[1]).max() * 2.0 ** -11


@pytest.mark.parametrize("bound", [-1, -2 ** 32, -2 ** 32 + 7])
def test_bounds_below_zero_are_refused(gq, bound):
    table = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    lens = torch.full((2,), 40, dtype=torch.int32, device="cuda")
    with pytest.raises(gq.GqaError):
        gq.kv_pages_groups(table, lens, bound)
    cache, _ = shared.pool("bf16", 2, 2, 64, 63, gq)
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gq.GqaError):
        gq.gqa_decode_shared(cache, q, table, lens, 0.1, gq.kv_pages_groups(table, lens), max_group=bound)
