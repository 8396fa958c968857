"""The groups of rows that share pages, against the same found entry by entry."""
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


def same(gq, table, lens, min_blocks=1, flag=0, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.kv_pages_groups(torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), min_blocks, err=err, **kw)
    want = shared.plan_of(table, lens, min_blocks)
    for name, w in zip(("count", "start", "blocks", "rows", "slot", "group"), want):
        assert getattr(got, name).tolist() == w, name
    assert int(err) == flag
    return got


def forest(rng, B, wide, roots, cut=0.3):
    """Rows that follow a root for a while and then go their own ways, some to a second level."""
    pages = iter(rng.permutation(B * wide * 2 + roots * wide * 3).tolist())
    base = [[next(pages) for _ in range(wide)] for _ in range(roots)]
    second = [[r[:rng.integers(0, wide)] for _ in range(3)] for r in base]
    second = [[s + [next(pages) for _ in range(wide - len(s))] for s in rows] for rows in second]
    table = np.full((B, wide), -1, dtype=np.int32)
    lens = np.zeros(B, dtype=np.int32)
    for b in range(B):
        r = int(rng.integers(roots))
        src = base[r] if rng.random() < 0.5 else second[r][int(rng.integers(3))]
        keep = int(rng.integers(0, wide + 1))
        n = int(rng.integers(0, wide + 1))
        row = (src[:keep] + [next(pages) for _ in range(wide)])[:n]
        table[b, :n] = row
        lens[b] = max(0, 16 * n - int(rng.integers(0, 16)))
        if rng.random() < cut and n:
            lens[b] = int(rng.integers(0, 16 * n + 1))
    return table, lens


@pytest.mark.parametrize("B,wide,roots", [(1, 1, 1), (2, 1, 1), (2, 5, 1), (7, 3, 2), (33, 9, 3), (64, 40, 4), (130, 17, 20),
                                          (300, 6, 3), (1030, 5, 11), (40, 700, 2), (9, 1500, 1)])
@pytest.mark.parametrize("min_blocks", [0, 1, 4])
def test_forests(gq, B, wide, roots, min_blocks):
    rng = np.random.default_rng(B * 1000 + wide)
    same(gq, *forest(rng, B, wide, roots), min_blocks)


@pytest.mark.parametrize("B", [16, 127, 128, 129, 255, 256, 257, 511, 513])
def test_one_launch_and_several(gq, B):
    """Around the sizes where a warp takes another row and where a launch per step begins."""
    rng = np.random.default_rng(B)
    same(gq, *forest(rng, B, 150, max(1, B // 17)))
    table, lens = forest(rng, B, 3, B)                       # hardly anything shared
    lens[::5] = 16 * 3 + 1                                   # past the table
    same(gq, table, lens, flag=gq.GQA_DEVERR_CONTEXT_LEN)


def test_nothing_shared(gq):
    table = np.arange(50 * 7, dtype=np.int32).reshape(50, 7)
    got = same(gq, table, np.full(50, 100, dtype=np.int32))
    assert got.count.tolist() == [0, 0]


def test_everything_shared(gq):
    table = np.tile(np.arange(600, dtype=np.int32), (300, 1))
    got = same(gq, table, np.full(300, 9600, dtype=np.int32))
    assert got.blocks.tolist()[0] == 600 and got.count.tolist() == [1, 300]


def test_largest_batch(gq):
    table = np.tile(np.arange(3, dtype=np.int32), (8192, 1))
    table[1::2] += 3
    table[5, 2] = 9
    got = same(gq, table, np.full(8192, 48, dtype=np.int32))
    assert got.count.tolist() == [2, 8191]


def test_equal_savings_take_more_pages(gq):
    # P = 2 for four rows saves 6 pages, P = 3 for three 6, P = 6 for two 6
    table = np.arange(4 * 6, dtype=np.int32).reshape(4, 6) + 100
    table[:, :2] = [0, 1]
    table[:3, 2] = 2
    table[:2, 3:] = [3, 4, 5]
    got = same(gq, table, np.full(4, 96, dtype=np.int32))
    assert got.blocks.tolist()[0] == 6 and got.rows.tolist()[:2] == [0, 1]


def test_entries_without_pages(gq):
    table = np.full((6, 4), -1, dtype=np.int32)
    table[0, :2] = [4, -1]
    table[1, :3] = [4, -1, 7]
    table[2] = table[3] = [5, 6, -1, 8]
    got = same(gq, table, np.full(6, 64, dtype=np.int32))
    assert got.blocks.tolist()[:2] == [1, 2]


def test_lengths_out_of_range(gq):
    table = np.tile(np.arange(4, dtype=np.int32), (5, 1))
    lens = np.array([64, -1, 64, 65, 40], dtype=np.int32)
    same(gq, table, lens, flag=gq.GQA_DEVERR_CONTEXT_LEN)


def test_plan_made_again_in_place_and_in_a_graph(gq):
    rng = np.random.default_rng(5)
    table, lens = forest(rng, 40, 12, 2)
    plan = same(gq, table, lens)
    same(gq, *forest(rng, 40, 12, 2), groups=plan)
    t, L = torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = gq.kv_pages_groups(t, L)
    for _ in range(3):
        table, lens = forest(rng, 40, 12, 2)
        t.copy_(torch.from_numpy(table))
        L.copy_(torch.from_numpy(lens))
        g.replay()
        want = shared.plan_of(table, lens)
        for name, w in zip(("count", "start", "blocks", "rows", "slot", "group"), want):
            assert getattr(kept, name).tolist() == w, name


def test_fewer_rows_than_the_table(gq):
    rng = np.random.default_rng(6)
    table, lens = forest(rng, 20, 8, 2)
    got = gq.kv_pages_groups(torch.from_numpy(table).cuda(), torch.from_numpy(lens[:12]).cuda())
    want = shared.plan_of(table[:12], lens[:12])
    assert got.rows.tolist() == want[3] and got.start.tolist() == want[1]
