"""The read-back without a bound on the rows of a sequence, and with bounds past 32 bits."""
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


@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("bound", [{}, {"max_tokens": 2 ** 31 - 1}, {"max_tokens": 2 ** 32}, {"max_tokens": 2 ** 33 + 5}])
def test_rows_by_token_start_alone(gq, kind, bound):
    """Every row is read, and no err flag is needed to learn it."""
    lens, reads = [333, 17, 100], [(0, 333), (16, 1), (20, 60)]
    bt = shared.batch([], lens, 5)
    table = bt.table[np.argsort(bt.order)]
    cache, values = shared.pool(kind, bt.pages, 2, 64, 6, gq)
    start = np.concatenate([[0], np.cumsum([n for _, n in reads])]).astype(np.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = (torch.from_numpy(table).cuda(), torch.tensor([p for p, _ in reads], dtype=torch.int32, device="cuda"))
    for out in (dict(total_tokens=int(start[-1]), dtype=torch.float32),
                dict(k_out=torch.full((int(start[-1]) + 2, 2, 64), 7.0, device="cuda"))):
        k, v = gq.kv_read(cache, *at, token_start=torch.from_numpy(start).cuda(), err=err, **bound, **out)
        assert int(err) == 0
        for x, held in ((k, values[0]), (v, values[1])):
            for b, (p, n) in enumerate(reads):
                want = torch.from_numpy(shared.rows_of(held, table, b, p + n)[p:]).float()
                assert torch.equal(x[start[b]:start[b + 1]].cpu(), want), b
    assert (k[start[-1]:] == 7).all()


def test_one_row_of_every_sequence(gq):
    """Without token_start the bound is the number of rows: one where none is given."""
    bt = shared.batch([], [40, 33], 7)
    cache, values = shared.pool("f16", bt.pages, 2, 64, 8, gq)
    pos = torch.tensor([39, 0], dtype=torch.int32, device="cuda")
    k, _ = gq.kv_read(cache, torch.from_numpy(bt.table).cuda(), pos) if bt.lens[0] == 40 else \
        gq.kv_read(cache, torch.from_numpy(bt.table).cuda(), pos.flip(0).contiguous())
    assert k.shape == (2, 1, 2, 64)
    at = [39, 0] if bt.lens[0] == 40 else [0, 39]
    for b in range(2):
        assert (k[b, 0].double().cpu().numpy() == shared.rows_of(values[0], bt.table, b, at[b] + 1)[-1]).all()
