"""Cached rows read back, against code * scale in fp64 rounded once (exact: both are)."""
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


KINDS = ["f32", "f16", "bf16", "int8", "fp8", "int4", "int4kc"]


def ragged(gq, kind, K, d, lens, reads, out, seed=0, order="pktd", spare_rows=0):
    """reads: (first position, rows) of every sequence."""
    bt = shared.batch([], lens, seed)
    where = np.argsort(bt.order)                                  # rows in the order of `lens`
    table = bt.table[where]
    cache, values = shared.pool(kind, bt.pages, K, d, seed + 1, gq, order=order)
    start = np.concatenate([[0], np.cumsum([n for _, n in reads])]).astype(np.int32)
    total = int(start[-1]) + spare_rows
    outs = [torch.full((total, K, d), 77.0, dtype=out, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.kv_read(cache, torch.from_numpy(table).cuda(),
                     torch.tensor([p for p, _ in reads], dtype=torch.int32, device="cuda"),
                     torch.from_numpy(start).cuda(), max([n for _, n in reads] + [1]), k_out=outs[0], v_out=outs[1], err=err)
    assert int(err) == 0 and got[0] is outs[0]
    for o, v in zip(outs, values):
        want = np.full((total, K, d), 77.0)
        for b, (p, n) in enumerate(reads):
            want[start[b]:start[b + 1]] = shared.rows_of(v, table, b, p + n)[p:]
        assert torch.equal(o.cpu(), torch.from_numpy(want).to(out))


@pytest.mark.parametrize("out", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,d", [(1, 64), (2, 128), (8, 128), (5, 64)])
def test_ragged(gq, kind, K, d, out):
    lens = [1, 16, 17, 100, 333, 64, 5]
    reads = [(0, 1), (0, 16), (16, 1), (33, 50), (0, 333), (64, 0), (2, 2)]
    ragged(gq, kind, K, d, lens, reads, out, seed=K, spare_rows=3)


@pytest.mark.parametrize("order", ["ptkd", "kptd"])
def test_axis_orders(gq, order):
    ragged(gq, "bf16", 3, 64, [90, 40], [(5, 80), (0, 40)], torch.float32, order=order)


def test_wide_cache(gq):
    """More kv-heads than a CTA takes at once."""
    ragged(gq, "int8", 96, 128, [40, 7], [(3, 30), (0, 7)], torch.bfloat16)


@pytest.mark.parametrize("kind", ["int8", "fp8", "int4", "bf16"])
def test_round_trip_of_the_append(gq, kind):
    """append -> read -> append gives the same codes; a float cache the same bits."""
    K, d, n = 2, 128, 75
    dtype = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "bf16": torch.bfloat16}.get(kind, kind)
    caches = [gq.PagedKVCache.allocate(8, K, d, dtype) for _ in range(2)]
    for c in caches:
        for t in (c.k, c.v):
            t.view(torch.uint8).zero_()
        for t in (c.k_scale, c.v_scale):
            if t is not None:
                t.zero_()
    table = torch.tensor([[5, 1, 7, 0, 2]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 1, n, K, d, generator=torch.Generator().manual_seed(1)).cuda()
    x = x.bfloat16() if kind == "bf16" else x
    gq.kv_append(caches[0], x[0].contiguous(), x[1].contiguous(), table, zero)
    k, v = gq.kv_read(caches[0], table, zero, max_tokens=n)
    assert k.shape == (1, n, K, d) and k.dtype == (torch.bfloat16 if kind == "bf16" else torch.float32)
    gq.kv_append(caches[1], k, v, table, zero)
    for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_bits_of_the_same_type(gq):
    """NaN payloads, infinities and subnormals of a 16-bit cache come back bit for bit."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(16, 2, 16, 128)
    for dt in (torch.float16, torch.bfloat16):
        k = bits.view(dt).cuda()
        cache = gq.PagedKVCache(k, k.clone(), 16, 2, 128, 2 * 16 * 128, 16 * 128, 128)
        table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
        got, _ = gq.kv_read(cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"), max_tokens=256)
        want = bits.permute(0, 2, 1, 3).reshape(1, 256, 2, 128)
        assert torch.equal(got.view(torch.int16).cpu(), want)


def test_out_of_range(gq):
    cache, values = shared.pool("bf16", 6, 2, 64, 3, gq)
    table = torch.tensor([[0, 1, 9], [2, -1, 3], [4, 5, 0]], dtype=torch.int32, device="cuda")

    def read(pos, start, most, total):
        out = torch.full((2, total, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        gq.kv_read(cache, table, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                   torch.tensor(start, dtype=torch.int32, device="cuda"), most, k_out=out[0], v_out=out[1], err=err)
        return out[0].double().cpu().numpy(), int(err)

    k = values[0]
    got, err = read([10, 0, 0], [0, 30, 60, 70], 30, 70)             # entries 9 and -1 are no pages
    assert err == gq.GQA_DEVERR_BLOCK_INDEX
    assert (got[:22] == np.concatenate([k[0], k[1]])[10:32]).all() and (got[22:30] == 7).all()
    assert (got[30:46] == k[2]).all() and (got[46:60] == 7).all() and (got[60:70] == k[4][:10]).all()
    got, err = read([-3, 40, 47], [0, 5, 20, 25], 30, 25)            # before 0 and past the table
    assert err == gq.GQA_DEVERR_POSITION
    assert (got[:3] == 7).all() and (got[3:5] == k[0][:2]).all()
    assert (got[5:13] == k[3][8:]).all() and (got[13:20] == 7).all()
    assert (got[20:21] == k[0][15:]).all() and (got[21:] == 7).all()
    for start in ([0, 31, 32, 33], [0, -1, 5, 6], [-2, 3, 4, 5], [0, 5, 10, 41]):
        got, err = read([0, 0, 0], start, 30, 40)
        assert err == gq.GQA_DEVERR_POSITION
    got, err = read([2 ** 31 - 1, 0, 0], [0, 4, 4, 4], 30, 4)
    assert err == gq.GQA_DEVERR_POSITION and (got == 7).all()


def test_sequences_of_no_rows_stand_anywhere(gq):
    """No row is asked for, so neither a position nor a table entry of theirs is at fault."""
    cache, values = shared.pool("bf16", 4, 2, 64, 3, gq)
    table = torch.tensor([[-1, -1], [2, 1], [9, 9], [0, -1]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([-3, 5, 7, 50], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 0, 20, 20, 20], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = gq.kv_read(cache, table, pos, start, max_tokens=24, total_tokens=20, err=err)
    assert int(err) == 0
    assert (k.double().cpu().numpy() == np.concatenate([values[0][2], values[0][1]])[5:25]).all()
    assert (v.double().cpu().numpy() == np.concatenate([values[1][2], values[1][1]])[5:25]).all()


def test_prefill_over_a_coded_cache(gq):
    """A coded context read back as an un-paged 16-bit cache, then prefilled over."""
    import math
    K, G, d, L, n = 2, 4, 128, 96, 20
    bt = shared.batch([], [L, L], 4)
    cache, values = shared.pool("int8", bt.pages, K, d, 5, gq)
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    k, v = gq.kv_read(cache, table, torch.zeros_like(lens), max_tokens=L, dtype=torch.float16)
    wide = gq.PagedKVCache(k, v, 2 * L // 16, K, d, 16 * K * d, d, K * d)
    flat = torch.arange(2 * L // 16, dtype=torch.int32, device="cuda").view(2, -1)
    q = torch.randn(2, n, K * G, d, generator=torch.Generator().manual_seed(6)).half()
    got = gq.gqa_prefill(wide, q.view(-1, K * G, d).cuda(), torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda"),
                         n, flat, lens, 1 / math.sqrt(d))
    # values rounded to f16 once: the softmax over them
    want = shared.attend(q.double().numpy(), [x.astype(np.float16).astype(np.float64) for x in values], bt.table, bt.lens,
                         1 / math.sqrt(d))
    assert float((got.view(want.shape).double().cpu() - torch.from_numpy(want)).abs().max()) <= \
        np.abs(values[1]).max() * 2.0 ** -11


def test_on_a_side_stream_and_in_a_graph(gq):
    cache, values = shared.pool("fp8", 20, 2, 128, 7, gq)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    want = torch.from_numpy(values[0].reshape(2, 160, 2, 128)).float()
    s = torch.cuda.Stream()
    a, _ = gq.kv_read(cache, table, pos, max_tokens=160, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b, _ = gq.kv_read(cache, table, pos, max_tokens=160)
    b.zero_()
    g.replay()
    assert torch.equal(a.cpu(), want) and torch.equal(b.cpu(), want)
