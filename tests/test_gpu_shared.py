"""Decode attention over shared prefixes against the softmax written out in fp64.

Bound of an fp32 output, relative to the largest |v|: a score of d <= 128 products that are
exact in fp32 has an accumulation error of at most 128 * 2^-23 * sum |q_i k_i| * scale, with
N(0,1) inputs below 8 * 128 * 2^-23 = 2^-13; it enters a weight and the sum of weights, so
2^-12. Weights in two 16-bit parts add 2^-16 each, exp2 and the merges 2^-20. Together below
2^-11. An output of a 16-bit type adds half its step."""
import math

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


def run(gq, kind, K, G, d, T, groups, alone, seed=0, q_dtype=None, out=torch.float32, order="pktd", max_group=0,
        columns=1, plan=None, tweak=None, amp=1.0, scale=None):
    bt = shared.batch(groups, alone, seed, columns=columns)
    cache, values = shared.pool(kind, bt.pages, K, d, seed + 1, gq, order=order, amp=amp)
    if tweak:
        tweak(bt, cache, values)
    qt = q_dtype or shared.DTYPES.get(kind, torch.bfloat16)
    q = torch.randn(len(bt.lens), T, K * G, d, generator=torch.Generator().manual_seed(seed + 2)).to(qt)
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = gq.kv_pages_groups(table, lens, err=err) if plan is None else plan(table, lens)
    scale = 1 / math.sqrt(d) if scale is None else scale
    got = gq.gqa_decode_shared(cache, q.cuda() if T > 1 else q[:, 0].contiguous().cuda(), table, lens, scale, plan,
                               out_dtype=out, max_group=max_group, err=err)
    torch.cuda.synchronize()
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, scale)
    return got.view(q.shape).double().cpu().numpy(), want, int(err), values, plan


def check(got, want, values, out=torch.float32):
    bound = np.nanmax(np.abs(values[1])) * 2.0 ** -11 + (
        np.abs(want) * torch.finfo(out).eps / 2 if out != torch.float32 else 0)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) - bound).max())


SHAPES = [
    # K, G, d, T, groups (shared blocks, lengths), alone
    (1, 1, 128, 1, [(1, [17, 16])], []),
    (2, 4, 128, 1, [(3, [49, 50, 70])], [5, 0]),
    (2, 4, 64, 1, [(4, [64, 65, 66, 100])], []),
    (2, 3, 128, 2, [(5, [82, 99, 81])], [1, 2, 300]),
    (8, 4, 128, 1, [(64, [1025, 1040, 1100, 1024])], [7]),
    (4, 8, 64, 3, [(17, [275, 290, 300]), (2, [35, 60]), (40, [700, 650])], [0, 33]),
    (1, 8, 128, 4, [(33, [532] * 9)], []),                       # 288 rows: more than a CTA's tiles
    (2, 8, 128, 1, [(20, [321 + i for i in range(40)])], []),    # 320 rows
    (1, 16, 64, 1, [(9, [150] * 9)], [3]),                       # 144 rows
    (2, 2, 128, 16, [(6, [112, 130])], [40]),
    (3, 5, 128, 1, [(7, [113, 120]), (7, [115, 200, 131])], []),
    (1, 64, 128, 1, [(11, [177, 190, 201])], [20]),              # 64 query rows a kv-head
    (1, 12, 64, 5, [(70, [1130, 1125, 1200, 1140])], []),        # 60, over two tiles of rows
    (8, 1, 128, 1, [(1, [17] * 30)], [1] * 3),                   # no groups of heads
    (2, 2, 64, 1, [(2, [33, 34])] * 20, [9]),                    # many small groups
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("K,G,d,T,groups,alone", SHAPES)
def test_against_fp64(gq, kind, K, G, d, T, groups, alone):
    got, want, err, values, plan = run(gq, kind, K, G, d, T, groups, alone)
    assert err == 0
    assert plan.count.tolist()[0] == len(groups)
    check(got, want, values)


@pytest.mark.parametrize("kind,q_dtype", [("int8", torch.bfloat16), ("int8", torch.float16), ("fp8", torch.bfloat16),
                                          ("fp8", torch.float16), ("int4", torch.bfloat16)])
@pytest.mark.parametrize("K,G,d,T,groups,alone", SHAPES)
def test_coded_against_fp64(gq, kind, q_dtype, K, G, d, T, groups, alone):
    """The values are code * scale exactly, and so are the products in fp16."""
    got, want, err, values, plan = run(gq, kind, K, G, d, T, groups, alone, q_dtype=q_dtype)
    assert err == 0
    assert plan.count.tolist()[0] == len(groups)
    check(got, want, values)


@pytest.mark.parametrize("kind", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_sizes_of_v_in_coded_caches(gq, kind, order):
    """V's scales from 2^-22 to 2^4, rising, falling and mixed along the prefix: the error goes by the
    largest |v| that a row sees, and rows of tiny V keep their bits."""
    n = 60
    size = {"rising": np.linspace(-20, 4, n), "falling": np.linspace(4, -20, n),
            "mixed": np.random.default_rng(1).uniform(-20, 4, n)}[order]
    for top in (4.0, -14.0):
        amp = 2.0 ** (size - 4 + top)

        def tweak(bt, cache, values):
            lead = max(range(len(bt.lens)), key=lambda b: bt.lens[b])
            scale = cache.v_scale.clone()
            for j in range(n):
                p = int(bt.table[lead, j])
                old = scale[p].clone()
                scale[p] = (old.float() * float(amp[j])).half()
                f = scale[p].double().cpu().numpy() / old.double().cpu().numpy()      # [K, 16]
                values[1][p] *= f.T[:, :, None]
            scale_small = [int(x) for b in range(len(bt.lens)) for x in bt.table[b, n:] if x >= 0]
            for p in scale_small:
                old = scale[p].clone()
                scale[p] = (old.float() * 2.0 ** (top - 8)).half()
                f = scale[p].double().cpu().numpy() / old.double().cpu().numpy()
                values[1][p] *= f.T[:, :, None]
            cache.v_scale.copy_(scale)

        got, want, err, values, _ = run(gq, kind, 2, 8, 128, 1, [(n, [16 * n + 5, 16 * n + 30, 16 * n + 1] * 3)], [],
                                        tweak=tweak)
        assert err == 0
        seen = 2.0 ** top * 4.5
        assert (np.abs(got - want) <= seen * 2.0 ** -11).all(), float(np.abs(got - want).max() / seen)


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_poisoned_scales_behind_the_rows(gq, kind):
    """Scales of slots that no row owns are NaN."""
    def tweak(bt, cache, values):
        owned = np.zeros((bt.pages, 16), dtype=bool)
        for b, L in enumerate(bt.lens):
            for t in range(L):
                owned[bt.table[b, t // 16], t % 16] = True
        at = torch.from_numpy(~owned)
        for t in (cache.k_scale, cache.v_scale):
            x = t.cpu()                                             # [pages, K, 16]
            x[at[:, None, :].expand(-1, x.shape[1], -1)] = float("nan")
            t.copy_(x)

    got, want, err, values, _ = run(gq, kind, 2, 4, 128, 1, [(5, [81, 95, 90]), (6, [97, 98])], [3, 0, 18], tweak=tweak)
    assert err == 0
    check(got, want, values)


@pytest.mark.parametrize("kind", ["int8", "fp8", "int4"])
def test_bad_pages_of_coded_caches_are_flagged(gq, kind):
    bt = shared.batch([(9, [150, 160])], [40], 14)
    cache, values = shared.pool(kind, bt.pages, 2, 128, 15, gq)
    q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(16)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    lead = plan.rows.tolist()[0]
    for bad in (-1, bt.pages, 2 ** 31 - 1):
        broken = table.clone()
        broken[lead, 4] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), broken, lens, 0.1, plan, err=err)
        assert int(err) == gq.GQA_DEVERR_BLOCK_INDEX
        assert torch.isfinite(got).all()


@pytest.mark.parametrize("max_group", [1, 4, 500])
@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16, torch.float32])
def test_forms_and_outputs(gq, max_group, out):
    """The hint picks one or two tiles per CTA whatever the groups are."""
    got, want, err, values, _ = run(gq, "bf16", 2, 8, 128, 1, [(20, [321 + i for i in range(40)]), (9, [150, 151])], [11],
                                    out=out, max_group=max_group)
    assert err == 0
    check(got, want, values, out)


@pytest.mark.parametrize("order", ["ptkd", "kptd", "pktd"])
def test_axis_orders(gq, order):
    got, want, err, values, _ = run(gq, "f16", 4, 2, 128, 1, [(10, [161, 170, 200])], [30], order=order)
    assert err == 0
    check(got, want, values)


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_axis_orders_of_coded_caches(gq, kind):
    """Codes as [page][slot][head][row]: the scales stay [page][head][slot]."""
    bt = shared.batch([(10, [161, 170, 200])], [30], 3)
    cache, values = shared.pool(kind, bt.pages, 4, 128, 4, gq)
    wide = 64 if kind == "int4" else 128
    turned = [t.permute(0, 2, 1, 3).contiguous() for t in (cache.k, cache.v)]
    other = gq.PagedKVCache(*turned, bt.pages, 4, 128, 4 * 16 * 128, 128, 4 * 128, cache.k_scale, cache.v_scale,
                            cache.dtype_code)
    assert turned[0].shape[-1] == wide
    q = torch.randn(4, 1, 8, 128, generator=torch.Generator().manual_seed(5)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    got = gq.gqa_decode_shared(other, q[:, 0].contiguous().cuda(), table, lens, 0.09, gq.kv_pages_groups(table, lens))
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.09)
    check(got.view(q.shape).double().cpu().numpy(), want, values)


def test_more_groups_than_threads(gq):
    """A plan of 900 groups: the kernels scan it in rounds."""
    groups = [(1 + i % 3, [16 * (1 + i % 3) + 1 + i % 5, 16 * (1 + i % 3) + 2]) for i in range(900)]
    got, want, err, values, plan = run(gq, "bf16", 1, 2, 64, 1, groups, [3] * 7, max_group=2)
    assert err == 0 and plan.count.tolist() == [900, 1800]
    check(got, want, values)


def test_replays_of_a_growing_batch(gq):
    """One captured call serves later lengths: the division of the work is the device's."""
    K, G, d, B = 2, 4, 128, 5
    bt = shared.batch([(20, [321 + 40] * B)], [], 29)
    cache, values = shared.pool("f16", bt.pages, K, d, 30, gq)
    q = torch.randn(B, 1, K * G, d, generator=torch.Generator().manual_seed(31)).half()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan, dq = gq.kv_pages_groups(table, lens), q[:, 0].contiguous().cuda()
    gq.gqa_decode_shared(cache, dq, table, lens, 0.1, plan)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gq.gqa_decode_shared(cache, dq, table, lens, 0.1, plan)
    for now in ([321] * B, [361, 0, 17, 320, 340], [0] * B, [361] * B):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        want = shared.attend(q.double().numpy(), values, bt.table, np.array(now), 0.1)
        check(out.view(q.shape).double().cpu().numpy(), want, values)


def test_short_and_empty_rows_of_a_group(gq):
    """Rows that went back behind the shared pages attend alone, with the plan they were in."""
    for T in (1, 2):
        bt = shared.batch([(10, [161, 170, 200, 165, 190, 177])], [], 0)
        cache, values = shared.pool("bf16", bt.pages, 2, 128, 1, gq)
        table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
        plan_ = gq.kv_pages_groups(table, lens)
        now = bt.lens.copy()
        now[0], now[2], now[3] = 0, 33, 160
        lens.copy_(torch.from_numpy(now))
        q = torch.randn(6, T, 8, 128, generator=torch.Generator().manual_seed(3)).bfloat16()
        got = gq.gqa_decode_shared(cache, q.cuda(), table, lens, 0.09, plan_)
        want = shared.attend(q.double().numpy(), values, bt.table, now, 0.09)
        check(got.double().cpu().numpy(), want, values)
        assert (got[0] == 0).all()


def test_no_groups_and_one_row(gq):
    got, want, err, values, plan = run(gq, "bf16", 2, 4, 128, 1, [], [100])
    assert err == 0 and plan.count.tolist() == [0, 0]
    check(got, want, values)


def test_no_rows(gq):
    cache, _ = shared.pool("bf16", 3, 2, 64, 0, gq)
    table = torch.full((0, 4), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    plan = gq.kv_pages_groups(table, lens)
    assert plan.count.tolist() == [0, 0]
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan).shape == q.shape


def test_poison_behind_the_rows(gq):
    """Slots behind a row's end and pages of no row hold NaN; nothing of them is seen."""
    def tweak(bt, cache, values):
        owned = np.zeros((bt.pages, 16), dtype=bool)
        for b, L in enumerate(bt.lens):
            for t in range(L):
                owned[bt.table[b, t // 16], t % 16] = True
        at = torch.from_numpy(~owned)
        for t in (cache.k, cache.v):
            x = t.cpu()                                             # [pages, K, 16, d]
            x[at[:, None, :].expand(-1, x.shape[1], -1)] = float("nan")
            t.copy_(x)

    for d in (64, 128):
        got, want, err, values, _ = run(gq, "bf16", 2, 4, d, 1, [(5, [81, 95, 90]), (6, [97, 98])], [3, 0, 18], tweak=tweak)
        assert err == 0
        check(got, want, values)


def test_same_pages_elsewhere_in_the_tables(gq):
    """A page that another row holds at another place is no shared prefix."""
    def tweak(bt, cache, values):
        bt.table[0, 3] = bt.table[1, 2]

    got, want, err, values, plan = run(gq, "f16", 2, 2, 64, 1, [(2, [60, 64, 50])], [], tweak=tweak)
    assert err == 0 and plan.blocks.tolist()[0] == 2
    check(got, want, values)


def test_large_and_small_scores(gq):
    """Scores far apart: the running maximum is rescaled step by step."""
    for amp, scale in ((4.0, 0.5), (1.0, 0.0), (1.0, -0.1)):
        bt = shared.batch([(40, [641, 700, 655])], [], 5)
        cache, values = shared.pool("bf16", bt.pages, 2, 128, 6, gq, amp=amp)
        q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(7)).bfloat16()
        table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
        got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, scale, gq.kv_pages_groups(table, lens))
        want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, scale)
        # scores up to amp * scale * sqrt(d) times larger than the bound above allows for
        bound = np.abs(values[1]).max() * 2.0 ** -11 * max(1.0, amp * abs(scale) * math.sqrt(128))
        assert (np.abs(got.view(q.shape).double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "int8"])
def test_many_small_weights_beside_a_large_one(gq, kind):
    """One token whose score is 18 above all others': a weight of e^-18 each, whose sum over
    the prefix is all that the output holds. Two 16-bit parts lose 2^-16 of a bf16 weight, at
    most 2^-32 of the largest from an fp16 one (2^-6 of e^-18), 2^-30 with int8 codes (2^-4)."""
    bt = shared.batch([(256, [4100, 4097])], [], 40)
    cache, values = shared.pool(kind, bt.pages, 1, 64, 41, gq)
    first = int(bt.table[0, 0])
    if kind == "int8":
        cache.k.zero_()
        cache.k[first, 0, 0] = 1
        cache.k_scale.fill_(2.25)
        cache.v.fill_(1)
        cache.v_scale.fill_(1)
        cache.v[first, 0, 0] = 0
    else:
        cache.k.zero_()
        cache.k[first, 0, 0] = 2.25                             # page, kv-head, token
        cache.v.fill_(1)
        cache.v[first, 0, 0] = 0
    q = torch.ones(2, 2, 64, dtype=shared.DTYPES.get(kind, torch.bfloat16), device="cuda")
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    assert plan.blocks.tolist()[0] == 256
    got = gq.gqa_decode_shared(cache, q, table, lens, 0.125, plan).double().cpu().numpy()
    x = (bt.lens.astype(np.float64) - 1) * math.exp(-18.0)
    want = (x / (1 + x))[:, None, None]
    # 18 = 64 products of 2.25 / 8, exact; exp2 of 18 log2(e) rounded: 2^-24 * 26 * ln 2
    bound = {"bf16": 2.0 ** -16, "f16": 2.0 ** -6, "int8": 2.0 ** -4}[kind] + 2.0 ** -18
    assert (np.abs(got - want) <= bound * want).all(), float(np.abs(got / want - 1).max())


@pytest.mark.parametrize("kind", ["bf16", "f16", "int8"])
def test_nan_and_infinite_inputs(gq, kind):
    """A NaN query head gives NaN there and nowhere else; a V of infinity that is attended
    leaves its column alone not finite (NaN where a weight's low part is zero or negative), and
    a score of -inf takes its token out."""
    bt = shared.batch([(20, [330, 340, 350])], [30], 60)
    cache, values = shared.pool(kind, bt.pages, 2, 64, 61, gq)
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    q = torch.randn(4, 1, 8, 64, generator=torch.Generator().manual_seed(62)).to(shared.DTYPES.get(kind, torch.bfloat16))
    row = plan.rows.tolist()[1]
    bad = q.clone()
    bad[row, 0, 3] = float("nan")
    got = gq.gqa_decode_shared(cache, bad[:, 0].contiguous().cuda(), table, lens, 0.125, plan)
    got = got.view(q.shape).double().cpu().numpy()
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.125)
    assert np.isnan(got[row, 0, 3]).all()
    got[row, 0, 3] = want[row, 0, 3]
    check(got, want, values)
    if kind == "int8":
        return
    page = int(bt.table[row, 5])                                 # in all three rows
    cache.v[page, 1, 4, 7] = float("inf")
    got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, 0.125, plan)
    got = got.view(q.shape).double().cpu().numpy()
    for r in plan.rows.tolist()[:3]:
        assert not np.isfinite(got[r, 0, 4:, 7]).any()
        got[r, 0, 4:, 7] = want[r, 0, 4:, 7]
    check(got, want, values)
    # a key of -inf where the queries are positive
    cache.v[page, 1, 4, 7] = 0
    cache.k[page, 1, 4, 0] = -float("inf")
    pos = q.abs()
    held = values[0].copy()
    held[page, 4, 1, 0] = -1e6
    kept = values[1].copy()
    kept[page, 4, 1, 7] = 0
    want = shared.attend(pos.double().numpy(), [held, kept], bt.table, bt.lens, 0.125)
    got = gq.gqa_decode_shared(cache, pos[:, 0].contiguous().cuda(), table, lens, 0.125, plan)
    check(got.view(q.shape).double().cpu().numpy(), want, values)


def test_two_threads_on_two_streams(gq):
    """Calls of two host threads at once, each on its own stream with the workspace kept for it."""
    import threading
    bt = shared.batch([(60, [1000 + i for i in range(9)])], [70], 70)
    cache, values = shared.pool("bf16", bt.pages, 2, 128, 71, gq)
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    qs = [torch.randn(10, 16, 128, generator=torch.Generator().manual_seed(72 + i)).bfloat16().cuda() for i in range(2)]
    want = [gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan) for q in qs]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in qs]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(30):
                got[i].append(gq.gqa_decode_shared(cache, qs[i], table, lens, 0.1, plan))
        streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 30
        for x in got[i]:
            assert float((x - want[i]).abs().max()) <= 2 * np.abs(values[1]).max() * 2.0 ** -11


def test_equals_decode_and_shares_its_workspace(gq):
    bt = shared.batch([(30, [500 + i for i in range(7)]), (11, [200, 300])], [40, 0], 8)
    cache, values = shared.pool("bf16", bt.pages, 4, 128, 9, gq)
    B = len(bt.lens)
    q = torch.randn(B, 16, 128, generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    ws = torch.zeros(gq.decode_shared_workspace_size(B, 16, 4, 128), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(3):
        outs.append(gq.gqa_decode(cache, q, table, lens, 0.1, workspace=ws))
        outs.append(gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan, workspace=ws))
    for a in outs[2:]:
        assert torch.equal(a, outs[0]) or torch.equal(a, outs[1])
    assert float((outs[0] - outs[1]).abs().max()) <= 2 * np.abs(values[1]).max() * 2.0 ** -11


@pytest.mark.parametrize("kind,d,G,T", [("bf16", 128, 8, 1), ("f16", 64, 4, 3), ("int8", 64, 16, 1)])
def test_most_rows(gq, kind, d, G, T):
    """8191 rows in three groups, against plain decode."""
    B, K = 8191, 2
    cache, values = shared.pool(kind, 64, K, d, 80, gq)
    gen = torch.Generator().manual_seed(81)
    table = torch.randint(0, 64, (B, 4), generator=gen, dtype=torch.int32)
    table[:, 0] = torch.arange(B) % 3
    table[:, 1] = 3 + torch.arange(B) % 3
    lens = torch.randint(32 + T, 65, (B,), generator=gen, dtype=torch.int32).cuda()
    table = table.cuda()
    q = torch.randn(B, T, K * G, d, generator=gen).to(shared.DTYPES.get(kind, torch.bfloat16)).cuda()
    q = q if T > 1 else q[:, 0].contiguous()
    plan = gq.kv_pages_groups(table, lens)
    assert plan.count.tolist() == [3, B]
    got = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan)
    assert float((got - gq.gqa_decode(cache, q, table, lens, 0.1)).abs().max()) <= 2 * np.abs(values[1]).max() * 2.0 ** -11


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_pages_past_32_bits(gq, kind):
    """Pages whose elements lie past 2^31, shared and own, in a pool of 140000."""
    K, d, pages = 8, 128, 140000
    bt = shared.batch([(20, [330, 350, 321])], [40], 82)
    small, values = shared.pool(kind, bt.pages, K, d, 83, gq)
    cache = gq.PagedKVCache.allocate(pages, K, d, small.k.dtype)
    at = pages - bt.pages                                        # the last pages of the pool
    for name in ("k", "v", "k_scale", "v_scale"):
        if getattr(small, name) is not None:
            getattr(cache, name)[at:] = getattr(small, name)
    table = torch.from_numpy(np.where(bt.table >= 0, bt.table + at, -1).astype(np.int32)).cuda()
    lens = torch.from_numpy(bt.lens).cuda()
    q = torch.randn(4, 1, 4 * K, d, generator=torch.Generator().manual_seed(84)).bfloat16()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, 0.1, gq.kv_pages_groups(table, lens), err=err)
    assert int(err) == 0
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    check(got.view(q.shape).double().cpu().numpy(), want, values)
    k, v = gq.kv_read(cache, table, torch.zeros(4, dtype=torch.int32, device="cuda"), max_tokens=1, dtype=torch.float32)
    for b in range(4):
        assert (k[b, 0].double().cpu().numpy() == shared.rows_of(values[0], bt.table, b, 1)[0]).all()


def test_streams_and_graphs(gq):
    """Captured calls of one stream replayed on two, interleaved with eager ones."""
    bt = shared.batch([(30, [500 + i for i in range(7)])], [40], 11)
    cache, values = shared.pool("bf16", bt.pages, 4, 128, 12, gq)
    B = len(bt.lens)
    q = torch.randn(B, 1, 16, 128, generator=torch.Generator().manual_seed(13)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    q = q[:, 0].contiguous().cuda()
    plan = gq.kv_pages_groups(table, lens)
    gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p = gq.kv_pages_groups(table, lens)
            outs.append(gq.gqa_decode_shared(cache, q, table, lens, 0.1, p))
        graphs.append(g)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, g in zip(side, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan)
        on = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan, stream=side[0])
    torch.cuda.synchronize()
    for o in (*outs, eager, on):
        check(o.view(want.shape).double().cpu().numpy(), want, values)


def test_bad_pages_are_flagged(gq):
    """A shared entry that is no page: flagged; rows outside the group are as they were."""
    bt = shared.batch([(9, [150, 160])], [40], 14)
    cache, values = shared.pool("bf16", bt.pages, 2, 128, 15, gq)
    q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(16)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    lead = plan.rows.tolist()[0]
    for bad in (-1, bt.pages, 2 ** 31 - 1):
        broken = table.clone()
        broken[lead, 4] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), broken, lens, 0.1, plan, err=err)
        assert int(err) == gq.GQA_DEVERR_BLOCK_INDEX
        assert torch.isfinite(got).all()
        alone = [b for b in range(3) if b not in plan.rows.tolist()[:2]][0]
        want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
        check(got.view(q.shape).double().cpu().numpy()[[alone]], want[[alone]], values)


def test_lengths_out_of_range_are_flagged(gq):
    bt = shared.batch([(9, [150, 160, 170])], [], 17)
    cache, values = shared.pool("bf16", bt.pages, 2, 128, 18, gq)
    q = torch.randn(3, 1, 8, 128, generator=torch.Generator().manual_seed(19)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    for bad in (-5, 16 * bt.table.shape[1] + 1):
        now = lens.clone()
        now[1] = bad
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, now, 0.1, plan, err=err)
        assert int(err) == gq.GQA_DEVERR_CONTEXT_LEN
        check(got.view(q.shape).double().cpu().numpy()[[0, 2]], want[[0, 2]], values)


def test_plans_that_point_astray_share_nothing(gq):
    """Entries outside the plan or the tables: every row attends alone, or as its entries say."""
    bt = shared.batch([(9, [150, 160, 170])], [60], 20)
    cache, values = shared.pool("bf16", bt.pages, 2, 128, 21, gq)
    B = len(bt.lens)
    q = torch.randn(B, 1, 8, 128, generator=torch.Generator().manual_seed(22)).bfloat16()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    for part, value in (("count", 0), ("count", -3), ("start", -7), ("start", 10 ** 6), ("blocks", 0), ("blocks", -1),
                        ("blocks", 10 ** 6), ("slot", -1), ("slot", 10 ** 6), ("group", 10 ** 6), ("group", -2),
                        ("rows", 10 ** 6), ("rows", -9)):
        plan = gq.kv_pages_groups(table, lens)
        getattr(plan, part).fill_(value)
        got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, 0.1, plan)
        check(got.view(q.shape).double().cpu().numpy(), want, values)


def test_plan_of_overlapping_groups(gq):
    """Every group over all rows: what comes out is not defined, that nothing is read astray is."""
    B, blocks = 64, 40
    bt = shared.batch([(blocks, [16 * blocks + 1 + i for i in range(B)])], [], 26)
    cache, values = shared.pool("bf16", bt.pages, 2, 64, 27, gq)
    q = torch.randn(B, 8, 64, generator=torch.Generator().manual_seed(28)).bfloat16().cuda()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    good = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan)
    plan.count.fill_(B)
    plan.start.copy_(torch.tensor([0, B] * (B // 2) + [0]))
    plan.blocks.fill_(blocks)
    plan.group.copy_(2 * (torch.arange(B) // 2))
    bad = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan)
    torch.cuda.synchronize()
    assert bad.shape == good.shape
    assert torch.equal(gq.gqa_decode_shared(cache, q, table, lens, 0.1, gq.kv_pages_groups(table, lens)), good)


def test_plan_written_by_the_caller(gq):
    """Two of three rows that share pages, over fewer pages than they have in common."""
    bt = shared.batch([(9, [150, 160, 170])], [60], 23)
    cache, values = shared.pool("f16", bt.pages, 2, 64, 24, gq)
    B = len(bt.lens)
    q = torch.randn(B, 2, 8, 64, generator=torch.Generator().manual_seed(25)).half()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    kin = sorted(plan_rows for plan_rows in gq.kv_pages_groups(table, lens).rows.tolist() if plan_rows >= 0)
    a, b = kin[2], kin[0]
    plan = gq.kv_pages_groups(table, lens)
    plan.count.copy_(torch.tensor([1, 2]))
    plan.start.fill_(2)
    plan.start[0] = 0
    plan.blocks.fill_(0)
    plan.blocks[0] = 5
    plan.rows.copy_(torch.tensor([a, b] + [-1] * (B - 2)))
    plan.slot.fill_(-1)
    plan.group.fill_(-1)
    plan.slot[a], plan.slot[b] = 0, 1
    plan.group[a], plan.group[b] = 0, 0
    got = gq.gqa_decode_shared(cache, q.cuda(), table, lens, 0.1, plan)
    want = shared.attend(q.double().numpy(), values, bt.table, bt.lens, 0.1)
    check(got.double().cpu().numpy(), want, values)


def test_steps_after_a_fork(gq):
    """fork, the plan, then steps of append and shared decode, against plain decode."""
    K, G, d, B = 2, 4, 128, 6
    cache = gq.PagedKVCache.allocate(128, K, d, torch.bfloat16)
    refs = torch.zeros(128, dtype=torch.int32, device="cuda")
    table = torch.full((B, 24), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(26)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    n = torch.tensor([203] + [0] * (B - 1), dtype=torch.int32, device="cuda")
    gq.kv_pages_reserve(refs, table, lens, n)
    gq.kv_append_varlen(cache, rand(203, K, d), rand(203, K, d),
                        torch.tensor([0] + [203] * B, dtype=torch.int32, device="cuda"), 203, table, lens)
    lens += n
    child = torch.arange(1, B, dtype=torch.int32, device="cuda")
    copies = gq.kv_pages_fork(refs, table, lens, torch.zeros_like(child), child)
    gq.kv_copy_pages(cache, copies)
    plan = gq.kv_pages_groups(table, lens)
    assert plan.count.tolist() == [1, B] and plan.blocks.tolist()[0] == 203 // 16
    for step in range(20):
        gq.kv_pages_reserve(refs, table, lens, 1)
        gq.kv_append(cache, rand(B, K, d), rand(B, K, d), table, lens)
        lens += 1
        q = rand(B, K * G, d)
        a = gq.gqa_decode_shared(cache, q, table, lens, 0.09, plan)
        b = gq.gqa_decode(cache, q, table, lens, 0.09)
        assert float((a - b).abs().max()) <= 2 * 5 * 2.0 ** -11, step
