"""What a shared decode sees of the work in front of it: its three kernels overlap, and the
one over the rows' own blocks begins while the one over the shared blocks runs."""
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


@pytest.mark.parametrize("kind,T", [("bf16", 1), ("f16", 3), ("int8", 1)])
@pytest.mark.parametrize("captured", [False, True])
def test_inputs_written_right_before_the_call(gq, kind, T, captured):
    """Tables, lengths, queries and the plan change in the kernels right in front of every step,
    back to back: each step gives the bits that it gives alone."""
    K, G, d, B, steps = 2, 4, 128, 12, 60
    bt = shared.batch([(30, [490 + i for i in range(B)])], [], 90)
    wide = bt.table.shape[1]
    cache, values = shared.pool(kind, bt.pages, K, d, 91, gq)
    gen = torch.Generator().manual_seed(92)
    dt = shared.DTYPES.get(kind, torch.bfloat16)
    base, lens0 = torch.from_numpy(bt.table), torch.from_numpy(bt.lens)
    order = [torch.randperm(B, generator=gen) for _ in range(steps)]     # rows change places, lengths too
    tables = torch.stack([base[o] for o in order]).cuda()
    lens = torch.stack([lens0[o] - int(torch.randint(0, 8, (1,), generator=gen)) for o in order]).cuda()
    q = torch.randn(steps, B, T, K * G, d, generator=gen).to(dt).cuda()
    q = q if T > 1 else q[:, :, 0].contiguous()
    t, L, x = torch.empty_like(tables[0]), torch.empty_like(lens[0]), torch.empty_like(q[0])
    plan = gq.kv_pages_groups(tables[0], lens[0])
    out = torch.empty(steps, *x.shape, device="cuda")
    ws = torch.zeros(gq.decode_shared_workspace_size(B, K * G, K, d, tokens_per_seq=T), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(i, o):
        t.copy_(tables[i])
        L.copy_(lens[i])
        x.copy_(q[i])
        gq.kv_pages_groups(t, L, groups=plan, err=err)
        gq.gqa_decode_shared(cache, x, t, L, 0.09, plan, out=o, workspace=ws, err=err)

    alone = torch.empty_like(out)
    for i in range(steps):
        step(i, alone[i])
        torch.cuda.synchronize()
        assert not ws[160:164].any()                              # the word between the kernels is clear again
    run = lambda: [step(i, out[i]) for i in range(steps)]  # noqa: E731
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        run = g.replay
    for _ in range(5):
        out.fill_(float("nan"))
        run()
        torch.cuda.synchronize()
        assert int(err) == 0
        assert torch.equal(out, alone)
    i = steps - 1
    want = shared.attend(q[i].view(B, T, K * G, d).double().cpu().numpy(), values, tables[i].cpu().numpy(), lens[i].cpu().numpy(), 0.09)
    assert np.abs(out[i].view(want.shape).double().cpu().numpy() - want).max() <= np.abs(values[1]).max() * 2.0 ** -11


def test_a_workspace_serves_both_decodes_in_turn(gq):
    """Header words that one call leaves set would let the next begin early, or never."""
    bt = shared.batch([(30, [500 + i for i in range(7)])], [40], 8)
    cache, _ = shared.pool("bf16", bt.pages, 4, 128, 9, gq)
    B = len(bt.lens)
    q = torch.randn(B, 16, 128, generator=torch.Generator().manual_seed(10)).bfloat16().cuda()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    ws = torch.zeros(gq.decode_shared_workspace_size(B, 16, 4, 128), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = None
    for i in range(12):
        a = gq.gqa_decode(cache, q, table, lens, 0.1, workspace=ws, err=err)
        b = gq.gqa_decode_shared(cache, q, table, lens, 0.1, plan, workspace=ws, err=err)
        first = first or (a, b)
        assert torch.equal(a, first[0]) and torch.equal(b, first[1])
        assert int(ws[128:164].view(torch.int32)[0]) == 0 and int(ws[160:164].view(torch.int32)[0]) == 0
    assert int(err) == 0


def test_a_plan_of_no_rows_is_cleared_on_the_calls_stream(gq):
    table = torch.full((0, 4), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    plan = gq.kv_pages_groups(table, lens)
    assert plan.count.tolist() == [0, 0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)          # 10 ms
        plan.plan.fill_(7)
    gq.kv_pages_groups(table, lens, groups=plan, stream=side)
    torch.cuda.synchronize()
    assert plan.count.tolist() == [0, 0]
    made = gq.kv_pages_groups(table, lens, stream=side)
    side.synchronize()
    assert made.count.tolist() == [0, 0] and made.start.tolist() == [0]
