"""Attention with a sliding window whose first tokens stay visible, decode and
prefill, against the plain fp64 form, through the C ABI.

Bound on fp32 output. With N(0, 1) inputs a score in log2 units errs by at most
d 2^-24 sum |q_i k_i| scale log2(e) ~ 8e-5 (d = 128, sum ~ 82), so a weight by a
relative 1.1e-4; its row sum of n <= 4000 fp32 terms by n 2^-24 = 2.4e-4; P is
kept as two 16-bit parts (2^-16). Times max |v| ~ 5: 1.9e-3 < 2e-3."""
import numpy as np
import pytest
import torch

import gqa_inputs as gi
from helpers import TOL, max_abs_err
from plain import attend, attend_case, cached_rows

pytestmark = pytest.mark.gpu

LENS = [1, 5, 15, 16, 17, 31, 33, 100, 300, 0, 1000]
POISON = 1 << 20                  # a block index outside every pool


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def _decode(gq, case, table=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gq.gqa_decode(gq.cache_from_case(case), case.q, case.block_table if table is None else table,
                        case.context_lens, case.scale, err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


def _poisoned(case, window, sinks, new):
    """The case's table with every block that no query sees made unreadable."""
    table = case.block_table.clone()
    for b, (L, n) in enumerate(zip(case.context_lens.tolist(), new)):
        for j in range(table.shape[1]):
            if 16 * j >= sinks and 16 * (j + 1) <= L - n + 1 - window:
                table[b, j] = POISON
    return table


@pytest.mark.parametrize("window,sinks", [(1, 1), (5, 4), (16, 16), (17, 33), (40, 4), (100, 128), (40, 2000),
                                          (4096, 4)])
@pytest.mark.parametrize("dtype,kernel,d", [("bf16", 1, 128), ("bf16", 2, 128), ("f16", 1, 64), ("f32", 2, 64),
                                            ("i8", 1, 128), ("fp8", 1, 128), ("fp8", 2, 64), ("i4", 1, 128),
                                            ("i4kc", 1, 128), ("i4kc", 2, 128)])
def test_decode_matches_the_plain_form(gq, dtype, kernel, d, window, sinks):
    case = gi.make_case(len(LENS), 16, 4, d, LENS, dtype, seed=31, device="cuda")
    ref = attend_case(case, window, sinks)
    table = _poisoned(case, window, sinks, [1] * len(LENS))
    for mw in (0, 3):                                   # many and few splits of a sequence
        out = _decode(gq, case, table, kernel=kernel, window=window, sinks=sinks, max_warps=mw, min_blocks_per_warp=1)
        assert max_abs_err(out, ref) <= TOL, mw


@pytest.mark.parametrize("layout", [0, 1, 2])
@pytest.mark.parametrize("H,K,T,dtype,d", [(32, 8, 2, "bf16", 128), (64, 8, 8, "bf16", 128), (8, 8, 4, "f16", 64),
                                           (24, 8, 3, "fp8", 128), (32, 4, 8, "i8", 128), (6, 2, 5, "f32", 64)])
def test_several_new_tokens(gq, H, K, T, dtype, d, layout):
    lens = [1, T, 16, 40, 257, 0, 600]
    case = gi.make_case(len(lens), H, K, d, lens, dtype, seed=32, device="cuda", queries=T)
    for window, sinks in ((7, 3), (33, 20), (100, 16)):
        ref = attend_case(case, window, sinks)
        table = _poisoned(case, window, sinks, [T] * len(lens))
        out = _decode(gq, case, table, window=window, sinks=sinks, row_layout=layout)
        assert max_abs_err(out, ref) <= TOL, (window, sinks)


@pytest.mark.parametrize("H,K,T", [(36, 4, 1), (16, 1, 1), (20, 4, 3), (16, 2, 2), (2, 2, 11), (80, 8, 1)])
@pytest.mark.parametrize("dtype", ["i8", "fp8", "i4"])
def test_nine_to_sixteen_rows_of_coded_caches(gq, dtype, H, K, T):
    """One warp serves the 16 rows of a pair: every layout, few and many splits, tokens
    that nobody sees behind NaN scales, rows past G T, empty sequences."""
    lens = [1, T, 15, 16, 17, 40, 257, 0, 601, 90]
    case = gi.make_case(len(lens), H, K, 128, lens, dtype, seed=40 + H, device="cuda", queries=T)
    for window, sinks in ((1, 1), (7, 3), (33, 20), (100, 16), (40, 2000)):
        ref = attend_case(case, window, sinks)
        table = _poisoned(case, window, sinks, [T] * len(lens))
        for kw in (dict(), dict(max_warps=3, min_blocks_per_warp=1), dict(min_blocks_per_warp=1), dict(row_layout=2)):
            out = _decode(gq, case, table, window=window, sinks=sinks, **kw)
            assert max_abs_err(out, ref) <= TOL, (window, sinks, kw)
    W, S = 21, 5
    ref = attend_case(case, W, S)
    for b, L in enumerate(lens):
        seen_from = L - T + 1 - W
        for t in range(S, max(0, seen_from)):
            p = int(case.block_table[b, t // 16])
            case.k_scale[p, :, t % 16] = float("nan")
            case.v_scale[p, :, t % 16] = float("nan")
        for t in range(L, -(-L // 16) * 16):
            p = int(case.block_table[b, t // 16])
            case.k_scale[p, :, t % 16] = float("nan")
            case.v_scale[p, :, t % 16] = float("nan")
    assert max_abs_err(_decode(gq, case, window=W, sinks=S), ref) <= TOL
    for t, eps in ((torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)):
        got = _decode(gq, case, window=W, sinks=S, out_dtype=t).double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= TOL + np.abs(ref) * eps)


def test_a_scratch_without_room_for_the_sixteen_row_workers(gq):
    """880 x 8 pairs of 16 rows and 1216 workers exceed the 64 MB scratch, 608 do not."""
    lens = [5 + b % 60 for b in range(880)]
    case = gi.make_case(len(lens), 64, 8, 128, lens, "fp8", seed=39, device="cuda", queries=2)
    want = _decode(gq, case, window=30, sinks=4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.gqa_decode_noalloc(gq.cache_from_case(case), case.q, case.block_table, case.context_lens, case.scale,
                                window=30, sinks=4, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and float((got - want).abs().max()) <= TOL
    part = [0, 1, 30, 59, 879]
    ref = attend_case(case, 30, 4)
    assert max(float(np.abs(got[b].double().cpu().numpy() - ref[b]).max()) for b in part) <= TOL


def test_no_sinks_and_no_window_are_the_calls_without(gq):
    case = gi.make_case(len(LENS), 32, 8, 128, LENS, "bf16", seed=33, device="cuda")
    assert torch.equal(_decode(gq, case, window=40, sinks=0), _decode(gq, case, window=40))
    assert torch.equal(_decode(gq, case, window=0, sinks=7), _decode(gq, case))
    # a window or sinks that reach over everything: full attention
    full = attend_case(case)
    assert max_abs_err(_decode(gq, case, window=5, sinks=10 ** 9), full) <= TOL
    assert max_abs_err(_decode(gq, case, window=2000, sinks=3), full) <= TOL


@pytest.mark.parametrize("dtype,kernel", [("bf16", 1), ("bf16", 2), ("fp8", 1), ("i8", 1), ("i4", 1)])
def test_tokens_that_left_the_window_may_hold_anything(gq, dtype, kernel):
    """NaN in K, V or scales of tokens that no query sees, inside blocks that are read."""
    W, S = 21, 5
    lens = [100, 333, 64]
    case = gi.make_case(len(lens), 16, 4, 128, lens, dtype, seed=34, device="cuda")
    ref = attend_case(case, W, S)
    for b, L in enumerate(lens):
        for t in list(range(S, 16)) + list(range((L - W) // 16 * 16, L - W)):
            p = int(case.block_table[b, t // 16])
            if dtype == "bf16":
                case.k_cache[p, :, t % 16] = float("nan")
                case.v_cache[p, :, t % 16] = float("nan")
            else:
                case.k_scale[p, :, t % 16] = float("nan")
                case.v_scale[p, :, t % 16] = float("nan")
    assert max_abs_err(_decode(gq, case, kernel=kernel, window=W, sinks=S), ref) <= TOL


def test_long_streams_match_on_a_full_batch(gq):
    """Many sequences, the window far behind the sinks, half-precision output."""
    lens = [1500 + 37 * i for i in range(24)]
    case = gi.make_case(len(lens), 32, 8, 128, lens, "bf16", seed=35, device="cuda")
    out = _decode(gq, case, window=700, sinks=4, out_dtype=torch.bfloat16)
    ref = attend_case(case, 700, 4)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= TOL + np.abs(ref) * 2.0 ** -8)


def test_unpaged_layout(gq):
    lens = [77, 200, 3]
    case = gi.make_case(len(lens), 8, 2, 64, lens, "f32", seed=36, device="cuda", contiguous=True)
    assert max_abs_err(_decode(gq, case, window=30, sinks=9), attend_case(case, 30, 9)) <= TOL


def test_captured_decode_replays_on_new_inputs(gq):
    lens = [130, 400]
    case = gi.make_case(len(lens), 16, 4, 128, lens, "bf16", seed=37, device="cuda", extra_tokens=64)
    cache = gq.cache_from_case(case)
    ws = torch.zeros(gq.decode_workspace_size(2, 16, 4, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty(case.q.shape, device="cuda")
    call = lambda: gq.gqa_decode(cache, case.q, case.block_table, case.context_lens, case.scale, out=out,  # noqa: E731
                                 workspace=ws, window=60, sinks=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in (0, 1, 2):
        case.q.normal_(generator=torch.Generator(device="cuda").manual_seed(step))
        graph.replay()
        torch.cuda.synchronize()
        assert max_abs_err(out, attend_case(case, 60, 4)) <= TOL, step
        case.context_lens -= 17                          # the graph reads the lengths on the device


def test_graphs_captured_on_one_stream_do_not_share_a_workspace(gq):
    """Two graphs without a workspace of the caller's, the second replayed first and then
    both at once on streams of their own."""
    side = torch.cuda.Stream()
    made = []
    for seed, lens in ((51, [900, 3000]), (52, [2500, 40])):
        case = gi.make_case(2, 16, 4, 128, lens, "bf16", seed=seed, device="cuda")
        cache, out = gq.cache_from_case(case), torch.full(case.q.shape, float("nan"), device="cuda")
        gq.load()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            gq.gqa_decode(cache, case.q, case.block_table, case.context_lens, case.scale, out=out, window=600, sinks=4)
        made.append((graph, case, cache, out, attend_case(case, 600, 4)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    made[1][0].replay()
    torch.cuda.synchronize()
    assert max_abs_err(made[1][3], made[1][4]) <= TOL
    for _ in range(20):
        for s, (graph, *_rest) in zip(streams, made):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, _, out, ref in made:
        assert max_abs_err(out, ref) <= TOL


def test_noalloc_gives_the_same_bits(gq):
    case = gi.make_case(len(LENS), 32, 8, 128, LENS, "bf16", seed=38, device="cuda")
    a = _decode(gq, case, window=40, sinks=4)
    b = gq.gqa_decode_noalloc(gq.cache_from_case(case), case.q, case.block_table, case.context_lens, case.scale,
                              window=40, sinks=4)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


# --------------------------------------------------------------------------- prefill


def _prefill_case(lens, news, H, K, d, dtype, seed):
    case = gi.make_case(len(lens), H, K, d, lens, dtype, seed=seed, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn((sum(news), H, d), generator=g, device="cuda").to(gi.DTYPES[dtype])
    start = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    return case, q, start


def _prefill_reference(case, q, news, window, sinks, magnitude=False):
    """Output rows, or with ``magnitude`` the same weights over |v|."""
    qh = q.double().cpu().numpy()
    out, row = [], 0
    for b, n in enumerate(news):
        if n:
            v = cached_rows(case, "v", b)
            out.append(attend(qh[row:row + n], cached_rows(case, "k", b), np.abs(v) if magnitude else v, case.scale, window,
                              sinks))
        row += n
    return np.concatenate(out)


def _prefill(gq, case, q, start, news, table=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gq.gqa_prefill(gq.cache_from_case(case), q, start, max(news), case.block_table if table is None else table,
                         case.context_lens, case.scale, err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    return out


@pytest.mark.parametrize("kernel", [0, 3, 4, 1, 2])
@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (37, 20), (37, 100), (200, 64), (200, 65), (64, 5000)])
def test_prefill_matches_the_plain_form(gq, kernel, window, sinks):
    news = [3, 64, 129, 300, 0, 1]
    prior = [10, 0, 77, 456, 20, 391]
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, 8, 2, 128, "bf16", seed=41)
    ref = _prefill_reference(case, q, news, window, sinks)
    table = _poisoned(case, window, sinks, news)
    assert max_abs_err(_prefill(gq, case, q, start, news, table, window=window, sinks=sinks, kernel=kernel), ref) <= TOL


@pytest.mark.parametrize("H,K,d,dtype", [(12, 4, 64, "f16"), (24, 8, 128, "f16"), (8, 1, 64, "bf16"), (5, 5, 128, "bf16")])
@pytest.mark.parametrize("kernel", [0, 2])
def test_prefill_group_sizes_and_types(gq, H, K, d, dtype, kernel):
    news = [1, 40, 130, 7]
    prior = [200, 9, 333, 100]
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, H, K, d, dtype, seed=42)
    ref = _prefill_reference(case, q, news, 50, 6)
    assert max_abs_err(_prefill(gq, case, q, start, news, window=50, sinks=6, kernel=kernel), ref) <= TOL


@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (37, 20), (37, 100), (200, 64), (200, 65), (64, 5000)])
@pytest.mark.parametrize("H,K,dtype", [(12, 4, "f16"), (8, 2, "bf16")])
def test_prefill_of_64_element_heads(gq, H, K, dtype, window, sinks):
    news = [3, 64, 129, 300, 0, 1]
    prior = [10, 0, 77, 456, 20, 391]
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, H, K, 64, dtype, seed=47)
    ref = _prefill_reference(case, q, news, window, sinks)
    table = _poisoned(case, window, sinks, news)
    # a 16-bit output takes the weights rounded to the cache's type, each off by half a
    # step of itself: the output by half a step of sum w |v| at most, and of itself
    spread = _prefill_reference(case, q, news, window, sinks, magnitude=True)
    for out_dtype in (torch.float32, gi.DTYPES[dtype]):
        out = _prefill(gq, case, q, start, news, table, window=window, sinks=sinks, out_dtype=out_dtype)
        step = 0.0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2
        assert np.all(np.abs(out.double().cpu().numpy() - ref) <= TOL + step * (np.abs(ref) + spread))


@pytest.mark.parametrize("kernel,d", [(3, 128), (4, 128), (0, 64)])
def test_prefill_many_items_per_cta(gq, kernel, d):
    """More (tile, kv-head, sequence) items than CTAs: the walk over the sinks and
    the window starts anew for every item a CTA takes."""
    rng = np.random.default_rng(43)
    news = rng.integers(0, 121, size=40).tolist()
    news[3] = 120
    prior = rng.integers(0, 150, size=40).tolist()
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, 32, 8, d, "bf16", seed=44)
    ref = _prefill_reference(case, q, news, 33, 17)
    assert max_abs_err(_prefill(gq, case, q, start, news, window=33, sinks=17, kernel=kernel), ref) <= TOL


@pytest.mark.parametrize("kernel,d", [(0, 128), (1, 128), (2, 128), (4, 128), (0, 64), (1, 64)])
def test_prefill_hidden_tokens_may_hold_anything(gq, kernel, d):
    W, S = 21, 5
    news, lens = [9, 16], [120, 333]
    case, q, start = _prefill_case(lens, news, 8, 2, d, "bf16", seed=45)
    ref = _prefill_reference(case, q, news, W, S)
    for b, (L, n) in enumerate(zip(lens, news)):
        first = L - n + 1 - W
        for t in list(range(S, 16)) + list(range(first // 16 * 16, first)):
            p = int(case.block_table[b, t // 16])
            case.k_cache[p, :, t % 16] = float("nan")
            case.v_cache[p, :, t % 16] = float("inf")
    assert max_abs_err(_prefill(gq, case, q, start, news, window=W, sinks=S, kernel=kernel), ref) <= TOL


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", torch.bfloat16), ("f16", torch.float16), ("f16", torch.bfloat16)])
@pytest.mark.parametrize("kernel", [0, 3, 4, 1])
def test_prefill_half_outputs(gq, dtype, out_dtype, kernel):
    """Weights rounded once to the cache's type (see the 64-element heads above)."""
    news, prior = [70, 1, 200, 33], [100, 300, 0, 555]
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, 16, 4, 128, dtype, seed=48)
    ref = _prefill_reference(case, q, news, 90, 7)
    spread = _prefill_reference(case, q, news, 90, 7, magnitude=True)
    out = _prefill(gq, case, q, start, news, window=90, sinks=7, out_dtype=out_dtype, kernel=kernel)
    allowed = TOL + torch.finfo(out_dtype).eps / 2 * np.abs(ref) + torch.finfo(gi.DTYPES[dtype]).eps / 2 * spread
    assert np.all(np.abs(out.double().cpu().numpy() - ref) <= allowed)


@pytest.mark.parametrize("dtype", ["i8", "fp8", "i4", "i4kc"])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16])
def test_decode_half_outputs_of_code_caches(gq, dtype, T, out_dtype):
    """The fp32 output's bound and half a step of the output's own type."""
    lens = [1, 16, 40, 257, 0, 600]
    case = gi.make_case(len(lens), 32, 4, 128, lens, dtype, seed=39, device="cuda", queries=T)
    ref = attend_case(case, 50, 6)
    out = _decode(gq, case, window=50, sinks=6, out_dtype=out_dtype).double().cpu().numpy()
    assert np.all(np.abs(out - ref) <= TOL + torch.finfo(out_dtype).eps / 2 * np.abs(ref))


def test_prefill_last_token_is_the_decode(gq):
    news, lens = [50, 200], [360, 200]
    case, q, start = _prefill_case(lens, news, 32, 8, 128, "bf16", seed=46)
    out = _prefill(gq, case, q, start, news, window=70, sinks=4)
    case.q = torch.stack([q[int(start[b + 1]) - 1] for b in range(2)])
    one = _decode(gq, case, window=70, sinks=4)
    got = torch.stack([out[int(start[b + 1]) - 1] for b in range(2)])
    # the same sums in another order: twice the bound's sum and weight terms without the input rounding
    assert (got - one).abs().max().item() <= TOL
