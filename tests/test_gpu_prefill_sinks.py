"""Prefill with sink tokens: what the softmax weights are held to for every output type,
batches whose CTAs walk many items, and cache layouts other than the pool's.

Bound. A score errs by at most d 2^-24 sum |q_i k_i| scale (fp32 sums of exact products)
and by 2^-22 |s| where it is scaled, exp2 by 2^-22, the row's sum of n terms by n 2^-24; P
is kept as two 16-bit parts, 2^-16 of itself. Such a relative error e of every weight moves
the output by e (sum w |v| + |out|) at most, P.V's own fp32 sum by n 2^-24 sum w |v|, and the
store rounds by half a step of the output's type (below 2^-14, f16: 2^-25)."""
import numpy as np
import pytest
import torch

import gqa_inputs as gi
from helpers import TOL, max_abs_err
from plain import attend, cached_rows
from test_gpu_sinks import _prefill, _prefill_case, _prefill_reference, gq  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def _allowed(case, q, news, window, sinks, out_dtype, ref):
    spread = _prefill_reference(case, q, news, window, sinks, magnitude=True)
    qh, row, s_abs, longest = np.abs(q.double().cpu().numpy()), 0, 0.0, 0
    for b, n in enumerate(news):
        k = np.abs(cached_rows(case, "k", b))
        G = q.shape[1] // k.shape[1]
        for h in range(q.shape[1] if n else 0):
            s_abs = max(s_abs, float((qh[row:row + n, h] @ k[:, h // G].T).max()) * case.scale)
        row, longest = row + n, max(longest, k.shape[0])
    seen = min(longest, window + sinks)
    e = s_abs * (q.shape[2] * 2.0 ** -24 + 2.0 ** -22) + 2.0 ** -22 + seen * 2.0 ** -24 + 2.0 ** -16
    step = torch.finfo(out_dtype).eps / 2
    return 1.01 * (e * (spread + np.abs(ref)) + seen * 2.0 ** -24 * spread) * (1 + step) + step * np.abs(ref) + 2.0 ** -25


@pytest.mark.parametrize("kernel,d", [(0, 128), (3, 128), (4, 128), (1, 128), (2, 128), (0, 64), (1, 64)])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", torch.float16), ("bf16", torch.bfloat16), ("f16", torch.float16),
                                             ("f16", torch.bfloat16), ("bf16", torch.float32)])
def test_weights_hold_the_same_for_every_output_type(gq, dtype, out_dtype, kernel, d):  # noqa: F811
    news, prior = [70, 1, 200, 33], [100, 300, 0, 555]
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, 8, 2, d, dtype, seed=61)
    for window, sinks in ((1, 1), (4, 3), (90, 7)):
        ref = _prefill_reference(case, q, news, window, sinks)
        out = _prefill(gq, case, q, start, news, window=window, sinks=sinks, out_dtype=out_dtype, kernel=kernel)
        off = np.abs(out.double().cpu().numpy() - ref) - _allowed(case, q, news, window, sinks, out_dtype, ref)
        assert off.max() <= 0, (window, sinks, off.max())


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kernel,d", [(3, 128), (4, 128), (0, 128), (0, 64), (1, 128), (1, 64)])
def test_even_batches_walk_many_items_per_cta(gq, kernel, d, out_dtype):  # noqa: F811
    """Equal lengths and more (tile, kv-head, sequence) items than CTAs, so that a CTA
    carries its ring and its barriers from one item to the next; the items of a sequence
    that has seen nothing yet, of one behind its sinks and of one in between follow each other."""
    B, n, H, K = 40, 128, 32, 8
    prior = [(0, 33, 150, 7, 64)[b % 5] for b in range(B)]
    case, q, start = _prefill_case([n + p for p in prior], [n] * B, H, K, d, "bf16", seed=62)
    full = _prefill_reference(case, q, [n] * B, 33, 17)
    out = _prefill(gq, case, q, start, [n] * B, window=33, sinks=17, out_dtype=out_dtype, kernel=kernel)
    step = 0.0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2
    assert np.all(np.abs(out.double().cpu().numpy() - full) <= TOL + step * np.abs(full))


@pytest.mark.parametrize("kernel,d", [(3, 128), (4, 128), (0, 64)])
def test_the_schedule_changes_no_result(gq, kernel, d):  # noqa: F811
    """Ragged rows with and without the host's count of them: a CTA per item, and a few
    persistent CTAs with many items each."""
    import ctypes
    rng = np.random.default_rng(63)
    news = rng.integers(0, 121, size=40).tolist()
    news[3] = 120
    lens = [n + int(p) for n, p in zip(news, rng.integers(0, 150, size=40))]
    case, q, start = _prefill_case(lens, news, 32, 8, d, "bf16", seed=64)
    want = _prefill(gq, case, q, start, news, window=33, sinks=17, kernel=kernel)
    desc, out = gq.cache_from_case(case).desc(), torch.full_like(want, float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = gq.load().gqa_prefill_sinks(ctypes.byref(desc), q.data_ptr(), gq.DTYPE_CODE[q.dtype], 32, start.data_ptr(),
                                     max(news), case.block_table.data_ptr(), case.block_table.shape[1],
                                     case.context_lens.data_ptr(), len(news), case.scale, 33, 17, 0, out.data_ptr(), 0,
                                     kernel, err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and int(err.item()) == 0 and torch.equal(out, want)


def _permuted(gq, case, order):  # noqa: F811
    """The case's pool with its outer axes (block, kv-head, slot) laid out in `order`."""
    def lay(t):
        return t.permute(*order, 3).contiguous()
    k, v = lay(case.k_cache), lay(case.v_cache)
    stride = [0, 0, 0]
    for axis, at in zip(order, k.stride()):
        stride[axis] = at
    return gq.PagedKVCache(k, v, case.num_blocks, case.num_kv_heads, case.head_dim, *stride)


@pytest.mark.parametrize("order", [(0, 2, 1), (1, 0, 2), (2, 0, 1), (1, 2, 0), (2, 1, 0)])
@pytest.mark.parametrize("kernel,d", [(0, 64), (1, 64), (2, 64), (3, 128), (4, 128), (1, 128), (2, 128)])
def test_layouts_of_other_axis_orders(gq, kernel, d, order):  # noqa: F811
    news, prior = [40, 7, 100], [60, 300, 13]
    lens = [n + p for n, p in zip(news, prior)]
    case, q, start = _prefill_case(lens, news, 8, 4, d, "bf16", seed=65)
    ref = _prefill_reference(case, q, news, 50, 20)
    out = gq.gqa_prefill(_permuted(gq, case, order), q, start, max(news), case.block_table, case.context_lens, case.scale,
                         window=50, sinks=20, kernel=kernel)
    torch.cuda.synchronize()
    assert max_abs_err(out, ref) <= TOL


@pytest.mark.parametrize("kernel,d", [(0, 64), (1, 64), (3, 128), (4, 128)])
def test_the_unpaged_layout(gq, kernel, d):  # noqa: F811
    news, prior = [40, 7, 100], [60, 300, 13]
    lens = [n + p for n, p in zip(news, prior)]
    case = gi.make_case(3, 8, 2, d, lens, "bf16", seed=66, device="cuda", contiguous=True)
    q = torch.randn((sum(news), 8, d), generator=torch.Generator(device="cuda").manual_seed(67), device="cuda")
    q = q.to(torch.bfloat16)
    start = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    ref = np.concatenate([attend(q.double().cpu().numpy()[s:s + n], cached_rows(case, "k", b), cached_rows(case, "v", b),
                                 case.scale, 50, 20) for b, (s, n) in enumerate(zip(start.tolist(), news))])
    assert max_abs_err(_prefill(gq, case, q, start, news, window=50, sinks=20, kernel=kernel), ref) <= TOL
