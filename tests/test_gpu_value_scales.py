"""Decode over coded caches whose V rows are small, large or of mixed sizes: the softmax
weights times V's scales go through 16-bit parts, which must not depend on how large V is.

Bound. A score errs by at most d 2^-24 sum |q_i k_i| scale (fp32 sums) and 2^-22 of itself;
what q loses as fp16 below 2^-14, and with K's channel scales as two parts, is 2^-25 of an
element of K's row or of its codes (at most 7 each); exp2 errs by 2^-22 and its argument, below
27 + 8 for scales of 2^-24 and a maximum 2^8 times the one of the last rescale, by 2^-19, the
row's sum by n 2^-24; a weight times its scale is kept as two fp16 parts, 2^-21 of itself, or,
the largest scale being put above 2^3 and half the low part's step being 2^-25, 2^-28 of that
one. Weights off by e move the output by e (sum w |v| +
|out|), the sums of P.V and over the splits by n 2^-24 sum w |v|."""
import numpy as np
import pytest
import torch

import gqa_inputs as gi
from plain import attend, cached_rows

pytestmark = pytest.mark.gpu

LENS = [1, 5, 16, 33, 100, 0, 1000]


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def _scale_v(case, sizes):
    """Multiply V's scales by 2^sizes, a number or a rule of (sequence length, token)."""
    if not callable(sizes):
        case.v_scale.mul_(2.0 ** sizes)
        return
    for b, L in enumerate(case.context_lens.tolist()):
        for t in range(L):
            case.v_scale[int(case.block_table[b, t // 16]), :, t % 16] *= 2.0 ** sizes(L, t)


def _reference(case, window, sinks):
    """fp64 output and its bound, both [B, T, H, d]."""
    q = case.q.double().cpu().numpy()
    q = q[:, None] if q.ndim == 3 else q
    ref, bound = np.zeros(q.shape), np.zeros(q.shape)
    d, T, H = case.head_dim, q.shape[1], q.shape[2]
    for b, L in enumerate(case.context_lens.tolist()):
        if L == 0:
            continue
        k, v = cached_rows(case, "k", b), cached_rows(case, "v", b)
        n = min(T, L)
        qb = q[b, T - n:]
        out = attend(qb, k, v, case.scale, window, sinks)
        spread = attend(qb, k, np.abs(v), case.scale, window, sinks)
        G = H // k.shape[1]
        s_abs = max(float((np.abs(qb[:, h]) @ np.abs(k[:, h // G]).T).max()) for h in range(H)) * case.scale
        k_abs = float(np.abs(k).sum(-1).max()) + 7 * d
        seen = L if window == 0 else min(L, window + sinks + 16)
        e = s_abs * (d * 2.0 ** -24 + 2.0 ** -22) + k_abs * case.scale * 2.0 ** -25 + 2.0 ** -19 + 2.0 ** -22 + seen * 2.0 ** -24 \
            + 2.0 ** -21
        ref[b, T - n:] = out
        bound[b, T - n:] = 1.01 * e * (spread + np.abs(out)) + seen * (2.0 ** -24 * spread + 2.0 ** -28 * np.abs(v).max()) \
            + 2.0 ** -140
    return ref, bound


SIZES = {"2^-10": -10, "2^-16": -16, "2^10": 10, "2^16": 16,
         "grows": lambda L, t: -14 + t // 16 % 20, "shrinks": lambda L, t: 4 - t // 16 % 19,
         "mixed": lambda L, t: (t * 7919 % 21) - 16, "one large": lambda L, t: 0 if t == L // 2 else -14}


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("H,K,T,window,sinks,kw", [
    (16, 4, 1, 0, 0, {}), (16, 4, 1, 40, 0, {}), (16, 4, 1, 40, 20, dict(max_warps=3, min_blocks_per_warp=1)),   # <= 8 rows
    (24, 2, 1, 0, 0, {}), (32, 4, 2, 40, 0, dict(row_layout=1)), (32, 4, 2, 40, 20, {}),                         # 9 .. 16
    (32, 4, 2, 300, 4, dict(max_warps=3, min_blocks_per_warp=1)), (16, 2, 3, 0, 0, {}), (16, 2, 3, 40, 20, {})])  # 16, 24
@pytest.mark.parametrize("dtype", ["fp8", "i8", "i4", "i4kc"])
def test_weights_do_not_depend_on_the_size_of_v(gq, dtype, H, K, T, window, sinks, kw, sizes):
    case = gi.make_case(len(LENS), H, K, 128, LENS, dtype, seed=71, device="cuda", queries=T)
    _scale_v(case, SIZES[sizes])
    ref, bound = _reference(case, window, sinks)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = gq.gqa_decode(gq.cache_from_case(case), case.q, case.block_table, case.context_lens, case.scale, window=window,
                        sinks=sinks, err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    off = np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) - bound
    assert off.max() <= 0, off.max() / max(float(np.abs(ref).max()), 1e-30)


@pytest.mark.parametrize("dtype", ["fp8", "i8", "i4"])
def test_rows_as_the_append_quantises_them(gq, dtype):
    """V rows of amax ~7e-4 and ~7e-6 next to each other, written by the append; the
    reference reads the codes and scales that it left."""
    lens, K, d = [40, 200], 4, 128
    case = gi.make_case(2, 16, K, d, lens, dtype, seed=72, device="cuda", source="normal")
    case.v_src.mul_(2.5e-4)
    case.v_src[1::2].mul_(1e-2)
    from helpers import fill_from_source
    fill_from_source(gq, case)
    ref, bound = _reference(case, 0, 0)
    out = gq.gqa_decode(gq.cache_from_case(case), case.q, case.block_table, case.context_lens, case.scale)
    torch.cuda.synchronize()
    assert np.all(np.abs(out.double().cpu().numpy().reshape(ref.shape) - ref) <= bound)
