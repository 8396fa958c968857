"""Prefill with sink tokens: what the softmax weights are held to for every output type.

Bound. A score errs by at most d 2^-24 sum |q_i k_i| scale (fp32 sums of exact products)
and by 2^-22 |s| where it is scaled, exp2 by 2^-22, the row's sum of n terms by n 2^-24; P
is kept as two 16-bit parts, 2^-16 of itself. Such a relative error e of every weight moves
the output by e (sum w |v| + |out|) at most, P.V's own fp32 sum by n 2^-24 sum w |v|, and the
store rounds by half a step of the output's type (below 2^-14, f16: 2^-25)."""
import numpy as np
import pytest
import torch

from plain import cached_rows
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
