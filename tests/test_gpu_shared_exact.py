"""The shared decode on inputs whose arithmetic is exact or nearly so: that every token counts once,
with its own weight, in every form of the kernels; that tokens of small V scales keep theirs; and
that a call repeats itself bit for bit.

K and V hold one-hot rows: token x of the pool (page * 16 + slot) and kv-head g has its one at
element (x + 5 g) mod d of V, so that an output's element is the share of the L / d tokens that end
there. A token left out, or taken twice, moves one element by d / L of itself: 2^-8 and more below,
where the bound is 2^-14."""
import math

import numpy as np
import pytest
import torch

import shared

pytestmark = pytest.mark.gpu

LN2 = float(np.float32(math.log(2.0)))


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def cache_of(gq, kind, k, v, k_scale=None, v_scale=None):
    """A cache of whole numbers k, v [pages, 16, K, d] (|x| <= 7), with scales [pages, 16, K] (1) where
    it is coded; and the values it holds."""
    pages, _, K, d = k.shape
    lie = lambda x: torch.from_numpy(np.ascontiguousarray(x.transpose(0, 2, 1, 3)))  # noqa: E731
    stride = (pages, K, d, K * 16 * d, 16 * d, d)
    if kind in shared.DTYPES:
        return gq.PagedKVCache(*(lie(x).to(shared.DTYPES[kind]).cuda() for x in (k, v)), *stride), [k, v]
    store, scales, held = [], [], []
    for x, s in ((k, k_scale), (v, v_scale)):
        s = np.ones(x.shape[:3]) if s is None else s
        code = lie(x)
        if kind == "int4":
            n = code.to(torch.int32) & 15
            code = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
        else:
            code = code.to(torch.int8 if kind == "int8" else torch.float8_e4m3fn)
        store.append(code.cuda())
        scales.append(torch.from_numpy(np.ascontiguousarray(s.transpose(0, 2, 1))).to(torch.float16).cuda())
        held.append(x * s[..., None])
    return gq.PagedKVCache(*store, *stride, *scales, gq.GQA_DTYPE_I4 if kind == "int4" else None), held


def one_hot(pages, K, d, step=1):
    x = np.zeros((pages, 16, K, d))
    p, s, g = np.meshgrid(np.arange(pages), np.arange(16), np.arange(K), indexing="ij")
    x[p, s, g, (step * (16 * p + s) + 5 * g) % d] = 1
    return x


KINDS = ["bf16", "f16", "int8", "fp8", "int4"]
SHAPES = [
    # K, G, d, T, groups (shared blocks, lengths), alone
    (1, 8, 128, 4, [(33, [532 + i for i in range(9)])], [40]),              # 288 query rows: more than two tiles
    (2, 8, 64, 1, [(20, [321 + i for i in range(40)])], []),                # 320
    (1, 4, 128, 1, [(1000, [16001, 16020, 16100])], []),                    # one kv-head over all SMs: continued pieces
    (2, 8, 64, 2, [(500, [8002 + 3 * i for i in range(10)])], [3, 0]),      # 160 rows: two tiles, the second part empty
    (1, 16, 128, 1, [(300, [4801 + i for i in range(40)])], [9]),           # 640 rows: three CTAs' tiles, each continued
    (3, 5, 64, 3, [(7, [115, 120]), (90, [1443, 1500, 1466]), (41, [660] * 12)], [100, 1]),
    (8, 1, 128, 1, [(129, [2065] * 3)], [17]),                              # a prefix that ends inside a step
]


def build(gq, kind, K, G, d, T, groups, alone, seed):
    bt = shared.batch(groups, alone, seed)
    q_dtype = shared.DTYPES.get(kind, torch.bfloat16)
    return bt, q_dtype, torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("max_group", [0, 1])                               # the two-tile form, and one tile a CTA
@pytest.mark.parametrize("K,G,d,T,groups,alone", SHAPES)
def test_every_token_counts_once(gq, kind, max_group, K, G, d, T, groups, alone):
    """K = 0: all weights are equal. They are a power of two, or off by 2^-22 together, so that an element's
    c <= L / d + 1 equal terms and the sum of L / 32 a thread round to less than 2^-14."""
    bt, q_dtype, table, lens = build(gq, kind, K, G, d, T, groups, alone, 50)
    v = one_hot(bt.pages, K, d)
    cache, _ = cache_of(gq, kind, np.zeros_like(v), v)
    q = torch.randn(len(bt.lens), T, K * G, d, generator=torch.Generator().manual_seed(51)).to(q_dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.gqa_decode_shared(cache, q.cuda() if T > 1 else q[:, 0].contiguous().cuda(), table, lens, 0.1,
                               gq.kv_pages_groups(table, lens), max_group=max_group, err=err)
    assert int(err) == 0
    got = got.view(q.shape).double().cpu().numpy()
    for b, L in enumerate(bt.lens.tolist()):
        ids = (16 * bt.table[b, np.arange(L) // 16] + np.arange(L) % 16).astype(np.int64)
        for i in range(T):
            n = L - T + i + 1
            for h in range(K * G):
                want = np.bincount((ids[:max(0, n)] + 5 * (h // G)) % d, minlength=d) / max(1, n)
                assert (np.abs(got[b, i, h] - want) <= 2.0 ** -14 * want).all(), (b, i, h)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("max_group", [0, 1])
@pytest.mark.parametrize("K,G,d,T,groups,alone", SHAPES[:2] + SHAPES[3:])
def test_weights_go_with_their_tokens(gq, kind, max_group, K, G, d, T, groups, alone):
    """Token x has its one at element 3 x + 5 g of K, q holds 0 .. -8 and the scale is ln 2: weights of
    2^0 .. 2^-8. Their exponents are off by 2^-19 (scale, maximum, merge), ex2 by 2^-22, the two 16-bit
    parts by 2^-16, the sums of at most 256 products a CTA by 2^-15: below 2^-14."""
    bt, q_dtype, table, lens = build(gq, kind, K, G, d, T, groups, alone, 52)
    k, v = one_hot(bt.pages, K, d, 3), one_hot(bt.pages, K, d)
    cache, held = cache_of(gq, kind, k, v)
    q = -torch.randint(0, 9, (len(bt.lens), T, K * G, d), generator=torch.Generator().manual_seed(53)).to(q_dtype)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = gq.gqa_decode_shared(cache, q.cuda() if T > 1 else q[:, 0].contiguous().cuda(), table, lens, LN2,
                               gq.kv_pages_groups(table, lens), max_group=max_group, err=err)
    assert int(err) == 0
    want = shared.attend(q.double().numpy(), held, bt.table, bt.lens, LN2)
    off = np.abs(got.view(q.shape).double().cpu().numpy() - want)
    assert (off <= 2.0 ** -14 * want).all(), float((off / np.maximum(want, 1e-30)).max())


@pytest.mark.parametrize("kind", ["int8", "fp8", "int4"])
@pytest.mark.parametrize("order", ["large-small-large", "small-large-small", "mixed"])
@pytest.mark.parametrize("d", [64, 128])
def test_tokens_of_small_scales_keep_theirs(gq, kind, order, d):
    """The queries look at tokens whose V scale is 2^-20, among tokens of scale 2^4 whose weights are 2^-60.
    A weight is off by at most 2^-30 of the largest (1) times the largest scale (2^4), so that an output,
    the mean of n of them times codes up to 7, is by 2^-30 2^4 7 L / n; its sums add 2^-14 of itself."""
    blocks, K, G = 60, 2, 8
    bt = shared.batch([(blocks, [16 * blocks + 5, 16 * blocks + 30, 16 * blocks + 1])], [], 54)
    lead = max(range(3), key=lambda b: bt.lens[b])
    rng = np.random.default_rng(55)
    large = {"large-small-large": [j < 20 or j >= 40 for j in range(blocks)],
             "small-large-small": [20 <= j < 40 for j in range(blocks)],
             "mixed": list(rng.random(blocks) < 0.5)}[order]
    is_large = np.zeros(bt.pages, dtype=bool)
    is_large[bt.table[lead, :blocks]] = large
    k = np.zeros((bt.pages, 16, K, d))
    k[..., 0] = ~is_large[:, None, None]
    k[..., 1] = is_large[:, None, None]
    v = rng.integers(1, 8, k.shape).astype(np.float64)
    v_scale = np.where(is_large, 2.0 ** 4, 2.0 ** -20)[:, None, None] * np.ones(k.shape[:3])
    cache, held = cache_of(gq, kind, k, v, None, v_scale)
    q = torch.zeros(3, 1, K * G, d, dtype=torch.bfloat16)
    q[..., 1] = -60
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    assert plan.blocks.tolist()[0] == blocks
    got = gq.gqa_decode_shared(cache, q[:, 0].contiguous().cuda(), table, lens, LN2, plan).view(q.shape)
    want = shared.attend(q.double().numpy(), held, bt.table, bt.lens, LN2)
    n = 16 * (blocks - sum(large))
    bound = 2.0 ** -30 * 2.0 ** 4 * 7 * (16 * blocks + 30) / n + 2.0 ** -14 * want
    assert (bound < want / 4).all()                              # nothing lost passes
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= bound).all(), float((off / bound).max())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 3])
def test_a_call_repeats_itself(gq, kind, T):
    """Pieces and their order go by the plan and the lengths alone, whichever SM takes them."""
    bt = shared.batch([(200, [3300 + 17 * i for i in range(12)]), (30, [700, 500, 483])], [900, 40], 56)
    cache, _ = shared.pool(kind, bt.pages, 4, 128, 57, gq)
    B = len(bt.lens)
    q = torch.randn(B, T, 16, 128, generator=torch.Generator().manual_seed(58)).to(shared.DTYPES.get(kind, torch.bfloat16)).cuda()
    q = q if T > 1 else q[:, 0].contiguous()
    table, lens = torch.from_numpy(bt.table).cuda(), torch.from_numpy(bt.lens).cuda()
    plan = gq.kv_pages_groups(table, lens)
    first = gq.gqa_decode_shared(cache, q, table, lens, 0.09, plan)
    side, noise = torch.cuda.Stream(), torch.empty(16 << 20, device="cuda")
    for i in range(40):
        if i % 3 == 0:
            with torch.cuda.stream(side):
                noise.zero_()
        assert torch.equal(gq.gqa_decode_shared(cache, q, table, lens, 0.09, plan), first)
    torch.cuda.synchronize()
