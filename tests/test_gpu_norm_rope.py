"""Per-head norm, rotation and the paged append in one pass against the plain
fp64 form, through the C ABI.

Bounds. The fp32 chain (sum of d <= 128 squares by a tree of 16 + 3 terms, root,
two products, one rotation) errs by at most ~32 steps of 2^-24 relative to the
pair's size; rounding to the stored type adds half a step, finfo.eps / 2."""
import numpy as np
import pytest
import torch

import gqa_inputs as gi
from plain import attend

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def turned(x, w, eps, rope, pos, interleaved):
    """fp64 rows [tokens, heads, d] and the bound's pair sizes, from their definition."""
    y = x.double().cpu()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double().cpu()
    size = y.abs()
    if rope is not None:
        pairs = rope.shape[1]
        first = torch.arange(0, 2 * pairs, 2) if interleaved else torch.arange(pairs)
        second = first + (1 if interleaved else pairs)
        cos, sin = (rope.double().cpu()[pos.long().cpu(), :, i][:, None] for i in (0, 1))
        a, b = y[..., first].clone(), y[..., second].clone()
        y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
        size = size.clone()
        size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


def check(got, ref, size, dtype):
    eps = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0             # half a step of fp16's subnormals
    off = (got.double().cpu() - ref).abs()
    allowed = ref.abs() * eps + (32 * 2.0 ** -24) * size * (1 + eps) + tiny
    assert bool((off <= allowed).all()), float((off - allowed).max())


CASES = [(3, 32, 8, 128, 128), (7, 5, 3, 64, 64), (1, 1, 1, 128, 48), (65, 24, 8, 64, 16), (9, 17, 2, 128, 0),
         (2, 130, 33, 64, 32)]


@pytest.mark.parametrize("tokens,H,K,d,rot", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", ["both", "f32", "q", "none"])
def test_dense_rows(gq, tokens, H, K, d, rot, dtype, interleaved, weights):
    t = TYPES[dtype]
    q, k = randn((tokens, H, d), t, 1), randn((tokens, K, d), t, 2) * 3
    wt = torch.float32 if weights == "f32" else t
    wq = None if weights == "none" else randn((d,), wt, 3)
    wk = randn((d,), wt, 4) if weights in ("both", "f32") else None
    rope = gq.rope_table(500, rot, 10000.0) if rot else None
    pos = torch.randint(0, 500, (tokens,), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo, ko = gq.qk_norm_rope(q, k, pos, rope, wq, wk, 1e-5, interleaved, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    check(qo, *turned(q, wq, 1e-5, rope, pos, interleaved), t)
    check(ko, *turned(k, wk, 1e-5, rope, pos, interleaved), t)


def test_rope_table_of_far_positions(gq):
    """Half a step of fp32: the angle is fp64 (p 2^-53 off at most)."""
    table = gq.rope_table(300000, 64, 500000.0)
    torch.cuda.synchronize()
    p = torch.arange(300000, dtype=torch.float64)[:, None]
    ang = p * 500000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ref = torch.stack((ang.cos(), ang.sin()), -1)
    assert bool(((table.double().cpu() - ref).abs() <= ref.abs() * 2.0 ** -24 + 1e-9).all())


def test_in_place_and_views_of_a_fused_projection(gq):
    H, K, d = 8, 2, 128
    qkv = randn((11, H + 2 * K, d), torch.bfloat16, 6)
    q, k = qkv[:, :H], qkv[:, H:H + K]
    rope = gq.rope_table(64, 128)
    pos = torch.arange(11, dtype=torch.int32, device="cuda")
    w = randn((d,), torch.bfloat16, 7)
    keep = qkv.clone()
    a, b = gq.qk_norm_rope(q, k, pos, rope, w, w)
    torch.cuda.synchronize()
    assert torch.equal(qkv, keep)
    q2, k2 = q.contiguous(), k.contiguous()
    gq.qk_norm_rope(q2, k2, pos, rope, w, w, q_out=q2, k_out=k2)
    torch.cuda.synchronize()
    assert torch.equal(a, q2) and torch.equal(b, k2)
    with pytest.raises(ValueError, match="overlaps"):
        gq.qk_norm_rope(q2[1:], k2[1:], pos[1:], rope, w, w, q_out=q2[:-1])


def _setup(gq, news, pos, K, d, cache_dtype, seed, extra=0):
    lens = [p + n for p, n in zip(pos, news)]
    case = gi.make_case(len(news), 8 * K, K, d, lens, cache_dtype, seed=seed, device="cuda", spare_blocks=3,
                        extra_tokens=extra)
    start = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device="cuda")
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    seq = np.repeat(np.arange(len(news)), news)
    at = np.concatenate([np.arange(p, p + n) for p, n in zip(pos, news)]).astype(np.int64)
    return case, gq.cache_from_case(case), start, positions, torch.from_numpy(seq), torch.from_numpy(at)


@pytest.mark.parametrize("news,pos", [([1, 1, 1], [0, 15, 40]), ([3, 0, 17, 33, 0, 1], [5, 9, 0, 31, 0, 100]),
                                      ([200] + [1] * 70, [7] * 71)])
@pytest.mark.parametrize("dtype,H,K,d,rot", [("bf16", 32, 8, 128, 128), ("f16", 6, 3, 64, 32), ("f32", 4, 1, 128, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_to_plain_caches(gq, news, pos, dtype, H, K, d, rot, interleaved):
    t = TYPES[dtype]
    case, cache, start, positions, seq, at = _setup(gq, news, pos, K, d, dtype, 11)
    total = sum(news)
    qkv = randn((total + 2, H + 2 * K, d), t, 12)            # two rows behind the last sequence
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    wq, wk = randn((d,), t, 13), randn((d,), t, 14)
    rope = gq.rope_table(400, rot)
    before_k, before_v = case.k_cache.clone(), case.v_cache.clone()
    q_out = torch.full((total + 2, H, d), 77.0, dtype=t, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq.qk_norm_rope_append(cache, q, k, v, case.block_table, positions, rope, wq, wk, 1e-6, interleaved,
                           token_start=start, max_new_tokens=max(news), q_out=q_out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert bool((q_out[total:] == 77.0).all())
    check(q_out[:total], *turned(q[:total], wq, 1e-6, rope, at, interleaved), t)
    phys, slot = case.block_table.cpu().long()[seq, at // 16], at % 16
    check(case.k_cache.cpu()[phys, :, slot], *turned(k[:total], wk, 1e-6, rope, at, interleaved), t)
    assert torch.equal(case.v_cache.cpu()[phys, :, slot], v[:total].cpu())
    # every other slot is as it was
    before_k[phys, :, slot], before_v[phys, :, slot] = case.k_cache[phys, :, slot], case.v_cache[phys, :, slot]
    bits = torch.int32 if dtype == "f32" else torch.int16
    assert torch.equal(case.k_cache.view(bits), before_k.view(bits))
    assert torch.equal(case.v_cache.view(bits), before_v.view(bits))


@pytest.mark.parametrize("cache_dtype", ["i8", "fp8", "i4"])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 128), ("f16", 64)])
def test_append_to_coded_caches(gq, cache_dtype, dtype, d):
    """V: the codes of the separate append. K: with fp32 rows the codes of the
    two-call form bit for bit; else within half a code of the fp64 rows."""
    import oracle
    K, H, news, pos = 3, 6, [1, 20, 5], [16, 3, 60]
    t = TYPES[dtype]
    case, cache, start, positions, seq, at = _setup(gq, news, pos, K, d, cache_dtype, 21)
    other = gq.PagedKVCache.allocate(case.num_blocks, K, d, "int4" if cache_dtype == "i4" else gi.DTYPES[cache_dtype])
    for x in (case.k_cache, case.v_cache, other.k, other.v):
        x.view(torch.uint8).zero_()
    for x in (case.k_scale, case.v_scale, other.k_scale, other.v_scale):
        x.zero_()
    total = sum(news)
    q, k, v = (randn((total, h, d), t, s) for h, s in ((H, 1), (K, 2), (K, 3)))
    v[1, 0] = 0                                              # a row of zeros: scale and codes 0
    wq, wk = randn((d,), t, 4), randn((d,), t, 5)
    rope = gq.rope_table(128, 64)
    qa = gq.qk_norm_rope_append(cache, q, k, v, case.block_table, positions, rope, wq, wk, token_start=start,
                                max_new_tokens=max(news))
    qb, kb = gq.qk_norm_rope(q, k, at.int().cuda(), rope, wq, wk)
    gq.kv_append_varlen(other, kb, v, start, max(news), case.block_table, positions)
    torch.cuda.synchronize()
    assert torch.equal(qa, qb)
    raw = lambda x: x.view(torch.uint8)  # noqa: E731
    assert torch.equal(raw(case.v_cache), raw(other.v)) and torch.equal(case.v_scale, other.v_scale)
    if dtype == "f32":
        assert torch.equal(raw(case.k_cache), raw(other.k)) and torch.equal(case.k_scale, other.k_scale)
    ref, size = turned(k, wk, 1e-6, rope, at, False)
    phys, slot = case.block_table.cpu().long()[seq, at // 16], at % 16
    s = case.k_scale.cpu()[phys, :, slot].double()
    codes = raw(case.k_cache).cpu()[phys, :, slot].numpy()
    val = {"i8": lambda c: c.view(np.int8).astype(np.float64), "fp8": oracle.e4m3_to_f64,
           "i4": lambda c: oracle.unpack_int4(c).astype(np.float64)}[cache_dtype](codes)
    deq = torch.from_numpy(np.asarray(val, dtype=np.float64)).reshape(ref.shape) * s[..., None]
    qmax = {"i8": 127, "fp8": 448, "i4": 7}[cache_dtype]
    slack = 32 * 2.0 ** -24 * size.amax(-1)
    assert bool(((s - ref.abs().amax(-1) / qmax).abs() <= (s * 2.0 ** -11 + 2.0 ** -25 + slack / qmax)).all())
    if cache_dtype == "fp8":   # half a step 2^-4 of the value, 2^-10 of the scale below the normals; saturation
        allowed = ref.abs() * (2.0 ** -4 + 2.0 ** -11) + s[..., None] * 2.0 ** -10 + 2 * slack[..., None]
    else:                      # half a code; the clamped extreme by the scale's rounding
        allowed = s[..., None] * (0.5 + qmax * 2.0 ** -11) + 2 * slack[..., None]
    assert bool(((deq - ref).abs() <= allowed).all())


@pytest.mark.parametrize("cache_dtype", ["i8", "fp8", "i4"])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_and_scales_are_the_appends_at_every_magnitude(gq, cache_dtype, d):
    """Rows from 2^-140 to 2^120, ties (multiples of half a code), infinities and NaN: the
    reciprocal with its correction gives the append's divisions bit for bit."""
    K, n = 4, 1024
    g = torch.Generator().manual_seed(81)
    x = torch.randn((n, K, d), generator=g)
    x *= torch.exp2(torch.randint(-140, 120, (n, K, 1), generator=g).float())
    x[::7] = torch.randint(-254, 255, (len(range(0, n, 7)), K, d), generator=g).float() / 2   # halves of an int8 code
    x[::7, :, 0] = 127.0
    x[3, 0, 5], x[4, 1, 6], x[5, 2, 7] = float("inf"), float("-inf"), float("nan")
    x[6] = 0
    x = x.cuda()
    kind = "int4" if cache_dtype == "i4" else gi.DTYPES[cache_dtype]
    a, b = (gq.PagedKVCache.allocate(n // 16, K, d, kind) for _ in range(2))
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda").reshape(1, -1)
    pos, start = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = torch.zeros((n, K, d), device="cuda")
    gq.qk_norm_rope_append(a, q, x, x, table, pos, token_start=start, max_new_tokens=n)   # no norm, no rotation
    gq.kv_append_varlen(b, x, x, start, n, table, pos)
    torch.cuda.synchronize()
    for name in ("k", "v"):
        assert torch.equal(getattr(a, name + "_scale").view(torch.int16), getattr(b, name + "_scale").view(torch.int16))
        assert torch.equal(getattr(a, name).view(torch.uint8), getattr(b, name).view(torch.uint8)), name


@pytest.mark.parametrize("T", [1, 3])
def test_uniform_tokens_match_the_ragged_call(gq, T):
    B, H, K, d = 5, 8, 2, 128
    pos = [0, 14, 15, 16, 100]
    case, cache, start, positions, seq, at = _setup(gq, [T] * B, pos, K, d, "bf16", 31)
    q, k, v = (randn((B, T, h, d), torch.bfloat16, s) for h, s in ((H, 1), (K, 2), (K, 3)))
    if T == 1:
        q, k, v = q[:, 0], k[:, 0], v[:, 0]
    rope = gq.rope_table(256, 128)
    a = gq.qk_norm_rope_append(cache, q, k, v, case.block_table, positions, rope)
    ka, va = case.k_cache.clone(), case.v_cache.clone()
    case.k_cache.fill_(0), case.v_cache.fill_(0)
    ka.nan_to_num_(0), va.nan_to_num_(0)
    b = gq.qk_norm_rope_append(cache, q.reshape(-1, H, d), k.reshape(-1, K, d), v.reshape(-1, K, d), case.block_table,
                               positions, rope, token_start=start, max_new_tokens=T)
    torch.cuda.synchronize()
    assert torch.equal(a.reshape(-1, H, d), b)
    phys, slot = case.block_table.cpu().long()[seq, at // 16], at % 16
    assert torch.equal(ka[phys, :, slot], case.k_cache[phys, :, slot])
    assert torch.equal(va[phys, :, slot], case.v_cache[phys, :, slot])


def test_rope_positions_of_their_own(gq):
    case, cache, start, positions, seq, at = _setup(gq, [4, 2], [30, 0], 2, 64, "f32", 41)
    q, k, v = (randn((6, h, 64), torch.float32, s) for h, s in ((4, 1), (2, 2), (2, 3)))
    rope = gq.rope_table(1000, 64)
    turn = torch.tensor([999, 0, 5, 5, 17, 500], dtype=torch.int32, device="cuda")
    qo = gq.qk_norm_rope_append(cache, q, k, v, case.block_table, positions, rope, token_start=start, max_new_tokens=4,
                                rope_positions=turn)
    torch.cuda.synchronize()
    check(qo, *turned(q, None, 0, rope, turn, False), torch.float32)
    phys, slot = case.block_table.cpu().long()[seq, at // 16], at % 16
    check(case.k_cache.cpu()[phys, :, slot], *turned(k, None, 0, rope, turn, False), torch.float32)


def test_bad_positions_and_pages_are_skipped_and_flagged(gq):
    B, H, K, d = 4, 8, 2, 64
    case, cache, start, positions, seq, at = _setup(gq, [1] * B, [3, 20, 9, 30], K, d, "bf16", 51)
    q, k, v = (randn((B, h, d), torch.bfloat16, s) for h, s in ((H, 1), (K, 2), (K, 3)))
    rope = gq.rope_table(25, 64)                             # too short for the last token
    table = case.block_table.clone()
    table[1, 20 // 16] = case.num_blocks                     # outside the pool
    bad = positions.clone()
    bad[2] = table.shape[1] * 16                             # past the table, and past the rotations
    keep_k, keep_v = case.k_cache.clone(), case.v_cache.clone()
    q_out = torch.full((B, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq.qk_norm_rope_append(cache, q, k, v, table, bad, rope, q_out=q_out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == gq.GQA_DEVERR_POSITION | gq.GQA_DEVERR_BLOCK_INDEX
    check(q_out[:2], *turned(q[:2], None, 0, rope, at[:2], False), torch.bfloat16)
    assert bool((q_out[2:] == 5.0).all())
    p = int(table[0, 0])
    keep_k[p, :, 3], keep_v[p, :, 3] = case.k_cache[p, :, 3], case.v_cache[p, :, 3]
    assert torch.equal(case.k_cache.view(torch.int16), keep_k.view(torch.int16))
    assert torch.equal(case.v_cache.view(torch.int16), keep_v.view(torch.int16))
    assert torch.equal(case.v_cache[p, :, 3], v[0])
    # a sequence with more tokens than the bound
    err.zero_()
    s2 = torch.tensor([0, 3, 4, 4, 4], dtype=torch.int32, device="cuda")
    q_out.fill_(5.0)
    gq.qk_norm_rope_append(cache, q, k, v, case.block_table, positions, None, token_start=s2, max_new_tokens=2,
                           q_out=q_out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == gq.GQA_DEVERR_POSITION
    assert bool((q_out[:3] == 5.0).all()) and torch.equal(q_out[3], q[3])


def test_pages_past_32_bit_offsets(gq):
    """A pool of more than 2^31 elements: the last pages' offsets need 64 bits."""
    K, d, pages = 8, 128, 140000
    cache = gq.PagedKVCache.allocate(pages, K, d, torch.bfloat16)
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 15], dtype=torch.int32, device="cuda")
    q, k, v = (randn((2, h, d), torch.bfloat16, s) for h, s in ((8, 1), (K, 2), (K, 3)))
    gq.qk_norm_rope_append(cache, q, k, v, table, pos)
    torch.cuda.synchronize()
    assert torch.equal(cache.k[pages - 1, :, 3], k[0]) and torch.equal(cache.v[pages - 2, :, 15], v[1])


@pytest.mark.parametrize("dtype,H,K,d,interleaved,lens", [("bf16", 32, 8, 128, False, [7001, 1, 3050, 2300]),
                                                          ("f16", 24, 8, 64, True, [20001, 9007, 33]),
                                                          ("bf16", 16, 8, 128, False, [16384, 0, 16])])
def test_a_batch_that_streams_equals_its_parts(gq, dtype, H, K, d, interleaved, lens):
    """Batches of over 256 MB read and written run in shorter runs of tokens; a row's
    result does not depend on the run it is in, so the parts give the very same bits."""
    t, total, B = TYPES[dtype], sum(lens), len(lens)
    qkv = torch.randn((total, H + 2 * K, d), generator=torch.Generator("cuda").manual_seed(3), device="cuda").to(t)
    q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
    assert 2 * q.element_size() * qkv.numel() >= 256 << 20
    rope, wq, wk = gq.rope_table(max(lens) + 9, d), randn((d,), t, 4), randn((d,), t, 5)
    at = torch.randint(0, max(lens), (total,), generator=torch.Generator().manual_seed(6), dtype=torch.int32).cuda()
    blocks = max(lens) // 16 + 2
    table = torch.randperm(B * blocks, generator=torch.Generator().manual_seed(7)).to(torch.int32).view(B, blocks).cuda()
    pos = torch.tensor([9, 0, 5, 1][:B], dtype=torch.int32, device="cuda")
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    caches = []
    for c in range(2):
        caches.append(gq.PagedKVCache.allocate(B * blocks, K, d, t))
        caches[c].k.zero_(), caches[c].v.zero_()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole = gq.qk_norm_rope_append(caches[0], q, k, v, table, pos, rope, wq, wk, interleaved=interleaved,
                                   token_start=start, max_new_tokens=max(lens), err=err)
    dense = gq.qk_norm_rope(q, k, at, rope, wq, wk, interleaved=interleaved, err=err)
    for b, n in enumerate(lens):
        for lo in range(0, n, 4000):
            i, m = int(start[b]) + lo, min(4000, n - lo)
            one = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            part = gq.qk_norm_rope_append(caches[1], q[i:i + m], k[i:i + m], v[i:i + m], table[b:b + 1],
                                          pos[b:b + 1] + lo, rope, wq, wk, interleaved=interleaved,
                                          token_start=one, max_new_tokens=m, err=err)
            assert torch.equal(whole[i:i + m], part)
            for x, y in zip(dense, gq.qk_norm_rope(q[i:i + m], k[i:i + m], at[i:i + m], rope, wq, wk,
                                                   interleaved=interleaved, err=err)):
                assert torch.equal(x[i:i + m], y)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    few = torch.tensor([0, 1, 2, 3, total // 2, total - 2, total - 1])
    check(dense[0][few], *turned(q[few], wq, 1e-6, rope, at[few], interleaved), t)
    check(dense[1][few], *turned(k[few], wk, 1e-6, rope, at[few], interleaved), t)


def test_positions_without_a_table_change_nothing(gq):
    q, k = randn((9, 8, 128), torch.bfloat16, 1), randn((9, 2, 128), torch.bfloat16, 2)
    w = randn((128,), torch.bfloat16, 3)
    far = torch.full((9,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = gq.qk_norm_rope(q, k, far, None, w, w, err=err)
    c, e = gq.qk_norm_rope(q, k, None, None, w, w, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(a, c) and torch.equal(b, e)


def test_other_stream_and_captured_replay(gq):
    B, H, K, d = 3, 8, 2, 128
    case, cache, start, positions, seq, at = _setup(gq, [1] * B, [3, 20, 9], K, d, "bf16", 61, extra=40)
    q, k, v = (randn((B, h, d), torch.bfloat16, s) for h, s in ((H, 1), (K, 2), (K, 3)))
    rope = gq.rope_table(256, 128)
    w = randn((d,), torch.float32, 4)
    q_out = torch.empty_like(q)
    call = lambda s=None: gq.qk_norm_rope_append(cache, q, k, v, case.block_table, positions, rope, w, w,  # noqa: E731
                                                 q_out=q_out, stream=s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    side.synchronize()
    check(q_out, *turned(q, w, 1e-6, rope, at, False), torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        positions += 13
        q.normal_(generator=torch.Generator(device="cuda").manual_seed(step))
        graph.replay()
        torch.cuda.synchronize()
        check(q_out, *turned(q, w, 1e-6, rope, positions, False), torch.bfloat16)
        for b in range(B):
            p = int(positions[b])
            assert torch.equal(case.v_cache[int(case.block_table[b, p // 16]), :, p % 16], v[b])


@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 4)])
def test_steps_of_a_stream_from_the_projection_to_the_output(gq, window, sinks):
    """A prompt, then single steps: projection -> norm, rotation, append -> attention,
    against the same in fp64 (K rounded to the cache's type, as it is stored)."""
    H, K, d, steps = 8, 2, 128, 5
    news, pos = [37, 5], [0, 0]
    case, cache, start, positions, seq, at = _setup(gq, [n + steps for n in news], pos, K, d, "f32", 71)
    rope, w = gq.rope_table(64, 128), randn((d,), torch.float32, 9)
    rows = {b: ([], []) for b in range(2)}

    def remember(b, k, v, p):
        rows[b][0].append(turned(k, w, 1e-6, rope, p, False)[0])
        rows[b][1].append(v.double().cpu())

    x = randn((sum(news), H + 2 * K, d), torch.float32, 8)
    start = torch.tensor([0, 37, 42], dtype=torch.int32, device="cuda")
    gq.qk_norm_rope_append(cache, x[:, :H], x[:, H:H + K], x[:, H + K:], case.block_table, positions, rope, w, w,
                           token_start=start, max_new_tokens=37)
    for b, (lo, hi) in enumerate(((0, 37), (37, 42))):
        remember(b, x[lo:hi, H:H + K], x[lo:hi, H + K:], torch.arange(hi - lo))
    lens = torch.tensor(news, dtype=torch.int32, device="cuda")
    for s in range(steps):
        x = randn((2, H + 2 * K, d), torch.float32, 100 + s)
        q = gq.qk_norm_rope_append(cache, x[:, :H], x[:, H:H + K], x[:, H + K:], case.block_table, lens, rope, w, w)
        lens += 1
        out = gq.gqa_decode(cache, q, case.block_table, lens, d ** -0.5, window=window, sinks=sinks)
        torch.cuda.synchronize()
        for b in range(2):
            p = int(lens[b]) - 1
            remember(b, x[b:b + 1, H:H + K], x[b:b + 1, H + K:], torch.tensor([p]))
            qr = turned(x[b:b + 1, :H], w, 1e-6, rope, torch.tensor([p]), False)[0].numpy()
            ref = attend(qr, torch.cat(rows[b][0]).numpy(), torch.cat(rows[b][1]).numpy(), d ** -0.5, window, sinks)[0]
            # |q|, |k| rows of size ~sqrt(d) w^2: scores of tens, each 2^-20 off at most; weights times |v| < 5
            assert np.abs(out[b].double().cpu().numpy() - ref).max() <= 2e-3
