"""What the serving operators around the paged cache cost: the cases and their plain forms.

Five operators, as a decoding server calls them:

* ``decode``    -- attention of the new token(s) with a sliding window and sink tokens
* ``prefill``   -- the same mask for prompts and chunks of prompts
* ``norm_rope`` -- per-head norm of q and k, position rotation and the paged append in one pass
* ``fork``      -- free the children of the last round, fork parents into them, copy their
                   unfinished pages in every layer, reserve pages for the next tokens
* ``compact``   -- release the pages that left the window, move the remaining ones to the
                   front of the pool in every layer

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits (or whole
numbers); with ``own`` true it makes the library's calls.
"""
import math

import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one short chat on an idle server: latency of a single step
        dict(name="decode_one_chat", op="decode", B=1, T=1, H=32, K=8, d=128, cache="bf16", q="bf16",
             lo=700, hi=700, W=512, S=4),
        # a full batch of long streams, the library's 4096-token window workload with four sinks
        dict(name="decode_streams", op="decode", B=64, T=1, H=32, K=8, d=128, cache="bf16", q="bf16",
             lo=16384, hi=16384, W=4096, S=4),
        # ragged batch on an FP8 cache verifying one draft token each (two queries per sequence)
        dict(name="decode_fp8_verify", op="decode", B=48, T=2, H=64, K=8, d=128, cache="fp8", q="bf16",
             lo=300, hi=8192, W=1000, S=20),
        # whole prompts with a window well below their length
        dict(name="prefill_prompts", op="prefill", B=8, H=32, K=8, d=128, cache="bf16", q="bf16",
             n_lo=2048, n_hi=2048, c_lo=0, c_hi=0, W=1024, S=4),
        # ragged chunks of longer prompts behind an existing context, three heads per group
        dict(name="prefill_chunks", op="prefill", B=6, H=24, K=8, d=64, cache="f16", q="f16",
             n_lo=97, n_hi=512, c_lo=333, c_hi=4001, W=1000, S=20),
        # the step of a small decode batch: latency
        dict(name="norm_rope_step", op="norm_rope", B=4, n_lo=1, n_hi=1, c_lo=100, c_hi=9000, H=32, K=8, d=128,
             cache="bf16", q="bf16", rot=128, inter=False),
        # eight prompts of 2048 tokens, rows inside the fused projection's output
        dict(name="norm_rope_prompts", op="norm_rope", B=8, n_lo=2048, n_hi=2048, c_lo=0, c_hi=0, H=32, K=8, d=128,
             cache="bf16", q="bf16", rot=128, inter=False),
        # ragged chunks onto an FP8 cache, partial rotation of interleaved pairs
        dict(name="norm_rope_fp8_ragged", op="norm_rope", B=37, n_lo=1, n_hi=701, c_lo=0, c_hi=5000, H=24, K=8, d=64,
             cache="fp8", q="f16", rot=32, inter=True),
        # one answer sampled four ways
        dict(name="fork_one", op="fork", parents=1, children=4, lo=1000, hi=1000, layers=1, K=8, d=128, cache="bf16",
             spare=16),
        # four continuations of each of 64 requests, every layer's cache
        dict(name="fork_batch", op="fork", parents=64, children=4, lo=100, hi=700, layers=28, K=8, d=128, cache="bf16",
             spare=64),
        # a few short streams on a small model
        dict(name="compact_small", op="compact", rows=8, lo=600, hi=1500, layers=2, K=2, d=64, cache="f16", W=256, S=4),
        # 64 streams that ran past a 1024-token window
        dict(name="compact_streams", op="compact", rows=64, lo=3500, hi=4700, layers=4, K=8, d=128, cache="bf16",
             W=1024, S=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prefill", "norm_rope", "fork", "compact"])
    d = rng.choice([64, 128])
    cache = rng.choice(["bf16", "f16"])
    if op == "decode":
        if d == 128 and rng.random() < 0.4:
            cache = "fp8"
        K = rng.choice([1, 2, 4, 8])
        T = rng.choice([1, 1, 2, 3])
        G = rng.randint(1, 8)
        W = _log(rng, 16, 4096)
        S = _log(rng, 1, 128)
        lo = _log(rng, 1, 16384)
        hi = rng.randint(lo, 16384)
        B = max(1, min(_log(rng, 1, 128), 500_000 // (W + S + T) // K))
        return dict(op=op, B=B, T=T, H=G * K, K=K, d=d, cache=cache, q="bf16" if cache == "bf16" else "f16",
                    lo=lo, hi=hi, W=W, S=S)
    if op == "prefill":
        K = rng.choice([1, 2, 4, 8])
        G = rng.randint(1, 8)
        n_lo = _log(rng, 1, 1024)
        n_hi = rng.randint(n_lo, 1024)
        c_lo = _log(rng, 1, 3000)
        c_hi = rng.randint(c_lo, 3000)
        B = max(1, min(_log(rng, 1, 16), 500_000_000 // (K * G * n_hi * (n_hi + c_hi))))
        return dict(op=op, B=B, H=K * G, K=K, d=d, cache=cache, q=cache, n_lo=n_lo, n_hi=n_hi, c_lo=c_lo, c_hi=c_hi,
                    W=_log(rng, 16, 2048), S=_log(rng, 1, 128))
    if op == "norm_rope":
        if rng.random() < 0.4:
            cache = "fp8"
        K = rng.choice([1, 2, 4, 8])
        G = rng.randint(1, 8)
        n_lo = _log(rng, 1, 1000)
        n_hi = rng.randint(n_lo, 1500)
        c_lo = _log(rng, 1, 8000)
        return dict(op=op, B=max(1, min(_log(rng, 1, 128), 16384 // n_hi)), n_lo=n_lo, n_hi=n_hi, c_lo=c_lo,
                    c_hi=rng.randint(c_lo, 8000), H=K * G, K=K, d=d, cache=cache, q=rng.choice(["bf16", "f16"])
                    if cache == "fp8" else cache, rot=rng.choice([16, 32, 48, 64, d]), inter=rng.random() < 0.5)
    K = rng.choice([1, 2, 4, 8])
    layers = _log(rng, 1, 28)
    lo = _log(rng, 1, 700)
    if op == "fork":
        return dict(op=op, parents=_log(rng, 1, 64), children=rng.randint(1, 4), lo=lo, hi=rng.randint(lo, 700),
                    layers=layers, K=K, d=d, cache=cache, spare=rng.randint(8, 200))
    lo = _log(rng, 300, 4000)
    return dict(op=op, rows=_log(rng, 1, 64), lo=lo, hi=rng.randint(lo, 4500), layers=min(layers, 4), K=K, d=d,
                cache=cache, W=_log(rng, 16, 1024), S=_log(rng, 1, 64))


# ------------------------------------------------------------------ inputs


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the same for every seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _new_and_before(case):
    """(new tokens, tokens before them) of each sequence: the fewer new ones, the longer the context."""
    return list(zip(_spread(case["n_lo"], case["n_hi"], case["B"]), reversed(_spread(case["c_lo"], case["c_hi"], case["B"]))))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, dtype, gen):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _shuffled(values, seed):
    order = torch.randperm(len(values), generator=torch.Generator().manual_seed(seed)).tolist()
    return [values[i] for i in order]


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _table(needed, seed, spare=0):
    """Block table [rows, blocks]: a shuffled page for every needed entry, -1 elsewhere."""
    pages = int(needed.sum())
    perm = torch.randperm(pages + spare, generator=torch.Generator().manual_seed(seed), dtype=torch.int64)
    table = torch.full(needed.shape, -1, dtype=torch.int64)
    table[needed] = perm[:pages]
    return table.to(torch.int32).cuda(), pages + spare


def _quantise(x):
    """FP8 rows as the library's append makes them: codes and one fp16 scale per row."""
    s = (x.float().abs().amax(-1) / 448.0).clamp(max=65504.0).to(torch.float16)
    sf = s.float().unsqueeze(-1)
    y = torch.where(sf > 0, x.float() / torch.where(sf > 0, sf, torch.ones_like(sf)), torch.zeros_like(x.float()))
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _pool(case, pages, gen):
    """K and V of one paged cache, with scales where its type has them."""
    shape = (pages, case["K"], BLOCK, case["d"])
    if case["cache"] != "fp8":
        return [_normal(shape, DTYPES[case["cache"]], gen) for _ in range(2)] + [None, None]
    (k, ks), (v, vs) = (_quantise(_normal(shape, torch.float32, gen)) for _ in range(2))
    return [k, v, ks, vs]


def _cache(gq, k, v, ks=None, vs=None):
    n, K, _, d = k.shape
    return gq.PagedKVCache(k, v, n, K, d, K * BLOCK * d, BLOCK * d, d, ks, vs)


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case=case)
    if case["op"] in ("decode", "prefill"):
        B, K, d, W, S = (case[x] for x in ("B", "K", "d", "W", "S"))
        if case["op"] == "decode":
            new = [case["T"]] * B
            lens = _shuffled(_spread(case["lo"], case["hi"], B), seed)
        else:
            new, before = zip(*_shuffled(_new_and_before(case), seed))
            lens = [n + c for n, c in zip(new, before)]
        L, n = torch.tensor(lens), torch.tensor(new)
        blk = torch.arange(-(-max(lens) // BLOCK))
        # pages that no query of the call can see went back to the pool before it
        needed = (blk * BLOCK < L[:, None]) & ((blk * BLOCK < S) | ((blk + 1) * BLOCK > (L - n + 1 - W)[:, None]))
        st["table"], pages = _table(needed, seed)
        st["lens"], st["max_new"] = _i32(lens), max(new)
        st["pool"] = _pool(case, pages, gen)
        shape = (B, case["T"], case["H"], d) if case["op"] == "decode" else (sum(new), case["H"], d)
        st["q"] = _normal(shape, DTYPES[case["q"]], gen)
        if case["op"] == "decode" and case["T"] == 1:
            st["q"] = st["q"].view(B, case["H"], d)
        st["q_start"] = _i32([0] + torch.cumsum(n, 0).tolist())
        st["scale"] = 1.0 / math.sqrt(d)
        if own:
            import gqa_decode_attention_kv_gb300 as gq
            st["gq"], st["cache"] = gq, _cache(gq, *st["pool"])
    elif case["op"] == "norm_rope":
        B, H, K, d, rot = (case[x] for x in ("B", "H", "K", "d", "rot"))
        new, pos = zip(*_shuffled(_new_and_before(case), seed))
        P, n = torch.tensor(pos), torch.tensor(new)
        blk = torch.arange(int((P + n).max() + BLOCK - 1) // BLOCK)
        # the pages that the new tokens go to
        needed = (blk * BLOCK < (P + n)[:, None]) & ((blk + 1) * BLOCK > P[:, None])
        st["table"], pages = _table(needed, seed)
        st["pos"], st["start"], st["max_new"] = _i32(pos), _i32([0] + torch.cumsum(n, 0).tolist()), max(new)
        st["pool"] = _pool(case, pages, gen)
        # one fused projection: q, k and v of a token side by side
        qkv = _normal((sum(new), H + 2 * K, d), DTYPES[case["q"]], gen)
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        st["wq"], st["wk"] = (_normal((d,), DTYPES[case["q"]], gen) * 0.1 + 1 for _ in range(2))
        # (cos, sin) of every position: the angles in 64 bits, the table in 32
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(int((P + n).max()), dtype=torch.float64, device="cuda")[:, None] * inv
        st["rope"] = torch.stack((ang.cos(), ang.sin()), -1).float()
        st["eps"] = 1e-6
        if own:
            import gqa_decode_attention_kv_gb300 as gq
            st["gq"], st["cache"] = gq, _cache(gq, *st["pool"])
    else:
        lens = _shuffled(_spread(case["lo"], case["hi"], case["parents"] if case["op"] == "fork" else case["rows"]), seed)
        L = torch.tensor(lens)
        if case["op"] == "fork":
            p, c = case["parents"], case["children"]
            # rows: the parents, then their children, empty; a page for each parent's next token
            blocks = max(lens) // BLOCK + 2
            needed = torch.zeros(p * (1 + c), blocks, dtype=torch.bool)
            needed[:p] = torch.arange(blocks) * BLOCK < (L + 1)[:, None]
            st["table"], pages = _table(needed, seed, 2 * p * c + case["spare"])
            st["lens"] = _i32(lens + [0] * (p * c))
            st["src"], st["dst"] = _i32([i for i in range(p) for _ in range(c)]), _i32(list(range(p, p * (1 + c))))
        else:
            needed = torch.arange(-(-max(lens) // BLOCK)) * BLOCK < L[:, None]
            st["table0"], pages = _table(needed, seed, 7)
            st["lens"] = _i32(lens)
            # how many pages the call will move: a server sizes its list of moves once
            dead = _dead(st["table0"], st["lens"], case["W"], case["S"])
            live = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
            live[torch.where((st["table0"] >= 0) & ~dead, st["table0"], pages).long().reshape(-1)] = 1
            st["moves"] = max(1, int(live[int(live[:pages].sum()):pages].sum()))
            st["table"] = st["table0"].clone()
        refs = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
        refs[st["table"].clamp(min=-1).reshape(-1).long()] = 1
        st["refs"] = refs[:pages].clone()
        st["refs0"] = st["refs"].clone()
        # every layer's cache: [layers, pages, K, 16, d]
        shape = (case["layers"], pages, case["K"], BLOCK, case["d"])
        st["k"], st["v"] = (_normal(shape, DTYPES[case["cache"]], gen) for _ in range(2))
        if own:
            import gqa_decode_attention_kv_gb300 as gq
            st["gq"] = gq
            st["caches"] = [_cache(gq, st["k"][i], st["v"][i]) for i in range(case["layers"])]
    return st


# ------------------------------------------------------------------ plain forms


def _rows_of(pool, scales, table, pos):
    """Cached rows at positions pos [B, n] as fp32 [B, K, n, d] (positions must have a page)."""
    phys, slot = torch.gather(table.long(), 1, pos // BLOCK), pos % BLOCK
    if scales is None:
        return pool[phys, :, slot].float().transpose(1, 2)
    rows = pool.view(torch.uint8)[phys, :, slot].view(pool.dtype).float()
    return (rows * scales[phys, :, slot].float().unsqueeze(-1)).transpose(1, 2)


def _softmax_av(s, visible, v):
    """softmax over the visible scores, times v; rows that see nothing are zero."""
    s = torch.where(visible, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p @ v / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(st):
    c, q, L = st["case"], st["q"], st["lens"].long()
    B, T, H, K, d, W, S = (c[x] for x in ("B", "T", "H", "K", "d", "W", "S"))
    G = H // K
    # the sinks, then the window of the first query up to the last token
    lo = torch.maximum((L - T + 1 - W).clamp(min=0), torch.full_like(L, S))
    pos = torch.cat((torch.arange(S, device=q.device).expand(B, S),
                     lo[:, None] + torch.arange(W + T - 1, device=q.device)), 1)
    inside = pos < L[:, None]
    pos = torch.where(inside, pos, (L - 1).clamp(min=0)[:, None])
    k, v = (_rows_of(st["pool"][i], st["pool"][2 + i], st["table"], pos) for i in range(2))
    qf = q.view(B, T, K, G, d).permute(0, 2, 1, 3, 4).reshape(B, K, T * G, d).float()
    at = (L[:, None] - T + torch.arange(T, device=q.device))[:, :, None]
    see = inside[:, None] & (pos[:, None] <= at) & ((pos[:, None] > at - W) | (pos[:, None] < S))   # [B, T, n]
    see = see[:, None, :, None].expand(B, 1, T, G, pos.shape[1]).reshape(B, 1, T * G, -1)
    o = _softmax_av(qf @ k.transpose(2, 3) * st["scale"], see, v)
    return o.view(B, K, T, G, d).permute(0, 2, 1, 3, 4).reshape(q.shape).to(q.dtype)


def _plain_prefill(st):
    c, q, L, start = st["case"], st["q"], st["lens"].long(), st["q_start"].long()
    B, H, K, d, W, S = (c[x] for x in ("B", "H", "K", "d", "W", "S"))
    G, n = H // K, st["max_new"]
    count = start[1:] - start[:-1]
    t = torch.arange(st["table"].shape[1] * BLOCK, device=q.device)
    pages = st["table"].long().gather(1, (t // BLOCK).expand(B, -1))
    held = (pages >= 0) & (t < L[:, None])
    k, v = (torch.where(held[:, None, :, None], st["pool"][i][pages.clamp(min=0), :, t % BLOCK].float().transpose(1, 2),
                        torch.zeros((), device=q.device)) for i in range(2))
    i = torch.arange(n, device=q.device)
    rows = (start[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qf = q[rows].float().view(B, n, K, G, d).permute(0, 2, 3, 1, 4).reshape(B, K, G * n, d)
    at = ((L - count)[:, None] + i)[:, :, None]
    see = held[:, None] & (t <= at) & ((t > at - W) | (t < S))                                     # [B, n, t]
    see = see[:, None, None].expand(B, 1, G, n, -1).reshape(B, 1, G * n, -1)
    o = _softmax_av(qf @ k.transpose(2, 3) * st["scale"], see, v)
    o = o.view(B, K, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, H, d).to(q.dtype)
    token = torch.arange(q.shape[0], device=q.device)
    b = (token[:, None] >= start[1:]).sum(1)
    return o[b, token - start[b]]


def _rotate(x, rot, cos, sin, inter):
    """Rotation of the first rot elements of x [total, heads, d]."""
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_norm_rope(st):
    c, start = st["case"], st["start"].long()
    token = torch.arange(st["q"].shape[0], device=start.device)
    b = (token[:, None] >= start[1:]).sum(1)
    pos = st["pos"].long()[b] + token - start[b]
    cos, sin = st["rope"][pos][:, None].unbind(-1)

    def turned(x, w):
        x = x.float()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + st["eps"]) * w.float()
        return _rotate(x, c["rot"], cos, sin, c["inter"])

    phys, slot = st["table"].long()[b, pos // BLOCK], pos % BLOCK
    kp, vp, ks, vs = st["pool"]
    k = turned(st["k"], st["wk"])
    if ks is None:
        kp[phys, :, slot] = k.to(kp.dtype)
        vp[phys, :, slot] = st["v"]
    else:
        k, ks[phys, :, slot] = _quantise(k)
        v, vs[phys, :, slot] = _quantise(st["v"])
        kp.view(torch.uint8)[phys, :, slot] = k.view(torch.uint8)
        vp.view(torch.uint8)[phys, :, slot] = v.view(torch.uint8)
    return [turned(st["q"], st["wq"]).to(st["q"].dtype), kp, vp, ks, vs]


def _free_pages(refs, count):
    """The `count` lowest free pages, in order (the pool has as many)."""
    free = refs == 0
    rank = torch.cumsum(free, 0) - 1
    ids = torch.zeros(count + 1, dtype=torch.int64, device=refs.device)
    at = torch.where(free & (rank < count), rank, torch.full_like(rank, count))
    return ids.scatter_(0, at, torch.arange(len(refs), device=refs.device))[:count]


def _count(refs, pages, step):
    """Adds step to the count of every page listed (entries below zero are none)."""
    held = pages >= 0
    refs.index_add_(0, pages.clamp(min=0).reshape(-1).long(), (held * step).reshape(-1).to(refs.dtype))


def _plain_fork(st):
    table, lens, refs, src, dst = st["table"], st["lens"], st["refs"], st["src"].long(), st["dst"].long()
    blk = torch.arange(table.shape[1], device=table.device)
    _count(refs, table[dst], -1)                       # free the children
    # fork: shared pages, and a fresh one in the place of an unfinished last page
    L = lens[src].long()
    last, cut = torch.div(L, BLOCK, rounding_mode="floor"), L % BLOCK != 0
    rows = torch.where(blk < torch.div(L + BLOCK - 1, BLOCK, rounding_mode="floor")[:, None], table[src],
                       torch.full_like(table[src], -1))
    old = rows.long().gather(1, last[:, None])[:, 0]
    fresh = _free_pages(refs, len(src))[(torch.cumsum(cut, 0) - 1).clamp(min=0)]
    new = torch.where(cut, fresh, old)
    rows = torch.where(cut[:, None] & (blk == last[:, None]), new[:, None].int(), rows)
    _count(refs, rows, 1)
    lens[dst] = L.int()
    # the pages' data, in every layer (a fork without an unfinished page copies its first page onto itself)
    first = table[src, 0].long()
    frm, to = torch.where(cut, old, first), torch.where(cut, new, first)
    st["k"][:, to] = st["k"][:, frm]
    st["v"][:, to] = st["v"][:, frm]
    table[dst] = rows
    # reserve: a page for the next token of every sequence that has none
    nxt = torch.div(lens.long(), BLOCK, rounding_mode="floor")
    lack = table.gather(1, nxt[:, None])[:, 0] < 0
    page = _free_pages(refs, len(lens))[(torch.cumsum(lack, 0) - 1).clamp(min=0)].int()
    table.copy_(torch.where(lack[:, None] & (blk == nxt[:, None]), page[:, None], table))
    refs.index_add_(0, page.long(), lack.to(refs.dtype))
    return [table, lens, refs, st["k"], st["v"]]


def _dead(table, lens, W, S):
    """Entries whose page no later token sees: past the sinks and before the next token's window."""
    blk = torch.arange(table.shape[1], device=table.device)
    return (blk * BLOCK >= S) & ((blk + 1) * BLOCK <= (lens.long() + 1 - W)[:, None])


def _plain_compact(st):
    c, table, refs, lens = st["case"], st["table"], st["refs"], st["lens"]
    table.copy_(st["table0"])                          # the bookkeeping as it was before the trim
    refs.copy_(st["refs0"])
    dead = _dead(table, lens, c["W"], c["S"])
    _count(refs, torch.where(dead, table, torch.full_like(table, -1)), -1)
    table.masked_fill_(dead, -1)
    pages, moves = len(refs), st["moves"]
    live = refs > 0
    n = live.sum()
    at = torch.arange(pages, device=refs.device)
    before = torch.cumsum(live, 0) - live.long()
    none = torch.full_like(at, moves)
    # i-th highest live page past the first n -> i-th lowest hole among them
    up = torch.where(live & (at >= n), n - 1 - before, none)
    down = torch.where(~live & (at < n), at - before, none)
    frm, to = (torch.zeros(moves + 1, dtype=torch.int64, device=refs.device).scatter_(0, x, at)[:moves] for x in (up, down))
    real = torch.arange(moves, device=refs.device) < (live & (at >= n)).sum()
    frm, to = torch.where(real, frm, 0), torch.where(real, to, 0)
    name = at.clone()
    name[frm] = to
    table.copy_(torch.where(table >= 0, name[table.clamp(min=0).long()].int(), table))
    moved = torch.where(real, refs[frm], refs[to])
    refs[frm] = torch.where(real, torch.zeros_like(moved), moved)
    refs[to] = moved
    st["k"][:, to] = st["k"][:, frm]
    st["v"][:, to] = st["v"][:, frm]
    return [table, refs, st["k"], st["v"]]


# ------------------------------------------------------------------ run


def _own(st):
    gq, c = st["gq"], st["case"]
    if c["op"] == "decode":
        return gq.gqa_decode(st["cache"], st["q"], st["table"], st["lens"], st["scale"], out_dtype=st["q"].dtype,
                             window=c["W"], sinks=c["S"])
    if c["op"] == "prefill":
        return gq.gqa_prefill(st["cache"], st["q"], st["q_start"], st["max_new"], st["table"], st["lens"], st["scale"],
                              out_dtype=st["q"].dtype, window=c["W"], sinks=c["S"])
    if c["op"] == "norm_rope":
        q = gq.qk_norm_rope_append(st["cache"], st["q"], st["k"], st["v"], st["table"], st["pos"], rope=st["rope"],
                                   q_weight=st["wq"], k_weight=st["wk"], eps=st["eps"], interleaved=c["inter"],
                                   token_start=st["start"], max_new_tokens=st["max_new"])
        return [q, *st["pool"]]
    table, lens, refs = st["table"], st["lens"], st["refs"]
    if c["op"] == "fork":
        gq.kv_pages_free(refs, table, lens, st["dst"])
        copies = gq.kv_pages_fork(refs, table, lens, st["src"], st["dst"])
        gq.kv_copy_pages(st["caches"], copies)
        gq.kv_pages_reserve(refs, table, lens, 1)
        return [table, lens, refs, st["k"], st["v"]]
    table.copy_(st["table0"])                          # the bookkeeping as it was before the trim
    refs.copy_(st["refs0"])
    gq.kv_pages_trim(refs, table, lens, c["W"], c["S"])
    copies = gq.kv_pages_compact(refs, table, max_copies=st["moves"])
    gq.kv_copy_pages(st["caches"], copies)
    return [table, refs, st["k"], st["v"]]


def run(st):
    if own:
        return _own(st)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "norm_rope": _plain_norm_rope, "fork": _plain_fork,
            "compact": _plain_compact}[st["case"]["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without


def _seen(pos, W, S):
    """How many positions a query at pos sees."""
    return min(pos + 1, W + min(S, max(0, pos + 1 - W))) if pos >= 0 else 0


def work(case):
    if case["op"] in ("decode", "prefill"):
        B, H, K, d, W, S = (case[x] for x in ("B", "H", "K", "d", "W", "S"))
        if case["op"] == "decode":
            new, lens = [case["T"]] * B, _spread(case["lo"], case["hi"], B)
        else:
            new = [n for n, _ in _new_and_before(case)]
            lens = [n + c for n, c in _new_and_before(case)]
        row = 2 * d + 4 if case["cache"] == "fp8" else 4 * d      # K and V of one token and head, scales too
        tokens = sum(min(L, W + n - 1 + min(S, max(0, L - n + 1 - W))) for L, n in zip(lens, new))
        pairs = sum(_seen(p, W, S) for L, n in zip(lens, new) for p in range(L - n, L))
        return dict(bytes=tokens * K * row + 4 * sum(new) * H * d + 4 * tokens / BLOCK, flops=4.0 * d * H * pairs)
    if case["op"] == "norm_rope":
        H, K, d, rot = (case[x] for x in ("H", "K", "d", "rot"))
        n = sum(_spread(case["n_lo"], case["n_hi"], case["B"]))
        row = 2 * d + 4 if case["cache"] == "fp8" else 4 * d
        turns = min(n, case["c_hi"] + case["n_hi"])               # rows of the rotation table
        return dict(bytes=n * (2 * (H + 2 * K) * d + 2 * H * d + K * row) + 4 * rot * turns, flops=n * (H + K) * (4.0 * d + 3 * rot))
    page = 2 * case["K"] * BLOCK * case["d"] * 2 * case["layers"]
    if case["op"] == "fork":
        lens = _spread(case["lo"], case["hi"], case["parents"])
        cut = sum(L % BLOCK != 0 for L in lens) * case["children"]
        entries = sum(-(-L // BLOCK) for L in lens)
        return dict(bytes=2 * cut * page + 4 * entries * (1 + case["children"]), flops=0)
    lens = _spread(case["lo"], case["hi"], case["rows"])
    full = [-(-L // BLOCK) for L in lens]
    gone = [max(0, (L + 1 - case["W"]) // BLOCK - -(-case["S"] // BLOCK)) for L in lens]
    live, pages = sum(full) - sum(gone), sum(full) + 7
    return dict(bytes=2 * page * max(1.0, live * (1 - live / pages)) + 8 * sum(full), flops=0)


# ------------------------------------------------------------------ the definitions in 64 bits


def _sequence(st, which, b, L):
    """Rows 0 .. L-1 of sequence b in 64 bits [L, K, d]; zero where it holds no page."""
    pool, scales = st["pool"][which], st["pool"][2 + which]
    ids = st["table"][b, :-(-L // BLOCK)].long()
    x = pool[ids.clamp(min=0)] if scales is None else pool.view(torch.uint8)[ids.clamp(min=0)].view(pool.dtype)
    x = x.double()
    if scales is not None:
        x = x * scales[ids.clamp(min=0)].double().unsqueeze(-1)
    x[ids < 0] = 0
    return x.transpose(1, 2).reshape(-1, *pool.shape[1::2])[:L]


def _exact_attention(st):
    c = st["case"]
    q = st["q"].double().reshape(-1, c["H"], c["d"])
    out = torch.zeros_like(q)
    if c["op"] == "decode":
        bounds = [c["T"] * b for b in range(c["B"] + 1)]
    else:
        bounds = st["q_start"].tolist()
    for b, L in enumerate(st["lens"].tolist()):
        n = bounds[b + 1] - bounds[b]
        k, v = _sequence(st, 0, b, L), _sequence(st, 1, b, L)
        p = torch.arange(L - n, L, device=q.device)[:, None]
        t = torch.arange(L, device=q.device)
        hidden = (t > p) | ((t <= p - c["W"]) & (t >= c["S"]))
        for h in range(c["H"]):
            s = q[bounds[b]:bounds[b + 1], h] @ k[:, h * c["K"] // c["H"]].T * st["scale"]
            w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
            w = w.masked_fill(hidden.all(-1, keepdim=True), 0)
            out[bounds[b]:bounds[b + 1], h] = w @ v[:, h * c["K"] // c["H"]]
    return out.reshape(st["q"].shape)


def _exact_norm_rope(st):
    c, rot = st["case"], st["case"]["rot"]
    start, pos = st["start"].tolist(), st["pos"].tolist()
    at = torch.cat([torch.arange(p, p + start[b + 1] - start[b]) for b, p in enumerate(pos)]).cuda()
    seq = torch.cat([torch.full((start[b + 1] - start[b],), b) for b in range(len(pos))]).cuda()
    first = torch.arange(0, rot, 2, device="cuda") if c["inter"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if c["inter"] else rot // 2)
    turn = torch.view_as_complex(st["rope"].double())[at][:, None]          # the table that the call is given

    def turned(x, w):
        x = x.double()
        y = x * (x.square().sum(-1, keepdim=True) / c["d"] + st["eps"]).rsqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    page, slot = st["table"].long()[seq, at // BLOCK], at % BLOCK
    outs = [turned(st["q"], st["wq"])]
    scales = []
    for which, x in ((0, turned(st["k"], st["wk"])), (1, st["v"].double())):
        pool = st["pool"][which].double()
        if c["cache"] == "fp8":
            s = (x.abs().amax(-1) / 448).clamp(max=65504).to(torch.float16).double()
            full = st["pool"][2 + which].double()
            full[page, :, slot] = s
            scales.append(full)
            x = x / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(-1)
            x = x.clamp(-448, 448).to(torch.float8_e4m3fn).double()
        pool[page, :, slot] = x
        outs.append(pool)
    return outs + (scales or [None, None])


def _exact_pages(st):
    """The bookkeeping entry by entry, and the copies that follow from it."""
    c = st["case"]
    refs = st["refs"].tolist()
    pairs = []
    if c["op"] == "fork":
        table, lens = st["table"].tolist(), st["lens"].tolist()
        for i in st["dst"].tolist():                                        # the children are empty at first
            lens[i] = 0
        for s, t in zip(st["src"].tolist(), st["dst"].tolist()):
            lens[t] = lens[s]
            for j in range(-(-lens[s] // BLOCK)):
                page = table[s][j]
                if j == lens[s] // BLOCK:
                    pairs.append((page, refs.index(0)))
                    page = pairs[-1][1]
                table[t][j] = page
                refs[page] += 1
        for b, row in enumerate(table):
            if row[lens[b] // BLOCK] < 0:
                row[lens[b] // BLOCK] = refs.index(0)
                refs[row[lens[b] // BLOCK]] = 1
        heads = [_i32(table), _i32(lens), _i32(refs)]
    else:
        table = st["table0"].tolist()
        for row, L in zip(table, st["lens"].tolist()):
            for j in range(len(row)):
                if row[j] >= 0 and j * BLOCK >= c["S"] and j * BLOCK + BLOCK <= L + 1 - c["W"]:
                    refs[row[j]] -= 1
                    row[j] = -1
        live = [p for p, r in enumerate(refs) if r > 0]
        holes = [p for p in range(len(live)) if refs[p] == 0]
        pairs = list(zip([p for p in reversed(live) if p >= len(live)], holes))
        to = dict(pairs)
        table = [[to.get(p, p) for p in row] for row in table]
        for s, t in pairs:
            refs[s], refs[t] = 0, refs[s]
        heads = [_i32(table), _i32(refs)]
    k, v = st["k"].clone(), st["v"].clone()
    for x in (k, v):
        for s, t in pairs:
            x[:, t] = x[:, s]
    return heads + [k, v]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("decode", "prefill"):
        return _exact_attention(st)
    return _exact_norm_rope(st) if case["op"] == "norm_rope" else _exact_pages(st)
