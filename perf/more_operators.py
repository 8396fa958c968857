"""What the operators around shared pages cost: the cases and their plain forms.

Three operators, as a server calls them whose sequences share prompts:

* ``shared`` -- decode attention of a batch whose rows share long prefixes, each prefix
                attended once for all rows of its group
* ``groups`` -- which rows of the block tables share their first pages (the plan of ``shared``)
* ``read``   -- cached rows back as dense K and V, from any cache type

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits (or whole
numbers); with ``own`` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
LIMIT = {"int8": 127.0, "fp8": 448.0, "int4": 7.0, "int4kc": 7.0}     # largest code of each coded cache


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one answer sampled four ways on an idle server: latency of a step
        dict(name="shared_samples", op="shared", groups=1, m_lo=4, m_hi=4, p_lo=512, p_hi=512, t_lo=1, t_hi=40,
             alone=0, T=1, H=32, K=8, d=128, cache="bf16", q="bf16"),
        # a full batch of chats behind one system prompt
        dict(name="shared_system_prompt", op="shared", groups=1, m_lo=64, m_hi=64, p_lo=4096, p_hi=4096, t_lo=100,
             t_hi=700, alone=0, T=1, H=32, K=8, d=128, cache="bf16", q="bf16"),
        # questions about one long document, eight heads per group
        dict(name="shared_document", op="shared", groups=1, m_lo=32, m_hi=32, p_lo=32768, p_hi=32768, t_lo=30, t_hi=500,
             alone=0, T=1, H=64, K=8, d=128, cache="bf16", q="bf16"),
        # forked requests of several users verifying drafts, some rows on their own
        dict(name="shared_forks_verify", op="shared", groups=9, m_lo=2, m_hi=12, p_lo=300, p_hi=5001, t_lo=3, t_hi=333,
             alone=5, T=3, H=24, K=8, d=64, cache="f16", q="f16"),
        # a large batch on an int8 cache behind four prompts
        dict(name="shared_int8_batch", op="shared", groups=4, m_lo=32, m_hi=32, p_lo=8192, p_hi=8192, t_lo=100, t_hi=900,
             alone=0, T=1, H=64, K=8, d=128, cache="int8", q="bf16"),
        # the plan of a small batch, made after a fork
        dict(name="groups_small", op="groups", B=16, roots=2, p_lo=20, p_hi=40, sub=3, s_lo=1, s_hi=5, t_lo=1, t_hi=8),
        # a batch of forked conversations, two levels of shared pages
        dict(name="groups_batch", op="groups", B=256, roots=12, p_lo=50, p_hi=400, sub=4, s_lo=3, s_hi=100, t_lo=1,
             t_hi=60),
        # as many rows and as long contexts as a pool serves
        dict(name="groups_large", op="groups", B=2048, roots=40, p_lo=100, p_hi=1500, sub=8, s_lo=10, s_hi=200, t_lo=1,
             t_hi=100),
        # one chunk of a request's context
        dict(name="read_chunk", op="read", B=1, n_lo=512, n_hi=512, c_lo=100, c_hi=100, K=8, d=128, cache="int8",
             out="bf16"),
        # ragged contexts of a small model off an FP8 cache
        dict(name="read_fp8_ragged", op="read", B=37, n_lo=1, n_hi=4001, c_lo=0, c_hi=777, K=4, d=64, cache="fp8",
             out="f16"),
        # whole prompts of a cache whose K is scaled by channel
        dict(name="read_int4kc_prompts", op="read", B=16, n_lo=8192, n_hi=8192, c_lo=0, c_hi=0, K=8, d=128,
             cache="int4kc", out="bf16"),
        # whole prompts of a 16-bit cache, widened for a comparison in 32 bits
        dict(name="read_bf16_prompts", op="read", B=8, n_lo=3000, n_hi=8192, c_lo=0, c_hi=0, K=8, d=128, cache="bf16",
             out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "groups", "read"])
    d = rng.choice([64, 128])
    K = rng.choice([1, 2, 4, 8])
    if op == "shared":
        cache = rng.choice(["bf16", "f16", "bf16", "f16", "int8", "fp8", "int4"])
        T = rng.choice([1, 1, 1, 2, 3, 4])
        groups = _log(rng, 1, 12)
        m_lo = _log(rng, 2, 64)
        m_hi = rng.randint(m_lo, 64)
        p_lo = _log(rng, 16, 20000)
        p_hi = rng.randint(p_lo, 32768)
        t_lo = _log(rng, T, 900)
        groups = max(1, min(groups, 8_000_000 // ((p_hi + 1000) * K * m_hi), 128 // m_hi))
        m_hi = max(2, min(m_hi, 8_000_000 // ((p_hi + 1000) * K * groups)))
        return dict(op=op, groups=groups, m_lo=min(m_lo, m_hi), m_hi=m_hi, p_lo=p_lo, p_hi=p_hi, t_lo=t_lo,
                    t_hi=rng.randint(t_lo, 1000), alone=rng.choice([0, 0, 1, 5]), T=T, H=K * rng.randint(1, 8), K=K, d=d,
                    cache=cache, q=cache if cache in DTYPES else rng.choice(["bf16", "f16"]))
    if op == "groups":
        B = _log(rng, 1, 2048)
        p_lo, s_lo, t_lo = _log(rng, 1, 1000), _log(rng, 1, 150), _log(rng, 1, 80)
        return dict(op=op, B=B, roots=_log(rng, 1, max(2, B // 4)), p_lo=p_lo, p_hi=rng.randint(p_lo, 1500),
                    sub=rng.randint(1, 9), s_lo=s_lo, s_hi=rng.randint(s_lo, 200), t_lo=t_lo, t_hi=rng.randint(t_lo, 100))
    n_lo = _log(rng, 1, 4000)
    n_hi = rng.randint(n_lo, 8192)
    c_lo = _log(rng, 1, 1000)
    return dict(op=op, B=max(1, min(_log(rng, 1, 64), 131072 // n_hi)), n_lo=n_lo, n_hi=n_hi, c_lo=c_lo,
                c_hi=rng.randint(c_lo, 2000), K=K, d=d,
                cache=rng.choice(["bf16", "f16", "f32", "int8", "fp8", "int4", "int4kc"]),
                out=rng.choice(["bf16", "f16", "f32"]))


# ------------------------------------------------------------------ inputs


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the same for every seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _order(n, seed):
    return torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def _normal(shape, dtype, gen):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


def _pack(codes):
    """4-bit codes two to a byte, the even element in the low nibble."""
    c = codes.to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _quantise(x, kind, dim):
    """Codes of x and their fp16 scales, one per row of `dim`, as the library's appends make them."""
    s = (x.abs().amax(dim, keepdim=True) / LIMIT[kind]).clamp(max=65504.0).to(torch.float16)
    y = x / s.float().clamp(min=2.0 ** -24)
    y = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn) if kind == "fp8" else y.round().clamp(-LIMIT[kind], LIMIT[kind]).to(torch.int8)
    return _pack(y) if kind.startswith("int4") else y, s.squeeze(dim)


def _pool(case, pages, gen):
    """k, v and their scales (None for float types) of one paged cache."""
    kind, shape = case["cache"], (pages, case["K"], BLOCK, case["d"])
    if kind in DTYPES:
        return [_normal(shape, DTYPES[kind], gen) for _ in range(2)] + [None, None]
    k, ks = _quantise(_normal(shape, torch.float32, gen), kind, 2 if kind == "int4kc" else 3)
    v, vs = _quantise(_normal(shape, torch.float32, gen), kind, 3)
    return [k, v, ks, vs]


def _cache(gq, case, k, v, ks, vs):
    n, K, d = k.shape[0], case["K"], case["d"]
    code = {"int4": gq.GQA_DTYPE_I4, "int4kc": gq.GQA_DTYPE_I4_KC}.get(case["cache"])
    return gq.PagedKVCache(k, v, n, K, d, K * BLOCK * d, BLOCK * d, d, ks, vs, code)


def _fill(rows, seed):
    """Block table of rows given as runs [(name, pages)]: runs of one name are the same pages (the
    first ones of the longest), shuffled over the pool; -1 past a row's end."""
    longest = {}
    for name, n in (run for r in rows for run in r):
        longest[name] = max(n, longest.get(name, 0))
    ends = np.cumsum(list(longest.values()))
    first = dict(zip(longest, ends - list(longest.values())))
    perm = np.array(_order(int(ends[-1]), seed), dtype=np.int32)
    table = np.full((len(rows), max(sum(n for _, n in r) for r in rows) + 1), -1, dtype=np.int32)
    for b, r in enumerate(rows):
        ids = np.concatenate([np.arange(first[name], first[name] + n) for name, n in r])
        table[b, :len(ids)] = perm[ids]
    return torch.from_numpy(table).cuda(), int(ends[-1])


def _shared_rows(case):
    """(group or -1, shared tokens, context length) of every row, in order of the groups."""
    rows = []
    for g, (m, p) in enumerate(zip(_spread(case["m_lo"], case["m_hi"], case["groups"]),
                                   reversed(_spread(case["p_lo"], case["p_hi"], case["groups"])))):
        rows += [(g, p, p + t) for t in _spread(case["t_lo"], case["t_hi"], m)]
    if case["alone"]:
        rows += [(-1, 0, t) for t in _spread(case["t_lo"], case["p_lo"] + case["t_hi"], case["alone"])]
    return rows


def _forest(case):
    """(page runs [(name, pages)], full pages, tokens) of every row: a root's pages, those of a fork of it, its own.
    Every seventh row shares nothing, every eleventh was cut back into its root's pages."""
    B, roots = case["B"], case["roots"]
    p, s, t = _spread(case["p_lo"], case["p_hi"], roots), _spread(case["s_lo"], case["s_hi"], 5), _spread(case["t_lo"], case["t_hi"], 13)
    rows = []
    for i in range(B):
        r, k = i % roots, i // roots
        runs = [(("root", r), p[r]), (("fork", r, k // case["sub"]), s[k // case["sub"] % 5]), (("own", i), t[i % 13])]
        if i % 7 == 6:
            runs = [(("own", i), p[r] + t[i % 13])]
        elif i % 11 == 10:
            runs = [(("root", r), 1 + p[r] * (i % 5) // 5)]
        rows.append((runs, BLOCK * sum(n for _, n in runs) - i % 16))
    return rows


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case=case)
    if case["op"] == "groups":
        rows = _forest(case)
        rows = [rows[i] for i in _order(len(rows), seed)]
        st["table"], _ = _fill([runs for runs, _ in rows], seed)
        st["lens"] = _i32([L for _, L in rows])
        if own:
            import gqa_decode_attention_kv_gb300 as gq
            st["gq"] = gq
        return st
    if case["op"] == "shared":
        rows = _shared_rows(case)
        rows = [rows[i] for i in _order(len(rows), seed)]
        # a fork shares full pages: the tokens behind them are the row's own
        table, pages = _fill([[(("prefix", g), p // BLOCK), (("own", b), -(-L // BLOCK) - p // BLOCK)]
                              for b, (g, p, L) in enumerate(rows)], seed)
        st["lens"] = _i32([L for _, _, L in rows])
        shape = (len(rows), case["T"], case["H"], case["d"])
        st["q"] = _normal(shape if case["T"] > 1 else (shape[0], *shape[2:]), DTYPES[case["q"]], gen)
        st["scale"] = 1.0 / math.sqrt(case["d"])
    else:
        n = _spread(case["n_lo"], case["n_hi"], case["B"])
        c = list(reversed(_spread(case["c_lo"], case["c_hi"], case["B"])))
        order = _order(case["B"], seed)
        n, c = [n[i] for i in order], [c[i] for i in order]
        table, pages = _fill([[(b, -(-(n[b] + c[b]) // BLOCK))] for b in range(case["B"])], seed)
        st["pos"], st["start"] = _i32(c), _i32([0] + np.cumsum(n).tolist())
        st["max"], st["total"] = max(n), sum(n)
    st["table"], st["pool"] = table, _pool(case, pages, gen)
    if own:
        import gqa_decode_attention_kv_gb300 as gq
        st["gq"], st["cache"] = gq, _cache(gq, case, *st["pool"])
        if case["op"] == "shared":                     # made at the fork and kept for the steps that follow
            st["plan"] = gq.kv_pages_groups(table, st["lens"])
    return st


# ------------------------------------------------------------------ plain forms


def _unpack(w):
    """4-bit codes of packed bytes as whole numbers in 32 bits."""
    c = torch.stack((w & 15, w >> 4), -1).flatten(-2).to(torch.int32)
    return torch.where(c > 7, c - 16, c)


def _rows_of(st, which, page, slot):
    """Cached rows at (page, slot) as fp32 [..., K, d]."""
    kind, pool, scale = st["case"]["cache"], st["pool"][which], st["pool"][2 + which]
    if kind == "fp8":
        x = pool.view(torch.uint8)[page, :, slot].view(pool.dtype).float()
    else:
        x = pool[page, :, slot]
        x = _unpack(x).float() if kind.startswith("int4") else x.float()
    if scale is None:
        return x
    return x * (scale[page].float() if which == 0 and kind == "int4kc" else scale[page, :, slot].float().unsqueeze(-1))


def _plain_shared(st):
    c, q, L = st["case"], st["q"], st["lens"].long()
    T, H, K, d = (c[x] for x in ("T", "H", "K", "d"))
    B, G = q.shape[0], H // K
    t = torch.arange(int(st["table"].shape[1] - 1) * BLOCK, device=q.device)
    page = st["table"].long()[:, t // BLOCK].clamp(min=0)
    k, v = (_rows_of(st, i, page, (t % BLOCK).expand(B, -1)).transpose(1, 2) for i in range(2))
    qf = q.view(B, T, K, G, d).permute(0, 2, 1, 3, 4).reshape(B, K, T * G, d).float()
    at = L[:, None] - T + torch.arange(T, device=q.device)
    see = t <= at[:, :, None]                                                  # [B, T, t]
    see = see[:, None, :, None].expand(B, 1, T, G, -1).reshape(B, 1, T * G, -1)
    s = (qf @ k.transpose(2, 3) * st["scale"]).masked_fill(~see, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = p @ v / p.sum(-1, keepdim=True)
    return o.view(B, K, T, G, d).permute(0, 2, 1, 3, 4).reshape(q.shape).to(q.dtype)


def _plain_groups(st):
    table, full = st["table"], torch.div(st["lens"].long(), BLOCK, rounding_mode="floor")
    B = len(full)
    row = torch.arange(B, device=table.device)
    first = torch.where((full > 0) & (table[:, 0] >= 0), table[:, 0].long(), -1 - row)   # no full page: its own leader
    leader = torch.where(first[:, None] == first, row, B).amin(1)
    same = (table == table[leader]) & (table >= 0) & \
        (torch.arange(table.shape[1], device=table.device) < torch.minimum(full, full[leader])[:, None])
    run = torch.cumprod(same.to(torch.int32), 1).sum(1)                        # pages shared with the leader
    kin = leader[:, None] == leader
    count = (kin & (run >= run[:, None])).sum(1)                               # rows that share as many
    saved = run * (count - 1)
    best = torch.where(kin, saved, -1).amax(1)                                 # of the row's leader
    blocks = torch.where(kin & (saved == best[:, None]), run, 0).amax(1)
    member = (best > 0) & (run >= blocks)
    head = member & (leader == row)
    total = head.sum()
    group = torch.where(member, (torch.cumsum(head, 0) - 1)[leader], torch.full_like(row, -1))
    before = (kin & member & (row < row[:, None])).sum(1)                      # members of the group before the row
    size = torch.zeros(B, dtype=torch.int64, device=table.device).index_add_(0, group.clamp(min=0), member.long())
    ends = torch.cumsum(size, 0)
    start = torch.cat((torch.zeros_like(ends[:1]), ends))
    slot = torch.where(member, start[group.clamp(min=0)] + before, torch.full_like(row, -1))
    at = torch.where(member, slot, B)
    rows = torch.full((B + 1,), -1, dtype=torch.int64, device=table.device).scatter_(0, at, row)[:B]
    at = torch.where(head, group, B)
    shared = torch.zeros(B + 1, dtype=torch.int64, device=table.device).scatter_(0, at, blocks)[:B]
    return [x.int() for x in (torch.stack((total, member.sum())), start, shared, rows, slot, group)]


def _plain_read(st):
    start = st["start"].long()
    token = torch.arange(st["total"], device=start.device)
    b = torch.searchsorted(start, token, right=True) - 1
    pos = st["pos"].long()[b] + token - start[b]
    page = st["table"].long()[b, pos // BLOCK]
    return [_rows_of(st, i, page, pos % BLOCK).to(DTYPES[st["case"]["out"]]) for i in range(2)]


# ------------------------------------------------------------------ run


def _own(st):
    gq, c = st["gq"], st["case"]
    if c["op"] == "shared":
        return gq.gqa_decode_shared(st["cache"], st["q"], st["table"], st["lens"], st["scale"], st["plan"],
                                    out_dtype=st["q"].dtype, max_group=c["m_hi"])
    if c["op"] == "groups":
        plan = gq.kv_pages_groups(st["table"], st["lens"])
        return [plan.count, plan.start, plan.blocks, plan.rows, plan.slot, plan.group]
    return list(gq.kv_read(st["cache"], st["table"], st["pos"], token_start=st["start"], max_tokens=st["max"],
                           total_tokens=st["total"], dtype=DTYPES[c["out"]]))


def run(st):
    if own:
        return _own(st)
    return {"shared": _plain_shared, "groups": _plain_groups, "read": _plain_read}[st["case"]["op"]](st)


# ------------------------------------------------------------------ what a pass cannot do without


def _row_bytes(case):
    """K and V of one cached token and head, their scales too."""
    d = case["d"]
    return {"f32": 8.0 * d, "bf16": 4.0 * d, "f16": 4.0 * d, "int8": 2.0 * d + 4, "fp8": 2.0 * d + 4, "int4": d + 4.0,
            "int4kc": d + 2.0 + 2.0 * d / BLOCK}[case["cache"]]


def work(case):
    if case["op"] == "shared":
        rows = _shared_rows(case)
        held = {g: p // BLOCK * BLOCK for g, p, _ in rows if g >= 0}
        tokens = sum(held.values()) + sum(L - held.get(g, 0) for g, _, L in rows)
        T, H, d = case["T"], case["H"], case["d"]
        pairs = sum(max(0, p + 1) for _, _, L in rows for p in range(L - T, L))
        return dict(bytes=tokens * case["K"] * _row_bytes(case) + 4.0 * len(rows) * T * H * d + 4.0 * tokens / BLOCK,
                    flops=4.0 * d * H * pairs)
    if case["op"] == "groups":
        # the pages that a row has in common with its root, and the one after them
        pages = sum(1 + sum(n for name, n in runs if name[0] == "root") for runs, _ in _forest(case))
        return dict(bytes=4.0 * (pages + 6 * case["B"]), flops=0)
    n = sum(_spread(case["n_lo"], case["n_hi"], case["B"]))
    wide = 4 if case["out"] == "f32" else 2
    return dict(bytes=n * case["K"] * (_row_bytes(case) + 2.0 * wide * case["d"]), flops=0)


# ------------------------------------------------------------------ the definitions in 64 bits


def _decoded(st, which, pages):
    """Whole pages in 64 bits [pages, 16, K, d]."""
    kind = st["case"]["cache"]
    raw = st["pool"][which]
    raw = raw.view(torch.uint8)[pages].view(raw.dtype) if kind == "fp8" else raw[pages]
    if kind.startswith("int4"):
        both = torch.stack((raw.to(torch.int16) << 12 >> 12, raw.to(torch.int16) << 8 >> 12), -1)
        raw = both.reshape(*raw.shape[:-1], -1)
    x = raw.double()
    if kind not in DTYPES:
        s = st["pool"][2 + which][pages].double()
        x = x * (s[:, :, None, :] if which == 0 and kind == "int4kc" else s[..., None])
    return x.permute(0, 2, 1, 3)


def _context(st, which, b, lo, hi):
    """Cached rows lo .. hi-1 of sequence b in 64 bits [hi - lo, K, d]."""
    j0, j1 = lo // BLOCK, -(-hi // BLOCK)
    return _decoded(st, which, st["table"][b, j0:j1].long()).flatten(0, 1)[lo - j0 * BLOCK:hi - j0 * BLOCK]


def _exact_shared(st):
    c = st["case"]
    T, K, d = c["T"], c["K"], c["d"]
    q = st["q"].double().reshape(-1, T, K, c["H"] // K, d)
    out = torch.empty_like(q)
    for b, L in enumerate(st["lens"].tolist()):
        k, v = (_context(st, i, b, 0, L) for i in range(2))
        for i in range(T):
            n = L - T + i + 1
            w = torch.softmax(torch.einsum("khd,nkd->khn", q[b, i], k[:n]) * st["scale"], -1)
            out[b, i] = torch.einsum("khn,nkd->khd", w, v[:n])
    return out.reshape(st["q"].shape)


def _exact_groups(st):
    """Row by row from the tables' entries."""
    table, lens = st["table"].cpu().numpy(), st["lens"].tolist()
    rows = [table[b, :L // BLOCK] for b, L in enumerate(lens)]
    kin = {}
    for b, r in enumerate(rows):
        if len(r) and r[0] >= 0:
            kin.setdefault(int(r[0]), []).append(b)
    B = len(rows)
    groups = []
    for members in kin.values():
        lead = rows[members[0]]
        runs = {}
        for b in members:
            n = min(len(lead), len(rows[b]))
            ok = (lead[:n] == rows[b][:n]) & (lead[:n] >= 0)
            runs[b] = n if ok.all() else int(np.argmin(ok))
        shared = sorted(runs.values(), reverse=True)
        gain, blocks = max((p * i, p) for i, p in enumerate(shared))
        if gain > 0:
            groups.append((members[0], blocks, [b for b in members if runs[b] >= blocks]))
    groups.sort()
    start, blocks, order, slot, group = [0], [], [], [-1] * B, [-1] * B
    for g, (_, p, members) in enumerate(groups):
        for b in members:
            slot[b], group[b] = len(order), g
            order.append(b)
        start.append(len(order))
        blocks.append(p)
    return [_i32([len(groups), len(order)]), _i32(start + [len(order)] * (B - len(groups))),
            _i32(blocks + [0] * (B - len(groups))), _i32(order + [-1] * (B - len(order))), _i32(slot), _i32(group)]


def _exact_read(st):
    start, pos = st["start"].tolist(), st["pos"].tolist()
    return [torch.cat([_context(st, i, b, p, p + start[b + 1] - start[b]) for b, p in enumerate(pos)]) for i in range(2)]


def exact(case, seed):
    st = prepare(case, seed)
    return {"shared": _exact_shared, "groups": _exact_groups, "read": _exact_read}[case["op"]](st)
