"""Batches whose rows share pages, for the tests of the operators around them: tables,
caches and the values they hold, on the host in fp64."""
from __future__ import annotations

from types import SimpleNamespace

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LIMIT = {"int8": 127.0, "fp8": 448.0, "int4": 7.0, "int4kc": 7.0}


def pool(kind, pages, K, d, seed, gq, device="cuda", order="pktd", amp=1.0):
    """A cache of N(0, amp^2) values, and those values as it holds them: two fp64 arrays
    [pages, 16, K, d]. ``order`` places the page, kv-head and token axes in memory."""
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(pages, 16, K, d, generator=g) * amp for _ in range(2)]
    if kind in DTYPES:
        held = [t.to(DTYPES[kind]) for t in x]
        axes = {"p": 0, "t": 1, "k": 2, "d": 3}
        perm = [axes[c] for c in order]
        stored = [t.permute(perm).contiguous().to(device) for t in held]
        back = dict(zip(order, stored[0].stride()))
        cache = gq.PagedKVCache(stored[0], stored[1], pages, K, d, back["p"], back["k"], back["t"])
        return cache, [t.double().numpy() for t in held]
    held, store = [], []
    for i, t in enumerate(x):
        per_channel = kind == "int4kc" and i == 0
        dim = 1 if per_channel else 3
        s = (t.abs().amax(dim, keepdim=True) / LIMIT[kind]).to(torch.float16)
        y = (t / s.float()).clamp(-LIMIT[kind], LIMIT[kind])
        if kind == "fp8":
            code = y.to(torch.float8_e4m3fn)
            value = code.float().double()
        else:
            code = y.round().to(torch.int8)
            value = code.double()
        held.append((value * s.double()).numpy())
        code = code.view(torch.uint8) if kind == "fp8" else code
        code = code.permute(0, 2, 1, 3).contiguous()                 # [pages, K, 16, d]
        if kind.startswith("int4"):
            n = code.to(torch.int32) & 15
            code = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
        elif kind == "fp8":
            code = code.view(torch.float8_e4m3fn)
        scale = s.squeeze(dim) if per_channel else s.squeeze(3).permute(0, 2, 1).contiguous()
        store.append((code.to(device), scale.to(device)))
    dt = {"int4": gq.GQA_DTYPE_I4, "int4kc": gq.GQA_DTYPE_I4_KC}.get(kind)
    cache = gq.PagedKVCache(store[0][0], store[1][0], pages, K, d, K * 16 * d, 16 * d, d, store[0][1], store[1][1], dt)
    return cache, held


def batch(groups, alone, seed, spare=3, columns=1):
    """Tables of rows that share pages. groups: (shared blocks, [context lengths]) each,
    alone: context lengths. Rows are shuffled; entries past a row's end are -1."""
    rng = np.random.default_rng(seed)
    rows, n = [], 0
    for blocks, lens in groups:
        shared = list(range(n, n + blocks))
        n += blocks
        for L in lens:
            own = max(0, -(-L // 16) - blocks)
            rows.append((shared[:-(-L // 16)] + list(range(n, n + own)), L))
            n += own
    for L in alone:
        rows.append((list(range(n, n + -(-L // 16))), L))
        n += -(-L // 16)
    perm = rng.permutation(n + spare)
    order = rng.permutation(len(rows))
    wide = max([len(r) for r, _ in rows] + [1]) + columns
    table = np.full((len(rows), wide), -1, dtype=np.int32)
    lens = np.zeros(len(rows), dtype=np.int32)
    for i, o in enumerate(order):
        ids, lens[i] = rows[o]
        table[i, :len(ids)] = perm[ids]
    return SimpleNamespace(table=table, lens=lens, pages=n + spare, order=order)


def rows_of(values, table, b, L):
    """Rows 0 .. L-1 of sequence b from page values [pages, 16, K, d]."""
    return np.concatenate([values[p] for p in table[b, :-(-L // 16)]])[:L] if L else np.zeros((0, *values.shape[2:]))


def attend(q, values, table, lens, scale):
    """fp64 [B, T, H, d]: query i of row b at position L - T + i over its context."""
    B, T, H, d = q.shape
    K = values[0].shape[2]
    out = np.zeros(q.shape)
    for b in range(B):
        L = int(lens[b])
        k, v = rows_of(values[0], table, b, L), rows_of(values[1], table, b, L)
        for i in range(T):
            n = L - T + i + 1
            if n <= 0:
                continue
            s = np.einsum("kgd,nkd->kgn", q[b, i].reshape(K, H // K, d), k[:n]) * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            out[b, i] = np.einsum("kgn,nkd->kgd", w / w.sum(-1, keepdims=True), v[:n]).reshape(H, d)
    return out


def plan_of(table, lens, min_blocks=1):
    """The groups entry by entry: lists (count, start, blocks, rows, slot, group)."""
    B = len(lens)
    full = [L // 16 if 0 <= L <= 16 * table.shape[1] else 0 for L in lens.tolist()]
    leader, run = list(range(B)), [0] * B
    for b in range(B):
        if not full[b] or table[b, 0] < 0:
            continue
        leader[b] = next(r for r in range(b + 1) if full[r] and table[r, 0] == table[b, 0])
        while run[b] < min(full[b], full[leader[b]]) and 0 <= table[b, run[b]] == table[leader[b], run[b]]:
            run[b] += 1
    count, start, blocks, rows, slot, group = [0, 0], [0], [], [], [-1] * B, [-1] * B
    for lead in range(B):
        if leader[lead] != lead:
            continue
        kin = [b for b in range(B) if leader[b] == lead]
        best = (0, 0)
        for p in {run[b] for b in kin if run[b] >= max(1, min_blocks)}:
            best = max(best, (p * (sum(run[b] >= p for b in kin) - 1), p))
        if best[0] == 0:
            continue
        for b in kin:
            if run[b] >= best[1]:
                slot[b], group[b] = len(rows), count[0]
                rows.append(b)
        count[0] += 1
        blocks.append(best[1])
        start.append(len(rows))
    count[1] = len(rows)
    start += [len(rows)] * (B + 1 - len(start))
    blocks += [0] * (B - len(blocks))
    return count, start, blocks, rows + [-1] * (B - len(rows)), slot, group
