"""Plain fp64 forms the operator tests compare with: dense arrays, no paging,
nothing shared with the CUDA library."""
from __future__ import annotations

import numpy as np
import torch


def attend(q, k, v, scale, window=0, sinks=0):
    """Causal attention of the last T positions of one sequence, fp64.

    q [T, H, d] at positions L-T .. L-1 over k, v [L, K, d]; a query at p sees
    t <= p with t > p - window or t < sinks (window 0: every t <= p). A query
    that sees nothing (a negative position) gets zeros."""
    T, H, _ = q.shape
    L, K, _ = k.shape
    p = np.arange(L - T, L)[:, None]
    t = np.arange(L)[None, :]
    see = t <= p
    if window > 0:
        see &= (t > p - window) | (t < sinks)
    out = np.zeros((T, H, v.shape[2]))
    for h in range(H):
        g = h // (H // K)
        for i in range(T):
            idx = np.nonzero(see[i])[0]
            if idx.size == 0:
                continue
            s = k[idx, g].astype(np.float64) @ q[i, h].astype(np.float64) * scale
            w = np.exp(s - s.max())
            out[i, h] = (w / w.sum()) @ v[idx, g].astype(np.float64)
    return out


def cached_rows(case, which, b, L=None):
    """Rows 0 .. L-1 of sequence b's K or V as the cache holds them, fp64 [L, K, d]."""
    import oracle
    L = int(case.context_lens[b]) if L is None else L
    K, d = case.num_kv_heads, case.head_dim
    nblk = -(-L // 16)
    ids = case.block_table[b, :nblk].long().cpu()
    pool = (case.k_cache if which == "k" else case.v_cache).detach()
    sc = case.k_scale if which == "k" else case.v_scale
    if case.cache_dtype in ("bf16", "f16", "f32"):
        x = pool.float().cpu()
        if case.stride_token != case.head_dim:          # contiguous [B, S_pad, K, d]
            return x[b, :L].double().numpy()
        return x[ids].permute(0, 2, 1, 3).reshape(-1, K, d)[:L].double().numpy()
    scales = sc.cpu()[ids].double()
    raw = pool.view(torch.uint8).cpu()[ids].numpy()
    if case.cache_dtype == "i8":
        codes = raw.view(np.int8).astype(np.float64)
    elif case.cache_dtype == "fp8":
        codes = oracle.e4m3_to_f64(raw)
    else:
        codes = oracle.unpack_int4(raw).astype(np.float64)
    codes = torch.from_numpy(np.asarray(codes, dtype=np.float64)).reshape(nblk, K, 16, d)
    if which == "k" and case.cache_dtype == "i4kc":
        x = codes * scales[:, :, None, :]
    else:
        x = codes * scales[..., None]
    return x.permute(0, 2, 1, 3).reshape(-1, K, d)[:L].numpy()


def attend_case(case, window=0, sinks=0):
    """attend() for every sequence of a decode case: [B, (T,) H, d]."""
    q = case.q.detach().double().cpu().numpy()
    one = q.ndim == 3
    outs = []
    for b in range(case.batch):
        L = int(case.context_lens[b])
        qb = q[b][None] if one else q[b]
        if L == 0:
            outs.append(np.zeros_like(qb))
            continue
        k, v = cached_rows(case, "k", b), cached_rows(case, "v", b)
        T = qb.shape[0]
        n = min(T, L)                                    # queries before position 0 see nothing
        o = np.zeros_like(qb)
        o[T - n:] = attend(qb[T - n:], k, v, case.scale, window, sinks)
        outs.append(o)
    out = np.stack(outs)
    return out[:, 0] if one else out
