"""The pages of a pool (reserve, fork, free, trim, compact) and the copies of page
data, against the same written out entry by entry, through the C ABI. Everything here
is whole numbers or copied bits: results are compared exactly."""
import numpy as np
import pytest
import torch

import gqa_inputs as gi
from helpers import TOL, max_abs_err
from plain import attend_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    from gqa_decode_attention_kv_gb300 import build
    build.build()
    import gqa_decode_attention_kv_gb300 as m
    return m


class Pool:
    """The plain form: lists, lowest free page first."""

    def __init__(self, refs, table, lens):
        self.refs, self.table, self.lens = list(refs), [list(r) for r in table], list(lens)

    def lowest(self):
        return self.refs.index(0) if 0 in self.refs else None

    def reserve(self, new):
        flag, out = 0, False
        free = [p for p, r in enumerate(self.refs) if r == 0]
        for b, row in enumerate(self.table):
            L, n = self.lens[b], new[b]
            if L < 0 or n < 0 or L + n > 16 * len(row):
                flag |= 4
                continue
            need = [j for j in range(-(-L // 16), -(-(L + n) // 16)) if row[j] < 0]
            if not need:
                continue
            if out or len(need) > len(free):
                flag, out = flag | 32, True
                continue
            for j in need:
                row[j] = free.pop(0)
                self.refs[row[j]] = 1
        return flag

    def release(self, b, j):
        p, self.table[b][j] = self.table[b][j], -1
        if p < 0:
            return 0
        if p >= len(self.refs):
            return 1
        if self.refs[p] <= 0:
            return 64
        self.refs[p] -= 1
        return 0

    def free(self, rows):
        flag = 0
        for b in rows:
            if not 0 <= b < len(self.table):
                flag |= 16
                continue
            for j in range(len(self.table[b])):
                flag |= self.release(b, j)
            self.lens[b] = 0
        return flag

    def trim(self, W, S):
        flag = 0
        for b, row in enumerate(self.table):
            if not 0 <= self.lens[b] <= 16 * len(row):
                flag |= 2
                continue
            for j in range(len(row)):
                if 16 * j >= S and 16 * (j + 1) <= self.lens[b] + 1 - W:
                    flag |= self.release(b, j)
        return flag

    def fork(self, src, dst):
        flag, pairs, rows, done, out = 0, [], [], [], False
        claimed = {}
        for i, d in enumerate(dst):
            if 0 <= d < len(self.table):
                claimed.setdefault(d, i)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        for i, (s, d) in enumerate(zip(src, dst)):
            rows.append((-1, -1))
            if not (0 <= s < len(self.table) and 0 <= d < len(self.table)) or claimed[d] != i or s in claimed \
                    or self.lens[d] != 0 or self.table[d][0] >= 0:
                flag |= 16
                continue
            L = self.lens[s]
            if not 0 <= L <= 16 * len(self.table[s]):
                flag |= 2
                continue
            fresh = None
            if L % 16:
                last = self.table[s][L // 16]
                if not 0 <= last < len(self.refs):
                    flag |= 1
                    continue
                if out or not free:
                    flag, out = flag | 32, True
                    continue
                fresh = free.pop(0)
                pairs.append((last, fresh))
            rows[-1] = (s, d)
            done.append((s, d, L, fresh))
        for s, d, L, fresh in done:
            new = [-1] * len(self.table[d])
            for j in range(-(-L // 16)):
                p = self.table[s][j]
                if fresh is not None and j == L // 16:
                    p = fresh
                    self.refs[p] = 1
                elif p >= len(self.refs):
                    flag, p = flag | 1, -1
                elif p >= 0:
                    self.refs[p] += 1
                new[j] = p
            self.table[d], self.lens[d] = new, L
        return flag, pairs, rows

    def compact(self, most):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        pairs = list(zip([p for p in reversed(live) if p >= n], holes))[:most]
        to = dict(pairs)
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for s, t in pairs:
            self.refs[t], self.refs[s] = self.refs[s], 0
        return pairs, n


def cuda(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def random_pool(rng, pages, rows, blocks, fill=0.7, max_len=None):
    """A pool with shared pages, ragged rows and empty rows."""
    refs, table, lens = [0] * pages, [[-1] * blocks for _ in range(rows)], [0] * rows
    order = rng.permutation(pages).tolist()
    for b in range(rows):
        if rng.random() < 0.25:
            continue
        L = int(rng.integers(1, (max_len or 16 * blocks) + 1))
        for j in range(-(-L // 16)):
            if not order or len(order) < (1 - fill) * pages:
                L = 16 * j
                break
            p = order.pop()
            table[b][j] = p
            refs[p] += 1
        lens[b] = L
    return Pool(refs, table, lens)


def same(pool, refs, table, lens):
    assert refs.tolist() == pool.refs
    assert table.tolist() == pool.table
    assert lens.tolist() == pool.lens


def on_gpu(pool):
    return cuda(pool.refs), cuda(pool.table), cuda(pool.lens), torch.zeros(1, dtype=torch.int32, device="cuda")


# pools below one scan chunk, of odd sizes, and past a round of 32 chunks
SIZES = [(1, 2, 1), (37, 5, 4), (1000, 40, 31), (1024, 3, 400), (5000, 90, 63), (33000, 60, 700)]


@pytest.mark.parametrize("pages,rows,blocks", SIZES)
@pytest.mark.parametrize("new", [1, 0, 17, "ragged"])
def test_reserve(gq, pages, rows, blocks, new):
    rng = np.random.default_rng(pages + rows)
    pool = random_pool(rng, pages, rows, blocks, max_len=max(1, 16 * blocks - 40))
    refs, table, lens, err = on_gpu(pool)
    n = rng.integers(0, 60, size=rows).tolist() if new == "ragged" else [new] * rows
    flag = pool.reserve(n)
    gq.kv_pages_reserve(refs, table, lens, cuda(n) if new == "ragged" else new, err=err)
    assert int(err.item()) == flag
    same(pool, refs, table, lens)
    gq.kv_pages_reserve(refs, table, lens, cuda(n) if new == "ragged" else new)      # again: nothing to do
    pool.reserve(n)
    same(pool, refs, table, lens)


def test_reserve_runs_out_and_refuses_bad_rows(gq):
    pool = Pool([0, 1, 0, 0, 1], [[1, -1, -1], [4, -1, -1], [-1, -1, -1], [-1, -1, -1]], [16, 10, 0, 0])
    new = [20, 3, 40, 1]                       # two pages, none, three (one is left), one
    refs, table, lens, err = on_gpu(pool)
    flag = pool.reserve(new)
    assert flag == gq.GQA_DEVERR_NO_PAGES
    gq.kv_pages_reserve(refs, table, lens, cuda(new), err=err)
    assert int(err.item()) == flag
    same(pool, refs, table, lens)
    pool = Pool([0] * 9, [[-1] * 3] * 4, [-5, 40, 0, 2 ** 31 - 1])
    new = [1, 9, 48, 5]                        # length below zero, past the table, the whole table, overflow
    refs, table, lens, err = on_gpu(pool)
    flag = pool.reserve(new)
    gq.kv_pages_reserve(refs, table, lens, cuda(new), err=err)
    assert int(err.item()) == flag == gq.GQA_DEVERR_POSITION
    same(pool, refs, table, lens)


@pytest.mark.parametrize("pages,rows,blocks", SIZES)
def test_free_and_trim(gq, pages, rows, blocks):
    rng = np.random.default_rng(pages)
    pool = random_pool(rng, pages, rows, blocks)
    refs, table, lens, err = on_gpu(pool)
    flag = pool.trim(40, 20)
    gq.kv_pages_trim(refs, table, lens, 40, 20, err=err)
    same(pool, refs, table, lens)
    gone = [0, rows - 1, rows // 2, 0]                                  # a row named twice
    flag |= pool.free(gone)
    gq.kv_pages_free(refs, table, lens, cuda(gone), err=err)
    assert int(err.item()) == flag == 0
    same(pool, refs, table, lens)


@pytest.mark.parametrize("W,S", [(1, 0), (1, 17), (16, 16), (17, 1), (33, 100), (10 ** 6, 4)])
def test_trim_releases_what_no_later_token_sees(gq, W, S):
    rng = np.random.default_rng(5)
    pool = random_pool(rng, 4000, 50, 40)
    pool.lens[3] = 641                                                  # past its table
    refs, table, lens, err = on_gpu(pool)
    flag = pool.trim(W, S)
    gq.kv_pages_trim(refs, table, lens, W, S, err=err)
    assert int(err.item()) == flag == gq.GQA_DEVERR_CONTEXT_LEN
    same(pool, refs, table, lens)


def test_free_of_bad_rows_pages_and_counts(gq):
    pool = Pool([1, 0, 2], [[0, 1, 7], [2, 2, -1]], [40, 20])
    refs, table, lens, err = on_gpu(pool)
    rows = [0, -1, 2, 1]
    flag = pool.free(rows)
    gq.kv_pages_free(refs, table, lens, cuda(rows), err=err)
    assert int(err.item()) == flag == gq.GQA_DEVERR_ROW | gq.GQA_DEVERR_BLOCK_INDEX | gq.GQA_DEVERR_REF_COUNT
    same(pool, refs, table, lens)


@pytest.mark.parametrize("pages,rows,blocks", SIZES)
def test_fork(gq, pages, rows, blocks):
    rng = np.random.default_rng(pages + 7)
    pool = random_pool(rng, pages, rows, blocks, fill=0.6)
    empty = [b for b in range(rows) if pool.lens[b] == 0]
    full = [b for b in range(rows) if pool.lens[b] > 0] or [0]
    src = [full[int(i)] for i in rng.integers(0, len(full), size=len(empty))]
    refs, table, lens, err = on_gpu(pool)
    flag, pairs, row_pairs = pool.fork(src, empty)
    c = gq.kv_pages_fork(refs, table, lens, cuda(src), cuda(empty), err=err)
    assert int(err.item()) == flag
    same(pool, refs, table, lens)
    assert c.pairs[:int(c.count[0])].tolist() == [list(p) for p in pairs]
    assert c.rows.tolist() == [list(r) for r in row_pairs]
    # the parent ends: shared pages live on
    pool.free(src[:1])
    gq.kv_pages_free(refs, table, lens, cuda(src[:1]))
    same(pool, refs, table, lens)


def test_fork_refusals_leave_their_rows_alone(gq):
    table = [[0, 1, -1], [2, 99, -1], [-1] * 3, [-1] * 3, [3, -1, -1], [-1] * 3, [-1, 4, -1], [-1] * 3]
    pool = Pool([1, 1, 1, 1, 1, 0, 0, 0], table, [20, 20, 0, 0, 16, 0, 30, 0])
    # done, row taken, bad page, whole parent, not empty, row out of range, trimmed parent, a child's child
    src = [0, 0, 1, 4, 0, 9, 6, 2]
    dst = [2, 2, 3, 5, 4, 3, 7, 3]
    refs, tab, lens, err = on_gpu(pool)
    flag, pairs, rows = pool.fork(src, dst)
    c = gq.kv_pages_fork(refs, tab, lens, cuda(src), cuda(dst), err=err)
    assert int(err.item()) == flag
    same(pool, refs, tab, lens)
    assert c.pairs[:int(c.count[0])].tolist() == [list(p) for p in pairs]
    assert c.rows.tolist() == [list(r) for r in rows]


def test_fork_into_an_empty_row_with_reserved_pages_is_refused(gq):
    """Its pages would be nobody's afterwards."""
    pool = Pool([1, 0, 0], [[0, -1], [-1, -1]], [5, 0])
    refs, table, lens, err = on_gpu(pool)
    pool.reserve([1, 1])
    gq.kv_pages_reserve(refs, table, lens, 1)
    flag, _, rows = pool.fork([0], [1])
    c = gq.kv_pages_fork(refs, table, lens, cuda([0]), cuda([1]), err=err)
    assert int(err.item()) == flag == gq.GQA_DEVERR_ROW and c.rows.tolist() == [[-1, -1]] and int(c.count[0]) == 0
    same(pool, refs, table, lens)


def test_fork_without_pages(gq):
    pool = Pool([1, 1, 0, 1], [[0, 1], [3, -1], [-1, -1], [-1, -1], [-1, -1]], [20, 16, 0, 0, 0])
    refs, table, lens, err = on_gpu(pool)
    src, dst = [0, 0, 1], [2, 3, 4]            # one fresh page for two, none needed for the third
    flag, pairs, rows = pool.fork(src, dst)
    c = gq.kv_pages_fork(refs, table, lens, cuda(src), cuda(dst), err=err)
    assert int(err.item()) == flag == gq.GQA_DEVERR_NO_PAGES
    same(pool, refs, table, lens)
    assert c.pairs[:int(c.count[0])].tolist() == [[1, 2]] and c.rows.tolist() == [[0, 2], [-1, -1], [1, 4]]


def test_empty_calls(gq):
    pool = Pool([1, 0, 2], [[0, 2], [2, -1]], [20, 10])
    refs, table, lens, err = on_gpu(pool)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    c = gq.kv_pages_fork(refs, table, lens, none, none, err=err)
    assert int(c.count[0]) == 0
    gq.kv_pages_free(refs, table, lens, none, err=err)
    gq.kv_pages_reserve(refs, table, lens, 0, err=err)
    assert int(err.item()) == 0
    same(pool, refs, table, lens)


@pytest.mark.parametrize("pages,rows,blocks", SIZES + [(70001, 20, 900)])
@pytest.mark.parametrize("most", [None, 0, 5])
def test_compact(gq, pages, rows, blocks, most):
    rng = np.random.default_rng(pages + 3)
    pool = random_pool(rng, pages, rows, blocks, fill=0.5)
    src = [b for b in range(rows) if pool.lens[b]][:3]
    dst = [b for b in range(rows) if not pool.lens[b]][:len(src)]
    pool.fork(src[:len(dst)], dst)                                      # shared pages move once
    refs, table, lens, err = on_gpu(pool)
    c = gq.kv_pages_compact(refs, table, max_copies=most, err=err)
    pairs, live = pool.compact(len(pool.refs) if most is None else most)
    assert int(err.item()) == 0
    assert c.count.tolist() == [len(pairs), live]
    assert c.pairs[:len(pairs)].tolist() == [list(p) for p in pairs]
    same(pool, refs, table, lens)


@pytest.mark.parametrize("refs", [[0, 0, 0], [1, 1, 1], [0, 0, 4], [2, 0, 0], [1] * 40 + [0] * 5, [0] * 2000 + [1] * 2000])
def test_compact_ends(gq, refs):
    held = [p for p, r in enumerate(refs) if r]
    pool = Pool(refs, [held + [-1]], [0])
    r, t, lens, err = on_gpu(pool)
    c = gq.kv_pages_compact(r, t, err=err)
    pairs, live = pool.compact(len(refs))
    assert int(err.item()) == 0 and c.count.tolist() == [len(pairs), live]
    same(pool, r, t, lens)


def test_compact_flags_entries_outside_the_pool(gq):
    pool = Pool([0, 0, 1], [[2, 9, -1]], [30])
    refs, table, lens, err = on_gpu(pool)
    gq.kv_pages_compact(refs, table, err=err)
    assert int(err.item()) == gq.GQA_DEVERR_BLOCK_INDEX
    assert table.tolist() == [[0, 9, -1]] and refs.tolist() == [1, 0, 0]


# --------------------------------------------------------------------------- page data


def _bits(t):
    return t.view(torch.uint8)


@pytest.mark.parametrize("dtype,K,d", [("bf16", 8, 128), ("f16", 3, 64), ("f32", 1, 64), ("i8", 8, 128), ("fp8", 2, 64),
                                       ("i4", 4, 128), ("i4kc", 3, 64), ("bf16", 33, 128)])
@pytest.mark.parametrize("layers", [1, 3])
def test_copies_are_bit_exact(gq, dtype, K, d, layers):
    pages = 21
    kind = {"i4": "int4", "i4kc": "int4kc"}.get(dtype, gi.DTYPES[dtype])
    caches = [gq.PagedKVCache.allocate(pages, K, d, kind, residual_rows=6) for _ in range(layers)]
    parts = ("k", "v", "k_scale", "v_scale", "k_residual")
    for i, c in enumerate(caches):
        for x in parts:
            t = getattr(c, x)
            if t is not None:
                _bits(t).copy_(torch.randint(0, 256, _bits(t).shape, dtype=torch.uint8,
                                             generator=torch.Generator().manual_seed(i)))
    before = [{x: getattr(c, x).clone() for x in parts if getattr(c, x) is not None} for c in caches]
    pairs = [(3, 0), (3, 20), (7, 7), (19, 4), (1, 99), (-1, 2), (5, 6)]
    rows = [(0, 1), (-1, -1), (2, 5), (3, 7)]
    copies = gq.PageCopies(cuda(pairs), cuda([6]), cuda(rows))          # the seventh pair is past the count
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq.kv_copy_pages(caches, copies, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == gq.GQA_DEVERR_BLOCK_INDEX | (gq.GQA_DEVERR_ROW if dtype == "i4kc" else 0)
    for c, old in zip(caches, before):
        for x, want in old.items():
            want = want.clone()
            todo = [(0, 1), (2, 5)] if x == "k_residual" else [(3, 0), (3, 20), (19, 4)]
            for s, t in todo:
                want[t] = want[s]
            assert torch.equal(_bits(getattr(c, x)), _bits(want)), x


@pytest.mark.parametrize("layout", ["padded heads", "padded tokens", "token major", "all apart"])
def test_copies_of_other_layouts(gq, layout):
    """Pages whose rows do not lie behind one another, and memory between them."""
    K, d, pages = 3, 64, 9
    st, sh = {"padded heads": (d, 16 * d + 32), "padded tokens": (d + 8, 16 * (d + 8)), "token major": (K * d, d),
              "all apart": (K * (d + 16), d + 16)}[layout]
    sb = max(16 * st, K * sh) + 64
    buf = [torch.randn(pages * sb, device="cuda").to(torch.bfloat16) for _ in range(2)]
    cache = gq.PagedKVCache(buf[0], buf[1], pages, K, d, sb, sh, st)
    want = [b.clone() for b in buf]
    pairs = [(8, 0), (2, 5)]
    gq.kv_copy_pages(cache, gq.PageCopies(cuda(pairs), cuda([2])))
    torch.cuda.synchronize()
    for w in want:
        for s, t in pairs:
            for g in range(K):
                for i in range(16):
                    o = g * sh + i * st
                    w[t * sb + o:t * sb + o + d] = w[s * sb + o:s * sb + o + d]
    assert torch.equal(buf[0], want[0]) and torch.equal(buf[1], want[1])


def test_more_caches_than_one_launch_and_far_pages(gq):
    """70 layers; and a pool past 2^31 elements, whose offsets need 64 bits."""
    caches = [gq.PagedKVCache.allocate(4, 1, 64, torch.float16) for _ in range(70)]
    for i, c in enumerate(caches):
        c.k.fill_(i)
        c.k[2], c.v[2] = i + 0.5, -i
    gq.kv_copy_pages(caches, gq.PageCopies(cuda([(2, 3)]), cuda([1])))
    big = gq.PagedKVCache.allocate(140000, 8, 128, torch.bfloat16)
    big.k[139999], big.v[139999] = 1.5, 2.5
    gq.kv_copy_pages(big, gq.PageCopies(cuda([(139999, 139000)]), cuda([1])))
    torch.cuda.synchronize()
    for i, c in enumerate(caches):
        assert bool((c.k[3] == i + 0.5).all()) and bool((c.v[3] == -i).all()) and bool((c.k[1] == i).all())
    assert bool((big.k[139000] == 1.5).all()) and bool((big.v[139000] == 2.5).all())


# --------------------------------------------------------------------------- together


@pytest.mark.parametrize("cache_dtype", ["f32", "i4kc"])
def test_a_stream_of_steps_with_all_of_them(gq, cache_dtype):
    """Serving: reserve, append, attend; fork; append to the children; trim; compact; attend.
    Attention over the moved, shared and trimmed pages equals the plain form over each
    sequence's own rows."""
    K, H, d, W, S = 2, 4, 128 if cache_dtype == "i4kc" else 64, 40, 4
    rows, blocks, pages = 6, 12, 60
    coded = cache_dtype != "f32"
    gen = torch.Generator(device="cuda").manual_seed(3)
    caches = [gq.PagedKVCache.allocate(pages, K, d, "int4kc" if coded else torch.float32, residual_rows=rows)
              for _ in range(2)]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((rows, blocks), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = [[[] for _ in range(rows)] for _ in range(2)]                # plain rows (k, v) of each layer and sequence

    def append(n):
        n = [x if x else 0 for x in n]
        start = cuda(np.concatenate([[0], np.cumsum(n)]).tolist())
        gq.kv_pages_reserve(refs, table, lens, cuda(n), err=err)
        for layer, c in enumerate(caches):
            k, v = (torch.randn((sum(n), K, d), generator=gen, device="cuda") for _ in range(2))
            gq.kv_append_varlen(c, k, v, start, max(n), table, lens, err=err)
            for b in range(rows):
                lo, hi = int(start[b]), int(start[b + 1])
                kept[layer][b] += [(k[t], v[t]) for t in range(lo, hi)]
        lens.add_(cuda(n))

    def check():
        for layer, c in enumerate(caches):
            q = torch.randn((rows, H, d), generator=gen, device="cuda")
            q = q.to(torch.bfloat16) if coded else q
            out = gq.gqa_decode(c, q, table, lens, d ** -0.5, window=W, sinks=S, err=err)
            torch.cuda.synchronize()
            assert int(err.item()) == 0
            for b in range(rows):
                if not kept[layer][b]:
                    assert bool((out[b] == 0).all())
                    continue
                k, v = (torch.stack([x[i] for x in kept[layer][b]]).double().cpu().numpy() for i in range(2))
                if coded:
                    import oracle
                    k = oracle.quantised_sequence(k.astype(np.float32), "i4kc", True)[0]
                    v = oracle.quantised_sequence(v.astype(np.float32), "i4")[0]
                from plain import attend
                ref = attend(q[b:b + 1].double().cpu().numpy(), k, v, d ** -0.5, W, S)[0]
                assert np.abs(out[b].double().cpu().numpy() - ref).max() <= TOL, (layer, b)

    def fork(src, dst):
        copies = gq.kv_pages_fork(refs, table, lens, cuda(src), cuda(dst), err=err)
        gq.kv_copy_pages(caches, copies, err=err)
        for s, t in zip(src, dst):
            for layer in range(2):
                kept[layer][t] = list(kept[layer][s])

    append([70, 33, 0, 0, 0, 16])
    check()
    fork([0, 0, 5], [2, 3, 4])
    check()
    append([1, 1, 5, 9, 1, 0])                                          # children part from their parents
    check()
    gq.kv_pages_free(refs, table, lens, cuda([0]), err=err)
    for layer in range(2):
        kept[layer][0] = []
    append([0, 40, 30, 60, 1, 30])
    gq.kv_pages_trim(refs, table, lens, W, S, err=err)
    check()
    copies = gq.kv_pages_compact(refs, table, err=err)
    gq.kv_copy_pages(caches, copies, err=err)
    n, live = copies.count.tolist()
    assert n > 0 and live == int((refs > 0).sum()) and bool((refs[:live] > 0).all())
    for c in caches:                                                    # what the moves left behind is nobody's
        _bits(c.k)[live:] = 255
        _bits(c.v)[live:] = 255
    check()
    append([3, 1, 1, 1, 1, 1])
    check()


def test_captured_step_of_bookkeeping(gq):
    """A graph of trim and reserve replays on the lengths of each step."""
    pool = Pool([0] * 200, [[-1] * 40 for _ in range(7)], [0, 5, 16, 31, 100, 0, 250])
    refs, table, lens, err = on_gpu(pool)
    pool.reserve([250] * 7)
    gq.kv_pages_reserve(refs, table, lens, 250)
    ws = torch.empty(gq.load().gqa_kv_pages_workspace_size(200, 7), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq.kv_pages_trim(refs, table, lens, 30, 4, err=err)
        gq.kv_pages_reserve(refs, table, lens, 3, err=err, workspace=ws)
    for step in range(6):
        graph.replay()
        lens += 3
        pool.trim(30, 4)
        pool.reserve([3] * 7)
        pool.lens = [x + 3 for x in pool.lens]
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        same(pool, refs, table, lens)


def test_other_stream(gq):
    pool = random_pool(np.random.default_rng(1), 900, 20, 30, fill=0.5)
    refs, table, lens, err = on_gpu(pool)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    src, dst = ([b for b in range(20) if (pool.lens[b] > 0) == x][:3] for x in (True, False))
    n = min(len(src), len(dst))
    flag, pairs, _ = pool.fork(src[:n], dst[:n])
    s, d = cuda(src[:n]), cuda(dst[:n])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        gq.kv_pages_fork(refs, table, lens, s, d, err=err, stream=side)
        gq.kv_pages_trim(refs, table, lens, 20, 4, err=err)
    side.synchronize()
    pool.trim(20, 4)
    assert int(err.item()) == flag
    same(pool, refs, table, lens)
