// gqa_pages.cu -- the pages of a paged KV cache as a server moves them: reserving
// pages for new tokens, forking a sequence into others, releasing what ended or left
// the window, compacting the pool, and the copies of page data these ask for.
//
// The whole state is ref_counts[num_blocks] (entries of the tables that hold a page,
// 0 = free) next to the block tables and context lengths. Every choice of a page goes
// by index (the lowest free page first; the highest pages into the lowest holes), so
// equal calls on equal states give equal tables, whatever order the threads ran in.
// Bookkeeping is done once for all layers; gqa_kv_copy_pages then moves the data of
// every layer's cache by the list that the bookkeeping wrote.
//
// Bound: the bookkeeping by latency (kilobytes are read; one CTA finds the free pages,
// 32 warps scanning 1024 counts each a round; it also writes the tables where they are
// few entries, a second, wide launch where they are many), the copies by memory (every
// moved byte is read and written once).
#include <algorithm>
#include <climits>

#include "gqa_device.cuh"
#include "gqa_internal.h"

namespace gqa {

int device_sms(int device);   // gqa_capi.cu

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kChunk = 1024;                 // ref counts one warp scans at a time
constexpr int kWideThreads = 256;
// Table entries up to which the planning CTA writes them itself (four a thread): a
// second launch costs 4-5 us of host time and ~2 us on the GPU.
constexpr long long kFewEntries = 4 * kPlanThreads;

struct PageArgs {
    int32_t* refs;
    int32_t* tables;
    int32_t* lens;
    int num_blocks, table_rows, max_blocks, n;
    const int32_t* src;                      // fork: parents; free: rows
    const int32_t* dst;
    const int32_t* new_tokens;               // reserve: per row, or NULL: tokens
    int tokens;
    int window, sinks;                       // trim
    int32_t* pairs;                          // [max_copies][2] (from, to)
    int32_t* count;                          // fork: [1]; compact: [2] (copies, live pages)
    int32_t* row_pairs;                      // fork: [n][2] (from, to), -1: none
    int max_copies;
    int32_t* ws_hdr;                         // [0] free pages found, compact: [0] moves, [1] live
    int32_t* ws_rows;                        // [rows + 1]
    int32_t* ws_list;                        // [num_blocks]
    int32_t* err;
};

// ------------------------------------------------------------------ scans

// Exclusive prefix sum over the CTA's threads; total gets the sum. `tmp` holds
// kPlanWarps + 1 ints.
__device__ __forceinline__ int block_scan(int x, int* tmp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();                         // tmp may still be read from the last call
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int t = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, t, o);
            if (lane >= o) t += y;
        }
        tmp[lane] = t;
    }
    __syncthreads();
    total = tmp[kPlanWarps - 1];
    return (warp ? tmp[warp - 1] : 0) + incl - x;
}

// One warp's chunk of ref counts, 8 quads a lane: bit 4 q + e of the result says
// whether count base + 128 q + 4 lane + e is held (pages past the pool: not).
__device__ __forceinline__ uint32_t held_mask(const int32_t* refs, int base, int num_blocks, int lane) {
    int4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int p = base + 128 * q + 4 * lane;
        v[q] = make_int4(0, 0, 0, 0);
        if (p + 3 < num_blocks) {
            v[q] = *reinterpret_cast<const int4*>(refs + p);
        } else {
            if (p < num_blocks) v[q].x = refs[p];
            if (p + 1 < num_blocks) v[q].y = refs[p + 1];
            if (p + 2 < num_blocks) v[q].z = refs[p + 2];
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        m |= ((v[q].x > 0 ? 1u : 0u) | (v[q].y > 0 ? 2u : 0u) | (v[q].z > 0 ? 4u : 0u) | (v[q].w > 0 ? 8u : 0u)) << (4 * q);
    return m;
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}
__device__ __forceinline__ int warp_before(int x, int lane) {     // exclusive prefix sum
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    return incl - x;
}

// The first round's masks of find_free: loaded before anything else in the kernel, so
// that their latency goes by with the rows'.
__device__ __forceinline__ uint32_t first_held(const PageArgs& a) {
    const int base = (threadIdx.x >> 5) * kChunk;
    return base < a.num_blocks ? held_mask(a.refs, base, a.num_blocks, threadIdx.x & 31) : 0u;
}

// The `want` lowest free pages, in order, into list; returns how many there are
// (CTA-uniform). Rounds of 32 chunks until enough are found; `held` is first_held().
__device__ int find_free(const PageArgs& a, uint32_t held, int want, int32_t* list, int* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int found = 0;
    for (int round = 0; round < a.num_blocks && found < want; round += kPlanWarps * kChunk) {
        const int base = round + warp * kChunk;
        uint32_t free_m = 0;
        if (base < a.num_blocks) {
            free_m = ~(round == 0 ? held : held_mask(a.refs, base, a.num_blocks, lane));
            // pages past the pool are none
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int p = base + 128 * q + 4 * lane;
                const int in = min(max(a.num_blocks - p, 0), 4);
                free_m &= ~((0xFu & ~((1u << in) - 1u)) << (4 * q));
            }
        }
        int total;
        const int cnt = warp_sum(__popc(free_m));
        const int at = block_scan(lane == 0 ? cnt : 0, tmp, total);
        int rank = found + __shfl_sync(kFull, at, 0);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t nib = (free_m >> (4 * q)) & 0xFu;
            const int c = __popc(nib);
            int r = rank + warp_before(c, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!((nib >> e) & 1u)) continue;
                if (r < want) list[r] = base + 128 * q + 4 * lane + e;
                ++r;
            }
            rank += warp_sum(c);
        }
        found += total;
    }
    __syncthreads();                         // list is complete for this CTA
    return min(found, want);
}

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kBlock - 1) / kBlock; }

// Give back the page a table entry holds and empty the entry. Only one of several
// threads that try gets the page.
__device__ __forceinline__ void release(const PageArgs& a, int32_t* entry) {
    if (*entry < 0) return;
    const int p = atomicExch(entry, -1);
    if (p < 0) return;
    if (p >= a.num_blocks) {
        flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
        return;
    }
    if (atomicSub(a.refs + p, 1) <= 0) {     // nobody held it: leave the count as it was
        atomicAdd(a.refs + p, 1);
        flag_error(a.err, GQA_DEVERR_REF_COUNT);
    }
}

// ------------------------------------------------------------------ reserve

// Blocks row b lacks for its next tokens lie in [lo, hi); false (flagged) if the row's
// length or the tokens do not fit the table.
__device__ __forceinline__ bool reserve_range(const PageArgs& a, int b, int& lo, int& hi) {
    const int L = a.lens[b], n = a.new_tokens ? a.new_tokens[b] : a.tokens;
    lo = hi = 0;
    if (L < 0 || n < 0 || (long long)L + n > (long long)a.max_blocks * kBlock) return false;
    lo = blocks_of(L);
    hi = blocks_of(L + n);
    return true;
}

// kAll: the CTA also hands the pages out, a thread per row (host: few blocks a row).
template <bool kAll>
__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(const PageArgs a) {
    __shared__ int tmp[kPlanWarps + 1];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t held = first_held(a);
    int carry = 0;
    for (int base = 0; base < a.n; base += kPlanThreads) {
        const int b = base + threadIdx.x;
        int lo = 0, hi = 0, lack = 0;
        if (b < a.n && !reserve_range(a, b, lo, hi)) flag_error(a.err, GQA_DEVERR_POSITION);
        const int32_t* row = a.tables + (long long)b * a.max_blocks;
        const bool wide = hi - lo > 4;
        if (!wide)
            for (int j = lo; j < hi; ++j) lack += row[j] < 0;
        // long ranges (prompts) by the whole warp
        for (uint32_t m = __ballot_sync(kFull, wide); m; m &= m - 1) {
            const int who = __ffs(m) - 1;
            const int wb = base + (int)(threadIdx.x & ~31u) + who;
            const int wlo = __shfl_sync(kFull, lo, who), whi = __shfl_sync(kFull, hi, who);
            int c = 0;
            for (int j = wlo + lane; j < whi; j += 32) c += a.tables[(long long)wb * a.max_blocks + j] < 0;
            c = warp_sum(c);
            if (lane == who) lack = c;
        }
        int total;
        const int before = block_scan(lack, tmp, total);
        if (b < a.n) a.ws_rows[b] = carry + before;
        carry += total;
    }
    if (threadIdx.x == 0) a.ws_rows[a.n] = carry;
    const int found = find_free(a, held, carry, a.ws_list, tmp);
    if (threadIdx.x == 0) a.ws_hdr[0] = found;
    if constexpr (kAll) {
        for (int b = threadIdx.x; b < a.n; b += kPlanThreads) {
            int k = a.ws_rows[b], lo, hi;
            const int end = b + 1 < a.n ? a.ws_rows[b + 1] : carry;
            if (k == end) continue;
            if (end > found) {                   // not enough pages for the whole row: none
                flag_error(a.err, GQA_DEVERR_NO_PAGES);
                continue;
            }
            if (!reserve_range(a, b, lo, hi)) continue;
            int32_t* row = a.tables + (long long)b * a.max_blocks;
            for (int j = lo; j < hi; ++j) {
                if (row[j] >= 0) continue;
                const int p = a.ws_list[k++];
                row[j] = p;
                a.refs[p] = 1;
            }
        }
    }
}

__global__ void __launch_bounds__(kWideThreads) reserve_assign_kernel(const PageArgs a) {
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int b = (int)blockIdx.x * (kWideThreads / 32) + (threadIdx.x >> 5);
    if (b >= a.n) return;
    int k = a.ws_rows[b];
    const int end = a.ws_rows[b + 1];
    if (k == end) return;
    if (end > a.ws_hdr[0]) {                 // not enough pages for the whole row: none
        if (lane == 0) flag_error(a.err, GQA_DEVERR_NO_PAGES);
        return;
    }
    int lo, hi;
    if (!reserve_range(a, b, lo, hi)) return;
    int32_t* row = a.tables + (long long)b * a.max_blocks;
    for (int j0 = lo; j0 < hi && k < end; j0 += 32) {
        const int j = j0 + lane;
        const bool lack = j < hi && row[j] < 0;
        const uint32_t m = __ballot_sync(kFull, lack);
        if (lack) {
            const int p = a.ws_list[k + __popc(m & ((1u << lane) - 1u))];
            row[j] = p;
            a.refs[p] = 1;
        }
        k += __popc(m);
    }
}

// ------------------------------------------------------------------ fork

// ws_rows[i] of fork i: its rank among those that need a fresh page, or one of these.
enum ForkKind : int { kForkSkip = -1, kForkWhole = -2 };

// Table entries of the forks, from thread `at` on in steps of `step`.
__device__ __forceinline__ void fork_entries(const PageArgs& a, long long at, long long step) {
    const long long total = (long long)a.n * a.max_blocks;
    for (long long x = at; x < total; x += step) {
        const int i = (int)(x / a.max_blocks), j = (int)(x - (long long)i * a.max_blocks);
        const int kind = a.ws_rows[i];
        if (kind == kForkSkip) continue;
        const int s = a.src[i], L = a.lens[s];
        int p = -1;
        if (j < blocks_of(L)) {
            if (kind >= 0 && j == L / kBlock) {
                p = a.ws_list[kind];         // its count was set with the plan
            } else {
                p = a.tables[(long long)s * a.max_blocks + j];
                if (p >= a.num_blocks) {
                    flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                    p = -1;
                }
                if (p >= 0) atomicAdd(a.refs + p, 1);
                else p = -1;
            }
        }
        a.tables[(long long)a.dst[i] * a.max_blocks + j] = p;
    }
}

// kAll: the CTA writes the tables too (host: few entries).
template <bool kAll>
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PageArgs a) {
    extern __shared__ int claim[];           // [table_rows] the first fork that writes the row
    __shared__ int tmp[kPlanWarps + 1];
    grid_dependency_wait();
    launch_dependents();
    const uint32_t held = first_held(a);
    for (int r = threadIdx.x; r < a.table_rows; r += kPlanThreads) claim[r] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        const int d = a.dst[i];
        if (d >= 0 && d < a.table_rows) atomicMin(&claim[d], i);
    }
    __syncthreads();
    int carry = 0;
    for (int base = 0; base < a.n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int kind = kForkSkip;
        if (i < a.n) {
            const int s = a.src[i], d = a.dst[i];
            // a parent is no child of this call, a child has one parent and is empty
            const bool rows_ok = s >= 0 && s < a.table_rows && d >= 0 && d < a.table_rows;
            if (!rows_ok || claim[d] != i || claim[s] != INT_MAX || a.lens[d] != 0 ||
                a.tables[(long long)d * a.max_blocks] >= 0) {
                flag_error(a.err, GQA_DEVERR_ROW);
            } else {
                const int L = a.lens[s];
                if (L < 0 || L > (long long)a.max_blocks * kBlock) {
                    flag_error(a.err, GQA_DEVERR_CONTEXT_LEN);
                } else if (L % kBlock == 0) {
                    kind = kForkWhole;
                } else {
                    const int p = a.tables[(long long)s * a.max_blocks + L / kBlock];
                    if (p >= 0 && p < a.num_blocks) kind = 0;
                    else flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                }
            }
        }
        int total;
        const int rank = carry + block_scan(kind == 0 ? 1 : 0, tmp, total);
        if (i < a.n) a.ws_rows[i] = kind == 0 ? rank : kind;
        carry += total;
    }
    const int found = find_free(a, held, carry, a.ws_list, tmp);
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
        int kind = a.ws_rows[i];
        if (kind >= found) {                 // (found <= the number of ranks)
            flag_error(a.err, GQA_DEVERR_NO_PAGES);
            a.ws_rows[i] = kind = kForkSkip;
        }
        a.row_pairs[2 * i] = a.row_pairs[2 * i + 1] = -1;
        if (kind == kForkSkip) continue;
        const int s = a.src[i], d = a.dst[i], L = a.lens[s];
        if (kind >= 0) {
            const int p = a.ws_list[kind];
            a.pairs[2 * kind] = a.tables[(long long)s * a.max_blocks + L / kBlock];
            a.pairs[2 * kind + 1] = p;
            a.refs[p] = 1;
        }
        a.row_pairs[2 * i] = s;
        a.row_pairs[2 * i + 1] = d;
    }
    if (threadIdx.x == 0) a.count[0] = found;
    // the children's lengths last: lens[s] of every fork has been read (no s is a d)
    for (int i = threadIdx.x; i < a.n; i += kPlanThreads)
        if (a.ws_rows[i] != kForkSkip) a.lens[a.dst[i]] = a.lens[a.src[i]];
    if constexpr (kAll) {
        __syncthreads();
        fork_entries(a, threadIdx.x, kPlanThreads);
    }
}

__global__ void __launch_bounds__(kWideThreads) fork_tables_kernel(const PageArgs a) {
    grid_dependency_wait();
    launch_dependents();
    fork_entries(a, (long long)blockIdx.x * kWideThreads + threadIdx.x, (long long)gridDim.x * kWideThreads);
}

// ------------------------------------------------------------------ free, trim

__global__ void __launch_bounds__(kWideThreads) free_kernel(const PageArgs a) {
    grid_dependency_wait();
    launch_dependents();
    const long long total = (long long)a.n * a.max_blocks;
    for (long long x = (long long)blockIdx.x * kWideThreads + threadIdx.x; x < total;
         x += (long long)gridDim.x * kWideThreads) {
        const int i = (int)(x / a.max_blocks), j = (int)(x - (long long)i * a.max_blocks);
        const int r = a.src[i];
        if (r < 0 || r >= a.table_rows) {
            if (j == 0) flag_error(a.err, GQA_DEVERR_ROW);
            continue;
        }
        release(a, a.tables + (long long)r * a.max_blocks + j);
        if (j == 0) a.lens[r] = 0;
    }
}

__global__ void __launch_bounds__(kWideThreads) trim_kernel(const PageArgs a) {
    grid_dependency_wait();
    launch_dependents();
    const long long total = (long long)a.n * a.max_blocks;
    const int first = (int)(((long long)a.sinks + kBlock - 1) / kBlock);
    for (long long x = (long long)blockIdx.x * kWideThreads + threadIdx.x; x < total;
         x += (long long)gridDim.x * kWideThreads) {
        const int b = (int)(x / a.max_blocks), j = (int)(x - (long long)b * a.max_blocks);
        const int L = a.lens[b];
        if (L < 0 || L > (long long)a.max_blocks * kBlock) {
            if (j == 0) flag_error(a.err, GQA_DEVERR_CONTEXT_LEN);
            continue;
        }
        // the next token, at position L, sees t > L - window: blocks that end at or
        // before L + 1 - window are out of it and of every later one's
        if (j >= first && (long long)(j + 1) * kBlock <= (long long)L + 1 - a.window)
            release(a, a.tables + (long long)b * a.max_blocks + j);
    }
}

// ------------------------------------------------------------------ compact

// Pairs of one warp's chunk: `before` live pages precede it, `live` pages exist in
// all. The i-th hole below `live` receives the i-th highest live page from `live` on:
// both ranks follow from the number of live pages before a page, so every chunk
// writes its halves of the pairs by itself.
__device__ __forceinline__ void compact_chunk(const PageArgs& a, uint32_t held, int base, int before, int live, int lane) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint32_t nib = (held >> (4 * q)) & 0xFu;
        int lb = before + warp_before(__popc(nib), lane);            // live pages before page p
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int p = base + 128 * q + 4 * lane + e;
            const bool h = (nib >> e) & 1u;
            if (p < a.num_blocks) {
                if (p < live && !h) {
                    const int r = p - lb;
                    if (r < a.max_copies) a.pairs[2 * r + 1] = p;
                } else if (p >= live && h) {
                    const int r = live - 1 - lb;
                    a.ws_list[p] = r;
                    if (r < a.max_copies) a.pairs[2 * r] = p;
                }
                // every live page from `live` on fills one hole below it
                if (p == live) a.ws_hdr[0] = min(live - lb, a.max_copies);
            }
            lb += h;
        }
        before += warp_sum(__popc(nib));
    }
}

__device__ __forceinline__ void compact_header(const PageArgs& a, int live) {
    a.ws_hdr[1] = live;
    a.count[1] = live;
    if (live >= a.num_blocks) a.ws_hdr[0] = 0;   // a full pool has no holes
}

// Counts of the moved pages and the table entries that name them, from thread `at` on.
__device__ __forceinline__ void compact_apply(const PageArgs& a, int moves, int live, long long at, long long step) {
    if (at == 0) a.count[0] = moves;
    for (long long i = at; i < moves; i += step) {
        const int s = a.pairs[2 * i], d = a.pairs[2 * i + 1];
        a.refs[d] = a.refs[s];
        a.refs[s] = 0;
    }
    const long long total = (long long)a.table_rows * a.max_blocks;
    for (long long x = at; x < total; x += step) {
        const int p = a.tables[x];
        if (p < live) continue;
        if (p >= a.num_blocks) {
            flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
            continue;
        }
        // the list holds a rank for every live page from `live` on; an entry whose
        // page nobody holds finds an old word there, which names another page's pair
        const int r = a.ws_list[p];
        if (r >= 0 && r < moves && a.pairs[2 * r] == p) a.tables[x] = a.pairs[2 * r + 1];
    }
}

// Pools of at most 32 chunks: one CTA, the counts held in registers between the scans.
// kAll: it also applies the moves (host: few entries).
template <bool kAll>
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PageArgs a) {
    __shared__ int tmp[kPlanWarps + 1];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, base = (threadIdx.x >> 5) * kChunk;
    const uint32_t held = base < a.num_blocks ? held_mask(a.refs, base, a.num_blocks, lane) : 0u;
    int live;
    const int cnt = warp_sum(__popc(held));
    const int before = __shfl_sync(kFull, block_scan(lane == 0 ? cnt : 0, tmp, live), 0);
    if (base < a.num_blocks) compact_chunk(a, held, base, before, live, lane);
    if (threadIdx.x == 0) compact_header(a, live);
    if constexpr (kAll) {
        __syncthreads();
        compact_apply(a, a.ws_hdr[0], live, threadIdx.x, kPlanThreads);
    }
}

// Larger pools: the live pages of every chunk, then the same with the chunks' sums
// read by each CTA (ws_rows holds them).
__global__ void __launch_bounds__(kWideThreads) compact_count_kernel(const PageArgs a) {
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunk = (int)blockIdx.x * (kWideThreads / 32) + (threadIdx.x >> 5);
    if ((long long)chunk * kChunk >= a.num_blocks) return;
    const int cnt = warp_sum(__popc(held_mask(a.refs, chunk * kChunk, a.num_blocks, lane)));
    if (lane == 0) a.ws_rows[chunk] = cnt;
}
__global__ void __launch_bounds__(kWideThreads) compact_pairs_kernel(const PageArgs a, int chunks) {
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunk = (int)blockIdx.x * (kWideThreads / 32) + (threadIdx.x >> 5);
    if (chunk >= chunks) return;                 // no barrier below: every warp sums for itself
    int before = 0, live = 0;
    for (int c = lane; c < chunks; c += 32) {
        const int x = a.ws_rows[c];
        live += x;
        if (c < chunk) before += x;
    }
    before = warp_sum(before);
    live = warp_sum(live);
    compact_chunk(a, held_mask(a.refs, chunk * kChunk, a.num_blocks, lane), chunk * kChunk, before, live, lane);
    if (chunk == 0 && lane == 0) compact_header(a, live);
}

__global__ void __launch_bounds__(kWideThreads) compact_apply_kernel(const PageArgs a) {
    grid_dependency_wait();
    launch_dependents();
    compact_apply(a, a.ws_hdr[0], a.ws_hdr[1], (long long)blockIdx.x * kWideThreads + threadIdx.x,
                  (long long)gridDim.x * kWideThreads);
}

// ------------------------------------------------------------------ copies

constexpr int kCopyCaches = 64;              // caches one launch serves
constexpr int kCopyThreads = 256;
constexpr int kPiece = 4096;                 // bytes a warp moves at a time: 8 x 16 a lane

// A page of one tensor: n1 x n2 runs of `run` bytes, s1 and s2 bytes apart.
struct PageShape {
    long long stride, s1, s2;                // bytes between pages, runs
    int n1, n2, run, pieces;                 // pieces of kPiece bytes per run
};
struct CopyArgs {
    uint8_t* base[kCopyCaches][4];           // k, v, k_scale, v_scale
    uint8_t* residual[kCopyCaches];
    PageShape shape[3];                      // k and v; k_scale; v_scale
    int items[4];                            // pieces of a page of each tensor
    int caches, per_cache;                   // sum of items
    const int32_t* pairs;
    const int32_t* count;
    const int32_t* row_pairs;
    int max_copies, rows, residual_rows, row_pieces;
    long long row_bytes;
    int num_blocks;
    int32_t* err;
};

__device__ __forceinline__ void move_piece(uint8_t* to, const uint8_t* from, int bytes, int lane) {
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if ((i * 32 + lane) * 16 < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(from) + i * 32 + lane);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if ((i * 32 + lane) * 16 < bytes) __stcs(reinterpret_cast<uint4*>(to) + i * 32 + lane, v[i]);
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyArgs a) {
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long warp = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
    const int count = min(max(a.count[0], 0), a.max_copies);
    const int per_pair = a.per_cache * a.caches;
    const long long total = (long long)count * per_pair;
    for (long long x = warp; x < total; x += warps) {
        const int i = (int)(x / per_pair);
        int w = (int)(x - (long long)i * per_pair);
        const int c = w / a.per_cache;
        w -= c * a.per_cache;
        const int from = a.pairs[2 * i], to = a.pairs[2 * i + 1];
        if (from < 0 || from >= a.num_blocks || to < 0 || to >= a.num_blocks) {
            if (lane == 0) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
            continue;
        }
        if (from == to) continue;
        int t = 0;
        while (t < 3 && w >= a.items[t]) w -= a.items[t++];
        const PageShape& s = a.shape[t < 2 ? 0 : t - 1];
        const int run = w / s.pieces, piece = w - run * s.pieces;
        const int r1 = run / s.n2, r2 = run - r1 * s.n2;
        const long long off = r1 * s.s1 + r2 * s.s2 + (long long)piece * kPiece;
        uint8_t* base = a.base[c][t] + off;
        move_piece(base + to * s.stride, base + from * s.stride, min(kPiece, s.run - piece * kPiece), lane);
    }
    // residual rows (the KIVI-style cache's open blocks)
    const long long rtotal = (long long)a.rows * a.caches * a.row_pieces;
    for (long long x = warp; x < rtotal; x += warps) {
        const int i = (int)(x / (a.caches * a.row_pieces));
        const int w = (int)(x - (long long)i * a.caches * a.row_pieces);
        const int c = w / a.row_pieces, piece = w - c * a.row_pieces;
        const int from = a.row_pairs[2 * i], to = a.row_pairs[2 * i + 1];
        if (from < 0 || to < 0 || from == to) continue;              // a fork that was skipped
        if (from >= a.residual_rows || to >= a.residual_rows) {
            if (lane == 0) flag_error(a.err, GQA_DEVERR_ROW);
            continue;
        }
        const long long off = (long long)piece * kPiece;
        move_piece(a.residual[c] + to * a.row_bytes + off, a.residual[c] + from * a.row_bytes + off,
                   (int)min((long long)kPiece, a.row_bytes - off), lane);
    }
}

cudaError_t launch_pdl(const void* fn, unsigned grid, int threads, int smem, cudaStream_t stream, void** args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t launch_pages(void (*fn)(PageArgs), long long threads_wanted, int threads, int smem, const PageArgs& a,
                         cudaStream_t stream) {
    const int sms = device_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    const long long most = sms * 8LL;
    const long long grid = std::min(most, std::max(1LL, (threads_wanted + threads - 1) / threads));
    void* args[] = {const_cast<PageArgs*>(&a)};
    return launch_pdl(reinterpret_cast<const void*>(fn), (unsigned)grid, threads, smem, stream, args);
}

PageArgs page_args(const PagesLaunch& L) {
    PageArgs a = {};
    a.refs = L.ref_counts;
    a.tables = L.block_tables;
    a.lens = L.context_lens;
    a.num_blocks = (int)L.num_blocks;
    a.table_rows = L.table_rows;
    a.max_blocks = L.max_blocks;
    a.n = L.n;
    a.src = L.src_rows;
    a.dst = L.dst_rows;
    a.new_tokens = L.new_tokens;
    a.tokens = L.tokens;
    a.window = L.window;
    a.sinks = L.sinks;
    a.pairs = L.pairs;
    a.count = L.count;
    a.row_pairs = L.row_pairs;
    a.max_copies = L.max_copies;
    a.err = L.err;
    int32_t* ws = static_cast<int32_t*>(L.workspace);
    a.ws_hdr = ws;
    a.ws_rows = ws + 64;
    a.ws_list = ws != nullptr ? ws + 64 + pages_ws_rows(L.num_blocks, std::max(L.n, 0)) : nullptr;
    return a;
}

}  // namespace

// Ints of the workspace between its header and the page list: a word per row (and
// one), or per chunk of pages.
long long pages_ws_rows(long long num_blocks, int rows) {
    const long long chunks = (num_blocks + kChunk - 1) / kChunk;
    return (std::max<long long>(rows + 1, chunks) + 63) / 64 * 64;
}

cudaError_t launch_pages_reserve(const PagesLaunch& L) {
    const PageArgs a = page_args(L);
    // a thread per row hands out up to five pages; longer rows get a warp each
    if (a.new_tokens == nullptr && a.tokens <= 4 * kBlock)
        return launch_pages(&reserve_plan_kernel<true>, 1, kPlanThreads, 0, a, L.stream);
    cudaError_t e = launch_pages(&reserve_plan_kernel<false>, 1, kPlanThreads, 0, a, L.stream);
    if (e != cudaSuccess) return e;
    void* args[] = {const_cast<PageArgs*>(&a)};
    const unsigned grid = (unsigned)((a.n + kWideThreads / 32 - 1) / (kWideThreads / 32));   // a warp per row
    return launch_pdl(reinterpret_cast<const void*>(&reserve_assign_kernel), grid, kWideThreads, 0, L.stream, args);
}

cudaError_t launch_pages_fork(const PagesLaunch& L) {
    const PageArgs a = page_args(L);
    if ((long long)a.n * a.max_blocks <= kFewEntries)
        return launch_pages(&fork_plan_kernel<true>, 1, kPlanThreads, a.table_rows * 4, a, L.stream);
    cudaError_t e = launch_pages(&fork_plan_kernel<false>, 1, kPlanThreads, a.table_rows * 4, a, L.stream);
    if (e != cudaSuccess) return e;
    return launch_pages(&fork_tables_kernel, (long long)a.n * a.max_blocks, kWideThreads, 0, a, L.stream);
}

cudaError_t launch_pages_free(const PagesLaunch& L) {
    const PageArgs a = page_args(L);
    return launch_pages(&free_kernel, (long long)a.n * a.max_blocks, kWideThreads, 0, a, L.stream);
}

cudaError_t launch_pages_trim(const PagesLaunch& L) {
    const PageArgs a = page_args(L);
    return launch_pages(&trim_kernel, (long long)a.n * a.max_blocks, kWideThreads, 0, a, L.stream);
}

cudaError_t launch_pages_compact(const PagesLaunch& L) {
    PageArgs a = page_args(L);
    int chunks = (a.num_blocks + kChunk - 1) / kChunk;
    cudaError_t e;
    const long long entries = std::max<long long>((long long)a.table_rows * a.max_blocks, a.max_copies);
    if (chunks <= kPlanWarps) {
        if (entries <= kFewEntries) return launch_pages(&compact_plan_kernel<true>, 1, kPlanThreads, 0, a, L.stream);
        e = launch_pages(&compact_plan_kernel<false>, 1, kPlanThreads, 0, a, L.stream);
    } else {
        const unsigned grid = (unsigned)((chunks + kWideThreads / 32 - 1) / (kWideThreads / 32));
        void* args[] = {&a};
        e = launch_pdl(reinterpret_cast<const void*>(&compact_count_kernel), grid, kWideThreads, 0, L.stream, args);
        if (e != cudaSuccess) return e;
        void* args2[] = {&a, &chunks};
        e = launch_pdl(reinterpret_cast<const void*>(&compact_pairs_kernel), grid, kWideThreads, 0, L.stream, args2);
    }
    if (e != cudaSuccess) return e;
    return launch_pages(&compact_apply_kernel, entries, kWideThreads, 0, a, L.stream);
}

// Runs of a page of K or V: the head dimension, then the axes that lie right behind
// one another are merged into one run.
static PageShape page_shape(const gqa_kv_cache_t& c) {
    long long run = c.head_dim;
    long long n[2] = {GQA_BLOCK_SIZE, c.num_kv_heads}, s[2] = {c.stride_token, c.stride_head};
    if (s[1] < s[0]) {
        std::swap(s[0], s[1]);
        std::swap(n[0], n[1]);
    }
    for (int i = 0; i < 2; ++i) {            // the inner axis first
        if (n[i] > 1 && s[i] != run) break;
        run *= n[i];
        n[i] = 1;
    }
    PageShape p;
    p.stride = dtype_bytes(c.dtype, c.stride_block);
    p.s1 = dtype_bytes(c.dtype, s[1]);
    p.s2 = dtype_bytes(c.dtype, s[0]);
    p.n1 = (int)n[1];
    p.n2 = (int)n[0];
    p.run = (int)dtype_bytes(c.dtype, run);
    p.pieces = (p.run + kPiece - 1) / kPiece;
    return p;
}
static PageShape flat_shape(long long bytes) {
    return PageShape{bytes, 0, 0, 1, 1, (int)bytes, (int)((bytes + kPiece - 1) / kPiece)};
}

cudaError_t launch_copy_pages(const CopyPagesLaunch& L) {
    const gqa_kv_cache_t& c0 = L.caches[0];
    CopyArgs a = {};
    a.shape[0] = page_shape(c0);
    a.items[0] = a.items[1] = a.shape[0].n1 * a.shape[0].n2 * a.shape[0].pieces;
    if (dtype_coded(c0.dtype)) {
        const long long slots = (long long)c0.num_kv_heads * GQA_BLOCK_SIZE * 2;
        a.shape[1] = flat_shape(c0.dtype == GQA_DTYPE_I4_KC ? (long long)c0.num_kv_heads * c0.head_dim * 2 : slots);
        a.shape[2] = flat_shape(slots);
        a.items[2] = a.shape[1].pieces;
        a.items[3] = a.shape[2].pieces;
    }
    a.per_cache = a.items[0] + a.items[1] + a.items[2] + a.items[3];
    a.pairs = L.pairs;
    a.count = L.count;
    a.max_copies = L.max_copies;
    a.num_blocks = (int)c0.num_blocks;
    a.err = L.err;
    if (c0.dtype == GQA_DTYPE_I4_KC && L.row_pairs != nullptr) {
        a.row_pairs = L.row_pairs;
        a.rows = L.rows;
        a.residual_rows = c0.residual_rows;
        a.row_bytes = (long long)c0.num_kv_heads * GQA_BLOCK_SIZE * c0.head_dim * 4;
        a.row_pieces = (int)((a.row_bytes + kPiece - 1) / kPiece);
    }
    const int sms = device_sms(-1);
    if (sms < 1) return cudaErrorInvalidDevice;
    for (int first = 0; first < L.num_caches; first += kCopyCaches) {
        a.caches = std::min(kCopyCaches, L.num_caches - first);
        for (int i = 0; i < a.caches; ++i) {
            const gqa_kv_cache_t& c = L.caches[first + i];
            a.base[i][0] = static_cast<uint8_t*>(c.k);
            a.base[i][1] = static_cast<uint8_t*>(c.v);
            a.base[i][2] = static_cast<uint8_t*>(c.k_scale);
            a.base[i][3] = static_cast<uint8_t*>(c.v_scale);
            a.residual[i] = static_cast<uint8_t*>(c.k_residual);
        }
        const long long items = ((long long)L.max_copies * a.per_cache + (long long)a.rows * a.row_pieces) * a.caches;
        const long long ctas = (items + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
        const unsigned grid = (unsigned)std::min<long long>(sms * 6LL, std::max<long long>(1, ctas));
        void* args[] = {&a};
        const cudaError_t e = launch_pdl(reinterpret_cast<const void*>(&copy_pages_kernel), grid, kCopyThreads, 0,
                                         L.stream, args);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace gqa
