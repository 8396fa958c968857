// gqa_groups.cu -- which rows of the block tables share their first pages.
//
// With n_b the full pages of row b, its leader is the lowest row with the same first
// page, and m_b the number of leading entries it has in common with the leader's. Of a
// leader's rows a group takes P pages where P (c(P) - 1) is largest, c(P) the rows with
// m_b >= P: the pages that attending them once saves reading. Each step needs all of the
// one before:
//   runs    the leader of a row, then the run they have in common
//   counts  c(m_b) over all rows, the best P of each leader by one 64-bit maximum (the
//           saving, then fewer rows, so the larger P at equal saving)
//   places  groups in the order of their leaders, members by row
// The tables are read once as far as rows agree (the leaders' rows come from L2), which is
// a few microseconds at most: the steps' latencies bound this. Up to 256 rows one cluster
// of eight CTAs does all three, a warp for one or two rows, with one cluster barrier; more rows
// take a launch per step over the whole GPU, where the two passes over all pairs of rows run
// from shared memory. One launch | three, both in turn: replayed in a graph up to 96 rows 8.2 |
// 8.2 us, 128 and 129 10.3 | 8.2, 160 to 224 12.3 | 10.3, 256 12.6 | 10.2; a call from Python
// with its views 25 | 32 at any of these, into a plan's old memory (back to back) 7.0 | 11.4 up
// to 128, 8.5 | 11.5 at 129, 10.0 | 11.1 at 192, 11.4 | 11.3 at 256. A plan is made once for
// many steps, so the call's cost on the host sets the limit; a captured one pays 2 us for it
// from 128 rows on. 2048 rows of up to 1700 shared pages take 23 (50 with the passes over pairs
// from L2).
#include "gqa_groups.cuh"
#include "gqa_internal.h"

namespace gqa {

namespace {

struct GroupsArgs {
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* plan;
    int2* run;                    // [B] (leader, pages in common with it)
    unsigned long long* best;     // [B] by leader: saving << 14 | 16383 - rows
    int32_t* err;
    int B, max_blocks, min_blocks;
};

constexpr int kRunThreads = 128, kRunUnroll = 4;
constexpr int kPairThreads = 512, kPairRows = kPairThreads / 32;   // a warp per row
constexpr int kSmallCtas = 8, kSmallWarps = kSmallCtas * kPairRows, kSmallRows = 256;
constexpr int kRankBits = 14;
constexpr unsigned kRankMask = (1u << kRankBits) - 1;

// What a run of m pages that c > 1 rows share is worth, as a leader's best is kept.
__device__ __forceinline__ unsigned long long worth(int m, int c) {
    return ((unsigned long long)m * (unsigned)(c - 1) << kRankBits) | (kRankMask - (unsigned)c);
}
// The pages of a best, 0: no group.
__device__ __forceinline__ int pages_of(unsigned long long best) {
    if (best == 0ull) return 0;
    return (int)((best >> kRankBits) / (kRankMask - (unsigned)(best & kRankMask) - 1u));
}

// Shared memory of the last step: for every row the leader whose group it is in (-1: none),
// and for every leader its group's pages, then rows, then where they start, and its number.
struct Places {
    int *lead, *pages, *start, *number;
    __device__ __forceinline__ Places(int* p, int B) : lead(p), pages(p + B), start(p + 2 * B), number(p + 3 * B) {}
};

// Rows first_row + warp of the plan, and every `stride` after, from lead and pages (all of the
// block's threads).
__device__ __forceinline__ void place_rows(int32_t* plan, int B, const Places& s, int first_row, int stride, int2* s_sum) {
    constexpr int kWarps = kPairThreads / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int r = tid; r < B; r += kPairThreads) s.start[r] = 0;
    __syncthreads();
    for (int r = tid; r < B; r += kPairThreads)
        if (s.lead[r] >= 0) atomicAdd(s.start + s.lead[r], 1);
    __syncthreads();
    // exclusive sums over the leaders: each thread some neighbours
    const int per = (B + kPairThreads - 1) / kPairThreads, lo = min(B, tid * per), hi = min(B, lo + per);
    int2 mine = make_int2(0, 0);               // rows, groups
    for (int r = lo; r < hi; ++r) {
        mine.x += s.start[r];
        mine.y += s.start[r] > 0;
    }
    int2 run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, run.x, o), y = __shfl_up_sync(kFull, run.y, o);
        if (lane >= o) {
            run.x += x;
            run.y += y;
        }
    }
    if (lane == 31) s_sum[warp] = run;
    __syncthreads();
    int2 at = make_int2(run.x - mine.x, run.y - mine.y), all = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int2 x = s_sum[w];
        if (w < warp) {
            at.x += x.x;
            at.y += x.y;
        }
        all.x += x.x;
        all.y += x.y;
    }
    for (int r = lo; r < hi; ++r) {
        const int c = s.start[r];
        s.start[r] = at.x;
        s.number[r] = at.y;
        at.x += c;
        at.y += c > 0;
    }
    __syncthreads();
    const GroupsLayout l(B);
    for (int b = first_row + warp; b < B; b += stride) {
        const int lead = s.lead[b];
        int rank = 0;                          // members of the group before the row
        if (lead >= 0) {
#pragma unroll 4
            for (int r = lead + lane; r < b; r += 32) rank += s.lead[r] == lead;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) rank += __shfl_xor_sync(kFull, rank, o);
        }
        if (lane != 0) continue;
        const int slot = lead >= 0 ? s.start[lead] + rank : -1, number = lead >= 0 ? s.number[lead] : -1;
        if (b == 0) {
            plan[0] = all.y;
            plan[1] = all.x;
            plan[l.start + B] = all.x;
        }
        plan[l.slot + b] = slot;
        plan[l.group + b] = number;
        if (lead >= 0) plan[l.rows + slot] = b;
        if (lead == b) {
            plan[l.start + number] = slot;
            plan[l.blocks + number] = s.pages[b];
        }
        if (b >= all.x) plan[l.rows + b] = -1;
        if (b >= all.y) {
            plan[l.start + b] = all.x;
            plan[l.blocks + b] = 0;
        }
    }
}

__device__ __forceinline__ int full_pages(const GroupsArgs& a, int r) {   // -1: a length out of range
    const int L = a.context_lens[r];
    return L < 0 || L > a.max_blocks * kBlock ? -1 : L / kBlock;
}

__global__ void __launch_bounds__(kRunThreads) runs_kernel(const GroupsArgs a) {
    __shared__ int s_min;
    const int tid = threadIdx.x, b = blockIdx.x;
    launch_dependents();
    grid_dependency_wait();
    const int32_t* mine = a.block_tables + (long long)b * a.max_blocks;
    const int n = full_pages(a, b);
    if (tid == 0 && n < 0) flag_error(a.err, GQA_DEVERR_CONTEXT_LEN);
    const int key = n > 0 ? *mine : -1;
    if (tid == 0) a.best[b] = 0ull;
    if (key < 0) {                             // uniform: no page to share
        if (tid == 0) a.run[b] = make_int2(b, 0);
        return;
    }
    // the lowest row with the same first page, itself at the latest
    int leader = b;
    for (int base = 0; base < b; base += kRunThreads * kRunUnroll) {
        if (tid == 0) s_min = b;
        __syncthreads();
        int first[kRunUnroll], len[kRunUnroll];
#pragma unroll
        for (int i = 0; i < kRunUnroll; ++i) {
            const int r = base + i * kRunThreads + tid;
            first[i] = r < b ? a.block_tables[(long long)r * a.max_blocks] : -1;
            len[i] = r < b ? full_pages(a, r) : 0;
        }
#pragma unroll
        for (int i = kRunUnroll - 1; i >= 0; --i)
            if (first[i] == key && len[i] > 0) leader = min(leader, base + i * kRunThreads + tid);
        if (leader < b) atomicMin(&s_min, leader);
        __syncthreads();
        leader = s_min;
        __syncthreads();
        if (leader < b) break;
    }
    const int32_t* lead = a.block_tables + (long long)leader * a.max_blocks;
    const int most = min(n, full_pages(a, leader));
    int run = most;
    for (int base = 0; base < most; base += kRunThreads * kRunUnroll * 2) {
        if (tid == 0) s_min = most;
        __syncthreads();
        int x[2 * kRunUnroll], y[2 * kRunUnroll];
#pragma unroll
        for (int i = 0; i < 2 * kRunUnroll; ++i) {
            const int j = base + i * kRunThreads + tid;
            x[i] = j < most ? mine[j] : 0;
            y[i] = j < most ? lead[j] : 0;
        }
        int at = most;
#pragma unroll
        for (int i = 2 * kRunUnroll - 1; i >= 0; --i)
            if (x[i] != y[i] || x[i] < 0) at = base + i * kRunThreads + tid;
        if (at < most) atomicMin(&s_min, at);
        __syncthreads();
        run = s_min;
        __syncthreads();
        if (run < most) break;
    }
    if (tid == 0) a.run[b] = make_int2(leader, run);
}

__global__ void __launch_bounds__(kPairThreads) counts_kernel(const GroupsArgs a) {
    extern __shared__ int2 s_run[];            // [B]
    const int lane = threadIdx.x & 31, b = blockIdx.x * kPairRows + (threadIdx.x >> 5);
    launch_dependents();
    grid_dependency_wait();
    for (int r = threadIdx.x; r < a.B; r += kPairThreads) s_run[r] = a.run[r];
    __syncthreads();
    if (b >= a.B) return;
    const int2 me = s_run[b];
    if (me.y < max(a.min_blocks, 1)) return;
    int c = 0;
#pragma unroll 4
    for (int r = lane; r < a.B; r += 32) {
        const int2 o = s_run[r];
        c += o.x == me.x && o.y >= me.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(kFull, c, o);
    if (lane == 0 && c > 1) atomicMax(a.best + me.x, worth(me.y, c));
}

__global__ void __launch_bounds__(kPairThreads) places_kernel(const GroupsArgs a) {
    extern __shared__ int s_places[];          // [4][B]
    __shared__ int2 s_sum[kPairThreads / 32];
    const Places s(s_places, a.B);
    launch_dependents();
    grid_dependency_wait();
    for (int r = threadIdx.x; r < a.B; r += kPairThreads) s.pages[r] = pages_of(a.best[r]);
    __syncthreads();
    for (int r = threadIdx.x; r < a.B; r += kPairThreads) {
        const int2 o = a.run[r];
        s.lead[r] = s.pages[o.x] > 0 && o.y >= s.pages[o.x] ? o.x : -1;
    }
    __syncthreads();
    place_rows(a.plan, a.B, s, blockIdx.x * kPairRows, kMaxGroupRows, s_sum);
}

// All three steps for up to kSmallRows rows.
__global__ void __cluster_dims__(kSmallCtas) __launch_bounds__(kPairThreads) small_kernel(const GroupsArgs a) {
    __shared__ int2 s_run[kSmallRows];
    __shared__ unsigned long long s_best[kSmallRows];
    __shared__ int s_places[4 * kSmallRows];
    __shared__ int2 s_sum[kPairThreads / 32];
    const Places s(s_places, a.B);
    const int tid = threadIdx.x, lane = tid & 31, row0 = blockIdx.x * kPairRows;
    launch_dependents();
    grid_dependency_wait();
    for (int b = row0 + (tid >> 5); b < a.B; b += kSmallWarps) {
        const int32_t* mine = a.block_tables + (long long)b * a.max_blocks;
        const int n = full_pages(a, b);
        if (lane == 0 && n < 0) flag_error(a.err, GQA_DEVERR_CONTEXT_LEN);
        const int key = n > 0 ? mine[0] : -1;
        int leader = b, run = 0;
        if (key >= 0) {                        // uniform per warp
            for (int base = 0; base < b && leader == b; base += 32 * kRunUnroll) {
                int first = b;
#pragma unroll
                for (int i = kRunUnroll - 1; i >= 0; --i) {
                    const int r = base + 32 * i + lane;
                    if (r < b && a.block_tables[(long long)r * a.max_blocks] == key && full_pages(a, r) > 0) first = r;
                }
                leader = __reduce_min_sync(kFull, first);
            }
            const int32_t* lead = a.block_tables + (long long)leader * a.max_blocks;
            const int most = min(n, full_pages(a, leader));
            run = most;
            for (int base = 0; base < most && run == most; base += 32 * 2 * kRunUnroll) {
                int x[2 * kRunUnroll], y[2 * kRunUnroll];
#pragma unroll
                for (int i = 0; i < 2 * kRunUnroll; ++i) {
                    const int j = base + 32 * i + lane;
                    x[i] = j < most ? mine[j] : 0;
                    y[i] = j < most ? lead[j] : 0;
                }
                int at = most;
#pragma unroll
                for (int i = 2 * kRunUnroll - 1; i >= 0; --i)
                    if (x[i] != y[i] || x[i] < 0) at = base + 32 * i + lane;
                run = __reduce_min_sync(kFull, at);
            }
        }
        if (lane == 0) a.run[b] = make_int2(leader, run);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // every CTA counts for all rows, then places its own
    for (int r = tid; r < a.B; r += kPairThreads) {
        s_run[r] = __ldcg(a.run + r);
        s_best[r] = 0ull;
    }
    __syncthreads();
    constexpr int kParts = 4;                  // neighbouring threads that count for a row
    for (int r0 = 0; r0 < a.B; r0 += kPairThreads / kParts) {
        const int r = r0 + tid / kParts;
        int c = 0;
        int2 me = make_int2(0, 0);
        if (r < a.B) {
            me = s_run[r];
            for (int o = tid % kParts; o < a.B; o += kParts) {
                const int2 x = s_run[o];
                c += x.x == me.x && x.y >= me.y;
            }
        }
        c += __shfl_xor_sync(kFull, c, 1);
        c += __shfl_xor_sync(kFull, c, 2);
        if (tid % kParts == 0 && me.y >= max(a.min_blocks, 1) && c > 1) atomicMax(&s_best[me.x], worth(me.y, c));
    }
    __syncthreads();
    for (int r = tid; r < a.B; r += kPairThreads) {
        const int2 o = s_run[r];
        const int pages = pages_of(s_best[o.x]);
        s.pages[r] = pages_of(s_best[r]);
        s.lead[r] = pages > 0 && o.y >= pages ? o.x : -1;
    }
    __syncthreads();
    place_rows(a.plan, a.B, s, row0, kSmallWarps, s_sum);
}

}  // namespace

long long prefix_groups_ints(int batch) {
    const GroupsLayout l(batch);
    return (long long)l.scratch + 4LL * batch;
}

cudaError_t launch_pages_groups(const int32_t* block_tables, int max_blocks, const int32_t* context_lens, int batch,
                                int min_blocks, int32_t* plan, int32_t* err, cudaStream_t stream) {
    GroupsArgs a;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.plan = plan;
    const GroupsLayout l(batch);
    a.run = reinterpret_cast<int2*>(plan + l.scratch);
    a.best = reinterpret_cast<unsigned long long*>(a.run + batch);
    a.err = err;
    a.B = batch;
    a.max_blocks = max_blocks;
    a.min_blocks = min_blocks;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (batch <= kSmallRows) {
        cfg.gridDim = dim3(kSmallCtas);
        cfg.blockDim = dim3(kPairThreads);
        return cudaLaunchKernelEx(&cfg, small_kernel, a);
    }
    cfg.gridDim = dim3(batch);
    cfg.blockDim = dim3(kRunThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, runs_kernel, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((batch + kPairRows - 1) / kPairRows);
    cfg.blockDim = dim3(kPairThreads);
    const int run_bytes = batch * (int)sizeof(int2), places_bytes = 4 * batch * (int)sizeof(int);   // 64 and 128 KB at most
    if (ctas_per_sm(reinterpret_cast<const void*>(&counts_kernel), kPairThreads, run_bytes) < 1 ||
        ctas_per_sm(reinterpret_cast<const void*>(&places_kernel), kPairThreads, places_bytes) < 1)
        return cudaErrorInvalidConfiguration;
    cfg.dynamicSmemBytes = run_bytes;
    if ((e = cudaLaunchKernelEx(&cfg, counts_kernel, a)) != cudaSuccess) return e;
    cfg.dynamicSmemBytes = places_bytes;
    return cudaLaunchKernelEx(&cfg, places_kernel, a);
}

}  // namespace gqa
