// gqa_groups.cu -- which rows of the block tables share their first pages.
//
// With n_b the full pages of row b, its leader is the lowest row with the same first
// page, and m_b the number of leading entries it has in common with the leader's. Of a
// leader's rows a group takes P pages where P (c(P) - 1) is largest, c(P) the rows with
// m_b >= P: the pages that attending them once saves reading. Three short kernels, each
// with the whole GPU on it, because each needs all of the one before:
//   runs    one CTA per row: the leader, then the common run, 512 entries a step
//   counts  one warp per row: c(m_b) over all rows, the best P of each leader by one
//           64-bit maximum (saving, then fewer rows, so the larger P at equal saving)
//   places  one warp per row: groups in the order of their leaders, members by row
// The tables are read once as far as rows agree (the leaders' rows come from L2). The
// two passes over all pairs of rows are 8 bytes a pair from L2 or L1.
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
constexpr int kPairThreads = 256;
constexpr int kRankBits = 14;
constexpr unsigned kRankMask = (1u << kRankBits) - 1;

__global__ void __launch_bounds__(kRunThreads) runs_kernel(const GroupsArgs a) {
    __shared__ int s_min;
    const int tid = threadIdx.x, b = blockIdx.x;
    launch_dependents();
    grid_dependency_wait();
    auto full_pages = [&](int r) {
        const int L = a.context_lens[r];
        if (L < 0 || L > a.max_blocks * kBlock) return -1;
        return L / kBlock;
    };
    const int32_t* mine = a.block_tables + (long long)b * a.max_blocks;
    const int n = full_pages(b);
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
            len[i] = r < b ? full_pages(r) : 0;
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
    const int most = min(n, full_pages(leader));
    int run = most;
    for (int base = 0; base < most; base += kRunThreads * kRunUnroll) {
        if (tid == 0) s_min = most;
        __syncthreads();
        int x[kRunUnroll], y[kRunUnroll];
#pragma unroll
        for (int i = 0; i < kRunUnroll; ++i) {
            const int j = base + i * kRunThreads + tid;
            x[i] = j < most ? mine[j] : 0;
            y[i] = j < most ? lead[j] : 0;
        }
        int at = most;
#pragma unroll
        for (int i = kRunUnroll - 1; i >= 0; --i)
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
    const int lane = threadIdx.x & 31, b = blockIdx.x * (kPairThreads / 32) + (threadIdx.x >> 5);
    launch_dependents();
    grid_dependency_wait();
    if (b >= a.B) return;
    const int2 me = a.run[b];
    if (me.y < max(a.min_blocks, 1)) return;
    int c = 0;
#pragma unroll 4
    for (int r = lane; r < a.B; r += 32) {
        const int2 o = a.run[r];
        c += o.x == me.x && o.y >= me.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(kFull, c, o);
    if (lane == 0 && c > 1)
        atomicMax(a.best + me.x, ((unsigned long long)me.y * (unsigned)(c - 1) << kRankBits) | (kRankMask - (unsigned)c));
}

__global__ void __launch_bounds__(kPairThreads) places_kernel(const GroupsArgs a) {
    const int lane = threadIdx.x & 31, b = blockIdx.x * (kPairThreads / 32) + (threadIdx.x >> 5);
    launch_dependents();
    grid_dependency_wait();
    if (b >= a.B) return;
    // pages of a leader's group, 0: none
    auto pages = [&](int leader) -> int {
        const unsigned long long k = a.best[leader];
        if (k == 0ull) return 0;
        return (int)((k >> kRankBits) / (kRankMask - (unsigned)(k & kRankMask) - 1u));
    };
    const int2 me = a.run[b];
    const int shared = pages(me.x);
    const bool member = shared > 0 && me.y >= shared;
    int groups = 0, total = 0, before_groups = 0, before = 0;
#pragma unroll 4
    for (int r = lane; r < a.B; r += 32) {
        const int2 o = a.run[r];
        const int p = pages(o.x);
        if (p == 0 || o.y < p) continue;
        const bool head = o.x == r;
        ++total;
        groups += head;
        before_groups += head && r < me.x;
        before += o.x < me.x || (o.x == me.x && r < b);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        groups += __shfl_xor_sync(kFull, groups, o);
        total += __shfl_xor_sync(kFull, total, o);
        before_groups += __shfl_xor_sync(kFull, before_groups, o);
        before += __shfl_xor_sync(kFull, before, o);
    }
    if (lane != 0) return;
    const GroupsLayout l(a.B);
    int32_t* plan = a.plan;
    if (b == 0) {
        plan[0] = groups;
        plan[1] = total;
        plan[l.start + a.B] = total;           // where every row leads a group: unused otherwise
    }
    plan[l.slot + b] = member ? before : -1;
    plan[l.group + b] = member ? before_groups : -1;
    if (member) {
        plan[l.rows + before] = b;
        if (me.x == b) {
            plan[l.start + before_groups] = before;
            plan[l.blocks + before_groups] = shared;
        }
    }
    if (b >= total) plan[l.rows + b] = -1;
    if (b >= groups) {
        plan[l.start + b] = total;
        plan[l.blocks + b] = 0;
    }
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
    cfg.gridDim = dim3(batch);
    cfg.blockDim = dim3(kRunThreads);
    cudaError_t e = cudaLaunchKernelEx(&cfg, runs_kernel, a);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((batch + kPairThreads / 32 - 1) / (kPairThreads / 32));
    cfg.blockDim = dim3(kPairThreads);
    if ((e = cudaLaunchKernelEx(&cfg, counts_kernel, a)) != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, places_kernel, a);
}

}  // namespace gqa
