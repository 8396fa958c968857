// gqa_groups.cuh -- the groups of rows that share their first blocks, as
// gqa_kv_pages_groups lays them out and the shared decode reads them.
#pragma once

#include "gqa_device.cuh"

namespace gqa {

// int32 offsets of the arrays in a plan for B rows (counts at 0 and 1).
struct GroupsLayout {
    int start, blocks, rows, slot, group, scratch;
    __host__ __device__ explicit GroupsLayout(int B)
        : start(2), blocks(3 + B), rows(3 + 2 * B), slot(3 + 3 * B), group(3 + 4 * B), scratch((3 + 5 * B + 3) & ~3) {}
};

struct PrefixGroups {
    const int32_t *count, *start, *blocks, *rows, *slot, *group;
    int B;
    __device__ __forceinline__ PrefixGroups(const int32_t* p, int batch) : B(batch) {
        const GroupsLayout l(batch);
        count = p;
        start = p + l.start;
        blocks = p + l.blocks;
        rows = p + l.rows;
        slot = p + l.slot;
        group = p + l.group;
    }
    __device__ __forceinline__ int groups() const { return min(max(*count, 0), B); }
};

// Group i: its first slot, rows and shared blocks. A group whose entries lie outside the
// plan or the tables has none, so that no plan leads a read astray.
struct GroupSpan {
    int first, rows, blocks;
};
__device__ __forceinline__ GroupSpan group_span(const PrefixGroups& p, int i, int max_blocks) {
    const int a = p.start[i], e = p.start[i + 1], n = p.blocks[i];
    const bool good = a >= 0 && e > a && e <= p.B && n > 0 && n <= max_blocks;
    return good ? GroupSpan{a, e - a, n} : GroupSpan{0, 0, 0};
}

// A row's part in a plan and its length, in two trips to memory: every load of a trip is
// issued before the first branch.
struct SharedRow {
    int len, blocks, group, member;           // a length out of range: -1, blocks 0
    GroupSpan span;
};
__device__ __forceinline__ SharedRow shared_row(const PrefixGroups& p, const int32_t* lens, int b, int T, int max_blocks) {
    const int L = lens[b], s = p.slot[b], i = p.group[b], n_groups = p.groups();
    const int sc = min(max(s, 0), p.B - 1), ic = min(max(i, 0), p.B - 1);
    const int row = p.rows[sc];
    SharedRow r{L, 0, ic, 0, group_span(p, ic, max_blocks)};
    if (L < 0 || L > max_blocks * kBlock) {
        r.len = -1;
        return r;
    }
    // all the blocks that the group shares where every query of the row sees them whole,
    // else none: the row then attends its context alone
    if (s == sc && i == ic && i < n_groups && row == b && s >= r.span.first && s < r.span.first + r.span.rows &&
        (long long)r.span.blocks * kBlock + T - 1 <= L) {
        r.blocks = r.span.blocks;
        r.member = s - r.span.first;
    }
    return r;
}

// ---- how the shared decode divides the GPU
//
// The kernel that attends the shared blocks and the one that attends the rows' own run side
// by side: the first takes as many SMs as make both end together, as far as their work can
// be told from the plan and the lengths. Times are per SM.
constexpr int kStepTokens = 64;                   // tokens of a step of the prefix kernel
struct SplitModel {
    int sms, ctas_per_sm, cta_rows, min_steps;    // of the prefix kernel; fewest steps of a CTA
    float step_us, prefix_us;                     // a step of an SM's CTAs, the kernel's start and end
    float unit_us, pair_us, tail_us;              // a (block, kv-head) of the tail, a (row, kv-head), its start
};

// One group's rows for one kv-head, and how its steps lie.
struct Problem {
    int rows, tiles, chunks, units;
};
__device__ __forceinline__ Problem problem_of(const GroupSpan& s, int K, int GT, int cta_rows) {
    Problem p;
    p.rows = s.rows * GT;
    p.tiles = (p.rows + cta_rows - 1) / cta_rows;
    p.chunks = (s.blocks * kBlock + kStepTokens - 1) / kStepTokens;
    p.units = p.tiles * p.chunks * K;
    return p;
}

// SMs for `steps` steps of the prefix beside `units` blocks of `pairs` rows' own: those with
// which the later of the two ends first, in whole pairs of SMs (see the launch) and no more
// than its CTAs have min_steps each for. Called by whole warps: the lanes try 32 numbers at a
// time (one after the other, by halving, takes 1.1 us before the first copy).
__device__ __forceinline__ int prefix_sms(const SplitModel& m, int steps, int units, int pairs) {
    if (steps <= 0) return 0;                     // (below 0: the sum of a plan of overlapping groups)
    const int per_sm = m.min_steps * m.ctas_per_sm, most = min(m.sms, (steps + per_sm - 1) / per_sm);
    if (units == 0) return most;
    const int lane = threadIdx.x & 31, cap = max(1, min(most, m.sms - 2));
    const float wp = steps * m.step_us / m.ctas_per_sm, wt = units * m.unit_us + pairs * m.pair_us;
    auto prefix_end = [&](int x) { return m.prefix_us + __fdividef(wp, (float)x); };
    auto tail_end = [&](int x) { return m.tail_us + __fdividef(wt, (float)(m.sms - x)); };
    int lo = 0;                                   // there the prefix ends last
    for (int step = (cap + 31) / 32;; step = (step + 31) / 32) {
        const int x = min(lo + (lane + 1) * step, cap);
        const bool first = x >= cap || prefix_end(x) <= tail_end(x);
        const int n = __ffs(__ballot_sync(kFull, first)) - 1;                // some lane's x is the cap, or past the answer
        if (step > 1) {
            lo += n * step;
            continue;
        }
        const int hi = min((lo + n + 2) & ~1, cap), less = (hi - 1) & ~1;    // the tail ends last; the prefix
        return less > 0 && prefix_end(less) < fmaxf(prefix_end(hi), tail_end(hi)) ? less : hi;
    }
}

}  // namespace gqa
