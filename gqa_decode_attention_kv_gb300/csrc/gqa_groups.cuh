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
    int first, rows, blocks, leader;
};
__device__ __forceinline__ GroupSpan group_span(const PrefixGroups& p, int i, int max_blocks) {
    GroupSpan s{0, 0, 0, 0};
    const int a = p.start[i], e = p.start[i + 1], n = p.blocks[i];
    if (a < 0 || e <= a || e > p.B || n <= 0 || n > max_blocks) return s;
    const int lead = p.rows[a];
    if (lead < 0 || lead >= p.B) return s;
    return GroupSpan{a, e - a, n, lead};
}

// Blocks that its group attends for row b of length L (T new tokens included): all that
// the group shares where every query of the row sees them whole, else none, and the row
// attends its context alone. g and slot: its group and place in it.
__device__ __forceinline__ int shared_blocks(const PrefixGroups& p, int b, int L, int T, int max_blocks, int* g = nullptr,
                                             int* member = nullptr) {
    const int s = p.slot[b], i = p.group[b];
    if (s < 0 || s >= p.B || i < 0 || i >= p.groups() || p.rows[s] != b) return 0;
    const GroupSpan span = group_span(p, i, max_blocks);
    if (s < span.first || s >= span.first + span.rows) return 0;
    if ((long long)span.blocks * kBlock + T - 1 > L) return 0;
    if (g) *g = i;
    if (member) *member = s - span.first;
    return span.blocks;
}

}  // namespace gqa
