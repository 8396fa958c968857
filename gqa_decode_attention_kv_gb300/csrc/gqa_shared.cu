// gqa_shared.cu -- decode attention for a batch whose rows share long prefixes. A group
// of rows holds the same pages at the front of their block tables; its K and V are read
// and multiplied with the queries of all of them, one (kv-head, group) being a problem of
// rows * G * T query rows: once for every 256 of those (a CTA's two tiles), or every 128 in
// the form for groups of no more. Three kernels, one behind the other:
//   prefix   (here) the shared blocks, for all rows of a group at once
//   tail     (gqa_decode_tail.cu) every row's own blocks; runs beside the prefix kernel
//   merge    (here) a row's pieces of both, with their log-sum-exp weights
// Softmax over a set of positions is the merge of softmaxes over its parts: a part is
// (m, l, o) = (max s, sum 2^(s-m), sum 2^(s-m) v), and parts join as M = max m_i,
// o / l = sum o_i 2^(m_i-M) / sum l_i 2^(m_i-M), all of it in fp32.
//
// The prefix kernel works on the 5th-generation tensor cores, 128 query rows (the MMA's M)
// a tile, the K/V of 64 tokens (4 pages) a step:
//   S[128 x 64]  = Q K^T     Q and K in shared memory, S in tensor memory
//   softmax                  two threads per row, 32 of the step's tokens each; the weights
//                            as a high and a low 16-bit part over S (a 16-bit weight alone
//                            would round it to the cache's type)
//   O[128 x d]  += P V       P from tensor memory, V from shared memory
// Coded caches (int8, e4m3, int4) take the same products in fp16: their copy warps widen
// the codes of a step on the way (exact), K's scales go into the scores and V's into the
// weights, which a power of two keeps where fp16 has its bits.
// The (group, kv-head, tile) problems are laid out one behind the other in steps and cut
// into equal runs, one per CTA of a single resident wave, so a long prefix is split over
// the whole GPU however few rows share it, and the pieces are joined by the merge.
//
// What bounds it: with 256 rows a step's products (S, and P V for both parts of P) are 1536
// cycles at the 8192 flop a cycle of an SM's tensor cores, and a step takes 1790, in which the
// softmax issues about as long: dropping the exponentials, one part of P or S alone changes
// that by less than 5%. Coded steps take 2900 cycles, bound by the instructions that widen and
// scale: over 48 int8 steps a scheduler issues 2475 a step. From 32768 to 98304 shared tokens
// a step adds 1.10 us (bf16, fp16), 1.43 (int8), 1.49 (int4), 1.51 (e4m3). With few rows K and
// V arrive at the copy rate (two CTAs of 128 rows: 64 KB in 1.4 us an SM, 6.9 TB/s). Around the
// steps: 8 to 10 us until the first (launch, sums of the plan, table, K), 4 for the last step's
// output, 4 to 6 for the merge. 32 rows of H=64, K=8, d=128 behind 32768 tokens take 56 us
// (gqa_decode 464), 64 rows of H=32 behind 4096 and 100 to 700 of their own 36, 128 rows of H=64
// in four groups behind 8192 and 100 to 900 over int8 106, e4m3 108, int4 107 (gqa_decode 484,
// 496, 418), bf16 95 (500).
#include <algorithm>
#include <climits>

#include "gqa_decode_kernels.cuh"
#include "gqa_groups.cuh"
#include "gqa_internal.h"

namespace gqa {

namespace {

using dec::DecodeArgs;
using dec::Partition;

constexpr int kRows = 128;                       // query rows of a tile: the MMA's M, one TMEM lane each
constexpr int kChunk = kStepTokens;              // tokens of a step: N of S, K of P.V
constexpr int kChunkBlocks = kChunk / kBlock;
constexpr int kBufs = 4;                         // per-step barrier copies (G & 3)
constexpr uint32_t kColTile = 256;               // tile t: S buffers at columns 256t, 256t + 64,
constexpr uint32_t kColO = 128;                  //         O at 256t + 128
constexpr int kHalf = kChunk / 2;                // tokens of a step that a softmax thread takes
constexpr float kSlackLog2 = 8.f;                // headroom before (m, l, O) are rescaled

// Barrier of the two warps that share rows; pair_any: whether any of their threads says so.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(int id, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)mine)
        : "memory");
    return r != 0;
}

// Two weights as a high and a low 16-bit part each. bf16's high part is the value cut
// off, which takes no conversion (together 2^-16 of the weight; rounded 2^-17). fp16's
// parts are exact to half its smallest step, 2^-25, so its weights come kUpF16 powers of
// two up (at most 2^15 with the slack): what is lost is 2^-32 of a row's largest weight.
constexpr float kUpF16 = 7.f;
template <bool kBf16>
__device__ __forceinline__ void split2(float x, float y, uint64_t xy, uint32_t& hi, uint32_t& lo) {
    float2 h;
    if constexpr (kBf16) {
        const uint32_t u = __float_as_uint(x), v = __float_as_uint(y);
        hi = __byte_perm(u, v, 0x7632);
        h = make_float2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u));
    } else {
        hi = pack2<false>(x, y);
        h = unpack2<false>(hi);
    }
    const float2 r = f2_split(f2_sub(xy, f2_make(h.x, h.y)));
    lo = pack2<kBf16>(r.x, r.y);
}

struct SharedArgs {
    const void* q;
    const __half *k_scale, *v_scale;
    int q_dtype;
    const int32_t* groups;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* err;
    long long num_blocks;
    int B, H, K, G, T, GT, max_blocks;
    int map_perm[3], page_perm[2];
    float scale_log2;
    SplitModel split;
    int32_t* begun;      // for the tail kernel: everything before this one has ended
    int32_t* hdr;        // [0] steps per CTA, [1] all steps, [2] rows of a CTA
    int32_t* first_unit; // [groups] first step of each group, INT_MIN where its first row is outside the batch
    float2 *ml_a, *ml_b; // (m, l) of a problem's first piece by row, and of CTA j's continued one
    float *o_a, *o_b;    // their un-normalised outputs
};

// kTiles query tiles per CTA: two (one CTA per SM, all 512 tensor-memory columns, K/V read
// once for 256 rows) or one (two CTAs per SM).
template <typename T, int kTiles, int D>
struct SharedCfg {
    static constexpr bool kI8 = std::is_same<T, int8_t>::value;
    static constexpr bool kFp8 = std::is_same<T, __nv_fp8_e4m3>::value;
    static constexpr bool kI4 = std::is_same<T, int4x2>::value;
    static constexpr bool kCoded = kI8 || kFp8 || kI4;
    static_assert(!kCoded || kTiles == 2, "coded caches have the two-tile form alone");
    static constexpr int kHalves = D / 64;               // 128-byte column halves of a row
    static constexpr int kCtaRows = kTiles * kRows;
    static constexpr int kSoftWarps = 8 * kTiles;        // four for each half of a step's tokens
    static constexpr int kCopyWarps = kCoded ? 4 : 2;    // K, V: one each, or two that also widen
    static constexpr int kThreads = 32 * (kSoftWarps + 2 * kTiles + kCopyWarps);   // + S and P.V warps per tile
    static constexpr int kStages = kCoded ? 2 : kTiles == 2 || D == 64 ? 4 : 2;    // K and V stages
    static constexpr int kRaw = kCoded ? 4 : 0;          // stages of codes
    static constexpr int kCtasPerSm = kTiles == 2 ? 1 : 2;
    static constexpr uint32_t kTmemCols = 256u * kTiles;
    static constexpr int kQt = kRows * D * 2;            // one Q tile: halves x 128 rows x 128 B
    static constexpr int kKc = kChunk * D * 2;           // K chunk: halves x 64 rows x 128 B
    static constexpr int kVb = kBlock * D * 2;           // one V page
    static constexpr int kVc = kChunkBlocks * kVb;
    static constexpr int kCodeRow = kI4 ? D / 2 : D;     // bytes of a row of codes
    static constexpr int kCodes = kHalf * kCodeRow;      // a copy warp's codes of a step, then the step's scales
    static constexpr int kRawStage = kCodes + kChunk * 2;
    static constexpr int kOffK = kTiles * kQt, kOffV = kOffK + kStages * kKc, kOffRaw = kOffV + kStages * kVc,
                         kOffBar = kOffRaw + 4 * kRaw * kRawStage;
    static constexpr int kOffEx = kOffBar + 1024;        // [tile][half][row]: maxima, then sums
    static constexpr int kOffSc = kOffEx + kCtaRows * 8; // coded: kSlots x (scales of K, of V, {factor, unlift})
    static constexpr int kSlots = 4, kSlotF = 2 * kChunk + 4;
    static constexpr int kSmem = 1024 + kOffSc + (kCoded ? kSlots * kSlotF * 4 : 0);
    static_assert((kSmem + 1024) * kCtasPerSm <= 228 * 1024, "CTAs per SM fit the shared memory");
};

// 16 codes of a row -> 8 words of two fp16 values each, exactly. w: 4 words of 8-bit
// codes, 2 of 4-bit ones.
template <class C>
__device__ __forceinline__ void widen16(const uint32_t* w, uint32_t (&o)[8]) {
    if constexpr (C::kI8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) i8x4_to_f16x4(w[i], o[2 * i], o[2 * i + 1]);
    } else if constexpr (C::kFp8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = e4m3x2_to_f16x2(w[i / 2] >> (16 * (i & 1)));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {          // bytes 0 and 2, then 1 and 3
                const uint32_t lo = i4_lo_pair(w[i] >> (8 * e)), hi = i4_hi_pair(w[i] >> (8 * e));
                o[4 * i + e] = __byte_perm(lo, hi, 0x5410);
                o[4 * i + 2 + e] = __byte_perm(lo, hi, 0x7632);
            }
        }
    }
}

// V's scales in the weights: w = p vs 2^lift, with the lift that puts the largest scale so
// far into [2^5, 2^6), kept until a scale passes 2^7: p is at most 2^8, so that w stays
// within fp16's range, and what its parts lose is 2^-30 of that scale and p's largest.
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }
constexpr int kLiftNone = 29;                     // before any scale: the least fp16 one is 2^-24

template <typename T, int kTiles, int D>
__global__ void __launch_bounds__(SharedCfg<T, kTiles, D>::kThreads, SharedCfg<T, kTiles, D>::kCtasPerSm)
shared_prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const SharedArgs a) {
    using C = SharedCfg<T, kTiles, D>;
    constexpr int kS = C::kStages;
    constexpr bool kCoded = C::kCoded;
    constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
    constexpr float kUp = std::is_same<T, __half>::value ? kUpF16 : 0.f;   // log2 of the weights' scaling
    constexpr uint32_t kIdescS = mma_idesc_f16(kRows, kChunk, kB, false, false);
    constexpr uint32_t kIdescO = mma_idesc_f16(kRows, D, kB, false, true);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t* gb = smem_raw + (sb - raw);
    const uint32_t sQ = sb, sK = sb + C::kOffK, sV = sb + C::kOffV;
    // Barriers, 8 B each: K stages, V stages (stage G % kS), then per tile t "S_t(G)
    // done", "P_t(G).V(G) done", "P_t(G) ready" (copy G & 3), "Q_t stored"; the TMEM
    // address; the scan's scratch; a coded cache's copies; warps that gave up. G counts the
    // CTA's steps across its segments. Per-step barriers come in four copies, so that no
    // parity wait can fall two phases behind.
    const uint32_t bar0 = sb + C::kOffBar;
    auto stage = [](int c) { return c % kS; };
    auto par_st = [](int c) { return (uint32_t)(c / kS) & 1u; };
    auto bar_k = [&](int c) { return bar0 + 8 * stage(c); };
    auto bar_v = [&](int c) { return bar0 + 32 + 8 * stage(c); };
    auto bar_s = [&](int t, int c) { return bar0 + 64 + 96 * t + 8 * (c & 3); };
    auto bar_o = [&](int t, int c) { return bar0 + 96 + 96 * t + 8 * (c & 3); };
    auto bar_p = [&](int t, int c) { return bar0 + 128 + 96 * t + 8 * (c & 3); };
    auto bar_q = [&](int t) { return bar0 + 256 + 8 * t; };
    const uint32_t tslot = bar0 + 272;
    // [128] sums by warp (word 24: groups overlap), then where the run begins: group, its step, its span, its leader
    int* scan = reinterpret_cast<int*>(gb + C::kOffBar + 288);
    auto bar_full = [&](int cw, int c) { return bar0 + 832 + 32 * cw + 8 * (c & 3); };   // coded: copy warp cw's codes landed
    float* scales = reinterpret_cast<float*>(gb + C::kOffSc);
    auto par4 = [](int c) { return (uint32_t)(c >> 2) & 1u; };

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(kFull, tid >> 5, 0);               // uniform: addresses from it stay so
    const bool softmax = warp < C::kSoftWarps, loader = warp >= C::kSoftWarps + 2 * kTiles;
    const bool mma_warp = !softmax && !loader;
    const int tt = warp >> 3, hf = (warp >> 2) & 1;             // softmax warps: their tile and half
    if (tid == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
        for (int i = 0; i < kS; ++i) {
            mbar_init(bar_k(i), kCoded ? 2 : 1);   // K, V stages: the copy, or two warps that widen
            mbar_init(bar_v(i), kCoded ? 2 : 1);
        }
        for (int i = 0; i < 4 * C::kRaw; ++i) mbar_init(bar_full(i >> 2, i), 33);   // the copies, and each lane's scales
        for (int t = 0; t < kTiles; ++t) {
            for (int i = 0; i < kBufs; ++i) {
                mbar_init(bar_s(t, i), 1);
                mbar_init(bar_o(t, i), 1);
                mbar_init(bar_p(t, i), 8);     // one arrival per softmax warp of the tile
            }
            mbar_init(bar_q(t), 8);
        }
        for (int i = 0; i < 2 * 4 * kTiles; ++i) scan[168 + i] = 0;      // "this pair's warp gave up"
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(tslot, C::kTmemCols);
    // The tail kernel behind this one does not wait for it: it may start only once
    // everything before this kernel has ended, which this wait makes sure of.
    grid_dependency_wait();
    if (blockIdx.x == 0 && tid == 0) store_release(a.begun, 1);
    launch_dependents();

    // ---- the steps of all problems and the rows' own blocks, from them the CTAs that take
    // part, and where this CTA's run of steps begins. Each thread takes a group of a round;
    // the first round's stay in registers.
    const PrefixGroups plan(a.groups, a.B);
    const int n_groups = plan.groups();
    // CTAs are numbered SM by SM, as a grid of one wave is dealt out: those that take no
    // part then leave whole SMs to the tail kernel
    const int j = (int)blockIdx.x % a.split.sms * C::kCtasPerSm + (int)blockIdx.x / a.split.sms;
    constexpr int kWarps = C::kThreads / 32;
    auto span_of = [&](int i) { return group_span(plan, min(i, a.B - 1), a.max_blocks); };
    auto units_of = [&](const GroupSpan& x, int i) {
        return i < n_groups ? problem_of(x, a.K, a.GT, C::kCtaRows).units : 0;
    };
    auto blocks_of = [&](int b) {
        const SharedRow r = shared_row(plan, a.context_lens, min(b, a.B - 1), a.T, a.max_blocks);
        return b < a.B && r.len > 0 ? (r.len + kBlock - 1) / kBlock - r.blocks : 0;
    };
    GroupSpan mine = span_of(tid);
    // a group's first row, -1: outside the batch, and its pages then count as missing (the merge flags it)
    auto leader_of = [&](const GroupSpan& x) {
        const int r = plan.rows[x.first];
        return r < a.B ? max(r, -1) : -1;
    };
    int lead = leader_of(mine);
    static_assert(kWarps <= 24, "the sums by warp leave word 24 of the scan");
    int U = 0, own = 0, own_rows = 0;
    {
        const int x0 = blocks_of(tid);
        int blocks = x0, rows = x0 > 0, sum = units_of(mine, tid), grouped = tid < n_groups ? mine.rows : 0;
        for (int i = tid + C::kThreads; i < n_groups; i += C::kThreads) {
            const GroupSpan x = span_of(i);
            sum += units_of(x, i);
            grouped += x.rows;                 // at most B * B < 2^26 in all
        }
        for (int b = tid + C::kThreads; b < a.B; b += C::kThreads) {
            const int x = blocks_of(b);
            blocks += x;
            rows += x > 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(kFull, sum, o);
            blocks += __shfl_xor_sync(kFull, blocks, o);
            rows += __shfl_xor_sync(kFull, rows, o);
        }
        grouped = __reduce_add_sync(kFull, grouped);
        if (lane == 0) {
            scan[warp] = sum;
            scan[32 + warp] = blocks;
            scan[96 + warp] = rows | min(grouped, kMaxBatch + 1) << 13;      // kWarps of them stay below 2^31
        }
        __syncthreads();
        U = __reduce_add_sync(kFull, lane < kWarps ? scan[lane] : 0);
        own = __reduce_add_sync(kFull, lane < kWarps ? scan[32 + lane] : 0);
        own_rows = __reduce_add_sync(kFull, lane < kWarps ? scan[96 + lane] : 0);
    }
    // Groups of more rows than there are overlap. Their steps could pass 32 bits, and the walk
    // below the plan's end: nothing is shared then, and the merge flags it. (By way of shared
    // memory: held in a register it costs the coded kernels spills.)
    if (tid == 0) scan[24] = own_rows >> 13 > a.B;
    own_rows &= kMaxBatch;
    const int P = max(1, prefix_sms(a.split, U, own * a.K, own_rows * a.K) * C::kCtasPerSm);
    const int R = max((U + P - 1) / P, a.split.min_steps);
    const int u_lo = (int)min((long long)U, (long long)j * R), u_hi = (int)min((long long)U, (long long)(j + 1) * R);
    if (j == 0 && tid == 0) {
        a.hdr[0] = R;
        a.hdr[1] = scan[24] ? 0 : U;
        a.hdr[2] = C::kCtaRows;
    }
    int carry = 0;
    for (int base = 0; base < n_groups; base += C::kThreads) {
        if (base > 0) {
            mine = span_of(base + tid);
            lead = leader_of(mine);
        }
        const int x = units_of(mine, base + tid);
        int y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(kFull, y, o);
            if (lane >= o) y += z;
        }
        if (base > 0) __syncthreads();         // the round before has been read
        if (lane == 31) scan[64 + warp] = y;
        __syncthreads();
        int before = carry;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += scan[64 + i];
            carry += scan[64 + i];
        }
        const int first = before + y - x;
        if (x > 0 && first <= u_lo && u_lo < first + x) {     // the group that the run begins in
            scan[128] = base + tid;
            scan[129] = first;
            scan[130] = mine.first;
            scan[131] = mine.rows;
            scan[132] = mine.blocks;
            scan[133] = lead;
        }
        if (j == 0 && base + tid < n_groups) a.first_unit[base + tid] = lead < 0 ? INT_MIN : first;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, *reinterpret_cast<volatile uint32_t*>(gb + (tslot - sb)), 0);
    if (u_lo >= u_hi || scan[24]) {            // uniform per CTA
        if (warp == 0) tmem_dealloc(tmem, C::kTmemCols);
        return;
    }
    bool ok = true;

    // ---- the CTA's segments: runs of steps [c0, c1) of one (group, kv-head, tile)
    struct Seg {
        GroupSpan span;
        int g, rows, row0, c0, c1;
    };
    struct Walk {
        int group, base, u;
        GroupSpan span;
    };
    Walk walk{scan[128], scan[129], u_lo, GroupSpan{scan[130], scan[131], scan[132]}};
    auto step_seg = [&](Walk& w, Seg& s) -> bool {
        if (w.u >= u_hi) return false;
        for (;;) {
            const Problem p = problem_of(w.span, a.K, a.GT, C::kCtaRows);
            const int rel = w.u - w.base;
            if (rel >= p.units) {              // steps are left, so a group is
                w.base += p.units;
                w.span = group_span(plan, ++w.group, a.max_blocks);
                continue;
            }
            const int pair = rel / p.chunks;
            s.span = w.span;
            s.c0 = rel - pair * p.chunks;
            s.g = pair / p.tiles;
            s.row0 = (pair - s.g * p.tiles) * C::kCtaRows;
            s.rows = p.rows;
            s.c1 = min(p.chunks, s.c0 + (u_hi - w.u));
            w.u += s.c1 - s.c0;
            return true;
        }
    };
    auto next_seg = [&](Seg& s) { return step_seg(walk, s); };
    Seg it;
    bool have = next_seg(it);

    if (kCoded && loader) {
        // ================================================== copy warps of a coded cache: two for K,
        // two for V. Each asks for the codes of two of a step's pages, kRaw steps ahead,
        // widens them into the stage that the tensor cores read, and puts the scales where the
        // softmax warps find them. A missing block lands as zero codes with zero scales.
        constexpr int kRaw = C::kRaw > 0 ? C::kRaw : 1;
        const int cw = warp - (C::kSoftWarps + 2 * kTiles), v = cw >> 1, part = cw & 1;
        const uint32_t raw0 = sb + C::kOffRaw + cw * kRaw * C::kRawStage;
        const __half* gscale = v ? a.v_scale : a.k_scale;
        const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_last();
        auto par_raw = [](int c) { return (uint32_t)(c / kRaw) & 1u; };
        Walk iw = walk;                            // the segment being asked for, and its next step
        Seg is = it;
        bool iss_have = have;
        int iss_c = is.c0, issued = 0;
        const int32_t* table = a.block_tables + (long long)scan[133] * a.max_blocks;
        if (scan[133] < 0) is.span.blocks = 0;
        int win = -(1 << 30), entries = -1;        // lane l: the page of entry win + l, -1: none
        auto issue = [&]() {                       // codes and scales of step `issued`
            const uint64_t pol = is.rows > C::kCtaRows ? again : once;
            const uint32_t dst = raw0 + (issued % kRaw) * C::kRawStage, bar = bar_full(cw, issued);
            const int blk = kChunkBlocks * iss_c;
            if (blk - win >= 32 || blk < win) {
                win = blk;
                entries = -1;
                if (blk + lane < is.span.blocks) {
                    const int p = table[blk + lane];
                    if (p < 0 || p >= a.num_blocks) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                    else entries = p;
                }
            }
            const int sp = __shfl_sync(kFull, entries, (blk - win + lane / 8) & 31);
            fence_proxy_async_smem();              // the stage's codes have been read
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(bar, C::kCodes);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ph = __shfl_sync(kFull, entries, blk - win + 2 * part + i);
                auto coord = [&](int which) { return which == 0 ? 0 : (which == 1 ? is.g : ph); };
                tma_load_4d_elect(dst + i * kBlock * C::kCodeRow, v ? &vmap : &kmap, 0, coord(a.map_perm[0]),
                                  coord(a.map_perm[1]), coord(a.map_perm[2]), bar, pol);
            }
            // lane l: the scales of tokens 2l and 2l + 1 of the step
            cp_async4(dst + C::kCodes + 4 * lane, gscale + ((long long)max(sp, 0) * a.K + is.g) * kBlock + 2 * (lane & 7),
                      sp >= 0 ? 4u : 0u);
            cp_async_arrive(bar);
            ++issued;
            if (++iss_c == is.c1 && (iss_have = step_seg(iw, is))) {
                iss_c = is.c0;
                const int leader = leader_of(is.span);
                table = a.block_tables + (long long)leader * a.max_blocks;
                if (leader < 0) is.span.blocks = 0;
                win = -(1 << 30);
            }
        };
        while (iss_have && issued < kRaw) issue();
        int G = 0;
        while (have && ok) {
            int lift = kLiftNone;
            for (int c = it.c0; c < it.c1 && ok; ++c, ++G) {
                // the codes are here; the stage's last step has been read by both tiles
                bool w = mbar_wait_tries(bar_full(cw, G), par_raw(G));
                if (G >= kS)
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        w = w && mbar_wait_tries(v ? bar_o(t, G - kS) : bar_s(t, G - kS), par4(G - kS));
                ok = __all_sync(kFull, w);
                if (!ok) break;
                const uint32_t src = raw0 + (G % kRaw) * C::kRawStage;
                const uint32_t to = (v ? sV : sK) + stage(G) * C::kKc;
                constexpr int kLanes = D / 16;         // lanes of a row, 16 codes each
                constexpr int kBatch = 4;              // loads of codes on their way together
#pragma unroll 1
                for (int i0 = 0; i0 < 32 * kLanes; i0 += 32 * kBatch) {
                    uint32_t codes[kBatch][4];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int i = i0 + 32 * k + lane, tok = i / kLanes, x = i % kLanes;
                        if constexpr (C::kI4) {
                            const uint2 r = lds64(src + tok * C::kCodeRow + 8 * x);
                            codes[k][0] = r.x; codes[k][1] = r.y;
                        } else {
                            const uint4 r = lds128(src + tok * C::kCodeRow + 16 * x);
                            codes[k][0] = r.x; codes[k][1] = r.y; codes[k][2] = r.z; codes[k][3] = r.w;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int i = i0 + 32 * k + lane, tok = 32 * part + i / kLanes, x = i % kLanes;
                        uint32_t o[8];
                        widen16<C>(codes[k], o);
                        // 16-byte chunks 2x, 2x + 1 of the row, swizzled; the lanes of the second
                        // half begin with the other one, so that both halves' banks differ
                        const int h = x >> 2, ck = 2 * (x & 3);
                        const uint32_t row = v ? to + (tok / kBlock) * C::kVb + h * (kBlock * 128) + (tok % kBlock) * 128
                                               : to + h * (kChunk * 128) + tok * 128;
                        const uint4 c0 = make_uint4(o[0], o[1], o[2], o[3]), c1 = make_uint4(o[4], o[5], o[6], o[7]);
                        const int s7 = tok & 7;
                        sts128(row + (((ck + h) ^ s7) << 4), h ? c1 : c0);
                        sts128(row + (((ck + 1 - h) ^ s7) << 4), h ? c0 : c1);
                    }
                }
                float2 sc = unpack2<false>(lds32(src + C::kCodes + 4 * lane));   // of tokens 2l and 2l + 1
                float* slot = scales + (G & 3) * C::kSlotF + v * kChunk;
                if (v) {
                    float most = fmaxf(sc.x, sc.y);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
                    float factor = 1.f;
                    if (most > power2(7 - lift)) {
                        const int now = 5 - ((int)(__float_as_uint(most) >> 23) - 127);
                        factor = power2(now - lift);
                        lift = now;
                    }
                    const float up = power2(lift);
                    sc.x *= up;
                    sc.y *= up;
                    if (part == 0 && lane == 0) {
                        scales[(G & 3) * C::kSlotF + 2 * kChunk] = factor;
                        scales[(G & 3) * C::kSlotF + 2 * kChunk + 1] = power2(-lift);
                    }
                } else {
                    sc.x *= a.scale_log2;
                    sc.y *= a.scale_log2;
                }
                if (lane / 16 == part) *reinterpret_cast<float2*>(slot + 2 * lane) = sc;
                fence_proxy_async_smem();          // the widened rows visible to the tensor core
                __syncwarp();
                if (lane == 0) mbar_arrive(v ? bar_v(G) : bar_k(G));
                if (iss_have) issue();             // into the stage just read
            }
            if (ok) have = next_seg(it);
        }
        if (!ok && lane == 0) {
            // let this warp's copies land before the shared memory goes
            flag_error(a.err, GQA_DEVERR_TIMEOUT);
            for (int c = max(0, issued - kRaw); c < issued; ++c) mbar_wait_tries(bar_full(cw, c), par_raw(c), kWaitTries / 4);
        }
        cp_async_wait_all();
        __syncwarp();
    } else if (loader) {
        // ================================================== copy warps: K, then V
        // A block that is missing (behind the prefix's last, or an entry that is no page) is
        // asked for at coordinate -1 and lands as zeros.
        const bool k_warp = warp == C::kSoftWarps + 2 * kTiles;
        const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_last();
        int issued = 0, G = 0;
        while (have && ok) {
            const uint64_t pol = it.rows > C::kCtaRows ? again : once;   // other tiles read the same pages
            // the first segment's leader came with the scan
            const int leader = G == 0 ? scan[133] : leader_of(it.span);
            const int32_t* table = a.block_tables + (long long)leader * a.max_blocks;
            if (leader < 0) it.span.blocks = 0;
            int win_base = -(1 << 30), win_phys = -1;
            for (int c = it.c0; c < it.c1 && ok; ++c, ++G) {
                const int v0 = kChunkBlocks * c;
                if (v0 - win_base >= 32 || v0 < win_base) {       // 32 entries: whole chunks
                    win_base = v0;
                    win_phys = -1;
                    if (v0 + lane < it.span.blocks) {
                        const int p = table[v0 + lane];
                        if (p < 0 || p >= a.num_blocks) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                        else win_phys = p;
                    }
                }
                if (G >= kS) {
                    // K(G) once every tile's S(G-kS) has read K(G-kS); V(G) once
                    // every tile's P(G-kS).V(G-kS) has read V(G-kS)
                    bool w = true;
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        w = w && mbar_wait_tries(k_warp ? bar_s(t, G - kS) : bar_o(t, G - kS), par4(G - kS));
                    ok = __all_sync(kFull, w);
                    if (!ok) break;
                }
                const uint32_t bar = k_warp ? bar_k(G) : bar_v(G);
                if (lane == 0) mbar_arrive_expect_tx(bar, C::kVc);
                __syncwarp();
                // K: a box per (block, 64-element half); V: one per page (head_dim 128: the page
                // map lands it as [half][slot][128 B]). One elected lane issues them with operands
                // that are the warp's: from a lane's own registers a box takes 180 cycles.
#pragma unroll
                for (int q = 0; q < kChunkBlocks; ++q) {
                    const int pq = __shfl_sync(kFull, win_phys, v0 - win_base + q);
                    auto coord = [&](int which) { return which == 0 ? 0 : (which == 1 ? it.g : pq); };
                    const int y = coord(a.map_perm[0]), z = coord(a.map_perm[1]), w = coord(a.map_perm[2]);
                    if (k_warp) {
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            tma_load_4d_elect(sK + stage(G) * C::kKc + h * (kChunk * 128) + q * (kBlock * 128), &kmap, h * 64,
                                              y, z, w, bar, pol);
                    } else {
                        const uint32_t dst = sV + stage(G) * C::kVc + q * C::kVb;
                        if constexpr (C::kHalves == 2)
                            tma_load_5d_elect(dst, &vmap, 0, 0, 0, coord(a.page_perm[0]), coord(a.page_perm[1]), bar, pol);
                        else
                            tma_load_4d_elect(dst, &vmap, 0, y, z, w, bar, pol);
                    }
                }
                ++issued;
            }
            have = next_seg(it);
        }
        if (!ok && lane == 0) {
            // let this CTA's copies land before the shared memory goes
            flag_error(a.err, GQA_DEVERR_TIMEOUT);
            for (int c = max(0, issued - kS); c < issued; ++c)
                mbar_wait_tries(k_warp ? bar_k(c) : bar_v(c), par_st(c), kWaitTries / 4);
        }
    } else if (mma_warp) {
        // ================================================== MMA warps: two per tile, one for S and
        // one for P.V, so that neither waits in the other's place (a step of 1790 cycles; of
        // 1817 with one warp for both). A whole warp walks along and one elected lane issues:
        // from a branch of one lane the operands go through vector registers, 144 cycles a
        // P.V product for 38.
        const int t = (warp - C::kSoftWarps) >> 1;
        const bool s_warp = ((warp - C::kSoftWarps) & 1) == 0;
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(kFull, mbar_wait_tries(bar, parity)); };
        int G = 0, qi = 0;                         // commits issued, segments
        while (have && ok) {
            // a tile past the group's rows takes part in the barriers alone
            const bool live = it.row0 + kRows * t < it.rows;
            const int n = it.c1 - it.c0;
            if (s_warp) {
                ok = wait(bar_q(t), (uint32_t)qi & 1u);           // Q_t of this segment stored
                ++qi;
                for (int c = 0; c < n && ok; ++c, ++G) {
                    // K(G) landed; P_t(G-2), which S_t(G) overwrites, read by its product
                    ok = wait(bar_k(G), par_st(G)) && (G < 2 || wait(bar_o(t, G - 2), par4(G - 2)));
                    tc_fence_after();
                    if (!ok) break;
                    if (live) {                    // S_t(G) = Q_t K(G)^T into buffer G & 1
                        const uint32_t kb = sK + stage(G) * C::kKc, qb = sQ + t * C::kQt;
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint64_t ad = smem_desc_sw128(qb + (ks >> 2) * (kRows * 128) + (ks & 3) * 32, 16, 1024);
                            const uint64_t bd = smem_desc_sw128(kb + (ks >> 2) * (kChunk * 128) + (ks & 3) * 32, 16, 1024);
                            tc_mma_f16_elect(tmem + kColTile * t + kChunk * (G & 1), ad, bd, kIdescS, ks > 0);
                        }
                    }
                    tc_commit_elect(bar_s(t, G));
                }
            } else {
                for (int c = 0; c < n && ok; ++c, ++G) {
                    ok = wait(bar_v(G), par_st(G)) && wait(bar_p(t, G), par4(G));   // V(G) landed, P_t(G) over S_t(G)
                    tc_fence_after();
                    if (!ok) break;
                    if (live) {                    // O_t (+)= P_t(G) V(G), high part then low part per block
                        const uint32_t vb = sV + stage(G) * C::kVc, pb = tmem + kColTile * t + kChunk * (G & 1);
#pragma unroll
                        for (int jl = 0; jl < kChunkBlocks; ++jl)
#pragma unroll
                            for (int part = 0; part < 2; ++part)
                                tc_mma_f16_ta_elect(tmem + kColTile * t + kColO, pb + 16 * jl + 8 * part,
                                                    smem_desc_sw128(vb + jl * C::kVb, kBlock * 128, 1024), kIdescO,
                                                    !(c == 0 && jl == 0 && part == 0));
                    }
                    tc_commit_elect(bar_o(t, G));
                }
            }
            if (ok) have = next_seg(it);
        }
        if (!ok) {
            // let this warp's MMAs land before the tensor memory goes, each barrier's events
            // in order
            if (lane == 0) flag_error(a.err, GQA_DEVERR_TIMEOUT);
            for (int k = max(0, G - kBufs); k < G; ++k) mbar_wait_tries(s_warp ? bar_s(t, k) : bar_o(t, k), par4(k), kWaitTries / 4);
        }
        __syncwarp();
    } else {
        // ================================================== softmax warps: two threads per row
        const int quad = warp & 3;                 // the tile's rows 32 quad .. +31, one a lane
        const int row_t = 32 * quad + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16) + kColTile * tt;
        const uint32_t t_o = t_lane + kColO + hf * (D / 2);
        const uint32_t qt = sQ + tt * C::kQt;
        float* ex = reinterpret_cast<float*>(gb + C::kOffEx) + tt * 2 * kRows;
        const int pair_bar = 1 + 4 * tt + quad;    // the two warps that hold the same rows
        // A warp whose wait ran out says so at the pair's next vote (of step c, or behind the
        // last one), so that its partner leaves with it: a word for odd and one for even steps,
        // as the other may still read the last.
        auto gone = [&](int c) -> volatile int& { return scan[168 + 2 * (4 * tt + quad) + (c & 1)]; };
        auto give_up = [&](int c) {
            if (lane == 0) gone(c) = 1;
            __syncwarp();
            pair_any(pair_bar, true);
            pair_sync(pair_bar);
        };
        auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(kFull, mbar_wait_tries(bar, parity)); };
        // This warp's 16 Q rows of segment x into its tile's swizzled K-major layout by
        // cp.async (16 bytes a lane; rows past the group's are zero-filled), then "Q_t
        // stored" once they have landed. All of their places are looked up first.
        auto load_q = [&](const Seg& x) {
            constexpr int kLanesPerRow = D / 8, kRowsPerStep = 32 / kLanesPerRow, kSteps = 16 / kRowsPerStep;
            const int c16 = lane % kLanesPerRow;
            const int rl0 = 16 * (warp & 7) + lane / kLanesPerRow;
            const int rq0 = x.row0 + kRows * tt + rl0;
            int src[kSteps];                       // rows of q
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int rq = rq0 + i * kRowsPerStep;
                const int member = rq / a.GT, w = rq - member * a.GT, tok = w / a.G;
                const int b = rq < x.rows ? plan.rows[x.span.first + member] : -1;
                src[i] = b >= 0 && b < a.B ? (b * a.T + tok) * a.H + x.g * a.G + (w - tok * a.G) : -1;
            }
            if constexpr (kCoded) {                // q as fp16
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int rl = rl0 + i * kRowsPerStep;
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (src[i] >= 0) {
                        x = dec::ldg128(static_cast<const uint16_t*>(a.q) + (long long)src[i] * D + 8 * c16);
                        if (a.q_dtype == GQA_DTYPE_BF16) {
                            x.x = dec::bf16x2_to_f16x2(x.x);
                            x.y = dec::bf16x2_to_f16x2(x.y);
                            x.z = dec::bf16x2_to_f16x2(x.z);
                            x.w = dec::bf16x2_to_f16x2(x.w);
                        }
                    }
                    sts128(qt + (c16 >> 3) * (kRows * 128) + rl * 128 + (((c16 & 7) ^ (rl & 7)) << 4), x);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const int rl = rl0 + i * kRowsPerStep;
                    cp_async16(qt + (c16 >> 3) * (kRows * 128) + rl * 128 + (((c16 & 7) ^ (rl & 7)) << 4),
                               static_cast<const uint16_t*>(a.q) + (long long)max(src[i], 0) * D + 8 * c16,
                               src[i] >= 0 ? 16u : 0u);
                }
            }
        };
        auto q_stored = [&]() {
            cp_async_wait_all();
            fence_proxy_async_smem();          // Q visible to the tensor core
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q(tt));
        };
        if (have) {
            load_q(it);
            q_stored();
        }
        int gc = 0;
        while (have) {
            const int n = it.c1 - it.c0;
            const bool tile_live = it.row0 + kRows * tt < it.rows;
            float m = -INFINITY, l = 0.f;      // the row's maximum, this half's sum
            float unlift = 1.f;                // coded: what takes the lift out of O
            for (int c = 0; c < n; ++c) {
                const int G = gc + c;
                if (!wait(bar_s(tt, G), par4(G))) {        // S_t(G) done
                    if (tile_live) give_up(c);
                    goto gave_up;
                }
                tc_fence_after();
                if (!tile_live) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_p(tt, G));
                    continue;
                }
                const uint32_t t_buf = t_lane + kChunk * (G & 1) + kHalf * hf;
                uint32_t r[kHalf / 16][16];
#pragma unroll
                for (int u = 0; u < kHalf / 16; ++u) tmem_ld16(t_buf + 16 * u, r[u]);
                tmem_wait_ld();
                float scl = a.scale_log2;
                float factor = 1.f;                // coded: of O, where V's lift changes
                const float* slot = scales + (G & 3) * C::kSlotF + kHalf * hf;
                if constexpr (kCoded) {            // scores by K's scales (the softmax scale is in them)
#pragma unroll
                    for (int u = 0; u < kHalf / 16; ++u)
#pragma unroll
                        for (int q = 0; q < 16; q += 4) {
                            const float4 ks = *reinterpret_cast<const float4*>(slot + 16 * u + q);
                            const float2 x = f2_split(f2_mul(
                                f2_make(__uint_as_float(r[u][q]), __uint_as_float(r[u][q + 1])), f2_make(ks.x, ks.y)));
                            const float2 y = f2_split(f2_mul(
                                f2_make(__uint_as_float(r[u][q + 2]), __uint_as_float(r[u][q + 3])), f2_make(ks.z, ks.w)));
                            r[u][q] = __float_as_uint(x.x);
                            r[u][q + 1] = __float_as_uint(x.y);
                            r[u][q + 2] = __float_as_uint(y.x);
                            r[u][q + 3] = __float_as_uint(y.y);
                        }
                    scl = 1.f;
                    if (!wait(bar_v(G), par_st(G))) {      // V's are there as well
                        give_up(c);
                        goto gave_up;
                    }
                    factor = slot[2 * kChunk - kHalf * hf];
                    unlift = slot[2 * kChunk + 1 - kHalf * hf];
                }
                const int blocks = it.span.blocks - kChunkBlocks * (it.c0 + c);   // of this step and after
                if (blocks < kChunkBlocks || !(scl > 0.f)) {      // the prefix's last step; or no positive scale
#pragma unroll
                    for (int u = 0; u < kHalf / 16; ++u) {
                        const bool here = kHalf / kBlock * hf + u < blocks;
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            r[u][q] = __float_as_uint(here ? __uint_as_float(r[u][q]) * scl : -INFINITY);
                    }
                    scl = 1.f;
                }
                float mx;
                {
                    float mx2[kHalf / 16];                        // short chains of 3-input maxima
#pragma unroll
                    for (int u = 0; u < kHalf / 16; ++u) {
                        float v0 = fmaxf(__uint_as_float(r[u][0]), __uint_as_float(r[u][1]));
                        float v1 = fmaxf(__uint_as_float(r[u][2]), __uint_as_float(r[u][3]));
#pragma unroll
                        for (int q = 4; q < 16; q += 4) {
                            v0 = fmax3(v0, __uint_as_float(r[u][q]), __uint_as_float(r[u][q + 1]));
                            v1 = fmax3(v1, __uint_as_float(r[u][q + 2]), __uint_as_float(r[u][q + 3]));
                        }
                        mx2[u] = fmaxf(v0, v1);
                    }
                    mx = fmaxf(mx2[0], mx2[1]) * scl;
                }
                // lazy rescale: keep the stale maximum while the new one stays within 2^slack
                // of it for all rows of the two warps
                if (pair_any(pair_bar, mx > m + kSlackLog2 || factor != 1.f)) {
                    ex[hf * kRows + row_t] = mx;
                    pair_sync(pair_bar);
                    if (gone(c)) goto gave_up;
                    mx = fmaxf(mx, ex[(hf ^ 1) * kRows + row_t]);
                    const bool old_live = m != -INFINITY;
                    const bool resc = mx > m + kSlackLog2;
                    const float alpha = !resc ? 1.f : old_live ? fast_exp2(m - mx) : 0.f;
                    if (resc) m = mx;
                    l *= alpha;
                    if (c > 0 && __any_sync(kFull, (resc && old_live) || factor != 1.f)) {   // O holds earlier steps: scale it
                        // once P_t(G-1).V(G-1) has landed in it, this half its columns
                        if (!wait(bar_o(tt, G - 1), par4(G - 1))) {
                            give_up(c + 1);
                            goto gave_up;
                        }
                        tc_fence_after();
                        const float f = (resc && old_live ? alpha : 1.f) * factor;
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            uint32_t r16[16];
                            tmem_ld16(t_o + 16 * q, r16);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) r16[k] = __float_as_uint(__uint_as_float(r16[k]) * f);
                            tmem_st16(t_o + 16 * q, r16);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.f : kUp - m;   // a row with nothing attended yet: p = 0
                const uint64_t mu2 = f2_make(mu, mu), sc2 = f2_make(scl, scl);
                uint64_t ps2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
                // P over S: a block's 16 tokens to its own columns, 8 high then 8 low ones
#pragma unroll
                for (int u = 0; u < kHalf / 16; ++u) {
                    uint32_t w16[16];
                    float4 vs = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 d = f2_split(
                            f2_fma(f2_make(__uint_as_float(r[u][2 * e]), __uint_as_float(r[u][2 * e + 1])), sc2, mu2));
                        const float x = fast_exp2(d.x), y = fast_exp2(d.y);
                        const uint64_t xy = f2_make(x, y);
                        ps2[e & 1] = f2_add(ps2[e & 1], xy);
                        if constexpr (kCoded) {
                            if (e % 2 == 0) vs = *reinterpret_cast<const float4*>(slot + kChunk + 16 * u + 2 * e);
                            const uint64_t w2 = f2_mul(xy, e % 2 ? f2_make(vs.z, vs.w) : f2_make(vs.x, vs.y));
                            const float2 w = f2_split(w2);
                            split2<false>(w.x, w.y, w2, w16[e], w16[8 + e]);
                        } else {
                            split2<kB>(x, y, xy, w16[e], w16[8 + e]);
                        }
                    }
                    tmem_st16(t_buf + 16 * u, w16);
                }
                tmem_wait_st();
                {
                    const float2 p0 = f2_split(ps2[0]), p1 = f2_split(ps2[1]);
                    l += (p0.x + p1.x) + (p0.y + p1.y);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p(tt, G));
            }
            // every S_t of the segment is done, so Q_t's buffer is free: with the next one's
            // rows in it, its MMA warp may start on it
            Seg nx;
            const bool have_nx = next_seg(nx);
            if (have_nx) {
                load_q(nx);
                q_stored();
            }
            // ---- wait for this tile's last P.V, then leave the row's state: a problem's
            // first piece by its row, a continued one (only a CTA's first can be) by CTA
            const int G_last = gc + n - 1;
            if (!wait(bar_o(tt, G_last), par4(G_last))) {
                if (tile_live) give_up(n);
                goto gave_up;
            }
            tc_fence_after();
            if (tile_live) {
                const int row = it.row0 + kRows * tt + row_t;
                const bool first = it.c0 == 0;
                const long long base = first ? (long long)it.span.first * a.GT * a.K + (long long)it.g * it.rows
                                             : (long long)j * C::kCtaRows - it.row0;
                ex[hf * kRows + row_t] = l;
                // Four neighbouring lanes turn the 16 columns of their four rows around, so that
                // they write 64 bytes of one row after the other.
                const int l4 = lane & 3, row_4 = row - l4;
                float* dst = (first ? a.o_a : a.o_b) + (base + row_4) * D + hf * (D / 2) + 4 * l4;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t x[16];                // quarter k of this lane's row: x[4k ..]
                    tmem_ld16(t_o + 16 * q, x);
                    tmem_wait_ld();
                    if constexpr (kCoded)
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * unlift);
                    // quarter k of lane i goes to lane k as its piece i: exchange by bits
#pragma unroll
                    for (int s = 1; s < 4; s <<= 1) {
                        const bool up = l4 & s;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (k & s) continue;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t& lo = x[4 * k + i];
                                uint32_t& hi = x[4 * (k + s) + i];
                                const uint32_t got = __shfl_xor_sync(kFull, up ? lo : hi, s);
                                if (up) lo = got;
                                else hi = got;
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (row_4 + k < it.rows)
                            *reinterpret_cast<float4*>(dst + k * D + 16 * q) =
                                make_float4(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1]),
                                            __uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3]));
                }
                if (pair_any(pair_bar, false)) {   // the other half's sums are there; or its warp gave up
                    pair_sync(pair_bar);
                    goto gave_up;
                }
                if (hf == 0 && row < it.rows)
                    (first ? a.ml_a : a.ml_b)[base + row] = make_float2(m - kUp, l + ex[kRows + row_t]);
                pair_sync(pair_bar);               // ex has been read
            }
            gc += n;
            it = nx;
            have = have_nx;
        }
        if (false) {
        gave_up:
            if (lane == 0) flag_error(a.err, GQA_DEVERR_TIMEOUT);
        }
        cp_async_wait_all();                   // nothing of this warp's still lands in shared memory
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, C::kTmemCols);
}

// ------------------------------------------------------------------ merge

// Row bh of [B, T, H]: its pieces of the tail (split slots, as dec::combine_kernel finds
// them) and of the prefix (its problem's first piece, then the continued pieces of the
// CTAs after), merged with their log-sum-exp weights. kRowWarps warps share a row, each
// an even share of the pieces. A piece that saw nothing holds m = -inf and o = 0.
template <int D, int kRowWarps, int kCtaRows>
__global__ void __launch_bounds__(kRowWarps * kCtaRows * 32) shared_merge_kernel(const DecodeArgs a, const SharedArgs p) {
    __shared__ float s_m[kCtaRows][kRowWarps], s_l[kCtaRows][kRowWarps];
    __shared__ float s_acc[kRowWarps > 1 ? kCtaRows : 1][kRowWarps > 1 ? kRowWarps : 1][kRowWarps > 1 ? D : 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int sub = warp % kRowWarps;
    const int bh = (int)blockIdx.x * kCtaRows + warp / kRowWarps;   // rows < 2^31 (host-checked)
    launch_dependents();
    const int TH = a.T * a.H;
    const int b = min(bh / TH, a.B - 1), ih = bh - b * TH;
    const int i = ih / a.H, h = ih - i * a.H, g = h / a.G;
    const int rr = i * a.G + (h - g * a.G);                           // row of the pair
    const int rg = a.NRG > 1 ? rr / dec::kHeadsPerWarp : 0;
    const int gv = g * a.NRG + rg, hh = rr - rg * dec::kHeadsPerWarp;
    const long long orow = (long long)bh * D;
    // What the earlier kernels read too needs no wait for them where their word is seen; where
    // it is not, CTA 0 has cleared it already and the wait is over at once.
    const bool begun = load_acquire(a.ws_hdr + kWsBegun) != 0;
    if (!begun) grid_dependency_wait();
    const SharedRow sr = shared_row(PrefixGroups(p.groups, a.B), a.context_lens, b, a.T, a.max_blocks);
    if (begun) grid_dependency_wait();         // the tail kernel, which ends after the prefix kernel
    if (blockIdx.x == 0 && tid == 0) {
        *a.ws_ctr = 0ull;
        a.ws_hdr[kWsBegun] = 0;
    }
    if (bh >= a.B * TH) return;                // uniform per warp, and per CTA where warps share a row
    const int p0 = a.ws_pref[b], nb = a.ws_pref[b + 1] - p0;
    const int R = p.hdr[0], U = p.hdr[1], cta_rows = p.hdr[2], unit0 = p.first_unit[sr.group];
    Partition pt;
    pt.R = a.ws_hdr[0];
    pt.U = a.ws_hdr[1];
    pt.Rs = a.ws_hdr[2];
    pt.Cz = a.ws_hdr[3];
    pt.P = a.ws_hdr[4];
    pt.cpw = a.ws_hdr[5];

    // the tail's pieces, then the prefix's
    long long first = 0;
    int n1 = 0;
    if (nb > 0) {
        const int u0 = a.Kv * p0 + gv * nb, s0 = pt.segment_of(u0);
        n1 = pt.segment_of(u0 + nb - 1) - s0 + 1;
        first = (long long)b * a.Kv + gv + s0;
    }
    int n2 = 0, j0 = 0, in_tile = 0;
    bool astray = false;
    long long row_a = 0;
    if (sr.blocks > 0) {
        const Problem pr = problem_of(sr.span, a.K, a.GT, cta_rows);
        const int row = sr.member * a.GT + rr, tile = row / cta_rows;
        in_tile = row - tile * cta_rows;
        row_a = (long long)sr.span.first * a.GT * a.K + (long long)g * pr.rows + row;
        const int u0 = unit0 + (g * pr.tiles + tile) * pr.chunks;
        j0 = u0 / R;
        n2 = (u0 + pr.chunks - 1) / R - j0 + 1;
        astray = u0 < 0 || pr.chunks > U - u0; // a first row outside the batch; overlapping groups: no steps
        if (astray) n2 = 0;
    }
    if (astray && lane == 0) flag_error(a.err, GQA_DEVERR_ROW);      // (in the branch it costs the merge 1 us)
    const int n = n1 + n2;
    auto piece_ml = [&](int x) -> const float2* {
        if (x < n1) return a.ws_ml + (first + x) * a.RS + hh;
        return x == n1 ? p.ml_a + row_a : p.ml_b + (long long)(j0 + x - n1) * cta_rows + in_tile;
    };
    auto piece_o = [&](int x) -> const float* {
        if (x < n1) return a.ws_o + ((first + x) * a.RS + hh) * D;
        return x == n1 ? p.o_a + row_a * D : p.o_b + ((long long)(j0 + x - n1) * cta_rows + in_tile) * D;
    };
    // Each warp an even share, four pieces at a time: their outputs and, lane x, piece x's
    // (m, l), all on the way before the first is used.
    const int per = (n + kRowWarps - 1) / kRowWarps;
    const int lo = min(n, sub * per), hi = min(n, lo + per);
    const bool has_dims = 4 * lane < D;
    float Mw = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = lo; base < hi; base += 4) {
        const int cnt = min(4, hi - base);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < cnt) ml = __ldcg(piece_ml(base + lane));
        float4 o[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (x < cnt && has_dims) o[x] = __ldcg(reinterpret_cast<const float4*>(piece_o(base + x) + 4 * lane));
        float mc = ml.x;
#pragma unroll
        for (int s = 2; s > 0; s >>= 1) mc = fmaxf(mc, __shfl_xor_sync(kFull, mc, s));
        const float Mn = fmaxf(Mw, __shfl_sync(kFull, mc, 0));
        if (Mn == -INFINITY) {                 // warp-uniform: nothing seen yet, or NaN alone
            L += ml.y;
            continue;
        }
        const float sc = fast_exp2(Mw - Mn);   // 0 while Mw = -inf, 1 if unchanged
        acc.x *= sc; acc.y *= sc; acc.z *= sc; acc.w *= sc;
        L *= sc;
        Mw = Mn;
        const float e = fast_exp2(ml.x - Mw);
        L += ml.y * e;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float ex = __shfl_sync(kFull, e, x);
            if (x < cnt && has_dims) {
                acc.x += o[x].x * ex; acc.y += o[x].y * ex; acc.z += o[x].z * ex; acc.w += o[x].w * ex;
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(kFull, L, o);
    if constexpr (kRowWarps > 1) {
        const int rw = warp / kRowWarps;
        if (has_dims) *reinterpret_cast<float4*>(&s_acc[rw][sub][4 * lane]) = acc;
        if (lane == 0) {
            s_m[rw][sub] = Mw;
            s_l[rw][sub] = L;
        }
        // the row's warps alone: rows of a CTA may have left
        asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(1 + rw), "r"(32 * kRowWarps) : "memory");
        float M = s_m[rw][0];
#pragma unroll
        for (int w = 1; w < kRowWarps; ++w) M = fmaxf(M, s_m[rw][w]);
        auto share = [&](int w) { return s_m[rw][w] == -INFINITY ? 0.f : fast_exp2(s_m[rw][w] - M); };   // (0 NaN is NaN)
        float Lt = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) Lt += s_l[rw][w] * share(w);
        const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
        for (int x = tid % (32 * kRowWarps); x < D; x += 32 * kRowWarps) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) v += s_acc[rw][w][x] * share(w);
            dec::store1(a.out, a.out_dtype, orow + x, v * inv);
        }
    } else if (has_dims) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        dec::store1(a.out, a.out_dtype, orow + 4 * lane + 0, acc.x * inv);
        dec::store1(a.out, a.out_dtype, orow + 4 * lane + 1, acc.y * inv);
        dec::store1(a.out, a.out_dtype, orow + 4 * lane + 2, acc.z * inv);
        dec::store1(a.out, a.out_dtype, orow + 4 * lane + 3, acc.w * inv);
    }
}

// ------------------------------------------------------------------ host side

// One form of the prefix kernel.
struct Form {
    const void* fn;
    int threads, smem, ctas_per_sm, rows;
    int code_row;                                    // bytes of a row of codes
};

template <typename T, int kTiles, int D>
Form form() {
    using C = SharedCfg<T, kTiles, D>;
    return Form{reinterpret_cast<const void*>(&shared_prefix_kernel<T, kTiles, D>), C::kThreads, C::kSmem, C::kCtasPerSm,
                C::kCtaRows, C::kCodeRow};
}

template <typename T>
Form pick_tiles(int d, bool two) {
    if (d == 64) return two ? form<T, 2, 64>() : form<T, 1, 64>();
    return two ? form<T, 2, 128>() : form<T, 1, 128>();
}
template <typename T>
Form pick_coded(int d) {
    return d == 64 ? form<T, 2, 64>() : form<T, 2, 128>();
}

// The form: two tiles a CTA where a group has more than 128 query rows, else one, twice an SM.
// K=8, behind 32768 tokens, one tile | two: d=128 with 32 rows 37 | 43 us, 128 rows 43 | 47 (a
// second tile that is empty), 136 rows 61 | 52, 256 rows 69 | 57; d=64 with 32 rows 31 | 37, 128
// rows 38 | 39, 136 rows 48 | 45, 256 rows 62 | 47. Behind 2048 tokens they differ by 2 us
// (d=64, 256 rows: 29 | 25). Coded caches have two tiles alone: their copy warps need the SM's
// issue slots that a second CTA would take.
bool pick_form(const DecodeLaunch& L, Form& f) {
    const int GT = L.num_heads / L.cache->num_kv_heads * L.tokens_per_seq, d = L.cache->head_dim;
    const long long rows = (long long)std::min(L.shared->max_group > 0 ? L.shared->max_group : L.batch, L.batch) * GT;
    const bool two = rows > kRows;
    switch (L.cache->dtype) {
        case GQA_DTYPE_F16: f = pick_tiles<__half>(d, two); return true;
        case GQA_DTYPE_BF16: f = pick_tiles<__nv_bfloat16>(d, two); return true;
        case GQA_DTYPE_I8: f = pick_coded<int8_t>(d); return true;
        case GQA_DTYPE_FP8_E4M3: f = pick_coded<__nv_fp8_e4m3>(d); return true;
        case GQA_DTYPE_I4: f = pick_coded<int4x2>(d); return true;
        default: return false;
    }
}

template <int D>
const void* pick_merge(int warps) {
    switch (warps) {
        case 1: return reinterpret_cast<const void*>(&shared_merge_kernel<D, 1, 8>);
        case 2: return reinterpret_cast<const void*>(&shared_merge_kernel<D, 2, 4>);
        case 4: return reinterpret_cast<const void*>(&shared_merge_kernel<D, 4, 2>);
        case 8: return reinterpret_cast<const void*>(&shared_merge_kernel<D, 8, 1>);
        case 16: return reinterpret_cast<const void*>(&shared_merge_kernel<D, 16, 1>);
        default: return reinterpret_cast<const void*>(&shared_merge_kernel<D, 32, 1>);
    }
}

constexpr int kMaxCtaRows = 2 * kRows;               // rows a CTA holds times its CTAs per SM, in every form

struct PrefixWs {
    size_t first_unit, ml_a, ml_b, o_a, o_b, total;
};
PrefixWs prefix_ws(long long batch, long long rows, int d, int sms) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const long long b_rows = (long long)sms * kMaxCtaRows;
    PrefixWs w;
    w.first_unit = 256;                              // behind the header
    w.ml_a = w.first_unit + up((size_t)batch * 4);
    w.ml_b = w.ml_a + up((size_t)rows * 8);
    w.o_a = w.ml_b + up((size_t)b_rows * 8);
    w.o_b = w.o_a + up((size_t)rows * d * 4);
    w.total = w.o_b + up((size_t)b_rows * d * 4);
    return w;
}

// The times behind the GPU's division, in us of an SM, each from the difference of two lengths:
// a step of the prefix kernel; a (block, kv-head) and a (row, kv-head) of the rows' own, the
// latter most of it for rows that have just begun (17 rows of up to 2 blocks behind 32768
// tokens take 53 us where they count as blocks alone 82). By the split-KV kernel's warps per
// pair, 1 for up to 8 query rows; on the CUDA cores (codes at head_dim 64) by its rows. Rows
// take half as long again beside the prefix kernel, and so does a block of 9 to 16 rows at
// head_dim 64 by a quarter (12 query rows over bf16, d=64, 41 us, where it does not 44; 1 query
// row over int8, d=64, whose rows count a block besides, 39, where they do not 45). 125 rows of 50 blocks of int4 codes, d=64: 110 us, where a block
// counts 1.6 whatever the rows 296; over 28 batches of every type, steps or blocks that count a
// tenth more cost up to 2%. Rounding the prefix's time to whole steps of a CTA costs its two
// divisions, 1 us, and no batch gained that. The times pick how the SMs are dealt out and
// change no result.
SplitModel split_of(const DecodeLaunch& L, const Form& f, int sms) {
    const gqa_kv_cache_t& c = *L.cache;
    const int GT = L.num_heads / c.num_kv_heads * L.tokens_per_seq;
    const bool coded = dtype_coded(c.dtype), wide = c.head_dim == 128;
    const int w = GT <= 8 ? 0 : GT <= 16 ? 1 : GT <= 32 ? 2 : 3;
    static const float kUnit[4][4] = {{0.178f, 0.178f, 0.42f, 0.82f},      // 16-bit, d = 128
                                      {0.1f, 0.16f, 0.31f, 0.59f},      // d = 64
                                      {0.133f, 0.218f, 0.465f, 0.98f},     // 8-bit codes
                                      {0.122f, 0.206f, 0.425f, 0.9f}};     // 4-bit
    static const float kPair[3][4] = {{0.2f, 0.47f, 1.1f, 2.25f}, {0.12f, 0.28f, 0.68f, 1.35f}, {0.75f, 1.35f, 2.7f, 5.4f}};
    SplitModel m;
    m.sms = sms;
    m.ctas_per_sm = f.ctas_per_sm;
    m.cta_rows = f.rows;
    m.min_steps = 2;
    m.prefix_us = 9.f;
    m.tail_us = 4.f;
    if (coded) {
        m.step_us = wide ? 1.5f : 1.3f;
        m.unit_us = kUnit[dtype_bits(c.dtype) == 8 ? 2 : 3][w];
        m.pair_us = kPair[2][w];
        if (!wide) {
            m.unit_us = (GT + 7) / 8 * (0.16f + 0.177f * std::min(GT, 8));
            m.pair_us = (GT + 7) / 8 * 0.5f + m.unit_us;
        }
    } else {
        m.step_us = f.rows > kRows ? (wide ? 1.f : 0.8f) : (wide ? 1.4f : 1.f);
        m.unit_us = kUnit[wide ? 0 : 1][w];
        m.pair_us = kPair[wide ? 0 : 1][w];
    }
    return m;
}

SharedArgs make_args(const DecodeLaunch& L, const Form& f, uint8_t* ws, int sms) {
    const gqa_kv_cache_t& c = *L.cache;
    const PrefixWs w = prefix_ws(L.batch, (long long)L.batch * L.tokens_per_seq * L.num_heads, c.head_dim, sms);
    SharedArgs a = {};
    a.q = L.q;
    a.q_dtype = L.q_dtype;
    a.k_scale = static_cast<const __half*>(c.k_scale);
    a.v_scale = static_cast<const __half*>(c.v_scale);
    a.groups = L.shared->groups;
    a.block_tables = L.block_tables;
    a.context_lens = L.context_lens;
    a.err = L.err;
    a.num_blocks = c.num_blocks;
    a.B = L.batch;
    a.H = L.num_heads;
    a.K = c.num_kv_heads;
    a.G = L.num_heads / c.num_kv_heads;
    a.T = L.tokens_per_seq;
    a.GT = a.G * a.T;
    a.max_blocks = L.max_blocks;
    a.scale_log2 = L.scale * dec::kLog2e;
    a.split = split_of(L, f, sms);
    a.begun = static_cast<int32_t*>(L.workspace) + kWsBegun;
    a.hdr = reinterpret_cast<int32_t*>(ws);
    a.first_unit = reinterpret_cast<int32_t*>(ws + w.first_unit);
    a.ml_a = reinterpret_cast<float2*>(ws + w.ml_a);
    a.ml_b = reinterpret_cast<float2*>(ws + w.ml_b);
    a.o_a = reinterpret_cast<float*>(ws + w.o_a);
    a.o_b = reinterpret_cast<float*>(ws + w.o_b);
    return a;
}

int launch_pdl(const void* fn, unsigned grid, int threads, int smem, cudaStream_t stream, void** args, int cluster = 1) {
    cudaLaunchAttribute pdl[2];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    pdl[1].id = cudaLaunchAttributeClusterDimension;
    pdl[1].val.clusterDim.x = cluster;
    pdl[1].val.clusterDim.y = pdl[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

bool dec::split_model(const DecodeLaunch& L, int num_sms, SplitModel& m) {
    Form f;
    if (!pick_form(L, f)) return false;
    m = split_of(L, f, num_sms);
    return true;
}

bool shared_prefix_supported(int dtype) { return dtype != GQA_DTYPE_F32 && dtype != GQA_DTYPE_I4_KC; }

size_t shared_prefix_bytes(int batch, int num_heads, int head_dim, int tokens_per_seq, int num_sms) {
    return prefix_ws(batch, (long long)batch * std::max(1, tokens_per_seq) * num_heads, head_dim, num_sms).total;
}

int launch_shared_prefix(const DecodeLaunch& L, uint8_t* ws, int num_sms) {
    const gqa_kv_cache_t& c = *L.cache;
    Form f;
    if (!pick_form(L, f)) return GQA_ERR_UNSUPPORTED;
    SharedArgs a = make_args(L, f, ws, num_sms);
    CUtensorMap kmap, vmap;
    const bool coded = dtype_coded(c.dtype);          // whole rows of codes, as they lie
    const int inner = coded ? f.code_row : 64, swizzle = coded ? 0 : 128;
    if (!encode_cache_map(&kmap, c, c.k, inner, swizzle, a.map_perm) ||
        !encode_cache_map(&vmap, c, c.v, inner, swizzle, a.map_perm))
        return GQA_ERR_UNSUPPORTED;
    if (!coded && c.head_dim == 128 && !encode_page_map(&vmap, c, c.v, a.page_perm)) return GQA_ERR_UNSUPPORTED;   // V a page per box
    if (ctas_per_sm(f.fn, f.threads, f.smem) < 1) return GQA_ERR_CUDA;
    void* args[] = {&kmap, &vmap, &a};
    // Clusters of two CTAs, which land on the two SMs of a pair: a pair then works for one
    // kernel. Over int8 caches an SM whose neighbour runs the tail kernel takes 92 us where
    // one beside its like takes 77 (16-bit caches: no difference).
    return launch_pdl(f.fn, (unsigned)(num_sms * f.ctas_per_sm), f.threads, f.smem, L.stream, args, num_sms % 2 ? 1 : 2);
}

int dec::launch_shared_merge(const DecodeArgs& tail, const DecodeLaunch& L, uint8_t* ws, int num_sms) {
    Form f;
    if (!pick_form(L, f)) return GQA_ERR_UNSUPPORTED;
    SharedArgs p = make_args(L, f, ws, num_sms);
    DecodeArgs a = tail;
    // Warps per row from the expected pieces: about 1.5 workers' worth of the tail's
    // segments per pair, and the prefix kernel's CTAs over the groups' problems.
    const long long group = std::min(L.shared->max_group > 0 ? L.shared->max_group : L.batch, L.batch);
    const long long problems = (group * a.GT + f.rows - 1) / f.rows * a.K * (L.batch / group);
    const long long est = (3LL * a.P) / (2LL * a.B * a.Kv) + 1 + num_sms * f.ctas_per_sm / problems + 1;
    // As many warps per row as all rows together have room for at once (64 registers a
    // thread: 32 warps an SM) and as there are pieces: a second wave costs what the first
    // does, 4 us.
    const long long all = (long long)L.batch * a.T * a.H;
    int warps = 32;
    while (warps > 1 && (warps > est || all * warps > 32LL * num_sms)) warps >>= 1;
    const bool d64 = L.cache->head_dim == 64;
    const void* fn = d64 ? pick_merge<64>(warps) : pick_merge<128>(warps);
    const int per_cta = std::max(1, 8 / warps);
    void* args[] = {&a, &p};
    return launch_pdl(fn, (unsigned)((all + per_cta - 1) / per_cta), per_cta * warps * 32, 0, L.stream, args);
}

}  // namespace gqa
