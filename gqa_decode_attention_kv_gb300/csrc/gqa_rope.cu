// gqa_rope.cu -- what a new token's projections go through before attention,
// in one pass: the norm of every query and key head, the rotation by the
// token's position, and the write of K and V into their paged cache slots.
//
// For a head row x of d elements (q and k; v goes to the cache as it is):
//   y = x / sqrt(mean(x^2) + eps) * w                       (skipped without w)
//   (a, b) -> (a cos - b sin, b cos + a sin)                for the pairs of the
//   first rotary_dim elements: (i, i + rotary_dim/2), or (2i, 2i+1) interleaved;
//   cos and sin come from row `position` of an fp32 table.
// Everything is held in fp32 and rounded once, into q_out or the cache; a coded
// cache quantises the fp32 rows by the rules of the append (gqa_append.cu), so V
// gets that call's very codes.
//
// Bound: memory. Per token (H + 2K) d elements are read and written and one
// table row is read; the arithmetic is ~10 flops an element. Layout: a lane
// holds two 8-element chunks of a row, lane l's first ones lying side by side over the
// lanes and its second ones too (adjacent chunks in one lane leave half of every
// sector to another instruction: 94 against 70 us where 16384 tokens are only moved).
// For split pairs the second chunk holds the first one's partners, so both elements of
// every pair are in one lane; the norm takes log2(d/16) shuffles; a warp step covers
// 512/d rows. A warp serves one part of a token (kRopeSteps query steps, or kKvSteps
// steps of K and of V) for a run of consecutive tokens, so the sequence is looked up
// once a run. The rows, the table
// row and the page entry of the next tokens are in flight while one is worked on:
// each lane copies the row pieces that it will read itself into a ring of stages
// with cp.async (the table row and the page entry once for the warp), which needs no
// registers for data in flight and no barrier.
#include <algorithm>
#include <type_traits>

#include "gqa_device.cuh"
#include "gqa_internal.h"

namespace gqa {

int device_sms(int device);   // gqa_capi.cu

namespace {

constexpr int kRopeWarps = 4;     // warps per CTA
constexpr int kRopeSteps = 4;     // query row steps one warp holds
constexpr int kMost = 4;          // steps a stage holds

// Where K (and V) rows go.
enum KvOut : int { kOutDense = 0, kOutCache = 1, kOutI8 = 2, kOutFp8 = 3, kOutI4 = 4 };

// K steps (and as many V steps) one warp holds
constexpr int kv_steps(int out) { return out > kOutCache ? 1 : 2; }
static_assert(kRopeSteps <= kMost && 2 * kv_steps(0) <= kMost, "a stage holds a part");

struct RopeArgs {
    const void* q;
    const void* k;
    const void* v;
    long long q_stride, k_stride, v_stride;   // elements between tokens
    const void* q_weight;
    const void* k_weight;
    int weight_dtype;
    float eps;
    const float2* rope;                       // [rope_rows][rotary_dim / 2] (cos, sin)
    int rope_rows, rotary_dim, interleaved;
    const int32_t* rope_positions;            // NULL: the cache position
    void* q_out;                              // [tokens, H, d]
    void* k_out;                              // kOutDense: [tokens, K, d]
    // cache destination
    void* k_cache;
    void* v_cache;
    __half* k_scale;
    __half* v_scale;
    const int32_t* block_tables;
    const int32_t* positions;
    const int32_t* token_start;               // NULL: token = b * T + i
    long long num_blocks, sb, sh, st;
    int batch, T, max_blocks;
    int32_t* err;
    long long tokens;
    int H, K, q_parts, parts;                 // warps per token: q_parts, then K/V parts
    int runs, run, longer;                    // runs of `run` consecutive tokens, the first `longer` of one more
};

// Stages of a warp's ring, and their layout: the rows of kMost steps in 16-byte
// slots of 32 lanes, then the table row (64 bytes a lane of a row), then the page
// entry. Two stages, so that four CTAs share an SM: the kernel waits on its own
// instruction latencies more than on memory (in one wave of 16384 tokens three stages and
// three CTAs took 81 us, these 67).
template <typename T>
struct RopeCfg {
    static constexpr int kPieces = sizeof(T) / 2;                 // 16-byte pieces per chunk
    static constexpr int kRowSlots = kMost * 2 * kPieces;
    static constexpr int kTable = kRowSlots * 512, kEntry = kTable + 512;
    static constexpr int kStage = kEntry + 16;
    static constexpr int kStages = 2;
    static constexpr int kSmem = kRopeWarps * kStages * kStage;
};

// Rows a lane works on at a time, CTAs per SM the registers are cut for, and K (and V)
// steps of a warp. Two rows overlap their shuffles and roots and need 128 registers (4
// CTAs); quantised rows go one by one, their compensated arithmetic taking the registers.
// Measured, 16384 tokens of 32 + 8 bf16 heads, d = 128, one row at 5 / two at 4 / two at
// 5 CTAs: 69.3 / 67.3 / 70 us; 14.3k tokens of 24 + 8 heads, d = 64, onto an FP8
// cache, one row at 5 / 4 CTAs, two at 4: 47.8 / 27.6 / 38.1 us. A
// quantised step of K and V takes a warp longer than four query steps, so its warp holds
// one: two make it the last to finish (16384 tokens, d = 128, FP8: 86.9 against 68.0 us).
template <typename T, int kOut>
struct RopeShape {
    static constexpr bool kTwo = sizeof(T) == 2 && kOut <= kOutCache;
    static constexpr int kPair = kTwo ? 2 : 1;
    static constexpr int kCtas = sizeof(T) == 4 ? 3 : 4;
    static constexpr int kKvSteps = kv_steps(kOut);
};

template <int kDst, int kSrc>
__device__ __forceinline__ void async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;" ::"r"(dst), "l"(src), "n"(kDst), "n"(kSrc) : "memory");
}
template <int kBegin, int kEnd, class F>
__device__ __forceinline__ void static_for(F&& f) {
    if constexpr (kBegin < kEnd) {
        f(std::integral_constant<int, kBegin>{});
        static_for<kBegin + 1, kEnd>(f);
    }
}
__device__ __forceinline__ void async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Eight elements of a row as loaded.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ void store8r(T* p, const Raw8<T>& r) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = r.w[i];
}
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&x)[8]) {
    const uint4 w = r.w[0];
    if constexpr (sizeof(T) == 4) {
        const uint4 v = r.w[sizeof(T) / 2 - 1];
        const uint32_t u[8] = {w.x, w.y, w.z, w.w, v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<kB>(u[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ Raw8<T> narrow8(const float (&x)[8]) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        r.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        r.w[sizeof(T) / 2 - 1] =
            make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        r.w[0] = make_uint4(pack2<kB>(x[0], x[1]), pack2<kB>(x[2], x[3]), pack2<kB>(x[4], x[5]), pack2<kB>(x[6], x[7]));
    }
    return r;
}

// Sequence b and index i of packed token `tok` among batch sequences that begin at
// token_start[0 .. batch]; false if the token belongs to none, or to one whose
// count is out of [0, T] (flagged). Warp-collective: 32 entries a round.
__device__ __forceinline__ bool sequence_of(const RopeArgs& a, long long tok, int lane, int& b, int& i, int& cnt) {
    int lo = 0, n = a.batch + 1;                   // the last entry <= tok lies in [lo - 1, lo + n - 1]
    while (n > 32) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool below = lane * step < n && (long long)a.token_start[at] <= tok;
        const int hits = __popc(__ballot_sync(kFull, below));
        if (hits == 0) return false;
        lo += (hits - 1) * step;
        n = min(step, n - (hits - 1) * step);
    }
    const bool below = lane < n && (long long)a.token_start[lo + lane] <= tok;
    const int hits = __popc(__ballot_sync(kFull, below));
    b = lo + hits - 1;
    if (b < 0 || b >= a.batch) return false;
    const int t0 = a.token_start[b];
    cnt = a.token_start[b + 1] - t0;
    i = (int)(tok - t0);
    if (cnt < 0 || cnt > a.T) {
        if (lane == 0) flag_error(a.err, GQA_DEVERR_POSITION);
        return false;
    }
    return i < cnt;
}

// The norm of kN rows, each held by kLanes lanes, x <- x / sqrt(mean(x^2) + eps) * w;
// the rows' shuffles and roots go by together, which hides their latency. kExact
// carries what fp32 products round away (the inverse root's low part by one Newton
// step, the products' remainders), to about half a step of fp32: for rows that stay
// fp32 or are quantised next, where a code next to a border, or a scale next to one of
// fp16, then falls where the exact value puts it. Rows rounded to 16 bits do not need
// it, and the kernel is bound by issue as much as by memory (carried everywhere it took
// 16384 tokens from 72 to 95 us). Packed fp32x2 instructions do not pay here: the moves
// that pair the operands made it 913 instructions per warp and token, against 667.
template <bool kExact, int kLanes, int D, int kN>
__device__ __forceinline__ void norm_rows(float (&x0)[kN][8], float (&x1)[kN][8], const float (&w0)[8],
                                          const float (&w1)[8], float eps) {
    float ss[kN];
#pragma unroll
    for (int u = 0; u < kN; ++u) {
        float sa = x0[u][0] * x0[u][0], sb = x1[u][0] * x1[u][0], sc = x0[u][1] * x0[u][1], sd = x1[u][1] * x1[u][1];
#pragma unroll
        for (int e = 2; e < 8; e += 2) {
            sa = fmaf(x0[u][e], x0[u][e], sa);
            sb = fmaf(x1[u][e], x1[u][e], sb);
            sc = fmaf(x0[u][e + 1], x0[u][e + 1], sc);
            sd = fmaf(x1[u][e + 1], x1[u][e + 1], sd);
        }
        ss[u] = (sa + sb) + (sc + sd);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < kN; ++u) ss[u] += __shfl_xor_sync(kFull, ss[u], o);
#pragma unroll
    for (int u = 0; u < kN; ++u) {
        const float m = fmaf(ss[u], 1.f / D, eps);
        if constexpr (kExact) {
            const float r = rsqrtf(m);
            const float mr = m * r, mr_lo = fmaf(m, r, -mr);
            float r_lo = 0.5f * r * (fmaf(-mr, r, 1.f) - mr_lo * r);   // r (1 - m r^2) / 2
            if (!(fabsf(r_lo) < r)) r_lo = 0.f;                        // m = 0 or not finite: r alone
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p0 = x0[u][e] * r, p1 = x1[u][e] * r;
                const float q0 = fmaf(x0[u][e], r_lo, fmaf(x0[u][e], r, -p0));
                const float q1 = fmaf(x1[u][e], r_lo, fmaf(x1[u][e], r, -p1));
                x0[u][e] = fmaf(p0, w0[e], q0 * w0[e]);
                x1[u][e] = fmaf(p1, w1[e], q1 * w1[e]);
            }
        } else {
            const float r = rsqrtf(m);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x0[u][e] = x0[u][e] * r * w0[e];
                x1[u][e] = x1[u][e] * r * w1[e];
            }
        }
    }
}

// (a, b) -> (a cos - b sin, b cos + a sin), kExact with what the products that are
// rounded first lose.
template <bool kExact>
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
    const float bs = b * s, as = a * s;
    float x = fmaf(a, c, -bs), y = fmaf(b, c, as);
    if constexpr (kExact) {
        x -= fmaf(b, s, -bs);
        y += fmaf(a, s, -as);
    }
    a = x;
    b = y;
}

// Codes and scales of kN rows (two 8-element chunks a lane, kLanes lanes a row), by the
// append's rule: s = fp16(min(amax / qmax, 65504)), code = x / s rounded to nearest
// even and clamped. The quotient is the correctly rounded one: with y = RN(1/s), once
// a row, q = RN(x y) and the exact remainder x - q s, RN(q + (x - q s) y) is RN(x / s)
// (Markstein's theorem; s has 11 significant bits, so its mantissa is not all ones,
// and no step leaves fp32's range where the code is not zero), at three instructions
// instead of a division; amax / qmax goes the same way (an infinite amax ends at 65504
// as its quotient would); an infinity and a NaN are their own quotients. The rows' maxima
// and reciprocals go by together, which hides their latency.
template <int kOut, int kLanes, int kN>
__device__ __forceinline__ void quantise_store(const float (&x0)[kN][8], const float (&x1)[kN][8], bool live,
                                               uint8_t* const (&row)[kN], int c0, int c1, __half* const (&scale)[kN],
                                               bool first) {
    constexpr float kQmax = kOut == kOutFp8 ? 448.0f : kOut == kOutI4 ? 7.0f : 127.0f;
    float amax[kN] = {};
#pragma unroll
    for (int u = 0; u < kN; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax[u] = fmaxf(amax[u], fmaxf(fabsf(x0[u][e]), fabsf(x1[u][e])));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < kN; ++u) amax[u] = fmaxf(amax[u], __shfl_xor_sync(kFull, amax[u], o));
    if (!live) return;
    __half sh[kN];
    float sf[kN], y[kN];
#pragma unroll
    for (int u = 0; u < kN; ++u) {
        constexpr float kInv = 1.0f / kQmax;     // RN(1 / qmax), folded by the compiler
        const float s0 = amax[u] * kInv;
        sh[u] = __float2half_rn(fminf(fmaf(fmaf(-s0, kQmax, amax[u]), kInv, s0), 65504.0f));
        sf[u] = __half2float(sh[u]);
        y[u] = __frcp_rn(sf[u]);
    }
#pragma unroll
    for (int u = 0; u < kN; ++u) {
        auto quotient = [&](float x) {
            const float q = x * y[u];
            return fabsf(x) < INFINITY ? fmaf(fmaf(-q, sf[u], x), y[u], q) : x;
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[2] = {0u, 0u};
            if (sf[u] != 0.f) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float t0 = quotient(h ? x1[u][e] : x0[u][e]), t1 = quotient(h ? x1[u][e + 1] : x0[u][e + 1]);
                    if constexpr (kOut == kOutFp8) {
                        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(t0, t1), __NV_SATFINITE, __NV_E4M3);
                        w[e / 4] |= two << (16 * (e / 2 % 2));
                    } else {
                        constexpr int qm = (int)kQmax;
                        const uint32_t a = (uint32_t)max(-qm, min(qm, __float2int_rn(t0)));
                        const uint32_t b = (uint32_t)max(-qm, min(qm, __float2int_rn(t1)));
                        if constexpr (kOut == kOutI4) w[0] |= ((a & 0xFu) | ((b & 0xFu) << 4)) << (4 * e);
                        else w[e / 4] |= ((a & 0xFFu) | ((b & 0xFFu) << 8)) << (16 * (e / 2 % 2));
                    }
                }
            }
            const int c = h ? c1 : c0;
            if constexpr (kOut == kOutI4) *reinterpret_cast<uint32_t*>(row[u] + 4 * c) = w[0];
            else *reinterpret_cast<uint2*>(row[u] + 8 * c) = make_uint2(w[0], w[1]);
        }
        if (first) *scale[u] = sh[u];
    }
}

// Where a token goes: its cache position and table row, or why it goes nowhere.
struct Place {
    int pos, turn;
    bool live;           // false: of no sequence, or without a table row
    bool slot;           // the position is inside the block table
};

template <typename T, int D, int kOut>
__global__ void __launch_bounds__(kRopeWarps * 32, RopeShape<T, kOut>::kCtas) norm_rope_kernel(const RopeArgs a) {
    using C = RopeCfg<T>;
    constexpr int kLanes = D / 16;                 // lanes per row
    constexpr int kRows = 32 / kLanes;             // rows per warp step
    constexpr bool kCached = kOut != kOutDense;
    constexpr bool kCoded = kOut > kOutCache;      // rows are quantised
    constexpr int kKvSteps = RopeShape<T, kOut>::kKvSteps;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = (int)blockIdx.x * kRopeWarps + warp;
    const int part = unit % a.parts;
    const int r = unit / a.parts;                  // run r: a.run tokens, the first a.longer one more
    if (r >= a.runs) return;                       // uniform per warp
    const long long t_lo = (long long)r * a.run + min(r, a.longer);
    const int n = a.run + (r < a.longer ? 1 : 0);
    const int li = lane % kLanes, grp = lane / kLanes;
    const int half = a.rotary_dim / 16;            // lanes of a row that rotate
    // this lane's chunks of a row, and whether they turn: split pairs, l and its partner
    // l + half, then the elements behind them; interleaved ones, l and l + kLanes
    int c0 = li, c1 = li + kLanes;
    bool turns0 = c0 < 2 * half, turns1 = c1 < 2 * half;
    if (!a.interleaved) {
        turns0 = turns1 = li < half;
        if (turns0) c1 = li + half;
        else c0 = li + half;
    }
    const bool is_q = part < a.q_parts;
    // this warp's first row, and its steps: query rows, or K rows and as many V rows
    const int hw = is_q ? part * kRopeSteps * kRows : (part - a.q_parts) * kKvSteps * kRows;
    const int rows = is_q ? min(kRopeSteps * kRows, a.H - hw) : min(kKvSteps * kRows, a.K - hw);
    const int h0 = hw + grp;                       // this lane's row of step 0; of step u: h0 + u kRows
    const uint32_t ring = smem_addr(smem_raw) + warp * (C::kStages * C::kStage);
    const int c01 = 8 * (c1 - c0);                 // elements between the chunks

    // ---- fetch: everything the run's next token needs, into stage s
    const T* src = static_cast<const T*>(is_q ? a.q : a.k) + t_lo * (is_q ? a.q_stride : a.k_stride) + (long long)h0 * D + 8 * c0;
    const T* vsrc = is_q || !kCached ? src : static_cast<const T*>(a.v) + t_lo * a.v_stride + (long long)h0 * D + 8 * c0;
    const long long src_step = is_q ? a.q_stride : a.k_stride;
    int b = 0, left = 0, pos = 0;                  // its sequence, tokens after it in there, its position
    // table row of the run's next token where it is given: loaded a token ahead
    int given = a.rope_positions != nullptr ? a.rope_positions[t_lo] : 0;
    auto fetch = [&](int j, int s) -> Place {
        const long long t = t_lo + j;
        const uint32_t st = ring + s * C::kStage;
        auto rows_in = [&](auto first, auto steps, const T* from) {
            static_for<0, decltype(steps)::value>([&](auto u) {
                constexpr int kSlot = 2 * C::kPieces * (decltype(first)::value + decltype(u)::value) * 512;
                constexpr int kFrom = decltype(u)::value * kRows * D * (int)sizeof(T);
                if (u * kRows + grp < rows) {
                    static_for<0, C::kPieces>([&](auto i) {
                        async16<kSlot + i * 512, kFrom + i * 16>(st + lane * 16, from);
                        async16<kSlot + (C::kPieces + i) * 512, kFrom + i * 16>(st + lane * 16, from + c01);
                    });
                }
            });
        };
        using std::integral_constant;
        if (is_q) {
            rows_in(integral_constant<int, 0>{}, integral_constant<int, kRopeSteps>{}, src);
        } else {
            rows_in(integral_constant<int, 0>{}, integral_constant<int, kKvSteps>{}, src);
            if constexpr (kCached) {
                rows_in(integral_constant<int, kKvSteps>{}, integral_constant<int, kKvSteps>{}, vsrc);
                vsrc += a.v_stride;
            }
        }
        src += src_step;
        Place p{0, 0, true, true};
        if constexpr (kCached) {
            if (left > 0) {                        // the token after the last one, same sequence
                --left;
                ++pos;
            } else {
                int i = 0, cnt = a.T;
                if (a.token_start == nullptr) {
                    b = (int)(t / a.T);
                    i = (int)(t - (long long)b * a.T);
                } else {
                    p.live = sequence_of(a, t, lane, b, i, cnt);
                }
                if (p.live) {
                    left = cnt - i - 1;
                    pos = a.positions[b] + i;
                }
            }
            p.pos = pos;
        }
        p.turn = pos;
        if (p.live && half > 0) {
            if (a.rope_positions != nullptr) p.turn = given;
            if (p.turn < 0 || p.turn >= a.rope_rows) {
                if (lane == 0 && part == 0) flag_error(a.err, GQA_DEVERR_POSITION);
                p.live = false;
            } else if (lane < 4 * half) {          // 16 bytes a lane: the row once for the warp
                async16<C::kTable, 0>(st + lane * 16,
                                      reinterpret_cast<const uint4*>(a.rope + (long long)p.turn * (a.rotary_dim / 2)) + lane);
            }
        }
        if (a.rope_positions != nullptr && j + 1 < n) given = a.rope_positions[t + 1];
        if constexpr (kCached) {
            if (p.live && !is_q) {
                p.slot = pos >= 0 && pos < a.max_blocks * kBlock;
                if (!p.slot) {
                    if (lane == 0 && part == a.q_parts) flag_error(a.err, GQA_DEVERR_POSITION);
                } else if (lane == 0) {
                    async4(st + C::kEntry, a.block_tables + (long long)b * a.max_blocks + pos / kBlock);
                }
            }
        }
        return p;
    };

    // ---- this lane's weights
    const void* wp = is_q ? a.q_weight : a.k_weight;
    float w0[8], w1[8];
    if (wp != nullptr) {
        if (a.weight_dtype == GQA_DTYPE_F32) {
            widen8(load8(static_cast<const float*>(wp) + 8 * c0), w0);
            widen8(load8(static_cast<const float*>(wp) + 8 * c1), w1);
        } else if (a.weight_dtype == GQA_DTYPE_BF16) {
            widen8(load8(static_cast<const __nv_bfloat16*>(wp) + 8 * c0), w0);
            widen8(load8(static_cast<const __nv_bfloat16*>(wp) + 8 * c1), w1);
        } else {
            widen8(load8(static_cast<const __half*>(wp) + 8 * c0), w0);
            widen8(load8(static_cast<const __half*>(wp) + 8 * c1), w1);
        }
    }

    // ---- norm, rotation and store of the run's token j from stage s
    auto finish = [&](const Place& p, int j, int s) {
        if (!p.live) return;                       // uniform per warp
        const long long t = t_lo + j;
        const uint32_t st = ring + s * C::kStage, mine = st + lane * 16;
        float cs[8], sn[8];
        if (turns0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {          // pairs 8 li .., or 4 c0 .. and 4 c1 ..
                if (a.interleaved && e >= 2 && !turns1) break;
                const int at = a.interleaved ? 2 * (e < 2 ? c0 : c1) + e % 2 : 4 * li + e;
                const uint4 f = lds128(st + C::kTable + at * 16);
                cs[2 * e] = __uint_as_float(f.x);
                sn[2 * e] = __uint_as_float(f.y);
                cs[2 * e + 1] = __uint_as_float(f.z);
                sn[2 * e + 1] = __uint_as_float(f.w);
            }
        }
        // row of slot u: raw, and normed and turned
        auto row_of = [&](int u, Raw8<T>& r0, Raw8<T>& r1) {
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {
                r0.w[i] = lds128(mine + (2 * C::kPieces * u + i) * 512);
                r1.w[i] = lds128(mine + (2 * C::kPieces * u + C::kPieces + i) * 512);
            }
        };
        // rows of steps u .. u + kN - 1, normed and turned
        auto turned = [&](auto exact, auto steps, int u0, float (&x0)[decltype(steps)::value][8],
                          float (&x1)[decltype(steps)::value][8]) {
            constexpr bool kExact = decltype(exact)::value;
            constexpr int kN = decltype(steps)::value;
#pragma unroll
            for (int u = 0; u < kN; ++u) {
                Raw8<T> r0, r1;
                row_of(u0 + u, r0, r1);
                widen8(r0, x0[u]);
                widen8(r1, x1[u]);
            }
            if (wp != nullptr) norm_rows<kExact, kLanes, D>(x0, x1, w0, w1, a.eps);
            if (turns0) {
#pragma unroll
                for (int u = 0; u < kN; ++u) {
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) rotate<kExact>(x0[u][2 * e], x0[u][2 * e + 1], cs[e], sn[e]);
                        if (!turns1) continue;
#pragma unroll
                        for (int e = 0; e < 4; ++e) rotate<kExact>(x1[u][2 * e], x1[u][2 * e + 1], cs[4 + e], sn[4 + e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) rotate<kExact>(x0[u][e], x1[u][e], cs[e], sn[e]);
                    }
                }
            }
        };
        constexpr int kPair = RopeShape<T, kOut>::kPair;
        using Pair = std::integral_constant<int, kPair>;
        static_assert(kMost % kPair == 0 && kKvSteps % kPair == 0, "steps come in whole groups");
        if (is_q || kOut == kOutDense) {           // rows of a dense output
            T* out = (is_q ? static_cast<T*>(a.q_out) + t * a.H * D : static_cast<T*>(a.k_out) + t * a.K * D) + h0 * D + 8 * c0;
#pragma unroll
            for (int u = 0; u < kMost; u += kPair) {
                if (u * kRows >= rows) break;      // uniform; a lane without a row works on what its slot holds
                float x0[kPair][8], x1[kPair][8];
                turned(std::integral_constant<bool, sizeof(T) == 4>{}, Pair{}, u, x0, x1);
#pragma unroll
                for (int v = 0; v < kPair; ++v) {
                    if ((u + v) * kRows + grp >= rows) continue;
                    store8r(out + (u + v) * kRows * D, narrow8<T>(x0[v]));
                    store8r(out + (u + v) * kRows * D + c01, narrow8<T>(x1[v]));
                }
            }
            return;
        }
        if constexpr (kCached) {                   // K and V rows of the cache
            if (!p.slot) return;
            const int ph = (int)lds32(st + C::kEntry);
            if (ph < 0 || ph >= a.num_blocks) {
                if (lane == 0 && part == a.q_parts) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                return;
            }
            // element offset of this lane's row of step 0, and of its scale
            long long off = (long long)ph * a.sb + (long long)(p.pos % kBlock) * a.st + (long long)h0 * a.sh;
            long long sidx = ((long long)ph * a.K + h0) * kBlock + p.pos % kBlock;
#pragma unroll
            for (int u = 0; u < kKvSteps; u += kPair) {
                if (u * kRows >= rows) break;
                float x0[kPair][8], x1[kPair][8];
                turned(std::integral_constant<bool, sizeof(T) == 4 || kCoded>{}, Pair{}, u, x0, x1);
#pragma unroll
                for (int v = 0; v < kPair; ++v, off += kRows * a.sh, sidx += kRows * kBlock) {
                    const bool in = (u + v) * kRows + grp < rows;
                    if constexpr (kCoded) {
                        if ((u + v) * kRows >= rows) break;
                        const long long at = kOut == kOutI4 ? off / 2 : off;
                        float y0[2][8], y1[2][8];        // the K row and the V row
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            y0[0][e] = x0[v][e];
                            y1[0][e] = x1[v][e];
                        }
                        Raw8<T> r0, r1;
                        row_of(kKvSteps + u + v, r0, r1);
                        widen8(r0, y0[1]);
                        widen8(r1, y1[1]);
                        uint8_t* const to[2] = {static_cast<uint8_t*>(a.k_cache) + at, static_cast<uint8_t*>(a.v_cache) + at};
                        __half* const scale[2] = {a.k_scale + sidx, a.v_scale + sidx};
                        quantise_store<kOut, kLanes, 2>(y0, y1, in, to, c0, c1, scale, li == 0);
                    } else if (in) {
                        T* ko = static_cast<T*>(a.k_cache) + off + 8 * c0;
                        store8r(ko, narrow8<T>(x0[v]));
                        store8r(ko + c01, narrow8<T>(x1[v]));
                        Raw8<T> r0, r1;
                        row_of(kKvSteps + u + v, r0, r1);
                        T* vo = static_cast<T*>(a.v_cache) + off + 8 * c0;
                        store8r(vo, r0);
                        store8r(vo + c01, r1);
                    }
                }
            }
        }
    };

    // ---- the run: kStages - 1 tokens ahead
    constexpr int kAhead = C::kStages - 1;
    Place q[C::kStages];
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
        q[s] = Place{0, 0, false, false};
        if (s < n) q[s] = fetch(s, s);
        async_commit();
    }
    int s = 0;
    for (int j = 0; j < n; ++j) {
        int s_next = s + kAhead;
        if (s_next >= C::kStages) s_next -= C::kStages;
        q[kAhead] = Place{0, 0, false, false};
        __syncwarp();                              // the warp has read the stage's table row and entry
        if (j + kAhead < n) q[kAhead] = fetch(j + kAhead, s_next);
        async_commit();
        async_wait<kAhead>();                      // this lane's copies of token j have landed,
        __syncwarp();                              // and the other lanes'
        finish(q[0], j, s);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = q[i + 1];
        if (++s == C::kStages) s = 0;
    }
    async_wait<0>();
}

template <typename T, int D>
const void* rope_fn(int out) {
    switch (out) {
        case kOutDense: return reinterpret_cast<const void*>(&norm_rope_kernel<T, D, kOutDense>);
        case kOutCache: return reinterpret_cast<const void*>(&norm_rope_kernel<T, D, kOutCache>);
        case kOutI8: return reinterpret_cast<const void*>(&norm_rope_kernel<T, D, kOutI8>);
        case kOutFp8: return reinterpret_cast<const void*>(&norm_rope_kernel<T, D, kOutFp8>);
        default: return reinterpret_cast<const void*>(&norm_rope_kernel<T, D, kOutI4>);
    }
}

template <typename T>
const void* rope_fn_d(int d, int out) {
    return d == 64 ? rope_fn<T, 64>(out) : rope_fn<T, 128>(out);
}

// (cos, sin) of position p and pair i, in fp64, rounded to fp32 once: far
// positions need the angle to more than fp32's 24 bits.
__global__ void __launch_bounds__(256) rope_table_kernel(float2* table, long long entries, int pairs, double log_base) {
    grid_dependency_wait();
    launch_dependents();
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
    if (e >= entries) return;
    const long long p = e / pairs;
    const int i = (int)(e - p * pairs);
    double s, c;
    sincos((double)p * exp(-log_base * ((double)i / (double)pairs)), &s, &c);
    table[e] = make_float2((float)c, (float)s);
}

cudaError_t launch_pdl(const void* fn, dim3 grid, int threads, int smem, cudaStream_t stream, void** args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& L) {
    RopeArgs a = {};
    const gqa_norm_rope_t& r = *L.desc;
    a.q = L.q;
    a.k = L.k;
    a.v = L.v;
    a.q_stride = L.q_stride;
    a.k_stride = L.k_stride;
    a.v_stride = L.v_stride;
    a.q_weight = r.q_weight;
    a.k_weight = r.k_weight;
    a.weight_dtype = r.weight_dtype;
    a.eps = r.eps;
    a.rope = reinterpret_cast<const float2*>(r.rope);
    a.rope_rows = r.rope_rows;
    a.rotary_dim = r.rope != nullptr ? r.rotary_dim : 0;
    a.interleaved = r.interleaved;
    a.rope_positions = r.rope != nullptr ? L.rope_positions : nullptr;   // read only where rows turn
    a.q_out = L.q_out;
    a.k_out = L.k_out;
    a.err = L.err;
    a.tokens = L.tokens;
    a.H = L.num_heads;
    a.K = L.num_kv_heads;
    int out = kOutDense;
    if (L.cache != nullptr) {
        const gqa_kv_cache_t& c = *L.cache;
        a.k_cache = c.k;
        a.v_cache = c.v;
        a.k_scale = static_cast<__half*>(c.k_scale);
        a.v_scale = static_cast<__half*>(c.v_scale);
        a.block_tables = L.block_tables;
        a.positions = L.positions;
        a.token_start = L.token_start;
        a.num_blocks = c.num_blocks;
        a.sb = c.stride_block;
        a.sh = c.stride_head;
        a.st = c.stride_token;
        a.batch = L.batch;
        a.T = L.tokens_per_seq;
        a.max_blocks = L.max_blocks;
        out = c.dtype == GQA_DTYPE_I8         ? kOutI8
              : c.dtype == GQA_DTYPE_FP8_E4M3 ? kOutFp8
              : c.dtype == GQA_DTYPE_I4       ? kOutI4
                                              : kOutCache;
    }
    const int rows = 512 / L.head_dim;                             // rows per warp step
    a.q_parts = (a.H + rows * kRopeSteps - 1) / (rows * kRopeSteps);
    a.parts = a.q_parts + (a.K + rows * kv_steps(out) - 1) / (rows * kv_steps(out));
    const void* fn = L.dtype == GQA_DTYPE_F32   ? rope_fn_d<float>(L.head_dim, out)
                     : L.dtype == GQA_DTYPE_F16 ? rope_fn_d<__half>(L.head_dim, out)
                                                : rope_fn_d<__nv_bfloat16>(L.head_dim, out);
    const int smem = L.dtype == GQA_DTYPE_F32 ? RopeCfg<float>::kSmem : RopeCfg<__half>::kSmem;
    const int sms = device_sms(-1), per_sm = ctas_per_sm(fn, kRopeWarps * 32, smem);
    if (sms < 1 || per_sm < 1) return cudaErrorInvalidConfiguration;
    if (a.tokens == 0) return cudaSuccess;
    // One wave of warps, each with an even share of consecutive tokens. Calls that stream
    // from DRAM (twice the L2's 129 MB read and written) take eight: shorter runs keep the
    // warps of the moment on fewer stretches of memory and even out parts of unequal work.
    // Not where most of the warps' rows are empty, nor for quantised rows: these are bound
    // by issue, and a run's start costs them more. Measured, one / eight waves, 32 + 8
    // heads, d = 128: 73.8 / 63.5 us for 400 MB, 37.3 / 36.3 for 200, 14.4 / 17.7 for 98;
    // 8 + 1 heads (31% of the rows), 334 MB: 83.9 / 88.7; FP8 cache, 370 MB: 68.0 / 74.1.
    const int esize = L.dtype == GQA_DTYPE_F32 ? 4 : 2;
    const bool streams = 2 * a.tokens * (a.H + 2 * a.K) * L.head_dim * esize >= (256LL << 20);
    const bool filled = 2 * (a.H + 2 * a.K) >= a.parts * rows * kRopeSteps;
    const int waves = streams && filled && out <= kOutCache ? 8 : 1;
    const long long runs =
        std::min(a.tokens, std::max<long long>(1, (long long)waves * sms * per_sm * kRopeWarps / a.parts));
    if (a.tokens / runs >= 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.runs = (int)runs;
    a.run = (int)(a.tokens / runs);
    a.longer = (int)(a.tokens % runs);
    const long long units = runs * a.parts;
    if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    void* args[] = {&a};
    return launch_pdl(fn, dim3((unsigned)((units + kRopeWarps - 1) / kRopeWarps)), kRopeWarps * 32, smem, L.stream, args);
}

cudaError_t launch_rope_table(float* table, int positions, int rotary_dim, double log_base, cudaStream_t stream) {
    int pairs = rotary_dim / 2;
    long long entries = (long long)positions * pairs;
    float2* t = reinterpret_cast<float2*>(table);
    if (entries == 0) return cudaSuccess;
    void* args[] = {&t, &entries, &pairs, &log_base};
    return launch_pdl(reinterpret_cast<const void*>(&rope_table_kernel), dim3((unsigned)((entries + 255) / 256)), 256,
                      0, stream, args);
}

}  // namespace gqa
