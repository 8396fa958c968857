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
// holds two 8-element chunks of a row, (c, c + rotary_dim/16) for split pairs and
// (2c, 2c + 1) for interleaved ones, so both elements of every pair are in one
// lane, the eight table pairs a lane needs are 64 contiguous bytes, and the norm
// takes log2(d/16) shuffles; a warp step covers 512/d rows. A warp serves one part
// of a token (kRopeSteps query steps, or kKvSteps steps of K and of V) for a run of
// consecutive tokens, so the sequence is looked up once a run. The rows, the table
// row and the page entry of the next tokens are in flight while one is worked on:
// each lane copies what it will read itself into a ring of stages with cp.async,
// which needs no registers for data in flight and no barrier.
#include <algorithm>
#include <type_traits>

#include "gqa_device.cuh"
#include "gqa_internal.h"

namespace gqa {

int device_sms(int device);   // gqa_capi.cu

namespace {

constexpr int kRopeWarps = 4;     // warps per CTA
constexpr int kRopeSteps = 4;     // query row steps one warp holds
constexpr int kKvSteps = 2;       // K steps (and as many V steps) one warp holds
constexpr int kMost = 4;          // steps a stage holds
static_assert(kRopeSteps <= kMost && 2 * kKvSteps <= kMost, "a stage holds a part");

// Where K (and V) rows go.
enum KvOut : int { kOutDense = 0, kOutCache = 1, kOutI8 = 2, kOutFp8 = 3, kOutI4 = 4 };

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
    int run;                                  // consecutive tokens a warp serves
};

// Stages of a warp's ring, and their layout: 16-byte slots of 32 lanes each (rows
// of kMost steps, then the table row), then 4 bytes a lane for the page entry.
template <typename T>
struct RopeCfg {
    static constexpr int kPieces = sizeof(T) / 2;                 // 16-byte pieces per chunk
    static constexpr int kRowSlots = kMost * 2 * kPieces;
    static constexpr int kStage = (kRowSlots + 4) * 512 + 128;
    static constexpr int kStages = sizeof(T) == 4 ? 2 : 3;
    static constexpr int kSmem = kRopeWarps * kStages * kStage;
};

__device__ __forceinline__ void async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
    if constexpr (sizeof(T) == 4) {
        const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
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
        r.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
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

// The norm of a row held by kLanes lanes, x <- x / sqrt(mean(x^2) + eps) * w, to
// about half a step of fp32: the squares are summed pairwise, the inverse root
// carries a low part (one Newton step's correction) and the products their exact
// remainders (as in rotate). A code next to a border, or a scale next to one of
// fp16, then falls where the exact value puts it far more often than with plain fp32
// products, at a few more instructions an element in a kernel that waits for memory.
template <int kLanes, int D>
__device__ __forceinline__ void norm_row(float (&x0)[8], float (&x1)[8], const float (&w0)[8], const float (&w1)[8],
                                         float eps) {
    float sq[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sq[e] = fmaf(x0[e], x0[e], x1[e] * x1[e]);
    float ss = ((sq[0] + sq[1]) + (sq[2] + sq[3])) + ((sq[4] + sq[5]) + (sq[6] + sq[7]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float m = fmaf(ss, 1.f / D, eps);
    const float r = 1.f / sqrtf(m);
    const float mr = m * r, mr_lo = fmaf(m, r, -mr);
    const float rest = fmaf(-mr, r, 1.f) - mr_lo * r;              // 1 - m r^2
    float r_lo = 0.5f * r * rest;
    if (!(fabsf(r_lo) < r)) r_lo = 0.f;                            // m = 0 or not finite: r alone
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float p0 = x0[e] * r, p1 = x1[e] * r;
        const float q0 = fmaf(x0[e], r_lo, fmaf(x0[e], r, -p0)), q1 = fmaf(x1[e], r_lo, fmaf(x1[e], r, -p1));
        x0[e] = fmaf(p0, w0[e], q0 * w0[e]);
        x1[e] = fmaf(p1, w1[e], q1 * w1[e]);
    }
}

// (a, b) -> (a cos - b sin, b cos + a sin), with the remainders of the products
// that are rounded first.
__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
    const float bs = b * cs.y, as = a * cs.y;
    const float x = fmaf(a, cs.x, -bs) - fmaf(b, cs.y, -bs);
    b = fmaf(b, cs.x, as) + fmaf(a, cs.y, -as);
    a = x;
}

// Codes and scale of one row (two 8-element chunks a lane, kLanes lanes a row),
// by the append's rule: s = fp16(min(amax / qmax, 65504)), code = x / s rounded to
// nearest even and clamped.
template <int kOut, int kLanes>
__device__ __forceinline__ void quantise_store(const float (&x0)[8], const float (&x1)[8], bool live, uint8_t* row,
                                               int c0, int c1, __half* scale, bool first) {
    constexpr float kQmax = kOut == kOutFp8 ? 448.0f : kOut == kOutI4 ? 7.0f : 127.0f;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const __half sh = __float2half_rn(fminf(__fdiv_rn(amax, kQmax), 65504.0f));
    const float sf = __half2float(sh);
    if (!live) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t code = 0;
            if (sf != 0.f) {
                const float t = __fdiv_rn(h ? x1[e] : x0[e], sf);
                if constexpr (kOut == kOutFp8) {
                    code = (uint32_t)__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
                } else {
                    constexpr int qm = (int)kQmax;
                    code = (uint32_t)max(-qm, min(qm, __float2int_rn(t)));
                }
            }
            if constexpr (kOut == kOutI4) w[0] |= (code & 0xFu) << (4 * e);
            else w[e / 4] |= (code & 0xFFu) << (8 * (e % 4));
        }
        const int c = h ? c1 : c0;
        if constexpr (kOut == kOutI4) *reinterpret_cast<uint32_t*>(row + 4 * c) = w[0];
        else *reinterpret_cast<uint2*>(row + 8 * c) = make_uint2(w[0], w[1]);
    }
    if (first) *scale = sh;
}

// Where a token goes: its cache position and table row, or why it goes nowhere.
struct Place {
    int pos, turn;
    bool live;           // false: of no sequence, or without a table row
    bool slot;           // the position is inside the block table
};

template <typename T, int D, int kOut>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeArgs a) {
    using C = RopeCfg<T>;
    constexpr int kLanes = D / 16;                 // lanes per row
    constexpr int kRows = 32 / kLanes;             // rows per warp step
    constexpr bool kCached = kOut != kOutDense;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = (int)blockIdx.x * kRopeWarps + warp;
    const int part = unit % a.parts;
    const long long t_lo = (long long)(unit / a.parts) * a.run;
    if (t_lo >= a.tokens) return;                  // uniform per warp
    const int n = (int)min((long long)a.run, a.tokens - t_lo);
    const int li = lane % kLanes, grp = lane / kLanes;
    const int half = a.rotary_dim / 16;            // lanes of a row that rotate
    const bool turns = li < half;
    // this lane's chunks of a row
    int c0 = 2 * li, c1 = 2 * li + 1;
    if (!a.interleaved && turns) {
        c0 = li;
        c1 = li + half;
    }
    const bool is_q = part < a.q_parts;
    // head of this lane's row in step u, -1: none. Steps of a K/V part: kKvSteps of
    // K, then the same heads' V.
    auto head = [&](int u) {
        const int h = is_q ? (part * kRopeSteps + u) * kRows + grp
                           : ((part - a.q_parts) * kKvSteps + u % kKvSteps) * kRows + grp;
        const bool in = is_q ? u < kRopeSteps && h < a.H : u < (kCached ? 2 : 1) * kKvSteps && h < a.K;
        return in ? h : -1;
    };
    const uint32_t ring = smem_addr(smem_raw) + warp * (C::kStages * C::kStage) + lane * 16;

    // ---- fetch: everything token t needs, into stage s
    int b = 0, left = 0, pos = 0;                  // its sequence, tokens after it in there, its position
    auto fetch = [&](int j, int s) -> Place {
        const long long t = t_lo + j;
        const uint32_t st = ring + s * C::kStage;
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            const int h = head(u);
            if (h < 0) continue;
            const T* src = is_q           ? static_cast<const T*>(a.q) + t * a.q_stride
                           : u < kKvSteps ? static_cast<const T*>(a.k) + t * a.k_stride
                                          : static_cast<const T*>(a.v) + t * a.v_stride;
            src += h * D;
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {
                async16(st + ((2 * u) * C::kPieces + i) * 512, reinterpret_cast<const uint4*>(src + 8 * c0) + i);
                async16(st + ((2 * u + 1) * C::kPieces + i) * 512, reinterpret_cast<const uint4*>(src + 8 * c1) + i);
            }
        }
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
            if (a.rope_positions != nullptr) p.turn = a.rope_positions[t];
            if (p.turn < 0 || p.turn >= a.rope_rows) {
                if (lane == 0 && part == 0) flag_error(a.err, GQA_DEVERR_POSITION);
                p.live = false;
            } else if (turns) {
                const uint4* src = reinterpret_cast<const uint4*>(a.rope + (long long)p.turn * (a.rotary_dim / 2) + 8 * li);
#pragma unroll
                for (int e = 0; e < 4; ++e) async16(st + (C::kRowSlots + e) * 512, src + e);
            }
        }
        if constexpr (kCached) {
            if (p.live && !is_q) {
                p.slot = pos >= 0 && pos < a.max_blocks * kBlock;
                if (p.slot)
                    async4(st + (C::kRowSlots + 4) * 512 - lane * 12,
                           a.block_tables + (long long)b * a.max_blocks + pos / kBlock);
                else if (lane == 0 && part == a.q_parts)
                    flag_error(a.err, GQA_DEVERR_POSITION);
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

    // ---- norm, rotation and store of token t from stage s
    auto finish = [&](const Place& p, int j, int s) {
        if (!p.live) return;                       // uniform per warp
        const long long t = t_lo + j;
        const uint32_t st = ring + s * C::kStage;
        long long dst = 0, sidx = 0;               // element offset of kv-head 0's slot; its scale
        if constexpr (kCached) {
            if (!is_q) {
                if (!p.slot) return;
                const int ph = (int)lds32(st + (C::kRowSlots + 4) * 512 - lane * 12);
                if (ph < 0 || ph >= a.num_blocks) {
                    if (lane == 0 && part == a.q_parts) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                    return;
                }
                dst = (long long)ph * a.sb + (long long)(p.pos % kBlock) * a.st;
                sidx = (long long)ph * a.K * kBlock + p.pos % kBlock;
            }
        }
        float2 cs[8];
        if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 f = lds128(st + (C::kRowSlots + e) * 512);
                cs[2 * e] = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
                cs[2 * e + 1] = make_float2(__uint_as_float(f.z), __uint_as_float(f.w));
            }
        }
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            const bool is_v = !is_q && u >= kKvSteps;
            if (is_v && !kCached) break;
            const int h = head(u);
            const bool live = h >= 0;
            if (!__any_sync(kFull, live)) continue;
            Raw8<T> r0, r1;
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {
                r0.w[i] = live ? lds128(st + ((2 * u) * C::kPieces + i) * 512) : make_uint4(0u, 0u, 0u, 0u);
                r1.w[i] = live ? lds128(st + ((2 * u + 1) * C::kPieces + i) * 512) : make_uint4(0u, 0u, 0u, 0u);
            }
            float x0[8], x1[8];
            widen8(r0, x0);
            widen8(r1, x1);
            if (!is_v) {
                if (wp != nullptr) norm_row<kLanes, D>(x0, x1, w0, w1, a.eps);
                if (turns) {
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            rotate(x0[2 * e], x0[2 * e + 1], cs[e]);
                            rotate(x1[2 * e], x1[2 * e + 1], cs[4 + e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) rotate(x0[e], x1[e], cs[e]);
                    }
                }
            }
            if (is_q || kOut == kOutDense) {
                if (live) {
                    T* out = is_q ? static_cast<T*>(a.q_out) + (t * a.H + h) * D
                                  : static_cast<T*>(a.k_out) + (t * a.K + h) * D;
                    store8r(out + 8 * c0, narrow8<T>(x0));
                    store8r(out + 8 * c1, narrow8<T>(x1));
                }
            } else if constexpr (kOut == kOutCache) {
                if (live) {
                    T* out = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + dst + (long long)h * a.sh;
                    store8r(out + 8 * c0, is_v ? r0 : narrow8<T>(x0));
                    store8r(out + 8 * c1, is_v ? r1 : narrow8<T>(x1));
                }
            } else if constexpr (kCached) {
                const long long off = dst + (long long)max(h, 0) * a.sh;
                uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (kOut == kOutI4 ? off / 2 : off);
                __half* sc = (is_v ? a.v_scale : a.k_scale) + sidx + (long long)max(h, 0) * kBlock;
                quantise_store<kOut, kLanes>(x0, x1, live, out, c0, c1, sc, li == 0);
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
        if (j + kAhead < n) q[kAhead] = fetch(j + kAhead, s_next);
        async_commit();
        async_wait<kAhead>();                      // this lane's copies of token j have landed
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
    a.rope_positions = L.rope_positions;
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
    a.parts = a.q_parts + (a.K + rows * kKvSteps - 1) / (rows * kKvSteps);
    const void* fn = L.dtype == GQA_DTYPE_F32   ? rope_fn_d<float>(L.head_dim, out)
                     : L.dtype == GQA_DTYPE_F16 ? rope_fn_d<__half>(L.head_dim, out)
                                                : rope_fn_d<__nv_bfloat16>(L.head_dim, out);
    const int smem = L.dtype == GQA_DTYPE_F32 ? RopeCfg<float>::kSmem : RopeCfg<__half>::kSmem;
    const int sms = device_sms(-1), per_sm = ctas_per_sm(fn, kRopeWarps * 32, smem);
    if (sms < 1 || per_sm < 1) return cudaErrorInvalidConfiguration;
    if (a.tokens == 0) return cudaSuccess;
    // one wave of warps: each serves as many consecutive tokens as it takes
    const long long runs = std::max<long long>(1, (long long)sms * per_sm * kRopeWarps / a.parts);
    const long long run = (a.tokens + runs - 1) / runs;
    if (run > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.run = (int)run;
    const long long units = (a.tokens + run - 1) / run * a.parts;
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
