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

// Stages of a warp's ring, and their layout: the rows of kMost steps in 16-byte
// slots of 32 lanes, then the table row (64 bytes a lane of a row), then the page
// entry. Two stages and at most 102 registers let five CTAs share an SM: the kernel
// waits on its own instruction latencies more than on memory (measured on 16384
// tokens of 32 + 8 heads, d = 128: KERNEL_FIGURES).
template <typename T>
struct RopeCfg {
    static constexpr int kPieces = sizeof(T) / 2;                 // 16-byte pieces per chunk
    static constexpr int kRowSlots = kMost * 2 * kPieces;
    static constexpr int kTable = kRowSlots * 512, kEntry = kTable + 512;
    static constexpr int kStage = kEntry + 16;
    static constexpr int kStages = 2;
    static constexpr int kWeights = kRopeWarps * kStages * kStage;   // fp32, q then k
    static constexpr int kSmem = kWeights + 2 * 128 * 4;
    static constexpr int kCtas = sizeof(T) == 4 ? 3 : 5;
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
// Eight elements as four packed fp32 pairs.
template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, uint64_t (&x)[4]) {
    const uint4 w = r.w[0];
    if constexpr (sizeof(T) == 4) {
        const uint4 v = r.w[sizeof(T) / 2 - 1];
        x[0] = f2_make(__uint_as_float(w.x), __uint_as_float(w.y));
        x[1] = f2_make(__uint_as_float(w.z), __uint_as_float(w.w));
        x[2] = f2_make(__uint_as_float(v.x), __uint_as_float(v.y));
        x[3] = f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2<kB>(u[i]);
            x[i] = f2_make(f.x, f.y);
        }
    }
}
template <typename T>
__device__ __forceinline__ Raw8<T> narrow8(const uint64_t (&x)[4]) {
    Raw8<T> r;
    const float2 a = f2_split(x[0]), b = f2_split(x[1]), c = f2_split(x[2]), d = f2_split(x[3]);
    if constexpr (sizeof(T) == 4) {
        r.w[0] = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
        r.w[sizeof(T) / 2 - 1] =
            make_uint4(__float_as_uint(c.x), __float_as_uint(c.y), __float_as_uint(d.x), __float_as_uint(d.y));
    } else {
        constexpr bool kB = std::is_same<T, __nv_bfloat16>::value;
        r.w[0] = make_uint4(pack2<kB>(a.x, a.y), pack2<kB>(b.x, b.y), pack2<kB>(c.x, c.y), pack2<kB>(d.x, d.y));
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

// The norm of a row held by kLanes lanes, x <- x / sqrt(mean(x^2) + eps) * w, two
// elements an instruction. kExact carries what fp32 products round away (the inverse
// root's low part by one Newton step, the products' remainders), to about half a step
// of fp32: for rows that stay fp32 or are quantised next, where a code next to a
// border, or a scale next to one of fp16, then falls where the exact value puts it.
// Rows rounded to 16 bits do not need it, and the kernel is bound by issue as much as
// by memory (carried everywhere it took 16384 tokens from 72 to 95 us).
template <bool kExact, int kLanes, int D>
__device__ __forceinline__ void norm_row(uint64_t (&x0)[4], uint64_t (&x1)[4], uint32_t wa, uint32_t wb, float eps) {
    uint64_t sq0 = f2_mul(x0[0], x0[0]), sq1 = f2_mul(x1[0], x1[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) {
        sq0 = f2_fma(x0[e], x0[e], sq0);
        sq1 = f2_fma(x1[e], x1[e], sq1);
    }
    const float2 sq = f2_split(f2_add(sq0, sq1));
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float m = fmaf(ss, 1.f / D, eps);
    const float r = kExact ? 1.f / sqrtf(m) : rsqrtf(m);
    const uint64_t r2 = f2_make(r, r);
    uint64_t w0[4], w1[4];                   // the chunks' weights, from shared memory at wa and wb
    {
        Raw8<float> f;
        f.w[0] = lds128(wa), f.w[1] = lds128(wa + 16);
        widen8(f, w0);
        f.w[0] = lds128(wb), f.w[1] = lds128(wb + 16);
        widen8(f, w1);
    }
    if constexpr (kExact) {
        const float mr = m * r, mr_lo = fmaf(m, r, -mr);
        float r_lo = 0.5f * r * (fmaf(-mr, r, 1.f) - mr_lo * r);   // r (1 - m r^2) / 2
        if (!(fabsf(r_lo) < r)) r_lo = 0.f;                        // m = 0 or not finite: r alone
        const uint64_t lo2 = f2_make(r_lo, r_lo), nr2 = f2_make(-r, -r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t p0 = f2_mul(x0[e], r2), p1 = f2_mul(x1[e], r2);
            const uint64_t q0 = f2_fma(x0[e], lo2, f2_fma(x0[e], r2, f2_mul(x0[e], nr2)));
            const uint64_t q1 = f2_fma(x1[e], lo2, f2_fma(x1[e], r2, f2_mul(x1[e], nr2)));
            x0[e] = f2_fma(p0, w0[e], f2_mul(q0, w0[e]));
            x1[e] = f2_fma(p1, w1[e], f2_mul(q1, w1[e]));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x0[e] = f2_mul(f2_mul(x0[e], r2), w0[e]);
            x1[e] = f2_mul(f2_mul(x1[e], r2), w1[e]);
        }
    }
}

// A lane's eight (cos, sin) pairs, two to a register pair, and -sin.
struct Turn {
    uint64_t c[4], s[4], n[4];
    __device__ __forceinline__ void set(int e, uint4 f) {
        c[e] = f2_make(__uint_as_float(f.x), __uint_as_float(f.z));
        s[e] = f2_make(__uint_as_float(f.y), __uint_as_float(f.w));
        n[e] = f2_make(-__uint_as_float(f.y), -__uint_as_float(f.w));
    }
};

// a c + b r, kExact with what the product b r rounds away (nr = -r).
template <bool kExact>
__device__ __forceinline__ uint64_t fma_rest(uint64_t a, uint64_t c, uint64_t b, uint64_t r, uint64_t nr) {
    const uint64_t x = f2_fma(a, c, f2_mul(b, r));
    if constexpr (kExact) return f2_add(x, f2_fma(b, r, f2_mul(b, nr)));
    else return x;
}
template <bool kExact>
__device__ __forceinline__ float fma_rest(float a, float c, float b, float r) {
    const float br = b * r, x = fmaf(a, c, br);
    if constexpr (kExact) return x + fmaf(b, r, -br);
    else return x;
}

// (a, b) -> (a cos - b sin, b cos + a sin) of a lane's eight pairs.
template <bool kExact>
__device__ __forceinline__ void rotate(uint64_t (&x0)[4], uint64_t (&x1)[4], const Turn& t, bool interleaved) {
    if (interleaved) {
        auto one = [&](uint64_t& x, float c, float s) {
            const float2 v = f2_split(x);
            x = f2_make(fma_rest<kExact>(v.x, c, v.y, -s), fma_rest<kExact>(v.y, c, v.x, s));
        };
#pragma unroll
        for (int e = 0; e < 4; ++e) {        // pairs 0 .. 3 are chunk 0's, 4 .. 7 chunk 1's
            const float2 c = f2_split(t.c[e / 2]), s = f2_split(t.s[e / 2]);
            const float2 d = f2_split(t.c[2 + e / 2]), u = f2_split(t.s[2 + e / 2]);
            one(x0[e], e % 2 ? c.y : c.x, e % 2 ? s.y : s.x);
            one(x1[e], e % 2 ? d.y : d.x, e % 2 ? u.y : u.x);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t a = x0[e], b = x1[e];
            x0[e] = fma_rest<kExact>(a, t.c[e], b, t.n[e], t.s[e]);
            x1[e] = fma_rest<kExact>(b, t.c[e], a, t.s[e], t.n[e]);
        }
    }
}

// Codes and scale of one row (two 8-element chunks a lane, kLanes lanes a row), by the
// append's rule: s = fp16(min(amax / qmax, 65504)), code = x / s rounded to nearest
// even and clamped. The quotient is the correctly rounded one: with y = RN(1/s), once
// a row, q = RN(x y) and the exact remainder x - q s, RN(q + (x - q s) y) is RN(x / s)
// (Markstein's theorem; s has 11 significant bits, so its mantissa is not all ones,
// and no step leaves fp32's range where the code is not zero), at three instructions
// instead of a division. A row with an infinity divides.
template <int kOut, int kLanes>
__device__ __forceinline__ void quantise_store(const uint64_t (&x0)[4], const uint64_t (&x1)[4], bool live, uint8_t* row,
                                               int c0, int c1, __half* scale, bool first) {
    constexpr float kQmax = kOut == kOutFp8 ? 448.0f : kOut == kOutI4 ? 7.0f : 127.0f;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = f2_split(x0[e]), b = f2_split(x1[e]);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const __half sh = __float2half_rn(fminf(__fdiv_rn(amax, kQmax), 65504.0f));
    const float sf = __half2float(sh);
    if (!live) return;
    const float y = __fdiv_rn(1.f, sf);
    const uint64_t y2 = f2_make(y, y), ns2 = f2_make(-sf, -sf);
    const bool finite = amax < INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w[2] = {0u, 0u};
        if (sf != 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t x = h ? x1[e] : x0[e];
                const uint64_t q = f2_mul(x, y2);
                float2 t = f2_split(f2_fma(f2_fma(q, ns2, x), y2, q));
                if (!finite) {
                    const float2 xs = f2_split(x);
                    t = make_float2(__fdiv_rn(xs.x, sf), __fdiv_rn(xs.y, sf));
                }
                if constexpr (kOut == kOutFp8) {
                    const uint32_t two = __nv_cvt_float2_to_fp8x2(t, __NV_SATFINITE, __NV_E4M3);
                    w[e / 2] |= two << (16 * (e % 2));
                } else {
                    constexpr int qm = (int)kQmax;
                    const uint32_t a = (uint32_t)max(-qm, min(qm, __float2int_rn(t.x)));
                    const uint32_t b = (uint32_t)max(-qm, min(qm, __float2int_rn(t.y)));
                    if constexpr (kOut == kOutI4) w[0] |= ((a & 0xFu) | ((b & 0xFu) << 4)) << (8 * e);
                    else w[e / 2] |= ((a & 0xFFu) | ((b & 0xFFu) << 8)) << (16 * (e % 2));
                }
            }
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
__global__ void __launch_bounds__(kRopeWarps * 32, RopeCfg<T>::kCtas) norm_rope_kernel(const RopeArgs a) {
    using C = RopeCfg<T>;
    constexpr int kLanes = D / 16;                 // lanes per row
    constexpr int kRows = 32 / kLanes;             // rows per warp step
    constexpr bool kCached = kOut != kOutDense;
    constexpr bool kCoded = kOut > kOutCache;      // rows are quantised
    extern __shared__ __align__(16) uint8_t smem_raw[];
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the weights as fp32, q's then k's
    const uint32_t weights = smem_addr(smem_raw) + C::kWeights;
    for (int i = threadIdx.x; i < 2 * D; i += kRopeWarps * 32) {
        const void* w = i < D ? a.q_weight : a.k_weight;
        if (w != nullptr)
            reinterpret_cast<float*>(smem_raw + C::kWeights)[i] =
                a.weight_dtype == GQA_DTYPE_F32    ? static_cast<const float*>(w)[i % D]
                : a.weight_dtype == GQA_DTYPE_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i % D])
                                                   : __half2float(static_cast<const __half*>(w)[i % D]);
    }
    __syncthreads();
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
    const bool normed = (is_q ? a.q_weight : a.k_weight) != nullptr;
    const uint32_t wbase = weights + (is_q ? 0 : D * 4);
    const uint32_t ring = smem_addr(smem_raw) + warp * (C::kStages * C::kStage);
    // rows of step u lie u * kRows heads past this lane's first one, of step 0
    const int h0 = (is_q ? part * kRopeSteps : (part - a.q_parts) * kKvSteps) * kRows + grp;
    const T* src0 = static_cast<const T*>(is_q ? a.q : a.k) + t_lo * (is_q ? a.q_stride : a.k_stride) + (long long)h0 * D;
    const T* vsrc0 = is_q || !kCached ? nullptr : static_cast<const T*>(a.v) + t_lo * a.v_stride + (long long)h0 * D;
    const long long src_step = is_q ? a.q_stride : a.k_stride;
    bool in[kMost];                                // this lane has a row in step u
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int h = h0 + (is_q ? u : u % kKvSteps) * kRows;
        in[u] = is_q ? u < kRopeSteps && h < a.H : u < (kCached ? 2 : 1) * kKvSteps && h < a.K;
    }

    // ---- fetch: everything token t needs, into stage s
    int b = 0, left = 0, pos = 0;                  // its sequence, tokens after it in there, its position
    auto fetch = [&](int j, int s) -> Place {
        const long long t = t_lo + j;
        const uint32_t st = ring + s * C::kStage;
        const T* row = src0 + j * src_step;
        const T* vrow = vsrc0 + (kCached ? j * a.v_stride : 0);
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            if (!in[u]) continue;
            const T* src = is_q ? row + u * kRows * D : u < kKvSteps ? row + u * kRows * D : vrow + (u - kKvSteps) * kRows * D;
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {
                async16(st + ((2 * u) * C::kPieces + i) * 512 + lane * 16, reinterpret_cast<const uint4*>(src + 8 * c0) + i);
                async16(st + ((2 * u + 1) * C::kPieces + i) * 512 + lane * 16, reinterpret_cast<const uint4*>(src + 8 * c1) + i);
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
            } else if (lane < 4 * half) {          // 16 bytes a lane: the row once for the warp
                async16(st + C::kTable + lane * 16,
                        reinterpret_cast<const uint4*>(a.rope + (long long)p.turn * (a.rotary_dim / 2)) + lane);
            }
        }
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

    // ---- norm, rotation and store of token t from stage s
    auto finish = [&](const Place& p, int j, int s) {
        if (!p.live) return;                       // uniform per warp
        const long long t = t_lo + j;
        const uint32_t st = ring + s * C::kStage;
        long long dst = 0, sidx = 0;               // element offset of kv-head 0's slot; its scale
        if constexpr (kCached) {
            if (!is_q) {
                if (!p.slot) return;
                const int ph = (int)lds32(st + C::kEntry);
                if (ph < 0 || ph >= a.num_blocks) {
                    if (lane == 0 && part == a.q_parts) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                    return;
                }
                dst = (long long)ph * a.sb + (long long)(p.pos % kBlock) * a.st;
                sidx = (long long)ph * a.K * kBlock + p.pos % kBlock;
            }
        }
        Turn turn;
        if (turns) {
#pragma unroll
            for (int e = 0; e < 4; ++e) turn.set(e, lds128(st + C::kTable + (4 * li + e) * 16));
        }
#pragma unroll
        for (int u = 0; u < kMost; ++u) {
            const bool is_v = !is_q && u >= kKvSteps;
            if (is_v && !kCached) break;
            if (!__any_sync(kFull, in[u])) continue;
            Raw8<T> r0, r1;
#pragma unroll
            for (int i = 0; i < C::kPieces; ++i) {       // (a lane without a row works on what the slot holds)
                r0.w[i] = lds128(st + ((2 * u) * C::kPieces + i) * 512 + lane * 16);
                r1.w[i] = lds128(st + ((2 * u + 1) * C::kPieces + i) * 512 + lane * 16);
            }
            uint64_t x0[4], x1[4];
            widen8(r0, x0);
            widen8(r1, x1);
            if (!is_v) {
                auto work = [&](auto exact) {
                    constexpr bool kExact = decltype(exact)::value;
                    if (normed) norm_row<kExact, kLanes, D>(x0, x1, wbase + 32 * c0, wbase + 32 * c1, a.eps);
                    if (turns) rotate<kExact>(x0, x1, turn, a.interleaved != 0);
                };
                if (sizeof(T) == 4 || (kCoded && !is_q)) work(std::true_type{});
                else work(std::false_type{});
            }
            const int h = h0 + (is_q ? u : u % kKvSteps) * kRows;
            if (is_q || kOut == kOutDense) {
                if (in[u]) {
                    T* out = is_q ? static_cast<T*>(a.q_out) + (t * a.H + h) * D : static_cast<T*>(a.k_out) + (t * a.K + h) * D;
                    store8r(out + 8 * c0, narrow8<T>(x0));
                    store8r(out + 8 * c1, narrow8<T>(x1));
                }
            } else if constexpr (kOut == kOutCache) {
                if (in[u]) {
                    T* out = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + dst + (long long)h * a.sh;
                    store8r(out + 8 * c0, is_v ? r0 : narrow8<T>(x0));
                    store8r(out + 8 * c1, is_v ? r1 : narrow8<T>(x1));
                }
            } else if constexpr (kCached) {
                const long long off = dst + (long long)h * a.sh;
                uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (kOut == kOutI4 ? off / 2 : off);
                __half* sc = (is_v ? a.v_scale : a.k_scale) + sidx + (long long)h * kBlock;
                quantise_store<kOut, kLanes>(x0, x1, in[u], out, c0, c1, sc, li == 0);
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
