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
// takes log2(d/16) shuffles; a warp step covers 512/d rows. A warp takes one batch
// of kRopeSteps query steps of one token, or one of its K and V steps, with every
// row load issued before the position is looked up. The warps of a token sit next
// to each other, so the table row comes from L1 for all but the first.
#include "gqa_device.cuh"
#include "gqa_internal.h"

namespace gqa {

namespace {

constexpr int kRopeWarps = 4;     // warps per CTA
constexpr int kRopeSteps = 4;     // query row steps one warp holds
constexpr int kKvSteps = 2;       // K steps (and as many V steps) one warp holds

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
};

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
__device__ __forceinline__ bool sequence_of(const RopeArgs& a, long long tok, int lane, int& b, int& i) {
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
    const int t0 = a.token_start[b], cnt = a.token_start[b + 1] - t0;
    i = (int)(tok - t0);
    if (cnt < 0 || cnt > a.T) {
        if (lane == 0) flag_error(a.err, GQA_DEVERR_POSITION);
        return false;
    }
    return i < cnt;
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

template <typename T, int D, int kOut>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(const RopeArgs a) {
    constexpr int kLanes = D / 16;                 // lanes per row
    constexpr int kRows = 32 / kLanes;             // rows per warp step
    constexpr bool kCached = kOut != kOutDense;
    grid_dependency_wait();
    launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const long long tok = unit / a.parts;
    const int part = (int)(unit - tok * a.parts);
    if (tok >= a.tokens) return;                   // uniform per warp
    const int li = lane % kLanes, grp = lane / kLanes;
    const int half = a.rotary_dim / 16;            // lanes of a row that rotate
    // this lane's chunks of a row
    int c0 = 2 * li, c1 = 2 * li + 1;
    if (!a.interleaved && li < half) {
        c0 = li;
        c1 = li + half;
    }
    const bool is_q = part < a.q_parts;

    // ---- the rows, before anything that depends on the position
    constexpr int kMost = kRopeSteps > 2 * kKvSteps ? kRopeSteps : 2 * kKvSteps;
    Raw8<T> raw[kMost][2];
    int row[kMost];                                // head of each step, -1: none
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const T* src = nullptr;
        row[u] = -1;
        if (is_q) {
            const int h = (part * kRopeSteps + u) * kRows + grp;
            if (u < kRopeSteps && h < a.H) {
                row[u] = h;
                src = static_cast<const T*>(a.q) + tok * a.q_stride + (long long)h * D;
            }
        } else {
            // steps 0 .. kKvSteps-1 are K rows, the next as many the same heads' V rows
            const int g = ((part - a.q_parts) * kKvSteps + u % kKvSteps) * kRows + grp;
            if (u < (kCached ? 2 * kKvSteps : kKvSteps) && g < a.K) {
                row[u] = g;
                src = u < kKvSteps ? static_cast<const T*>(a.k) + tok * a.k_stride + (long long)g * D
                                   : static_cast<const T*>(a.v) + tok * a.v_stride + (long long)g * D;
            }
        }
        if (row[u] >= 0) {
            raw[u][0] = load8(src + 8 * c0);
            raw[u][1] = load8(src + 8 * c1);
        } else {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) / 2); ++i) raw[u][0].w[i] = raw[u][1].w[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }

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

    // ---- the token's place: sequence, position, table row
    int b = 0, i = 0, pos = 0;
    if constexpr (kCached) {
        if (a.token_start == nullptr) {
            b = (int)(tok / a.T);
            i = (int)(tok - (long long)b * a.T);
        } else if (!sequence_of(a, tok, lane, b, i)) {
            return;                                // uniform per warp
        }
        pos = a.positions[b] + i;
    }
    int turn = pos;                                // row of the rotation table
    if (a.rope_positions != nullptr) turn = a.rope_positions[tok];
    float2 cs[8];
    const bool turns = li < half;
    if (half > 0) {
        if (turn < 0 || turn >= a.rope_rows) {
            if (lane == 0 && part == 0) flag_error(a.err, GQA_DEVERR_POSITION);
            return;                                // uniform per warp
        }
        if (turns) {
            const float4* p = reinterpret_cast<const float4*>(a.rope + (long long)turn * (a.rotary_dim / 2) + 8 * li);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 f = __ldg(p + e);
                cs[2 * e] = make_float2(f.x, f.y);
                cs[2 * e + 1] = make_float2(f.z, f.w);
            }
        }
    }
    long long dst = 0, sidx = 0;                   // element offset of kv-head 0's slot; its scale
    if constexpr (kCached) {
        if (!is_q) {
            if (pos < 0 || pos >= a.max_blocks * kBlock) {
                if (lane == 0 && part == a.q_parts) flag_error(a.err, GQA_DEVERR_POSITION);
                return;
            }
            const int ph = a.block_tables[(long long)b * a.max_blocks + pos / kBlock];
            if (ph < 0 || ph >= a.num_blocks) {
                if (lane == 0 && part == a.q_parts) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                return;
            }
            dst = (long long)ph * a.sb + (long long)(pos % kBlock) * a.st;
            sidx = (long long)ph * a.K * kBlock + pos % kBlock;
        }
    }

    // ---- norm, rotation, store
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const bool is_v = !is_q && u >= kKvSteps;
        if (is_v && !kCached) break;
        const bool live = row[u] >= 0;
        float x0[8], x1[8];
        if (!is_v || (kOut != kOutDense && kOut != kOutCache)) {
            widen8(raw[u][0], x0);
            widen8(raw[u][1], x1);
        }
        if (!is_v) {
            if (wp != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
                const float rs = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x0[e] = x0[e] * rs * w0[e];
                    x1[e] = x1[e] * rs * w1[e];
                }
            }
            if (turns) {
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a0 = x0[2 * e], b0 = x0[2 * e + 1], a1 = x1[2 * e], b1 = x1[2 * e + 1];
                        x0[2 * e] = a0 * cs[e].x - b0 * cs[e].y;
                        x0[2 * e + 1] = b0 * cs[e].x + a0 * cs[e].y;
                        x1[2 * e] = a1 * cs[4 + e].x - b1 * cs[4 + e].y;
                        x1[2 * e + 1] = b1 * cs[4 + e].x + a1 * cs[4 + e].y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float av = x0[e], bv = x1[e];
                        x0[e] = av * cs[e].x - bv * cs[e].y;
                        x1[e] = bv * cs[e].x + av * cs[e].y;
                    }
                }
            }
        }
        if (is_q || kOut == kOutDense) {
            if (live) {
                T* out = is_q ? static_cast<T*>(a.q_out) + (tok * a.H + row[u]) * D
                              : static_cast<T*>(a.k_out) + (tok * a.K + row[u]) * D;
                store8r(out + 8 * c0, narrow8<T>(x0));
                store8r(out + 8 * c1, narrow8<T>(x1));
            }
        } else if constexpr (kOut == kOutCache) {
            if (live) {
                T* out = static_cast<T*>(is_v ? a.v_cache : a.k_cache) + dst + (long long)row[u] * a.sh;
                store8r(out + 8 * c0, is_v ? raw[u][0] : narrow8<T>(x0));
                store8r(out + 8 * c1, is_v ? raw[u][1] : narrow8<T>(x1));
            }
        } else if constexpr (kCached) {
            const long long off = dst + (long long)max(row[u], 0) * a.sh;
            uint8_t* out = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (kOut == kOutI4 ? off / 2 : off);
            __half* sc = (is_v ? a.v_scale : a.k_scale) + sidx + (long long)max(row[u], 0) * kBlock;
            quantise_store<kOut, kLanes>(x0, x1, live, out, c0, c1, sc, li == 0);
        }
    }
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

cudaError_t launch_pdl(const void* fn, dim3 grid, int threads, cudaStream_t stream, void** args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
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
    const long long warps = a.tokens * a.parts;
    const long long grid = (warps + kRopeWarps - 1) / kRopeWarps;
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const void* fn = L.dtype == GQA_DTYPE_F32   ? rope_fn_d<float>(L.head_dim, out)
                     : L.dtype == GQA_DTYPE_F16 ? rope_fn_d<__half>(L.head_dim, out)
                                                : rope_fn_d<__nv_bfloat16>(L.head_dim, out);
    void* args[] = {&a};
    return launch_pdl(fn, dim3((unsigned)grid), kRopeWarps * 32, L.stream, args);
}

cudaError_t launch_rope_table(float* table, int positions, int rotary_dim, double log_base, cudaStream_t stream) {
    int pairs = rotary_dim / 2;
    long long entries = (long long)positions * pairs;
    float2* t = reinterpret_cast<float2*>(table);
    if (entries == 0) return cudaSuccess;
    void* args[] = {&t, &entries, &pairs, &log_base};
    return launch_pdl(reinterpret_cast<const void*>(&rope_table_kernel), dim3((unsigned)((entries + 255) / 256)), 256,
                      stream, args);
}

}  // namespace gqa
