// gqa_read.cu -- cached rows back as dense K and V: the inverse of the appends, for every
// cache type. Element i of a row is code * scale (exact in fp32: at most 8 x 11 bits),
// rounded once to the output's type; rows of the output's own type are copied bit for bit.
//
// Bound by memory: codes and scales are read once and the rows written once. A thread
// takes 8 elements of a row of one page (4 to 32 bytes in, 16 or 32 out), kUnroll of
// them at a time; the lanes of a row and the rows of a page are adjacent, so a warp's
// loads are whole lines of the page and its stores whole pieces of a token's row.
#include "gqa_device.cuh"
#include "gqa_internal.h"

namespace gqa {

namespace {

struct ReadArgs {
    const void *k, *v;
    const __half *k_scale, *v_scale;
    void *k_out, *v_out;
    const int32_t* token_start;   // NULL: every sequence reads max_tokens rows
    const int32_t* block_tables;
    const int32_t* positions;
    int32_t* err;
    long long num_blocks, total, sb, sh, st;
    int batch, K, max_tokens, max_blocks, pages_per_cta, ctas_per_seq;
};

constexpr int kReadThreads = 256, kUnroll = 4, kElems = 8;

// Cache formats as the kernel sees them.
enum ReadKind : int { kReadF32, kReadF16, kReadBf16, kReadI8, kReadFp8, kReadI4, kReadI4Kc };

template <int kKind>
struct Raw {                      // 8 elements as they lie in the cache
    static constexpr int kBits = kKind == kReadF32 ? 32 : kKind <= kReadBf16 ? 16 : kKind <= kReadFp8 ? 8 : 4;
    uint32_t w[kBits / 4];
    __device__ __forceinline__ void load(const uint8_t* p) {
        if constexpr (kBits == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (kBits == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x; w[1] = x.y;
        } else {
#pragma unroll
            for (int i = 0; i < kBits / 16; ++i) {
                const uint4 x = *(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
            }
        }
    }
    __device__ __forceinline__ void values(float (&f)[kElems]) const {
        if constexpr (kBits == 32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
        } else if constexpr (kBits == 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = unpack2<kKind == kReadBf16>(w[i]);
                f[2 * i] = x.x; f[2 * i + 1] = x.y;
            }
        } else if constexpr (kKind == kReadI8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (float)(int8_t)(w[i / 4] >> (8 * (i % 4)));
        } else if constexpr (kKind == kReadFp8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = unpack2<false>(e4m3x2_to_f16x2(w[i / 2] >> (16 * (i % 2))));
                f[2 * i] = x.x; f[2 * i + 1] = x.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (float)((int)(w[0] << (28 - 4 * i)) >> 28);
        }
    }
};

template <int kKind, int kOut>
__device__ __forceinline__ void put(void* out, long long at, const Raw<kKind>& raw, const float (&f)[kElems]) {
    if constexpr (kOut == kKind) {             // the same type: the same bits
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + at * (Raw<kKind>::kBits / 8));
#pragma unroll
        for (int i = 0; i < Raw<kKind>::kBits / 16; ++i)
            p[i] = make_uint4(raw.w[4 * i], raw.w[4 * i + 1], raw.w[4 * i + 2], raw.w[4 * i + 3]);
    } else if constexpr (kOut == kReadF32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        constexpr bool kB = kOut == kReadBf16;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack2<kB>(f[0], f[1]), pack2<kB>(f[2], f[3]), pack2<kB>(f[4], f[5]), pack2<kB>(f[6], f[7]));
    }
}

template <int kKind, int kOut, int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
    constexpr int kLanes = D / kElems;         // threads of a row
    constexpr bool kCoded = kKind >= kReadI8;
    launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x / a.ctas_per_seq, part = blockIdx.x - b * a.ctas_per_seq;
    const long long row0 = a.token_start ? a.token_start[b] : (long long)b * a.max_tokens;
    const long long n = a.token_start ? (long long)a.token_start[b + 1] - row0 : a.max_tokens;
    if (n < 0 || n > a.max_tokens || row0 < 0 || row0 + n > a.total) {
        if (part == 0 && threadIdx.x == 0) flag_error(a.err, GQA_DEVERR_POSITION);
        return;
    }
    const long long pos0 = a.positions[b], end = pos0 + n;
    // pages first .. last hold the rows; this CTA's are first + part * pages_per_cta ..
    const long long page0 = (pos0 >> 4) + (long long)part * a.pages_per_cta;
    const int pages = (int)min((long long)a.pages_per_cta, ((end + kBlock - 1) >> 4) - page0);
    if (pages <= 0) return;
    const int items = pages * 2 * a.K * kBlock * kLanes;
    for (int base = 0; base < items; base += kReadThreads * kUnroll) {
        Raw<kKind> raw[kUnroll];
        float s[kUnroll];
        uint4 kc[kUnroll];
        long long at[kUnroll];                 // element of the output, -1: none
        bool is_v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int item = base + i * kReadThreads + threadIdx.x;
            at[i] = -1;
            is_v[i] = false;
            s[i] = 1.f;
            if (item >= items) continue;
            const int e = (item % kLanes) * kElems, slot = item / kLanes % kBlock;
            const int tile = item / (kLanes * kBlock), side = tile / a.K, g = tile - side * a.K;
            is_v[i] = side & 1;
            const long long page = page0 + (side >> 1), pos = page * kBlock + slot;
            if (pos < pos0 || pos >= end) continue;
            if (pos < 0 || page >= a.max_blocks) {
                if (g == 0 && e == 0) flag_error(a.err, GQA_DEVERR_POSITION);
                continue;
            }
            const int ph = a.block_tables[(long long)b * a.max_blocks + page];
            if (ph < 0 || ph >= a.num_blocks) {
                if (g == 0 && e == 0) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
                continue;
            }
            const long long off = ph * a.sb + g * a.sh + slot * a.st + e;
            raw[i].load(static_cast<const uint8_t*>(is_v[i] ? a.v : a.k) + off * Raw<kKind>::kBits / 8);
            if constexpr (kCoded) {
                const long long tok = ((long long)ph * a.K + g) * kBlock + slot;
                if (kKind == kReadI4Kc && !is_v[i])
                    kc[i] = *reinterpret_cast<const uint4*>(a.k_scale + ((long long)ph * a.K + g) * D + e);
                else
                    s[i] = __half2float((is_v[i] ? a.v_scale : a.k_scale)[tok]);
            }
            at[i] = ((row0 + pos - pos0) * a.K + g) * D + e;
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (at[i] < 0) continue;
            float f[kElems];
            raw[i].values(f);
            if constexpr (kCoded) {
                if (kKind == kReadI4Kc && !is_v[i]) {
                    const uint32_t w[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = unpack2<false>(w[j]);
                        f[2 * j] *= x.x;
                        f[2 * j + 1] *= x.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kElems; ++j) f[j] *= s[i];
                }
            }
            put<kKind, kOut>(is_v[i] ? a.v_out : a.k_out, at[i], raw[i], f);
        }
    }
}

template <int kKind, int kOut>
const void* read_fn(int d) {
    return d == 64 ? reinterpret_cast<const void*>(&read_kernel<kKind, kOut, 64>)
                   : reinterpret_cast<const void*>(&read_kernel<kKind, kOut, 128>);
}
template <int kKind>
const void* pick_out(int out, int d) {
    return out == GQA_DTYPE_F32   ? read_fn<kKind, kReadF32>(d)
           : out == GQA_DTYPE_F16 ? read_fn<kKind, kReadF16>(d)
                                  : read_fn<kKind, kReadBf16>(d);
}

}  // namespace

cudaError_t launch_kv_read(const gqa_kv_cache_t& c, void* k_out, void* v_out, int out_dtype, long long total,
                           const int32_t* token_start, int max_tokens, const int32_t* block_tables, int max_blocks,
                           const int32_t* positions, int batch, int32_t* err, cudaStream_t stream) {
    const void* fn = nullptr;
    switch (c.dtype) {
        case GQA_DTYPE_F32: fn = pick_out<kReadF32>(out_dtype, c.head_dim); break;
        case GQA_DTYPE_F16: fn = pick_out<kReadF16>(out_dtype, c.head_dim); break;
        case GQA_DTYPE_BF16: fn = pick_out<kReadBf16>(out_dtype, c.head_dim); break;
        case GQA_DTYPE_I8: fn = pick_out<kReadI8>(out_dtype, c.head_dim); break;
        case GQA_DTYPE_FP8_E4M3: fn = pick_out<kReadFp8>(out_dtype, c.head_dim); break;
        case GQA_DTYPE_I4: fn = pick_out<kReadI4>(out_dtype, c.head_dim); break;
        default: fn = pick_out<kReadI4Kc>(out_dtype, c.head_dim); break;
    }
    ReadArgs a;
    a.k = c.k;
    a.v = c.v;
    a.k_scale = static_cast<const __half*>(c.k_scale);
    a.v_scale = static_cast<const __half*>(c.v_scale);
    a.k_out = k_out;
    a.v_out = v_out;
    a.token_start = token_start;
    a.block_tables = block_tables;
    a.positions = positions;
    a.err = err;
    a.num_blocks = c.num_blocks;
    a.total = total;
    a.sb = c.stride_block;
    a.sh = c.stride_head;
    a.st = c.stride_token;
    a.batch = batch;
    a.K = c.num_kv_heads;
    a.max_tokens = max_tokens;
    a.max_blocks = max_blocks;
    // a page of one kv-head is 2 * 16 * d / 8 items, 256 or 512: pages until a CTA's
    // threads have kUnroll of them each, where there are pages enough
    const int per_page = 2 * c.num_kv_heads * kBlock * c.head_dim / kElems;
    a.pages_per_cta = max(1, kReadThreads * kUnroll / per_page);
    const long long pages = ((long long)max_tokens + 2 * kBlock - 2) / kBlock;   // an unaligned run touches one more
    a.ctas_per_seq = (int)((pages + a.pages_per_cta - 1) / a.pages_per_cta);
    const long long grid = (long long)a.ctas_per_seq * batch;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kReadThreads);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    void* args[] = {&a};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace gqa
