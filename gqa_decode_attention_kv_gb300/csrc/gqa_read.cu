// gqa_read.cu -- cached rows back as dense K and V: the inverse of the appends, for every
// cache type. Element i of a row is code * scale (exact in fp32: at most 8 x 11 bits),
// rounded once to the output's type; rows of the output's own type are copied bit for bit.
//
// Bound by memory: codes and scales are read once and the rows written once. A warp takes
// the 16 rows of one (page, K or V, kv-head) at a time, all of its loads in flight before
// the first store; a lane holds 8 elements of every second or fourth row, so that a store
// instruction writes whole 128- to 256-byte pieces of a token's row. Of the copy rate: 16
// prompts of 8192 tokens to bf16 from a KIVI-style INT4 cache 0.92 (110 us), from int8 0.95
// (126), e4m3 0.94 (126), int4 0.92 (108), at d=64 to fp16 from int8 0.88 (68), e4m3 0.83 (72);
// 8 prompts of 3000 to 8192 tokens from bf16 to fp32 0.90 (90), 37 ragged ones of FP8, d=64, to
// fp16 0.67 (25).
#include <algorithm>

#include "gqa_device.cuh"
#include "gqa_internal.h"

namespace gqa {

int device_sms(int device);   // gqa_capi.cu

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

constexpr int kReadThreads = 256, kElems = 8;

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

// 8 elements as they go out: 32-bit words, 4 of a 16-bit type, 8 of fp32.
template <int kKind, int kOut>
struct Out {
    static constexpr int kWords = kOut == kReadF32 ? 8 : 4;
    uint32_t w[kWords];
    __device__ __forceinline__ Out(const Raw<kKind>& raw, const float (&f)[kElems]) {
        if constexpr (kOut == kKind) {         // the same type: the same bits
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = raw.w[i];
        } else if constexpr (kOut == kReadF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack2<kOut == kReadBf16>(f[2 * i], f[2 * i + 1]);
        }
        if constexpr (kWords == 8) {
            // lanes 2i and 2i + 1 swap halves, so that each of their two stores writes 32
            // bytes in a row, of the even lane's elements and then of the odd's
            const bool odd = threadIdx.x & 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t got = __shfl_xor_sync(kFull, odd ? w[i] : w[4 + i], 1);
                if (odd) w[i] = got;
                else w[4 + i] = got;
            }
        }
    }
    // at: the lane's own first element
    __device__ __forceinline__ void store(void* out, long long at) const {
        if constexpr (kWords == 4) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            uint32_t* p = static_cast<uint32_t*>(out) + at - 4 * (threadIdx.x & 1);
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
};

template <int kKind, int kOut, int D>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadArgs a) {
    constexpr int kLanes = D / kElems, kRowsPerStep = 32 / kLanes, kSteps = kBlock / kRowsPerStep;
    constexpr bool kCoded = kKind >= kReadI8;
    constexpr int kBits = Raw<kKind>::kBits;
    launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x / a.ctas_per_seq, part = blockIdx.x - b * a.ctas_per_seq;
    const long long row0 = a.token_start ? a.token_start[b] : (long long)b * a.max_tokens;
    const long long n = a.token_start ? (long long)a.token_start[b + 1] - row0 : a.max_tokens;
    if (n < 0 || n > a.max_tokens || row0 < 0 || row0 + n > a.total) {
        if (part == 0 && threadIdx.x == 0) flag_error(a.err, GQA_DEVERR_POSITION);
        return;
    }
    if (n == 0) return;                        // wherever it stands
    const long long pos0 = a.positions[b], end = pos0 + n;
    // pages (pos0 >> 4) .. (end - 1) >> 4 hold the rows; this CTA's are page0 ..
    const long long page0 = (pos0 >> 4) + (long long)part * a.pages_per_cta;
    const int pages = (int)min((long long)a.pages_per_cta, ((end + kBlock - 1) >> 4) - page0);
    const int tiles = pages * 2 * a.K;         // (page, K or V, kv-head), kv-heads adjacent
    const int lane = threadIdx.x & 31;
    const int e = lane % kLanes * kElems, slot0 = lane / kLanes;
    constexpr int kWarps = kReadThreads / 32;
    // tiles of a warp whose loads are on their way together: codes are few bytes a row
    constexpr int kTogether = kBits <= 8 ? 2 : 1;
    struct Tile {
        Raw<kKind> raw[kSteps];
        uint4 kc;                              // channel scales of this lane's elements
        float scale;                           // lane t: token t's
        int lo, hi;                            // slots [lo, hi) are asked for
        bool is_v;
        long long out0;                        // element of slot slot0's row
    };
    auto fetch = [&](int tile, Tile& x) {
        x.lo = x.hi = 0;
        if (tile >= tiles) return;
        const int side = tile / a.K, g = tile - side * a.K;
        x.is_v = side & 1;
        const long long page = page0 + (side >> 1);
        if (page < 0 || page >= a.max_blocks) {
            if (g == 0 && lane == 0) flag_error(a.err, GQA_DEVERR_POSITION);
            return;
        }
        const int ph = a.block_tables[(long long)b * a.max_blocks + page];
        if (ph < 0 || ph >= a.num_blocks) {
            if (g == 0 && lane == 0) flag_error(a.err, GQA_DEVERR_BLOCK_INDEX);
            return;
        }
        x.lo = (int)max(0ll, pos0 - page * kBlock);
        x.hi = (int)min((long long)kBlock, end - page * kBlock);
        const long long at = ph * a.sb + g * a.sh + slot0 * a.st + e;
        const uint8_t* src = static_cast<const uint8_t*>(x.is_v ? a.v : a.k) + at * kBits / 8;
        const long long step = kRowsPerStep * a.st * kBits / 8;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int slot = slot0 + i * kRowsPerStep;
            if (slot >= x.lo && slot < x.hi) x.raw[i].load(src + i * step);
        }
        if constexpr (kCoded) {
            const long long head = (long long)ph * a.K + g;
            if (kKind == kReadI4Kc && !x.is_v) x.kc = *reinterpret_cast<const uint4*>(a.k_scale + head * D + e);
            else if (lane < kBlock) x.scale = __half2float((x.is_v ? a.v_scale : a.k_scale)[head * kBlock + lane]);
        }
        // the row of slot s is row0 + 16 page + s - pos0
        x.out0 = ((row0 + page * kBlock - pos0 + slot0) * a.K + g) * D + e;
    };
    auto write = [&](const Tile& x) {
        if (x.hi <= x.lo) return;              // uniform
        void* out = x.is_v ? a.v_out : a.k_out;
        auto rows = [&](auto&& scaled) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int slot = slot0 + i * kRowsPerStep;
                float f[kElems];
                x.raw[i].values(f);
                scaled(f, i);
                const Out<kKind, kOut> o(x.raw[i], f);
                if (slot >= x.lo && slot < x.hi) o.store(out, x.out0 + (long long)i * kRowsPerStep * a.K * D);
            }
        };
        if constexpr (!kCoded) {
            rows([](float (&)[kElems], int) {});
        } else if (kKind == kReadI4Kc && !x.is_v) {
            float c[kElems];
            const uint32_t w[4] = {x.kc.x, x.kc.y, x.kc.z, x.kc.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 y = unpack2<false>(w[j]);
                c[2 * j] = y.x;
                c[2 * j + 1] = y.y;
            }
            rows([&](float (&f)[kElems], int) {
#pragma unroll
                for (int j = 0; j < kElems; ++j) f[j] *= c[j];
            });
        } else {
            rows([&](float (&f)[kElems], int i) {
                const float y = __shfl_sync(kFull, x.scale, slot0 + i * kRowsPerStep);
#pragma unroll
                for (int j = 0; j < kElems; ++j) f[j] *= y;
            });
        }
    };
    for (int tile = threadIdx.x >> 5; tile < tiles; tile += kWarps * kTogether) {
        Tile x[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) fetch(tile + i * kWarps, x[i]);
#pragma unroll
        for (int i = 0; i < kTogether; ++i) write(x[i]);
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
    // Four tiles a warp where that still gives every SM eight CTAs (two to three waves of them),
    // else fewer: a CTA first walks positions, table entry and data, one behind the other.
    const long long enough = 8LL * std::max(1, device_sms(-1));
    const long long pages = ((long long)max_tokens + 2 * kBlock - 2) / kBlock;   // an unaligned run touches one more
    a.pages_per_cta = std::max(1, 2 * kReadThreads / 32 / c.num_kv_heads);
    while (a.pages_per_cta > 1 && pages * batch < enough * a.pages_per_cta) a.pages_per_cta /= 2;
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
