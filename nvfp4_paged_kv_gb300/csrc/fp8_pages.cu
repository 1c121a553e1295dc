// Pages held as FP8 E4M3 with one FP32 scale for each page and KV head: from 16-bit pages, or from NVFP4 pages.
//
// Over the page's valid tokens, per KV head: a = max |x|, s = fp32(a / 448) (1 where that is below 2^-100), and every
// value becomes E4M3_rne_satfinite(fp32(x fp32(1 / s))); tokens past the valid ones become 0. Each (page, head) is one
// contiguous run of T x D values, so a CTA takes one run: it loads it once into registers (32 values a thread and
// step, two 16-value blocks), reduces the maximum through shared memory, and converts what it holds. A run of more than
// 32768 values is read twice instead, the second time out of L2. Maxima are taken over the bits of magnitudes, where NaN is above all
// else: NaN in a run makes its scale and its valid codes NaN, whatever the run's size.
//
// Bound: HBM, 3 bytes a value from 16 bits and 1.5625 from NVFP4. The maximum stands between the loads and the stores of a run,
// so a CTA alternates between the two; the CTAs of an SM (8 of 128 threads at 64 x 128) keep both under way. 4096 BF16 pages of
// 64 tokens, 8 heads, 128 dims (805 MB): 130 us, 6.2 TB/s, 0.91 of the copy rate. 1024 NVFP4 pages (105 MB): 24.0 us, 4.4 TB/s,
// 0.64 (in token pairs 30 us): 3 of it launch and the first loads, the rest 8.4 instructions a value and their waits (10.2 and 28 us
// with every value converted by itself; CTAs that go on to further runs, 2 us more, and load the next one ahead of the stores, the same).
#include <cstdint>
#include <type_traits>
#include <cuda_runtime.h>

#include "codec_core.cuh"
#include "host_util.h"

using namespace nvfp4kv;

namespace {

constexpr int kMaxThreads = 512;   // of a CTA: runs of up to 512 x 2 x 32 values are read once
constexpr int kPairs = NVFP4KV_NVFP4 + 1;  // NVFP4 in NVFP4KV_PACK_TOKEN_PAIRS, as a source of its own

constexpr int kKept = 2;           // steps of 32 values that a thread keeps in registers (of 1 to 4, 2 was the soonest for packed ones, by 0.1 to 1.3 us)

struct Fp8Params {
    const uint8_t* src;
    const uint8_t* src_scales;
    const float* g;
    const int32_t* src_ids;
    const int32_t* dst_ids;
    const int32_t* tokens;
    uint8_t* dst;
    float* dst_scales;
    int32_t* status;
    uint64_t row_magic;  // div_magic(D / 16)
    int32_t src_pages, dst_pages, H, T, nb;  // nb = D / 16
};

// Step i of a run covers blocks first and second (blocks of 16 values, numbered through the run).
template <int SRC>
__device__ __forceinline__ void blocks_of(const Fp8Params& p, uint32_t i, uint32_t& first, uint32_t& second) {
    if constexpr (SRC == kPairs) {  // one block of two tokens
        const uint32_t pair = fast_div(i, p.row_magic);
        first = 2 * pair * p.nb + (i - pair * p.nb);
        second = first + p.nb;
    } else {
        first = 2 * i;
        second = first + 1;
    }
}

// The two blocks of a step of a 16-bit source, as pairs of values.
struct Step {
    uint32_t w[16];
};

// A step of 16-bit values: what lies below the valid blocks' end (whole blocks, `one` and `two`); the rest is 0.
__device__ __forceinline__ void load_16bit(Step& s, const uint8_t* src, uint32_t i, bool one, bool two) {
    const uint8_t* a = src + static_cast<size_t>(i) * 64;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 v[4] = {zero, zero, zero, zero};
    if (one) {
        v[0] = ld_stream_16B(a);
        v[1] = ld_stream_16B(a + 16);
    }
    if (two) {
        v[2] = ld_stream_16B(a + 32);
        v[3] = ld_stream_16B(a + 48);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        s.w[4 * k] = v[k].x;
        s.w[4 * k + 1] = v[k].y;
        s.w[4 * k + 2] = v[k].z;
        s.w[4 * k + 3] = v[k].w;
    }
}

// The same of packed ones, as loaded.
struct Packed {
    uint4 codes;
    uint32_t scales;
};
template <int SRC>
__device__ __forceinline__ Packed load_packed(const uint8_t* src, const uint8_t* scales, uint32_t i, bool one, bool two, bool even) {
    Packed r{make_uint4(0u, 0u, 0u, 0u), 0u};
    const uint8_t* a = src + static_cast<size_t>(i) * 16;
    const uint8_t* sc = scales + static_cast<size_t>(i) * 2;
    if (SRC == kPairs || even) {  // 16 bytes of codes and 2 of scales, aligned (runs of an odd number of blocks are not)
        if (one) {
            r.codes = ld_stream_16B(a);
            uint16_t h;
            asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(sc));
            r.scales = h;
        }
        if (SRC == NVFP4KV_NVFP4 && !two) {  // (the second block may be past the valid ones, its scale anything)
            r.codes.z = r.codes.w = 0u;
            r.scales &= 0xFFu;
        }
    } else {
        if (one) {
            const uint2 x = ld_stream_8B(a);
            r.codes.x = x.x;
            r.codes.y = x.y;
            r.scales = ld_stream_1B(sc);
        }
        if (two) {
            const uint2 x = ld_stream_8B(a + 8);
            r.codes.z = x.x;
            r.codes.w = x.y;
            r.scales |= ld_stream_1B(sc + 1) << 8;
        }
    }
    return r;
}

// Two blocks of NVFP4 as codes, eight to a word in the order of the dims, and scales. (Token pairs: a byte holds two tokens of one
// dim, and a step is a block of each.)
struct Codes {
    uint32_t c[4];
    uint32_t scales;
};
template <int SRC>
__device__ __forceinline__ Codes unpack(const Packed& r, bool two) {
    Codes o{{r.codes.x, r.codes.y, r.codes.z, r.codes.w}, r.scales};
    if constexpr (SRC == kPairs) {
        const uint32_t w[4] = {r.codes.x, r.codes.y, r.codes.z, r.codes.w};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a = (w[2 * k] >> (4 * half)) & 0x0F0F0F0Fu, b = (w[2 * k + 1] >> (4 * half)) & 0x0F0F0F0Fu;
                const uint32_t lo = (a | (a >> 4)) & 0x00FF00FFu, hi = (b | (b >> 4)) & 0x00FF00FFu;
                o.c[2 * half + k] = half == 0 || two ? __byte_perm(lo, hi, 0x6420) : 0u;
            }
        if (!two) o.scales &= 0xFFu;
    }
    return o;
}

// Largest e2m1 * e4m3 magnitude of a block (exact), as bits.
__device__ __forceinline__ uint32_t largest(uint32_t c0, uint32_t c1, uint32_t scale) {
    uint32_t h[8];
    e2m1x8_to_f16x2x4(c0, *reinterpret_cast<uint32_t(*)[4]>(h));
    e2m1x8_to_f16x2x4(c1, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
    __half2 m = __habs2(*reinterpret_cast<const __half2*>(&h[0]));
#pragma unroll
    for (int k = 1; k < 8; ++k) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&h[k])));
    return __float_as_uint(fmaxf(__low2float(m), __high2float(m)) * e4m3_to_f32(scale & 0xFFu)) & 0x7FFFFFFFu;
}

// Largest magnitudes of a step's low and high halves: positive FP16 and BF16 values order as their bits do.
__device__ __forceinline__ uint32_t largest(const Step& s, uint32_t m) {
#pragma unroll
    for (int k = 0; k < 16; ++k) m = __vmaxu2(m, s.w[k] & 0x7FFF7FFFu);
    return m;
}

__device__ __forceinline__ void mul2(float& a, float& b, float c) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b) : "f"(c));
}

// FP8 codes of a block of 16-bit values.
template <int SRC>
__device__ __forceinline__ void store_16bit(uint8_t* dst, uint32_t block, const uint32_t* w, float r) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float x[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t v = w[2 * j + k];
            x[2 * k] = SRC == NVFP4KV_BF16 ? bf16_lo(v) : f16_lo(v);
            x[2 * k + 1] = SRC == NVFP4KV_BF16 ? bf16_hi(v) : f16_hi(v);
            mul2(x[2 * k], x[2 * k + 1], r);
        }
        o[j] = f32x2_to_e4m3x2(x[0], x[1]) | f32x2_to_e4m3x2(x[2], x[3]) << 16;
    }
    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(block) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
}

// FP8 codes of a block of NVFP4. A block has eight magnitudes, so their codes fp32(fp32(v g) r) are made once, and byte
// permutes look them up: an E2M1 code's low bits are the selector, its sign becomes the E4M3 sign. (Converting all 16 values
// took 10.2 instructions a value in all.)
__device__ __forceinline__ void store_packed(uint8_t* dst, uint32_t block, uint32_t c0, uint32_t c1, uint32_t scale, float g, float r) {
    const float sf = e4m3_to_f32(scale & 0xFFu);
    float x[8] = {0.0f, 0.5f * sf, sf, 1.5f * sf, 2.0f * sf, 3.0f * sf, 4.0f * sf, 6.0f * sf};  // exact
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        mul2(x[k], x[k + 1], g);
        mul2(x[k], x[k + 1], r);
    }
    const uint32_t lo = f32x2_to_e4m3x2(x[0], x[1]) | f32x2_to_e4m3x2(x[2], x[3]) << 16;
    const uint32_t hi = f32x2_to_e4m3x2(x[4], x[5]) | f32x2_to_e4m3x2(x[6], x[7]) << 16;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t c = (k < 2 ? c0 : c1) >> (16 * (k & 1));  // four codes
        o[k] = __byte_perm(lo, hi, c & 0x7777u) | __byte_perm(0x8000u, 0u, (c >> 3) & 0x1111u);
    }
    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(block) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int SRC, bool KEPT>
__global__ void __launch_bounds__(kMaxThreads) fp8_pages_kernel(const Fp8Params p) {
    pdl_enter();
    constexpr bool kPacked = SRC != NVFP4KV_BF16 && SRC != NVFP4KV_FP16;
    constexpr int N = KEPT ? kKept : 1;
    __shared__ uint32_t most[kMaxThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const uint32_t blocks = static_cast<uint32_t>(p.T) * p.nb, steps = (blocks + 1) / 2;
    const bool even = blocks % 2 == 0;
    const float g = p.g ? __ldg(p.g) : 1.0f;
    const uint32_t u = blockIdx.x;
    const uint32_t i = u / static_cast<uint32_t>(p.H);
    const int h = static_cast<int>(u - i * p.H);
    const int from = p.src_ids ? __ldg(p.src_ids + i) : static_cast<int>(i);
    const int to = p.dst_ids ? __ldg(p.dst_ids + i) : static_cast<int>(i);
    const int tokens = p.tokens ? __ldg(p.tokens + i) : p.T;
    int32_t bad = 0;
    if (from < 0 || from >= p.src_pages || to < 0 || to >= p.dst_pages) bad |= NVFP4KV_STATUS_PAGE_OOB;
    if (tokens < 0 || tokens > p.T) bad |= NVFP4KV_STATUS_BAD_SEQ_LEN;
    if (bad) {  // the same for every thread of the CTA
        if (tid == 0 && h == 0 && from != -1 && to != -1) flag_status(p.status, bad);
        return;
    }
    const uint32_t end = static_cast<uint32_t>(tokens) * p.nb;  // blocks of valid tokens
    const int64_t run = static_cast<int64_t>(from) * p.H + h, out = static_cast<int64_t>(to) * p.H + h;
    uint8_t* dst = p.dst + out * blocks * 16;

    // a step's values (16 bits) or codes
    using Held = std::conditional_t<kPacked, Packed, Step>;
    auto take = [&](Held& v, uint32_t j) {
        uint32_t b0, b1;
        blocks_of<SRC>(p, j, b0, b1);
        if constexpr (kPacked)
            v = load_packed<SRC>(p.src + run * blocks * 8, p.src_scales + run * blocks, j, b0 < end, b1 < end, even);
        else
            load_16bit(v, p.src + run * blocks * 32, j, b0 < end, b1 < end);
    };
    uint32_t bits = 0u;  // of 16-bit values: of the low and high halves; packed: of a float
    auto look = [&](const Held& v, uint32_t j) {
        if constexpr (kPacked) {
            uint32_t b0, b1;
            blocks_of<SRC>(p, j, b0, b1);
            const Codes c = unpack<SRC>(v, b1 < end);
            bits = max(bits, max(largest(c.c[0], c.c[1], c.scales), largest(c.c[2], c.c[3], c.scales >> 8)));
        } else {
            bits = largest(v, bits);
        }
    };
    auto put = [&](const Held& v, uint32_t j, float r) {
        uint32_t b0, b1;
        blocks_of<SRC>(p, j, b0, b1);
        if constexpr (kPacked) {
            const Codes c = unpack<SRC>(v, b1 < end);
            store_packed(dst, b0, c.c[0], c.c[1], c.scales, g, r);
            if (b1 < blocks) store_packed(dst, b1, c.c[2], c.c[3], c.scales >> 8, g, r);
        } else {
            store_16bit<SRC>(dst, b0, v.w, r);
            if (b1 < blocks) store_16bit<SRC>(dst, b1, v.w + 8, r);
        }
    };
    Held held[N];
    if constexpr (KEPT) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t j = tid + k * blockDim.x;
            if (j < steps) take(held[k], j);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t j = tid + k * blockDim.x;
            if (j < steps) look(held[k], j);
        }
    } else {
        for (uint32_t j = tid; j < steps; j += blockDim.x) {
            take(held[0], j);
            look(held[0], j);
        }
    }
    if constexpr (!kPacked) {
        bits = max(bits & 0xFFFFu, bits >> 16);
        bits = SRC == NVFP4KV_BF16 ? bits << 16 : __float_as_uint(f16_lo(bits)) & 0x7FFFFFFFu;
    }
    bits = __reduce_max_sync(0xFFFFFFFFu, bits);
    if (warps > 1) {
        if (lane == 0) most[warp] = bits;
        __syncthreads();
        for (int w = 0; w < warps; ++w) bits = max(bits, most[w]);
    }
    float a = __uint_as_float(bits);
    if constexpr (kPacked) a = __fmul_rn(a, fabsf(g));  // (the largest of fp32(|v| |g|))
    float s = __fdiv_rn(a, 448.0f);
    if (s < 7.8886090522101181e-31f) s = 1.0f;  // 2^-100: all values become 0
    const float r = __frcp_rn(s);
    if (tid == 0) p.dst_scales[out] = s;
    if (s != s) {
        for (uint32_t j = tid; j < blocks; j += blockDim.x) {
            const uint32_t w = j < end ? 0x7F7F7F7Fu : 0u;
            *reinterpret_cast<uint4*>(dst + static_cast<size_t>(j) * 16) = make_uint4(w, w, w, w);
        }
        return;
    }
    if constexpr (KEPT) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t j = tid + k * blockDim.x;
            if (j < steps) put(held[k], j, r);
        }
    } else {
        for (uint32_t j = tid; j < steps; j += blockDim.x) {
            take(held[0], j);
            put(held[0], j, r);
        }
    }
}

template <int SRC>
cudaError_t launch_fp8(const Fp8Params& p, uint32_t runs, cudaStream_t s) {
    const int64_t steps = (static_cast<int64_t>(p.T) * p.nb + 1) / 2;
    constexpr int N = kKept;
    int threads = 32;
    while (threads < kMaxThreads && static_cast<int64_t>(threads) * N < steps) threads *= 2;
    // a CTA for each run: runs are short, and CTAs that come and go keep an SM full without a tail of its own
    return static_cast<int64_t>(threads) * N >= steps ? launch_pdl(fp8_pages_kernel<SRC, true>, dim3(runs), dim3(threads), 0, s, p)
                                                      : launch_pdl(fp8_pages_kernel<SRC, false>, dim3(runs), dim3(threads), 0, s, p);
}

}  // namespace

extern "C" nvfp4kv_status nvfp4_kv_fp8_pages(
    const nvfp4kv_layout* layout, nvfp4kv_dtype src_dtype, const void* src, const uint8_t* src_scales,
    const float* src_global_scale, int32_t src_pool_pages, const int32_t* src_page_ids,
    const int32_t* page_tokens, uint8_t* dst, float* dst_scales, int32_t dst_pool_pages,
    const int32_t* dst_page_ids, int32_t num_pages, int32_t* status, nvfp4kv_stream_t stream) {
    const bool packed = src_dtype == NVFP4KV_NVFP4;
    if (!layout_ok(layout) || num_pages < 0 || (!packed && !dtype_ok(src_dtype))) return NVFP4KV_ERR_INVALID_ARG;
    const bool pairs = packed && layout->packing == NVFP4KV_PACK_TOKEN_PAIRS;
    if (packed && !pairs && layout->packing != NVFP4KV_PACK_DIM_PAIRS) return NVFP4KV_ERR_INVALID_ARG;
    if (pairs && layout->page_size % 2 != 0) return NVFP4KV_ERR_INVALID_ARG;
    if (src_dtype == NVFP4KV_FP8_E4M3) return NVFP4KV_ERR_UNSUPPORTED;
    if (num_pages == 0) return NVFP4KV_OK;
    if (!src || !dst || !dst_scales || src_pool_pages <= 0 || dst_pool_pages <= 0 || (packed && !src_scales))
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(src) || !aligned16(dst) || (packed && !aligned16(src_scales)) || src == dst)
        return NVFP4KV_ERR_INVALID_ARG;
    if ((!src_page_ids && num_pages > src_pool_pages) || (!dst_page_ids && num_pages > dst_pool_pages))
        return NVFP4KV_ERR_INVALID_ARG;
    const int nb = layout->head_dim / 16;
    // a run's blocks are numbered in 32 bits, and divided by nb with a multiply (fast_div); so are the runs
    if (static_cast<int64_t>(layout->page_size) * nb > (1 << 24) || nb > (1 << 12) ||
        static_cast<int64_t>(num_pages) * layout->num_kv_heads > (1 << 30))
        return NVFP4KV_ERR_UNSUPPORTED;
    Fp8Params p{};
    p.src = static_cast<const uint8_t*>(src);
    p.src_scales = packed ? src_scales : nullptr;
    p.g = packed ? src_global_scale : nullptr;
    p.src_ids = src_page_ids;
    p.dst_ids = dst_page_ids;
    p.tokens = page_tokens;
    p.dst = dst;
    p.dst_scales = dst_scales;
    p.status = status;
    p.row_magic = div_magic(static_cast<uint32_t>(nb));
    p.src_pages = src_pool_pages;
    p.dst_pages = dst_pool_pages;
    p.H = layout->num_kv_heads;
    p.T = layout->page_size;
    p.nb = nb;
    const uint32_t runs = static_cast<uint32_t>(num_pages) * p.H;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (pairs) return launched(launch_fp8<kPairs>(p, runs, s));
    switch (src_dtype) {
    case NVFP4KV_BF16: return launched(launch_fp8<NVFP4KV_BF16>(p, runs, s));
    case NVFP4KV_FP16: return launched(launch_fp8<NVFP4KV_FP16>(p, runs, s));
    default: return launched(launch_fp8<NVFP4KV_NVFP4>(p, runs, s));
    }
}
