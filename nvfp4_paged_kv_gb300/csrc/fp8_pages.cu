// Pages held as FP8 E4M3 with one FP32 scale for each page and KV head: from 16-bit pages, or from NVFP4 pages.
//
// Over the page's valid tokens, per KV head: a = max |x|, s = fp32(a / 448) (1 where that is below 2^-100), and every
// value becomes E4M3_rne_satfinite(fp32(x fp32(1 / s))); tokens past the valid ones become 0. Each (page, head) is one
// contiguous run of T x D values, so a CTA takes one run: it loads it once into registers (32 values a thread and
// step, two 16-value blocks), reduces the maximum through shared memory, and converts what it holds. A run of more than
// 32768 values is read twice instead, the second time out of L2.
//
// Bound: HBM, 3 bytes a value from 16 bits and 1.5625 from NVFP4. The maximum stands between the loads and the stores of a run,
// so a CTA alternates between the two; the 16 CTAs of an SM (128 threads at 64 x 128) are what keeps both under way.
#include <cstdint>
#include <cuda_runtime.h>

#include "codec_core.cuh"
#include "host_util.h"

using namespace nvfp4kv;

namespace {

constexpr int kKept = 2;           // steps of 32 values that a thread keeps in registers
constexpr int kMaxThreads = 512;   // of a CTA: runs of up to 512 x 2 x 32 values are read once
constexpr int kPairs = NVFP4KV_NVFP4 + 1;  // NVFP4 in NVFP4KV_PACK_TOKEN_PAIRS, as a source of its own

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
    int64_t units;
};

// Two blocks of 16 source values as loaded.
struct Raw {
    uint32_t w[16];
    uint32_t scales;
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

// Loads what of step i lies below block `end` (whole blocks); the rest reads as 0.
template <int SRC>
__device__ __forceinline__ Raw load_step(const uint8_t* src, const uint8_t* scales, uint32_t i, bool one, bool two) {
    Raw r;
#pragma unroll
    for (int k = 0; k < 16; ++k) r.w[k] = 0u;
    r.scales = 0u;
    if constexpr (SRC == NVFP4KV_BF16 || SRC == NVFP4KV_FP16) {
        const uint8_t* a = src + static_cast<size_t>(i) * 64;
        if (one) {
            const uint4 x = ld_stream_16B(a), y = ld_stream_16B(a + 16);
            r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
            r.w[4] = y.x; r.w[5] = y.y; r.w[6] = y.z; r.w[7] = y.w;
        }
        if (two) {
            const uint4 x = ld_stream_16B(a + 32), y = ld_stream_16B(a + 48);
            r.w[8] = x.x; r.w[9] = x.y; r.w[10] = x.z; r.w[11] = x.w;
            r.w[12] = y.x; r.w[13] = y.y; r.w[14] = y.z; r.w[15] = y.w;
        }
    } else if constexpr (SRC == NVFP4KV_NVFP4) {
        if (one) {
            const uint2 x = ld_stream_8B(src + static_cast<size_t>(i) * 16);
            r.w[0] = x.x; r.w[1] = x.y;
            r.scales = ld_stream_1B(scales + static_cast<size_t>(i) * 2);
        }
        if (two) {
            const uint2 x = ld_stream_8B(src + static_cast<size_t>(i) * 16 + 8);
            r.w[2] = x.x; r.w[3] = x.y;
            r.scales |= ld_stream_1B(scales + static_cast<size_t>(i) * 2 + 1) << 8;
        }
    } else if (one) {
        const uint4 x = ld_stream_16B(src + static_cast<size_t>(i) * 16);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
        r.scales = ld_stream_1B(scales + static_cast<size_t>(i) * 2);
        if (two) r.scales |= ld_stream_1B(scales + static_cast<size_t>(i) * 2 + 1) << 8;
    }
    return r;
}

// The 16 values of block `half` of a step, in FP32 (16-bit sources exactly, NVFP4 as fp32(v g)).
template <int SRC>
__device__ __forceinline__ void values_of(const Raw& r, int half, float g, float (&x)[16]) {
    if constexpr (SRC == NVFP4KV_BF16 || SRC == NVFP4KV_FP16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = r.w[8 * half + j];
            x[2 * j] = SRC == NVFP4KV_BF16 ? bf16_lo(w) : f16_lo(w);
            x[2 * j + 1] = SRC == NVFP4KV_BF16 ? bf16_hi(w) : f16_hi(w);
        }
    } else {
        uint2 code;
        if constexpr (SRC == NVFP4KV_NVFP4) {
            code = make_uint2(r.w[2 * half], r.w[2 * half + 1]);
        } else {  // a byte holds two tokens of one dim: this token's nibbles, two dims to a byte
            uint32_t n[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a = (r.w[2 * k] >> (4 * half)) & 0x0F0F0F0Fu, b = (r.w[2 * k + 1] >> (4 * half)) & 0x0F0F0F0Fu;
                const uint32_t lo = (a | (a >> 4)) & 0x00FF00FFu, hi = (b | (b >> 4)) & 0x00FF00FFu;
                n[k] = __byte_perm(lo, hi, 0x6420);
            }
            code = make_uint2(n[0], n[1]);
        }
        block_values(code, (r.scales >> (8 * half)) & 0xFFu, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = __fmul_rn(x[j], g);
    }
}

__device__ __forceinline__ void store_block(uint8_t* dst, uint32_t block, const float (&x)[16], float r) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = f32x2_to_e4m3x2(__fmul_rn(x[4 * j], r), __fmul_rn(x[4 * j + 1], r)) |
               f32x2_to_e4m3x2(__fmul_rn(x[4 * j + 2], r), __fmul_rn(x[4 * j + 3], r)) << 16;
    *reinterpret_cast<uint4*>(dst + static_cast<size_t>(block) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int SRC, bool KEPT>
__global__ void __launch_bounds__(kMaxThreads) fp8_pages_kernel(const Fp8Params p) {
    pdl_enter();
    __shared__ float most[2][kMaxThreads / 32];  // two sets: the next run's maxima do not wait for this one's readers
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const uint32_t blocks = static_cast<uint32_t>(p.T) * p.nb, steps = (blocks + 1) / 2;
    const float g = p.g ? __ldg(p.g) : 1.0f;
    int set = 0;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const int64_t i = u / p.H;
        const int h = static_cast<int>(u - i * p.H);
        const int from = p.src_ids ? __ldg(p.src_ids + i) : static_cast<int>(i);
        const int to = p.dst_ids ? __ldg(p.dst_ids + i) : static_cast<int>(i);
        const int tokens = p.tokens ? __ldg(p.tokens + i) : p.T;
        int32_t bad = 0;
        if (from < 0 || from >= p.src_pages || to < 0 || to >= p.dst_pages) bad |= NVFP4KV_STATUS_PAGE_OOB;
        if (tokens < 0 || tokens > p.T) bad |= NVFP4KV_STATUS_BAD_SEQ_LEN;
        if (bad) {  // the same for every thread of the CTA
            if (tid == 0 && h == 0 && !(from == -1 || to == -1)) flag_status(p.status, bad);
            continue;
        }
        const uint32_t end = static_cast<uint32_t>(tokens) * p.nb;  // blocks of valid tokens
        const int64_t run = static_cast<int64_t>(from) * p.H + h;
        constexpr int kBytes = SRC == NVFP4KV_BF16 || SRC == NVFP4KV_FP16 ? 32 : 8;  // of a block
        const uint8_t* src = p.src + run * blocks * kBytes;
        const uint8_t* scales = p.src_scales + run * blocks;
        uint8_t* dst = p.dst + (static_cast<int64_t>(to) * p.H + h) * blocks * 16;

        float a = 0.0f;
        auto take = [&](uint32_t j) {
            uint32_t b0, b1;
            blocks_of<SRC>(p, j, b0, b1);
            return load_step<SRC>(src, scales, j, b0 < end, b1 < end);
        };
        auto look = [&](const Raw& r, uint32_t j) {  // the maximum over the step's valid blocks
            uint32_t b0, b1;
            blocks_of<SRC>(p, j, b0, b1);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float x[16];
                values_of<SRC>(r, half, g, x);
                float m = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(x[k]));
                if ((half ? b1 : b0) < end) a = fmaxf(a, m);
            }
        };
        auto put = [&](const Raw& r, uint32_t j, float rs) {
            uint32_t b0, b1;
            blocks_of<SRC>(p, j, b0, b1);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint32_t b = half ? b1 : b0;
                float x[16];
                values_of<SRC>(r, half, g, x);
                if (b >= end)
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] = 0.0f;
                if (b < blocks) store_block(dst, b, x, rs);
            }
        };
        Raw kept[KEPT ? kKept : 1];
        if constexpr (KEPT) {
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                const uint32_t j = tid + k * blockDim.x;
                if (j < steps) kept[k] = take(j);
            }
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                const uint32_t j = tid + k * blockDim.x;
                if (j < steps) look(kept[k], j);
            }
        } else {
            for (uint32_t j = tid; j < steps; j += blockDim.x) look(take(j), j);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        if (warps > 1) {
            if (lane == 0) most[set][warp] = a;
            __syncthreads();
            for (int w = 0; w < warps; ++w) a = fmaxf(a, most[set][w]);
            set ^= 1;
        }
        float s = __fdiv_rn(a, 448.0f);
        if (s < 7.8886090522101181e-31f) s = 1.0f;  // 2^-100: all values become 0
        const float r = __frcp_rn(s);
        if (tid == 0) p.dst_scales[static_cast<int64_t>(to) * p.H + h] = s;
        if constexpr (KEPT) {
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                const uint32_t j = tid + k * blockDim.x;
                if (j < steps) put(kept[k], j, r);
            }
        } else {
            for (uint32_t j = tid; j < steps; j += blockDim.x) put(take(j), j, r);
        }
    }
}

template <int SRC>
cudaError_t launch_fp8(const Fp8Params& p, cudaStream_t s) {
    const int64_t steps = (static_cast<int64_t>(p.T) * p.nb + 1) / 2;
    int threads = 32;
    while (threads < kMaxThreads && static_cast<int64_t>(threads) * kKept < steps) threads *= 2;
    const bool kept = static_cast<int64_t>(threads) * kKept >= steps;
    // CTAs come and go: a run is short, and a CTA per run keeps an SM full without a tail of its own
    const int64_t most = (int64_t{1} << 31) - 1;
    const unsigned grid = static_cast<unsigned>(p.units < most ? p.units : most);
    return kept ? launch_pdl(fp8_pages_kernel<SRC, true>, dim3(grid), dim3(threads), 0, s, p)
                : launch_pdl(fp8_pages_kernel<SRC, false>, dim3(grid), dim3(threads), 0, s, p);
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
    // a run's blocks are numbered in 32 bits, and divided by nb with a multiply (fast_div)
    if (static_cast<int64_t>(layout->page_size) * nb > (1 << 24) || nb > (1 << 12)) return NVFP4KV_ERR_UNSUPPORTED;
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
    p.units = static_cast<int64_t>(num_pages) * p.H;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (pairs) return launched(launch_fp8<kPairs>(p, s));
    switch (src_dtype) {
    case NVFP4KV_BF16: return launched(launch_fp8<NVFP4KV_BF16>(p, s));
    case NVFP4KV_FP16: return launched(launch_fp8<NVFP4KV_FP16>(p, s));
    default: return launched(launch_fp8<NVFP4KV_NVFP4>(p, s));
    }
}
