// Page bounds and page selection of the sparse decode, for sm_103a.
//
// Bounds. For every (page, KV head), the largest and smallest value of each head dim over the
// page's tokens, as int8 steps of one FP32 scale: with v = e2m1 * e4m3 (exact in FP16),
//   a = max_d max(|max_t v|, |min_t v|),  s = fp32(a / 127),
//   hi_d = min(127, ceil(fp32(max_t v / s))),  lo_d = max(-127, floor(fp32(min_t v / s))),
// all 0 when a is 0. Rounding away from the interval keeps  lo_d s <= v <= hi_d s  (up to the two
// FP32 roundings), so the product of any vector with the nearer bound of each dim is at least its
// product with any key of the page.
//
// Scores and selection. The queries of a KV head's group are brought to integers of 9 bits,
//   q_i = rint(fp32(q / f)),  f = fp32(max|q| / 255)   (0 when max|q| is 0 or not finite),
// and the score of a page is the largest over the group of
//   fp32(fp32(S f) s),  S = sum_d (q_d > 0 ? q_d hi_d : q_d lo_d).
// This bounds the product of the rounded query f q_i; that of the query itself may be larger by up to
// f/2 sum_d max(|hi_d|, |lo_d|) s.
// S is an integer below 2^23 in magnitude, exact in FP32 in every order of summation, so the
// selection is the same bit for bit whatever the split of the work: the reason for integer bounds
// and integer queries, which also halve the bytes of 16-bit bounds.
//
// Bounds kernel: 4096 pages of 64 tokens x 8 heads x 128 (160 MB) take 37.0 us, 4.3 TB/s, bound by the
// conversions of two codes each, the products and the maxima: without any one of the three kinds it would be
// 2 to 3 us less (with the walk's 64-bit divisions and a ceil by conversions it was 38.9). Halves as large in
// flight for 32 warps an SM took 39 to 40, three slots 40, a grid of one wave 39.3. A chunk is copied whole as far
// as the page goes, whatever page_tokens says (one of few tokens costs the bytes of a chunk); what lies past the
// tokens is not looked at.
// Selection kernel: its bytes are few (2 D + 4 per scored page and head) and its time is latency: 256 pairs of 128
// pages (9 MB) 6.0 us, 64 pairs of up to 2048 pages (22 MB) 12.5 us, of which 2 us until the queries are integers,
// 3 to 5 us of scores, 3 us of radix passes and 1.5 us of writing the tables.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "codec_core.cuh"
#include "common.cuh"
#include "host_util.h"

namespace cg = cooperative_groups;

namespace nvfp4kv {
namespace {

// 16 bytes of a lane, 512 K bytes (K whole warps) behind both addresses.
template <int K>
__device__ __forceinline__ void cp_async_512(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%2], 16;" ::"r"(dst), "l"(src), "n"(512 * K) : "memory");
}
__device__ __forceinline__ void cp_async_commit_group() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
    uint32_t o;
    asm("max.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}
__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b) {
    uint32_t o;
    asm("min.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}

// ------------------------------------------------------------------------------------------
// Page bounds. One warp per (page, head), in chunks of 4608 bytes (128, 64 or 32 tokens of head_dim
// 64, 128 or 256) that it copies ahead into a ring of two shared-memory slots, so that the next
// chunk or page is on its way while this one is reduced. A lane owns 32 dims (16 code bytes) of every
// (32 / (D / 32))-th token and keeps the maxima and minima of its dims in FP16 pairs; the lanes that
// hold the same dims then exchange halves of what they have (a reduce-scatter), so each ends with a
// few finished dims to round and store.
// ------------------------------------------------------------------------------------------
constexpr int kBoundsThreads = 128;
constexpr int kBoundsChunk = 4608;  // bytes of a slot: codes, then scales

struct BoundsParams {
    const uint8_t* kd;
    const uint8_t* ks;
    const int32_t* page_ids;     // null: 0 .. num_pages-1
    const int32_t* page_tokens;  // null: T
    int8_t* bounds;
    float* scales;
    int32_t* status;
    int32_t pool_pages, num_pages, H, T;
};

// Maxima over the lanes that differ in the bits OFF, OFF / 2, .. LAST: with each bit a lane gives half of
// its CNT pairs away and keeps the other half, in m[0 ..]. Returns where the kept pairs began in m.
template <int CNT, int OFF, int LAST>
__device__ __forceinline__ int reduce_scatter(uint32_t (&m)[32], int lane) {
    if constexpr (OFF >= LAST) {
        constexpr int half = CNT / 2;
        const bool up = (lane & OFF) != 0;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const uint32_t give = up ? m[k] : m[k + half];
            const uint32_t keep = up ? m[k + half] : m[k];
            m[k] = max_f16x2(keep, __shfl_xor_sync(0xFFFFFFFFu, give, OFF));
        }
        return (up ? half : 0) + reduce_scatter<half, OFF / 2, LAST>(m, lane);
    } else {
        return 0;
    }
}

template <int D>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const BoundsParams p) {
    pdl_enter();
    constexpr int LPR = D / 32;    // lanes of a token row
    constexpr int RPP = 32 / LPR;  // token rows of a pass
    constexpr int NB = D / 16;
    constexpr int KEEP = 32 / RPP; // FP16 pairs a lane ends with
    constexpr int CH = 8 * RPP;    // token rows of a chunk
    static_assert(CH * (D / 2 + NB) == kBoundsChunk, "chunk size");
    __shared__ __align__(16) uint8_t ring[kBoundsThreads / 32][2][kBoundsChunk];
    const int lane = threadIdx.x & 31;
    const int l = lane % LPR, rr = lane / LPR;
    uint8_t(*slots)[kBoundsChunk] = ring[threadIdx.x >> 5];

    // the walk over the warp's chunks, one ahead of the reduction; the ids of the item after are
    // loaded while an item is walked. An item is a place in the list and a head, kept apart: one 64-bit
    // division for each item's place would cost as much as a quarter of its values
    const uint32_t H = static_cast<uint32_t>(p.H);
    const uint32_t first = blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
    const uint32_t step = gridDim.x * (kBoundsThreads / 32), step_i = step / H, step_h = step % H;
    uint32_t next_i = first / H, next_h = first % H;  // of the item after
    int id_page = -1, id_n = 0;
    int64_t ph = 0;                    // page * H + head of the item
    int n = 0, t0 = 0;                 // its tokens, first token of the chunk
    auto load_ids = [&]() {
        if (next_i >= static_cast<uint32_t>(p.num_pages)) return;
        id_page = p.page_ids ? __ldg(p.page_ids + next_i) : static_cast<int>(next_i);
        id_n = p.page_tokens ? __ldg(p.page_tokens + next_i) : p.T;
    };
    load_ids();
    auto advance = [&]() -> bool {  // to the next chunk; false: none left
        if (n - t0 > CH) {
            t0 += CH;
            return true;
        }
        for (;;) {
            if (next_i >= static_cast<uint32_t>(p.num_pages)) return false;
            const int page = id_page;
            const uint32_t head = next_h;
            n = id_n;
            next_i += step_i;
            next_h += step_h;
            if (next_h >= H) {
                next_h -= H;
                ++next_i;
            }
            load_ids();
            if (page == -1) continue;
            if (page < 0 || page >= p.pool_pages || n < 0 || n > p.T) {
                if (lane == 0)
                    flag_status(p.status, (page < 0 || page >= p.pool_pages) ? NVFP4KV_STATUS_PAGE_OOB
                                                                             : NVFP4KV_STATUS_BAD_SEQ_LEN);
                continue;
            }
            ph = static_cast<int64_t>(page) * p.H + head;
            t0 = 0;
            return true;
        }
    };
    // rows [t0, t0 + CH) of the page, as far as it has them
    auto copy = [&](uint8_t* slot) {
        const int rows = min(CH, p.T - t0);
        const int64_t r0 = ph * p.T + t0;
        const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(slot)) + 16 * lane;
        const uint8_t* codes = p.kd + r0 * (D / 2) + 16 * lane;
        const uint8_t* scales = p.ks + r0 * NB + 16 * lane;
        if (rows == CH) {
            cp_async_512<0>(dst, codes);
            cp_async_512<1>(dst, codes);
            cp_async_512<2>(dst, codes);
            cp_async_512<3>(dst, codes);
            cp_async_512<4>(dst, codes);
            cp_async_512<5>(dst, codes);
            cp_async_512<6>(dst, codes);
            cp_async_512<7>(dst, codes);
            cp_async_512<0>(dst + CH * (D / 2), scales);
        } else {
#pragma unroll 1
            for (int k = 0; 32 * k + lane < rows * (D / 32); ++k) cp_async_512<0>(dst + 512 * k, codes + 512 * k);
            if (16 * lane < rows * NB) cp_async_512<0>(dst + CH * (D / 2), scales);
        }
    };

    bool more = advance();
    if (more) copy(slots[0]);
    cp_async_commit_group();
    // maxima of dims (2j, 2j+1) in m[j], minima in m[16 + j]
    uint32_t m[32];
    for (int turn = 0; more; turn ^= 1) {
        const int64_t my_ph = ph;
        const int my_n = n, my_t0 = t0;
        more = advance();
        if (more) copy(slots[turn ^ 1]);
        cp_async_commit_group();
        cp_async_wait_group<1>();
        __syncwarp();
        if (my_t0 == 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) m[j] = j < 16 ? 0xFC00FC00u : 0x7C007C00u;
        }
        const uint8_t* codes = slots[turn] + 16 * l;
        const uint8_t* scales = slots[turn] + CH * (D / 2) + 2 * l;
        const int rows = min(CH, my_n - my_t0);
        // passes two at a time, so that their values meet in one three-way maximum; a row past the end
        // repeats the last one
        for (int r0 = rr; r0 - rr < rows; r0 += 2 * RPP) {
            uint4 w[2];
            uint32_t sa[2], sb[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = min(r0 + k * RPP, rows - 1);
                w[k] = *reinterpret_cast<const uint4*>(codes + t * (D / 2));
                const uint32_t sc = *reinterpret_cast<const uint16_t*>(scales + t * NB);
                sa[k] = e4m3x2_to_f16x2(__byte_perm(sc, 0u, 0x0000));
                sb[k] = e4m3x2_to_f16x2(__byte_perm(sc, 0u, 0x1111));
            }
            const uint32_t ww[2][4] = {{w[0].x, w[0].y, w[0].z, w[0].w}, {w[1].x, w[1].y, w[1].z, w[1].w}};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t v0[4], v1[4];
                e2m1x8_to_f16x2x4(ww[0][e], v0);
                e2m1x8_to_f16x2x4(ww[1][e], v1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x0 = hmul2_u32(v0[j], e < 2 ? sa[0] : sb[0]);
                    const uint32_t x1 = hmul2_u32(v1[j], e < 2 ? sa[1] : sb[1]);
                    m[4 * e + j] = max_f16x2(max_f16x2(m[4 * e + j], x0), x1);
                    m[16 + 4 * e + j] = min_f16x2(min_f16x2(m[16 + 4 * e + j], x0), x1);
                }
            }
        }
        __syncwarp();  // every lane is done with the slot before it refills
        if (my_n - my_t0 > CH) continue;
        // from here on the negated minima, so that both halves are maxima
#pragma unroll
        for (int j = 16; j < 32; ++j) m[j] ^= 0x80008000u;
        const int base = reduce_scatter<32, 16, LPR>(m, lane);
        float a = 0.0f;
        float y[2 * KEEP];
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            y[2 * k] = my_n > 0 ? f16_lo(m[k]) : 0.0f;
            y[2 * k + 1] = my_n > 0 ? f16_hi(m[k]) : 0.0f;
            a = fmaxf(a, fmaxf(fabsf(y[2 * k]), fabsf(y[2 * k + 1])));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
        const float s = __fdiv_rn(a, 127.0f);
        if (lane == 0) p.scales[my_ph] = s;
        const bool neg = base >= 16;
        uint32_t w[(2 * KEEP + 3) / 4];
#pragma unroll
        for (int k = 0; k < (2 * KEEP + 3) / 4; ++k) w[k] = 0u;
        // ceil(fp32(y / s)) by a product with 1 / s, off by less than 2^-15 at 127, as the whole number next to
        // x + 1/2; where x is next to a whole number itself by the division, but for those past 126, which end
        // at 127 either way (the largest value of the page always lies there). A non-zero s is at least 2^-17
        // (a at least 2^-10), so 1 / s is finite. Sums with 1.5 2^23 leave the whole number in the low bits
        const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
        const float sign = neg ? -1.0f : 1.0f;  // floor of a negated value is the negated ceil
        constexpr float kWhole = 12582912.0f;
        bool open = false;
#pragma unroll
        for (int k = 0; k < 2 * KEEP; ++k) {
            const float u = fminf(fmaf(y[k], inv, 0.5f), 127.4f);
            const float t = fmaf(u, sign, kWhole);
            const float d = fmaf(-sign, t - kWhole, u);
            open = open || (fabsf(d) > 0.4999f && y[k] != 0.0f);
            w[k / 4] = __byte_perm(w[k / 4], __float_as_uint(t), k % 4 == 0 ? 0x3214 : k % 4 == 1 ? 0x3240
                                                                 : k % 4 == 2 ? 0x3410 : 0x4210);
        }
        if (open) {
#pragma unroll
            for (int k = 0; k < (2 * KEEP + 3) / 4; ++k) w[k] = 0u;
#pragma unroll
            for (int k = 0; k < 2 * KEEP; ++k) {
                const int c = static_cast<int>(fminf(127.0f, ceilf(__fdiv_rn(y[k], s))));
                w[k / 4] |= static_cast<uint32_t>((neg ? -c : c) & 0xFF) << (8 * (k % 4));
            }
        }
        int8_t* dst = p.bounds + (my_ph * 2 + (neg ? 1 : 0)) * D + 32 * l + 2 * (base & 15);
        if constexpr (KEEP == 2) {
            *reinterpret_cast<uint32_t*>(dst) = w[0];
        } else if constexpr (KEEP == 4) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        } else {
            *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ------------------------------------------------------------------------------------------
// Selection. One thread-block cluster per (sequence, KV head) pair. Its warps score tiles of 16
// pages on the tensor cores (FP16, whose mma.sync runs 8 times as often per clock as the int8 one on
// this GPU; pages as M, the query group as N, head dims as K, once with the upper bounds and the
// positive queries, once with the lower and the negative) and put the scores as sortable keys into the
// shared memory of the cluster's first CTA, which then finds the smallest selected key by a radix selection
// that starts at the highest bit in which the keys differ and stops when a bin is taken whole. (Counting ranks
// was no faster for few pages, 6.1 against 6.0 us for 256 pairs of 128, nor among the keys of the last bin, 12.9
// against 12.3 us for 64 pairs of up to 2048: code that runs once costs its fetch.) The selected pages are written
// in ascending order, equal keys from the lowest page on.
// ------------------------------------------------------------------------------------------
constexpr int kSelMaxGroup = 8;
constexpr int kSelMaxCluster = 8;
constexpr int kSelMaxPages = 49152;  // keys of a pair: 192 KiB of shared memory
constexpr int kSelBins = 1024;

struct SelectParams {
    const uint16_t* q;
    const int8_t* bounds;
    const float* bscales;
    const int32_t* page_table;
    const int32_t* seq_lens;
    int32_t* sel_table;
    int32_t* sel_lens;
    int32_t* sel_index;  // or null
    float* scores;       // or null
    int32_t* status;
    int32_t B, H, G, T, pool_pages, max_pages, budget, sink, recent;
};

// Order-preserving map of a score to a key above 0; NaN (a page whose bounds were never written) below
// everything, 0 and -0 equal.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (!(x == x)) return 1u;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The four int8 of w plus 128, as FP16 pairs of the value times 2^-24: a byte in the low half of an
// FP16 mantissa is that subnormal, and the tensor cores take subnormals exactly.
__device__ __forceinline__ void s8x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = w ^ 0x80808080u;
    lo = __byte_perm(x, 0u, 0x4140);
    hi = __byte_perm(x, 0u, 0x4342);
}

// What the kernel has to know of one radix pass: the bin that holds the wanted key, how many keys
// are wanted from it and how many it has.
struct RadixBin {
    uint32_t bin, want, have;
};

// Inclusive sum over the CTA's threads (every thread calls); sums: one word per warp.
template <int NT>
__device__ __forceinline__ uint32_t cta_inclusive(uint32_t v, uint32_t* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sums[warp] = v;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NT / 32; ++k)
        if (k < warp) v += sums[k];
    return v;
}

template <int D, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) select_pages_kernel(const SelectParams p) {
    pdl_enter();
    constexpr int NW = NT / 32;
    constexpr int QROW = D + 8;  // FP16 of a query row in shared memory
    extern __shared__ __align__(16) uint32_t keys[];  // [max_pages rounded up to 32], then two masks of as many bits
    __shared__ __align__(16) uint32_t hist[kSelBins];
    __shared__ __align__(16) uint16_t q_s[kSelMaxGroup * QROW];
    __shared__ float f_s[kSelMaxGroup];   // step of each head's integers
    __shared__ float bias_s[kSelMaxGroup];  // 128 times their sum
    __shared__ uint32_t sums[2][NW];
    __shared__ RadixBin found;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    if (C > 1) cluster.barrier_arrive();  // waited for before the first remote store
    const int pair = blockIdx.x / C;
    const int b = pair / p.H, h = pair - b * p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;

    // loads that do not wait for one another: the length, the first page ids, the queries (a warp per
    // head of the group)
    const int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    auto id_at = [&](int i) { return i < p.max_pages ? __ldg(row + i) : -1; };
    const int first = (rank * NW + warp) * 16, stride = C * NW * 16;
    int id0 = id_at(first + r), id1 = id_at(first + r + 8);
    const int len = __ldg(p.seq_lens + b);
    uint32_t qw[D / 64];  // BF16 pairs: dims [lane D/32, lane D/32 + D/32) of head `warp`
    if (warp < p.G) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<int64_t>(pair) * p.G + warp) * D) + lane * (D / 64);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) qw[k] = __ldg(src + k);
    }

    const bool len_ok = len >= 0 && len <= static_cast<int64_t>(p.max_pages) * p.T;
    if (!len_ok && h == 0 && rank == 0 && tid == 0) flag_status(p.status, NVFP4KV_STATUS_BAD_SEQ_LEN);
    const int n = len_ok ? static_cast<int>((static_cast<int64_t>(len) + p.T - 1) / p.T) : 0;
    const int count = min(n, p.budget);
    const bool choose = n > p.budget;
    int32_t* out_table = p.sel_table + static_cast<int64_t>(pair) * p.budget;
    int32_t* out_index = p.sel_index ? p.sel_index + static_cast<int64_t>(pair) * p.budget : nullptr;

    if (choose || p.scores) {
        // tiles of 16 pages; lane (r, c) holds quarter c of the bounds of pages r and r + 8
        struct Tile {
            uint32_t hi0[D / 16], hi1[D / 16], lo0[D / 16], lo1[D / 16];
            float s0, s1;
            int a0, a1;  // page ids; -1: not scored, -2: outside the pool
        };
        auto load_ids = [&](int t, Tile& x) {  // those of tile t, loaded before; leaves the next one's
            auto checked = [&](int i, int id) {
                if (i >= n || i < p.sink || i >= n - p.recent) return -1;
                return id >= 0 && id < p.pool_pages ? id : -2;
            };
            x.a0 = checked(t + r, id0);
            x.a1 = checked(t + r + 8, id1);
            x.s0 = x.a0 >= 0 ? __ldg(p.bscales + static_cast<int64_t>(x.a0) * p.H + h) : 0.0f;
            x.s1 = x.a1 >= 0 ? __ldg(p.bscales + static_cast<int64_t>(x.a1) * p.H + h) : 0.0f;
            id0 = id_at(t + r + stride);
            id1 = id_at(t + r + 8 + stride);
        };
        // the upper (half 0) or lower (1) bounds of a page
        auto fetch = [&](int id, int half, uint32_t(&w)[D / 16]) {
            const uint4* src = reinterpret_cast<const uint4*>(
                p.bounds + ((static_cast<int64_t>(max(id, 0)) * p.H + h) * 2 + half) * D + c * (D / 4));
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                const uint4 v = id >= 0 ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
                w[4 * k] = v.x;
                w[4 * k + 1] = v.y;
                w[4 * k + 2] = v.z;
                w[4 * k + 3] = v.w;
            }
        };
        auto load_tile = [&](int t, Tile& x) {
            load_ids(t, x);
            fetch(x.a0, 0, x.hi0);
            fetch(x.a1, 0, x.hi1);
            fetch(x.a0, 1, x.lo0);
            fetch(x.a1, 1, x.lo1);
        };
        Tile cur;
        if (first < n) load_tile(first, cur);

        // ---- the group's queries as integers, exact in FP16
        for (int g = warp; g < kSelMaxGroup; g += NW) {  // (one round: there are at least 8 warps)
            float amax = 0.0f, x[D / 32];
            bool finite = true;
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                x[2 * k] = g < p.G ? bf16_lo(qw[k]) : 0.0f;
                x[2 * k + 1] = g < p.G ? bf16_hi(qw[k]) : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                finite = finite && fabsf(x[k]) < INFINITY;
                amax = fmaxf(amax, fabsf(x[k]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            const float f = __all_sync(0xFFFFFFFFu, finite) ? __fdiv_rn(amax, 255.0f) : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                x[k] = f > 0.0f ? rintf(__fdiv_rn(x[k], f)) : 0.0f;
                sum += x[k];
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            uint32_t* dst = reinterpret_cast<uint32_t*>(q_s + g * QROW + lane * (D / 32));
#pragma unroll
            for (int k = 0; k < D / 64; ++k) dst[k] = pack_f16x2(x[2 * k], x[2 * k + 1]);
            if (lane == 0) {
                f_s[g] = f;
                bias_s[g] = 128.0f * sum;
            }
        }
        __syncthreads();
        uint32_t q[D / 8];  // head r, dims [c D/4, c D/4 + D/4), which meet the same quarter of the bounds
        {
            const uint4* src = reinterpret_cast<const uint4*>(q_s + r * QROW + c * (D / 4));
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const uint4 v = src[k];
                q[4 * k] = v.x;
                q[4 * k + 1] = v.y;
                q[4 * k + 2] = v.z;
                q[4 * k + 3] = v.w;
            }
        }
        const float f0 = f_s[2 * c], f1 = f_s[2 * c + 1];
        const float bias0 = bias_s[2 * c], bias1 = bias_s[2 * c + 1];
        const bool has0 = 2 * c < p.G, has1 = 2 * c + 1 < p.G;
        uint32_t* pair_keys = keys;
        if (C > 1) {
            cluster.barrier_wait();
            pair_keys = cluster.map_shared_rank(keys, 0);
        }

        auto multiply = [](float(&sum)[4], uint32_t w0, uint32_t w1, uint32_t b0, uint32_t b1) {
            uint32_t a[4];
            s8x4_to_f16x2x2(w0, a[0], a[2]);
            s8x4_to_f16x2x2(w1, a[1], a[3]);
            mma_f16_16816(sum, a, b0, b1);
        };
        for (int t = first; t < n; t += stride) {
            Tile next;
            const bool more = t + stride < n;
            if constexpr (D <= 128) {
                if (more) load_tile(t + stride, next);
            } else {
                if (more) load_ids(t + stride, next);
            }
            // the positive parts of the queries meet the upper bounds, the negative the lower
            float up[4] = {0.0f, 0.0f, 0.0f, 0.0f}, down[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (D <= 128) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    multiply(up, cur.hi0[k], cur.hi1[k], max_f16x2(q[2 * k], 0u), max_f16x2(q[2 * k + 1], 0u));
                    multiply(down, cur.lo0[k], cur.lo1[k], min_f16x2(q[2 * k], 0u), min_f16x2(q[2 * k + 1], 0u));
                }
            } else {
                // at 256 the registers hold one tile, and each half of it makes room for the next one's (128 pairs
                // of 512 pages 12.8 us; with the next tile loaded after this one 14.7)
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    multiply(up, cur.hi0[k], cur.hi1[k], max_f16x2(q[2 * k], 0u), max_f16x2(q[2 * k + 1], 0u));
                if (more) {
                    fetch(next.a0, 0, cur.hi0);
                    fetch(next.a1, 0, cur.hi1);
                }
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    multiply(down, cur.lo0[k], cur.lo1[k], min_f16x2(q[2 * k], 0u), min_f16x2(q[2 * k + 1], 0u));
                if (more) {
                    fetch(next.a0, 1, cur.lo0);
                    fetch(next.a1, 1, cur.lo1);
                }
            }
            auto score = [&](float x0, float x1, float s) {
                float v = -INFINITY;
                if (has0) v = __fmul_rn(__fmul_rn(x0 * 16777216.0f - bias0, f0), s);
                if (has1) v = fmaxf(v, __fmul_rn(__fmul_rn(x1 * 16777216.0f - bias1, f1), s));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
            };
            const float v0 = score(up[0] + down[0], up[1] + down[1], cur.s0);
            const float v1 = score(up[2] + down[2], up[3] + down[3], cur.s1);
            if (c < 2) {
                const int i = t + r + 8 * c, id = c == 0 ? cur.a0 : cur.a1;
                float v = c == 0 ? v0 : v1;
                if (i < n) {
                    if (id == -1) v = INFINITY;
                    if (id == -2) {
                        v = -INFINITY;
                        flag_status(p.status, NVFP4KV_STATUS_PAGE_OOB);
                    }
                    if (choose) pair_keys[i] = id == -1 ? 0u : key_of(v);
                    if (p.scores) p.scores[static_cast<int64_t>(pair) * p.max_pages + i] = v;
                }
            }
            if constexpr (D <= 128) {
                cur = next;
            } else {
                cur.a0 = next.a0;
                cur.a1 = next.a1;
                cur.s0 = next.s0;
                cur.s1 = next.s1;
            }
        }
    } else if (C > 1) {
        cluster.barrier_wait();
    }

    if (choose) {  // (the same for all CTAs of the cluster) until every CTA's keys are written
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
    }
    if (rank != 0) return;
    for (int i = count + tid; i < p.budget; i += NT) {
        out_table[i] = -1;
        if (out_index) out_index[i] = -1;
    }
    // the last page is always taken, and it alone can be cut short
    if (tid == 0) p.sel_lens[pair] = n > 0 ? (count - 1) * p.T + (len - (n - 1) * p.T) : 0;
    if (!choose) {  // every page is taken
        for (int i = tid; i < n; i += NT) {
            out_table[i] = __ldg(row + i);
            if (out_index) out_index[i] = i;
        }
        return;
    }

    // ---- the always-taken pages are [0, lo) and [hi, n); `want` of the keys in [lo, hi) are taken:
    // those above `above`, and the first `equal` of those equal to it
    const int lo = p.sink, hi = n - p.recent;
    uint32_t want = static_cast<uint32_t>(count - p.sink - p.recent);
    uint32_t above = 0xFFFFFFFFu, equal = 0u;
    if (want > 0) {
        uint32_t top = 0u, low = 0xFFFFFFFFu;
        for (int i = lo + tid; i < hi; i += NT) {
            const uint32_t k = keys[i];
            top = max(top, k);
            low = min(low, k);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        low = __reduce_min_sync(0xFFFFFFFFu, low);
        if (lane == 0) {
            sums[0][warp] = top;
            sums[1][warp] = low;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            top = max(top, sums[0][k]);
            low = min(low, sums[1][k]);
        }
        // keys agree above bit `bits`; a pass looks at the next 10 bits below
        int bits = 32 - __clz(top ^ low);
        uint32_t prefix = bits < 32 ? (top >> bits) << bits : 0u;
        bool whole_bin = false;
        while (bits > 0) {
            const int shift = max(0, bits - 10);
            const uint32_t mask = bits < 32 ? ~((1u << bits) - 1u) : 0u;
#pragma unroll
            for (int i = 0; i < kSelBins / NT; ++i) hist[tid + i * NT] = 0u;
            __syncthreads();
#pragma unroll 1
            for (int i = lo + tid; i < hi; i += NT) {
                const uint32_t k = keys[i];
                if ((k & mask) == prefix) atomicAdd(&hist[(k & ~mask) >> shift], 1u);
            }
            __syncthreads();
            // thread t sums the bins below 1024 - PER t, from the top
            constexpr int PER = kSelBins / NT;
            const int b0 = kSelBins - PER - PER * tid;
            uint32_t mine = 0u;
#pragma unroll
            for (int k = 0; k < PER; ++k) mine += hist[b0 + k];
            uint32_t at = cta_inclusive<NT>(mine, sums[0]) - mine;
            if (at < want && want <= at + mine) {
#pragma unroll
                for (int k = PER - 1; k >= 0; --k) {
                    const uint32_t have = hist[b0 + k];
                    if (at < want && want <= at + have)
                        found = RadixBin{static_cast<uint32_t>(b0 + k), want - at, have};
                    at += have;
                }
            }
            __syncthreads();
            prefix |= found.bin << shift;
            want = found.want;
            bits = shift;
            whole_bin = found.have == want;
            if (whole_bin) break;
        }
        // a bin taken whole: every key from its lowest on (0 cannot be, it would be all the keys)
        above = whole_bin ? prefix - 1u : prefix;
        equal = whole_bin ? 0u : want;
    }

    // ---- the selected pages in ascending order: a warp takes consecutive keys, 32 at a time, and
    // leaves one mask of those above the threshold and one of those at it
    const int words = (n + 31) >> 5;
    uint32_t* over = keys + ((p.max_pages + 31) & ~31);
    uint32_t* same = over + ((p.max_pages + 31) >> 5);
    const int share = (words + NW - 1) / NW;
    const int w0 = min(words, warp * share), w1 = min(words, w0 + share);
    uint32_t bo = 0u, bs = 0u;
#pragma unroll 4
    for (int w = w0; w < w1; ++w) {
        const int i = 32 * w + lane;
        const bool forced = i < lo || i >= hi;
        const uint32_t k = i < n ? keys[i] : 0u;
        const uint32_t mo = __ballot_sync(0xFFFFFFFFu, i < n && (forced || k > above));
        const uint32_t ms = __ballot_sync(0xFFFFFFFFu, i < n && !forced && k == above);
        if (lane == 0) {
            over[w] = mo;
            same[w] = ms;
        }
        bo += __popc(mo);
        bs += __popc(ms);
    }
    __syncthreads();  // sums and keys are free, once every warp is here
    if (lane == 0) {
        sums[0][warp] = bo;
        sums[1][warp] = bs;
    }
    __syncthreads();
    bo = bs = 0u;
#pragma unroll
    for (int k = 0; k < NW; ++k)
        if (k < warp) {
            bo += sums[0][k];
            bs += sums[1][k];
        }
#pragma unroll 4
    for (int w = w0; w < w1; ++w) {
        const uint32_t mo = over[w], ms = same[w], less = (1u << lane) - 1u;
        const uint32_t es = bs + __popc(ms & less);
        if (((mo >> lane) & 1u) || (((ms >> lane) & 1u) && es < equal))
            keys[bo + __popc(mo & less) + min(es, equal)] = static_cast<uint32_t>(32 * w + lane);
        bo += __popc(mo);
        bs += __popc(ms);
    }
    __syncthreads();
    for (int j = tid; j < count; j += NT) {
        const int i = static_cast<int>(keys[j]);
        out_table[j] = __ldg(row + i);
        if (out_index) out_index[j] = i;
    }
}

template <int D, int NT>
cudaError_t launch_select(const SelectParams& p, int cluster, size_t smem, cudaStream_t s) {
    if (smem > 36 * 1024) {  // with the static arrays, past the 48 KiB a launch may use by default
        const cudaError_t e = cudaFuncSetAttribute(
            select_pages_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelMaxPages / 32 * 136);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.H * cluster));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_pages_kernel<D, NT>, p);
}

template <int D>
cudaError_t launch_select_for(const SelectParams& p, bool large, int cluster, size_t smem, cudaStream_t s) {
    return large ? launch_select<D, 512>(p, cluster, smem, s) : launch_select<D, 256>(p, cluster, smem, s);
}

}  // namespace
}  // namespace nvfp4kv

using namespace nvfp4kv;

extern "C" nvfp4kv_status nvfp4_kv_page_bounds(
    const nvfp4kv_layout* layout, const uint8_t* k_data, const uint8_t* k_scales,
    int32_t pool_pages, const int32_t* page_ids, const int32_t* page_tokens, int32_t num_pages,
    int8_t* bounds, float* bound_scales, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || num_pages < 0) return NVFP4KV_ERR_INVALID_ARG;
    const int D = layout->head_dim;
    if ((D != 64 && D != 128 && D != 256) || layout->page_size % 16 != 0)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (num_pages == 0) return NVFP4KV_OK;
    if (!k_data || !k_scales || !bounds || !bound_scales || pool_pages <= 0 ||
        !aligned16(k_data) || !aligned16(k_scales) || !aligned16(bounds) ||
        !aligned16(bound_scales) || (!page_ids && num_pages > pool_pages))
        return NVFP4KV_ERR_INVALID_ARG;
    BoundsParams p{};
    p.kd = k_data;
    p.ks = k_scales;
    p.page_ids = page_ids;
    p.page_tokens = page_tokens;
    p.bounds = bounds;
    p.scales = bound_scales;
    p.status = status;
    p.pool_pages = pool_pages;
    p.num_pages = num_pages;
    p.H = layout->num_kv_heads;
    p.T = layout->page_size;
    const int64_t items = static_cast<int64_t>(num_pages) * p.H;
    const int64_t ctas = (items + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
    const int64_t most = static_cast<int64_t>(num_sms()) * 32;
    const int grid = static_cast<int>(ctas < most ? ctas : most);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
    case 64: e = launch_pdl(page_bounds_kernel<64>, grid, kBoundsThreads, 0, s, p); break;
    case 128: e = launch_pdl(page_bounds_kernel<128>, grid, kBoundsThreads, 0, s, p); break;
    default: e = launch_pdl(page_bounds_kernel<256>, grid, kBoundsThreads, 0, s, p); break;
    }
    return launched(e);
}

extern "C" nvfp4kv_status nvfp4_kv_select_pages(
    const nvfp4kv_layout* layout, int32_t batch, int32_t num_q_heads, const void* q,
    const int8_t* bounds, const float* bound_scales, int32_t pool_pages,
    const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
    int32_t budget, int32_t sink_pages, int32_t recent_pages, int32_t* sel_page_table,
    int32_t* sel_lens, int32_t* sel_index, float* scores, int32_t* status,
    nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 ||
        pool_pages <= 0 || budget <= 0 || sink_pages < 0 || recent_pages < 1 ||
        static_cast<int64_t>(sink_pages) + recent_pages > budget)
        return NVFP4KV_ERR_INVALID_ARG;
    const int D = layout->head_dim, H = layout->num_kv_heads;
    if ((D != 64 && D != 128 && D != 256) || num_q_heads % H != 0 || num_q_heads / H > kSelMaxGroup)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0) return NVFP4KV_OK;
    if (!q || !bounds || !bound_scales || !page_table || !seq_lens || !sel_page_table || !sel_lens ||
        !aligned16(q) || !aligned16(bounds))
        return NVFP4KV_ERR_INVALID_ARG;
    const int64_t pairs = static_cast<int64_t>(batch) * H;
    if (pairs > 65535 || max_pages_per_seq > kSelMaxPages ||
        static_cast<int64_t>(max_pages_per_seq) * layout->page_size > INT32_MAX ||
        static_cast<int64_t>(budget) * layout->page_size > INT32_MAX)
        return NVFP4KV_ERR_UNSUPPORTED;
    // CTAs per pair: as many as the SMs allow while each still has a tile for every warp (64 pairs of up to
    // 2048 pages: 12.3 us with 2 CTAs, 12.8 with 4, 16.7 with 8). CTAs of 512 threads for the few pairs
    // that leave more than half of the SMs free even so (2 pairs of 6251 pages: 11.4 us against 13.0)
    int cluster = 1;
    while (cluster < kSelMaxCluster && pairs * cluster * 2 <= num_sms() && max_pages_per_seq > 128 * cluster)
        cluster *= 2;
    const bool large = pairs * cluster * 2 <= num_sms() && max_pages_per_seq > 128 * cluster;
    SelectParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.bounds = bounds;
    p.bscales = bound_scales;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.sel_table = sel_page_table;
    p.sel_lens = sel_lens;
    p.sel_index = sel_index;
    p.scores = scores;
    p.status = status;
    p.B = batch;
    p.H = H;
    p.G = num_q_heads / H;
    p.T = layout->page_size;
    p.pool_pages = pool_pages;
    p.max_pages = max_pages_per_seq;
    p.budget = budget;
    p.sink = sink_pages;
    p.recent = recent_pages;
    const size_t smem = static_cast<size_t>((max_pages_per_seq + 31) / 32) * (32 * 4 + 2 * 4);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
    case 64: e = launch_select_for<64>(p, large, cluster, smem, s); break;
    case 128: e = launch_select_for<128>(p, large, cluster, smem, s); break;
    default: e = launch_select_for<256>(p, large, cluster, smem, s); break;
    }
    return launched(e);
}
