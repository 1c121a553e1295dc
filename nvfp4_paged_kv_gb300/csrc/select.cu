// Page bounds and page selection of the sparse decode, for sm_103a.
//
// Bounds. For every (page, KV head), the largest and smallest value of each head dim over the
// page's tokens, as int8 steps of one FP32 scale: with v = e2m1 * e4m3 (exact in FP16),
//   a = max_d max(|max_t v|, |min_t v|),  s = fp32(a / 127),
//   hi_d = min(127, ceil(fp32(max_t v / s))),  lo_d = max(-127, floor(fp32(min_t v / s))),
// all 0 when a is 0. Rounding away from the interval keeps  lo_d s <= v <= hi_d s  (up to the two
// FP32 roundings), so a query's product with the nearer bound of each dim is at least its product
// with any key of the page.
//
// Scores and selection. The queries of a KV head's group are brought to integers of 9 bits,
//   q_i = rint(fp32(q / f)),  f = fp32(max|q| / 255)   (0 when max|q| is 0 or not finite),
// and the score of a page is the largest over the group of
//   fp32(fp32(S f) s),  S = sum_d (q_d > 0 ? q_d hi_d : q_d lo_d).
// S is an integer below 2^23 in magnitude, exact in FP32 in every order of summation, so the
// selection is the same bit for bit whatever the split of the work: the reason for integer bounds
// and integer queries, which also halve the bytes of 16-bit bounds.
//
// Bound: HBM for the bounds' bytes (2 D + 4 per page and head) in long contexts, latency elsewhere.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "codec_core.cuh"
#include "common.cuh"
#include "host_util.h"

namespace cg = cooperative_groups;

namespace nvfp4kv {
namespace {

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// ------------------------------------------------------------------------------------------
// Page bounds. One warp per (page, head): a lane owns 32 dims (16 code bytes) of every
// (32 / (D / 32))-th token, and keeps max v and max -v of its dims in FP16 pairs; the lanes that
// hold the same dims then exchange halves of what they have (a reduce-scatter), so each ends with
// a few finished dims to round and store.
// ------------------------------------------------------------------------------------------
constexpr int kBoundsThreads = 256;

struct BoundsParams {
    const uint8_t* kd;
    const uint8_t* ks;
    const int32_t* page_ids;     // null: 0 .. num_pages-1
    const int32_t* page_tokens;  // null: T
    int8_t* bounds;
    float* scales;
    int32_t* status;
    int32_t pool_pages, num_pages, H, T;
    int64_t items;
};

template <int D>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const BoundsParams p) {
    pdl_enter();
    constexpr int LPR = D / 32;    // lanes of a token row
    constexpr int RPP = 32 / LPR;  // token rows of a pass
    constexpr int NB = D / 16;
    constexpr int KEEP = 32 / RPP; // FP16 pairs a lane ends with
    const int lane = threadIdx.x & 31;
    const int l = lane % LPR, rr = lane / LPR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kBoundsThreads / 32);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kBoundsThreads / 32) + (threadIdx.x >> 5);
         item < p.items; item += step) {
        const int i = static_cast<int>(item / p.H);
        const int h = static_cast<int>(item - static_cast<int64_t>(i) * p.H);
        const int page = p.page_ids ? __ldg(p.page_ids + i) : i;
        if (page == -1) continue;
        const int n = p.page_tokens ? __ldg(p.page_tokens + i) : p.T;
        if (page < 0 || page >= p.pool_pages || n < 0 || n > p.T) {
            if (lane == 0)
                flag_status(p.status, (page < 0 || page >= p.pool_pages) ? NVFP4KV_STATUS_PAGE_OOB
                                                                         : NVFP4KV_STATUS_BAD_SEQ_LEN);
            continue;
        }
        const int64_t ph = static_cast<int64_t>(page) * p.H + h;
        const uint8_t* kd = p.kd + ph * p.T * (D / 2) + 16 * l;
        const uint8_t* ks = p.ks + ph * p.T * NB + 2 * l;
        __half2 m[32];  // max of dims (2j, 2j+1) in m[j], of their negatives in m[16 + j]
#pragma unroll
        for (int j = 0; j < 32; ++j) m[j] = as_h2(0xFC00FC00u);
#pragma unroll 4
        for (int t = rr; t < n; t += RPP) {
            const uint4 w = ld_stream_16B(kd + static_cast<int64_t>(t) * (D / 2));
            const uint32_t sc = *reinterpret_cast<const uint16_t*>(ks + static_cast<int64_t>(t) * NB);
            const uint32_t sa = e4m3x2_to_f16x2((sc & 0xFFu) * 0x0101u);
            const uint32_t sb = e4m3x2_to_f16x2((sc >> 8) * 0x0101u);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t v[4];
                e2m1x8_to_f16x2x4(ww[k], v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t x = hmul2_u32(v[j], k < 2 ? sa : sb);
                    m[4 * k + j] = __hmax2(m[4 * k + j], as_h2(x));
                    m[16 + 4 * k + j] = __hmax2(m[16 + 4 * k + j], as_h2(x ^ 0x80008000u));
                }
            }
        }
        int base = 0, cnt = 32;
#pragma unroll
        for (int off = 16; off >= LPR; off >>= 1) {
            cnt >>= 1;
            const bool up = (lane & off) != 0;
            if (up) base += cnt;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                if (k >= cnt) break;
                const uint32_t give = as_u32(up ? m[k] : m[k + cnt]);
                const __half2 keep = up ? m[k + cnt] : m[k];
                m[k] = __hmax2(keep, as_h2(__shfl_xor_sync(0xFFFFFFFFu, give, off)));
            }
        }
        float a = 0.0f;
        float y[2 * KEEP];
#pragma unroll
        for (int k = 0; k < KEEP; ++k) {
            const float2 f = __half22float2(m[k]);
            y[2 * k] = n > 0 ? f.x : 0.0f;
            y[2 * k + 1] = n > 0 ? f.y : 0.0f;
            a = fmaxf(a, fmaxf(fabsf(y[2 * k]), fabsf(y[2 * k + 1])));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
        const float s = __fdiv_rn(a, 127.0f);
        if (lane == 0) p.scales[ph] = s;
        const bool neg = base >= 16;
        uint32_t w[(2 * KEEP + 3) / 4];
#pragma unroll
        for (int k = 0; k < (2 * KEEP + 3) / 4; ++k) w[k] = 0u;
#pragma unroll
        for (int k = 0; k < 2 * KEEP; ++k) {
            // floor of a negated value is the negated ceil
            const int c = s > 0.0f ? static_cast<int>(fminf(127.0f, ceilf(__fdiv_rn(y[k], s)))) : 0;
            w[k / 4] |= static_cast<uint32_t>((neg ? -c : c) & 0xFF) << (8 * (k % 4));
        }
        int8_t* dst = p.bounds + (ph * 2 + (neg ? 1 : 0)) * D + 32 * l + 2 * (base & 15);
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
// Selection. One thread-block cluster per (sequence, KV head) pair; every CTA scores a contiguous
// share of the sequence's pages on the tensor cores (16 pages as M, the query group as N, the 2 D
// bounds as K) and keeps the scores as sortable keys in shared memory. The smallest selected key is
// found by a radix selection over the cluster's keys (8 bits a pass, histograms summed through
// distributed shared memory), and the selected pages are written in ascending order, equal keys
// from the lowest page on.
// ------------------------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxGroup = 8;
constexpr int kSelMaxCluster = 8;
constexpr int kSelMaxKeys = 49152;  // keys of a CTA: 192 KiB of shared memory

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

// Order-preserving map of a score to an unsigned key; NaN (a page whose bounds were never written)
// below everything, 0 and -0 equal.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (!(x == x)) return 0u;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The four int8 of w as FP16 pairs (exact): v + 128 placed in the mantissa of 1024 + (v + 128).
__device__ __forceinline__ void s8x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = w ^ 0x80808080u;
    const __half2 bias = as_h2(0x64806480u);  // 1152
    lo = as_u32(__hsub2(as_h2(__byte_perm(x, 0x64646464u, 0x4140)), bias));
    hi = as_u32(__hsub2(as_h2(__byte_perm(x, 0x64646464u, 0x4342)), bias));
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(const SelectParams p) {
    pdl_enter();
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t hist[4][256];
    __shared__ uint32_t warp_sum[kSelWarps][2];
    __shared__ uint32_t found[2];    // bin of the pass, keys still wanted from it
    __shared__ uint32_t cta_sum[2];  // this CTA's keys above and at the threshold
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    const int pair = blockIdx.x / C;
    const int b = pair / p.H, h = pair - b * p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;

    const int len = __ldg(p.seq_lens + b);
    const bool len_ok = len >= 0 && len <= static_cast<int64_t>(p.max_pages) * p.T;
    if (!len_ok && h == 0 && rank == 0 && tid == 0) flag_status(p.status, NVFP4KV_STATUS_BAD_SEQ_LEN);
    const int n = len_ok ? static_cast<int>((static_cast<int64_t>(len) + p.T - 1) / p.T) : 0;
    const int count = min(n, p.budget);
    const int per = ((n + C - 1) / C + 15) & ~15;
    const int lo = min(n, rank * per), hi = min(n, lo + per), m = hi - lo;
    const int32_t* row = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    int32_t* out_table = p.sel_table + static_cast<int64_t>(pair) * p.budget;
    int32_t* out_index = p.sel_index ? p.sel_index + static_cast<int64_t>(pair) * p.budget : nullptr;
    if (rank == 0) {
        for (int i = count + tid; i < p.budget; i += kSelThreads) {
            out_table[i] = -1;
            if (out_index) out_index[i] = -1;
        }
        // the last page is always taken, and it alone can be cut short
        if (tid == 0) p.sel_lens[pair] = n > 0 ? (count - 1) * p.T + (len - (n - 1) * p.T) : 0;
    }
    const bool choose = n > p.budget;

    if (choose || p.scores) {
        // ---- the group's queries as integers: lane (r, c) holds head r, dims [c D/4, c D/4 + D/4);
        // fragments of the positive parts (against hi) and of the negative parts (against lo)
        uint32_t qp[D / 16][2], qn[D / 16][2];
        float f = 0.0f;
        {
            uint32_t w[D / 8];
            float amax = 0.0f;
            if (r < p.G) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + (static_cast<int64_t>(pair) * p.G + r) * D + c * (D / 4));
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const uint4 v = __ldg(src + k);
                    w[4 * k] = v.x;
                    w[4 * k + 1] = v.y;
                    w[4 * k + 2] = v.z;
                    w[4 * k + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < D / 8; ++k) w[k] = 0u;
            }
            bool finite = true;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const float x0 = fabsf(bf16_lo(w[k])), x1 = fabsf(bf16_hi(w[k]));
                finite = finite && x0 < INFINITY && x1 < INFINITY;
                amax = fmaxf(amax, fmaxf(x0, x1));
            }
            if (!finite) amax = INFINITY;
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            f = amax < INFINITY ? __fdiv_rn(amax, 255.0f) : 0.0f;
            auto whole = [&](float x) { return f > 0.0f ? rintf(__fdiv_rn(x, f)) : 0.0f; };
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const float x0 = whole(bf16_lo(w[k])), x1 = whole(bf16_hi(w[k]));
                qp[k / 2][k % 2] = pack_f16x2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f));
                qn[k / 2][k % 2] = pack_f16x2(fminf(x0, 0.0f), fminf(x1, 0.0f));
            }
        }
        const float f0 = __shfl_sync(0xFFFFFFFFu, f, 8 * c), f1 = __shfl_sync(0xFFFFFFFFu, f, 8 * c + 4);
        const bool has0 = 2 * c < p.G, has1 = 2 * c + 1 < p.G;

        // ---- scores of this CTA's pages, 16 to a warp tile; lane (r, c) loads quarter c of the
        // bounds of pages r and r + 8
        auto page_at = [&](int i) -> int {  // page id of page i; -1: not scored, -2: outside the pool
            if (i >= hi || i < p.sink || i >= n - p.recent) return -1;
            const int id = __ldg(row + i);
            return id >= 0 && id < p.pool_pages ? id : -2;
        };
        for (int t = warp * 16; t < m; t += kSelWarps * 16) {
            const int i0 = lo + t + r, i1 = i0 + 8;
            const int id0 = page_at(i0), id1 = page_at(i1);
            uint32_t w0[D / 8], w1[D / 8];  // quarter c of hi, then of lo
            float s0 = 0.0f, s1 = 0.0f;
            auto fetch = [&](int id, uint32_t(&w)[D / 8], float& s) {
                const int64_t ph = static_cast<int64_t>(id) * p.H + h;
                if (id >= 0) {
                    const int8_t* a = p.bounds + ph * 2 * D + c * (D / 4);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            const uint4 v = __ldg(reinterpret_cast<const uint4*>(a + half * D) + k);
                            w[half * (D / 16) + 4 * k] = v.x;
                            w[half * (D / 16) + 4 * k + 1] = v.y;
                            w[half * (D / 16) + 4 * k + 2] = v.z;
                            w[half * (D / 16) + 4 * k + 3] = v.w;
                        }
                    s = __ldg(p.bscales + ph);
                } else {
#pragma unroll
                    for (int k = 0; k < D / 8; ++k) w[k] = 0u;
                }
            };
            fetch(id0, w0, s0);
            fetch(id1, w1, s1);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t a[4];
                s8x4_to_f16x2x2(w0[k], a[0], a[2]);
                s8x4_to_f16x2x2(w1[k], a[1], a[3]);
                mma_f16_16816(acc, a, qp[k][0], qp[k][1]);
                s8x4_to_f16x2x2(w0[D / 16 + k], a[0], a[2]);
                s8x4_to_f16x2x2(w1[D / 16 + k], a[1], a[3]);
                mma_f16_16816(acc, a, qn[k][0], qn[k][1]);
            }
            auto score = [&](float x0, float x1, float s) {
                float v = -INFINITY;
                if (has0) v = __fmul_rn(__fmul_rn(x0, f0), s);
                if (has1) v = fmaxf(v, __fmul_rn(__fmul_rn(x1, f1), s));
                v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
            };
            const float v0 = score(acc[0], acc[1], s0), v1 = score(acc[2], acc[3], s1);
            if (c < 2) {
                const int i = c == 0 ? i0 : i1, id = c == 0 ? id0 : id1;
                float v = c == 0 ? v0 : v1;
                if (i < hi) {
                    if (id == -1) v = INFINITY;
                    if (id == -2) {
                        v = -INFINITY;
                        flag_status(p.status, NVFP4KV_STATUS_PAGE_OOB);
                    }
                    if (choose) keys[i - lo] = id == -1 ? 0xFFFFFFFFu : key_of(v);
                    if (p.scores) p.scores[static_cast<int64_t>(pair) * p.max_pages + i] = v;
                }
            }
        }
    }

    if (!choose) {  // every page is taken (the same for all CTAs of the cluster)
        for (int i = lo + tid; i < hi; i += kSelThreads) {
            out_table[i] = __ldg(row + i);
            if (out_index) out_index[i] = i;
        }
        return;
    }

    // ---- the count-th largest key of the cluster
    for (int i = tid; i < 4 * 256; i += kSelThreads) (&hist[0][0])[i] = 0u;
    __syncthreads();
    uint32_t prefix = 0u, mask = 0u, want = static_cast<uint32_t>(count);
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        for (int i = tid; i < m; i += kSelThreads) {
            const uint32_t k = keys[i];
            if ((k & mask) == prefix) atomicAdd(&hist[pass][(k >> shift) & 255u], 1u);
        }
        cluster.sync();
        // thread t takes bin 255 - t: inclusive counts from the top bin down
        uint32_t mine = 0u, incl = 0u;
        if (tid < 256) {
            for (int k = 0; k < C; ++k) mine += cluster.map_shared_rank(&hist[pass][0], k)[255 - tid];
            incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) warp_sum[warp][0] = incl;
        }
        __syncthreads();
        if (tid < 256) {
            for (int k = 0; k < warp; ++k) incl += warp_sum[k][0];
            const uint32_t excl = incl - mine;
            if (excl < want && want <= incl) {
                found[0] = static_cast<uint32_t>(255 - tid);
                found[1] = want - excl;
            }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        mask |= 255u << shift;
        want = found[1];
        __syncthreads();  // found and warp_sum are free for the next pass
    }

    // ---- the selected pages in ascending order: thread t looks at a run of consecutive keys
    const int run = (m + kSelThreads - 1) / kSelThreads;
    const int j0 = min(m, tid * run), j1 = min(m, j0 + run);
    uint32_t above = 0u, equal = 0u;
    for (int j = j0; j < j1; ++j) {
        above += keys[j] > prefix;
        equal += keys[j] == prefix;
    }
    uint32_t ia = above, ie = equal;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t va = __shfl_up_sync(0xFFFFFFFFu, ia, o), ve = __shfl_up_sync(0xFFFFFFFFu, ie, o);
        if (lane >= o) {
            ia += va;
            ie += ve;
        }
    }
    if (lane == 31) {
        warp_sum[warp][0] = ia;
        warp_sum[warp][1] = ie;
    }
    __syncthreads();
    uint32_t ba = ia - above, be = ie - equal;
    for (int k = 0; k < warp; ++k) {
        ba += warp_sum[k][0];
        be += warp_sum[k][1];
    }
    if (tid == kSelThreads - 1) {
        cta_sum[0] = ba + above;
        cta_sum[1] = be + equal;
    }
    cluster.sync();
    for (int k = 0; k < rank; ++k) {
        const uint32_t* other = cluster.map_shared_rank(&cta_sum[0], k);
        ba += other[0];
        be += other[1];
    }
    for (int j = j0; j < j1; ++j) {
        const uint32_t k = keys[j];
        if (k > prefix || (k == prefix && be < want)) {
            const uint32_t at = ba + min(be, want);
            out_table[at] = __ldg(row + lo + j);
            if (out_index) out_index[at] = lo + j;
        }
        ba += k > prefix;
        be += k == prefix;
    }
    cluster.sync();  // no CTA leaves while another may still read its counts
}

template <int D>
cudaError_t launch_select(const SelectParams& p, int cluster, size_t smem, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(select_pages_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSelMaxKeys * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.H * cluster));
    cfg.blockDim = dim3(kSelThreads);
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
    return cudaLaunchKernelEx(&cfg, select_pages_kernel<D>, p);
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
    if (D != 64 && D != 128 && D != 256) return NVFP4KV_ERR_UNSUPPORTED;
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
    p.items = static_cast<int64_t>(num_pages) * p.H;
    const int64_t ctas = (p.items + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
    const int64_t most = static_cast<int64_t>(num_sms()) * 32;
    const int grid = static_cast<int>(ctas < most ? ctas : most);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
    case 64: e = launch_pdl(page_bounds_kernel<64>, grid, kBoundsThreads, 0, s, p); break;
    case 128: e = launch_pdl(page_bounds_kernel<128>, grid, kBoundsThreads, 0, s, p); break;
    default: e = launch_pdl(page_bounds_kernel<256>, grid, kBoundsThreads, 0, s, p); break;
    }
    return e == cudaSuccess ? launch_status() : NVFP4KV_ERR_CUDA;
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
    if (pairs > 65535 || max_pages_per_seq > kSelMaxKeys * kSelMaxCluster ||
        static_cast<int64_t>(max_pages_per_seq) * layout->page_size > INT32_MAX ||
        static_cast<int64_t>(budget) * layout->page_size > INT32_MAX)
        return NVFP4KV_ERR_UNSUPPORTED;
    // CTAs per pair: enough to fill the GPU when there are few pairs, but at least 128 pages (one
    // tile for every second warp) each, and no more keys than fit in shared memory
    int cluster = 1;
    while (cluster < kSelMaxCluster &&
           ((pairs * cluster < num_sms() && max_pages_per_seq > 128 * cluster) ||
            max_pages_per_seq > kSelMaxKeys * cluster))
        cluster *= 2;
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
    const size_t smem = static_cast<size_t>(((max_pages_per_seq + cluster - 1) / cluster + 15) & ~15) * 4;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
    case 64: e = launch_select<64>(p, cluster, smem, s); break;
    case 128: e = launch_select<128>(p, cluster, smem, s); break;
    default: e = launch_select<256>(p, cluster, smem, s); break;
    }
    return e == cudaSuccess ? launch_status() : NVFP4KV_ERR_CUDA;
}
