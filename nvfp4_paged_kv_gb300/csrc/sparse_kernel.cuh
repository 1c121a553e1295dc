// Split-KV decode attention over selected pages: every (sequence, KV head) pair has a page table and a length
// of its own. The mathematics, packings and per-warp pipeline are those of the dense decode (decode_kernel.cuh,
// whose helpers this file uses); what differs is how the pairs' stages are cut into warp runs. It is a kernel of
// its own because the dense one loses 1 to 2 % to the additional cases, of its 60 and 120 us.
//
// The cut. The selection makes all pairs of about one length, and the calls are short, so the join of a pair's
// runs counts: through records in global memory (a fence, a count, a last arrival that loads them all) it takes 4
// to 5 us. Pairs by clusters avoid it: a cluster of 1, 2, 4 or 8 CTAs holds a few pairs, or one, and joins their
// runs through its shared memory. But its SMs hold whole pairs (256 pairs are 2 on 104 of 152 SMs and 1 on the
// others), so long pairs, and pairs of very different lengths, are cut as in the dense decode: runs of equal
// length over all pairs and SMs. Both ways' times are estimated from the lengths (Times), on the host for the size
// of the cluster, in the kernel for the cut. Against runs over all pairs (head_dim 128, 4 heads): 64 pairs of 32
// pages 12.2 us, so 13.6; 256 pairs of 4 pages 7.7 and 11.1, of 16 pages 15.9 and 19.2, of 32 pages 24.2 and 26.3,
// of 64 pages 39.4 and 37.7.
//
// Bound: an SM's rate. One more stage (9216 bytes) takes it 0.24 us, with 12 warps (39 GB/s each SM: 5.9 TB/s on
// all of them, 0.87 of the copy peak), alone as well as with all others and with K and V in L2: it is the
// instructions, 352 to a 16-token tile with start and join (293 in the dense decode's longer runs). Of 128 pairs of
// 8192 tokens (151 MB in 38.7 us), a throwaway copy without the products by the scales took 31.4, without the E2M1
// conversions 33.5, without both 30.2 (5.0 TB/s over the whole call).
// 256 pairs of 2048 tokens (76 MB, 11.2 us at the copy peak) take 24.2 us: 6 until the first stages are
// computed, 64 stages on the fuller SMs, 1 for the join. 64 pairs of 8192 tokens with 8 heads, on clusters of 2,
// 24.9 us; 8 pairs of 4096 tokens, on clusters of 8, 9.3 us; 95 ragged pairs with head_dim 256 24.2 us. Measured
// and slower: one combined record per CTA and pair, runs of unequal length on every warp, 32-token stages (14 to 16
// warps, or more slots), tiles of a stage worked on two or one at a time, the scores of a stage interleaved with
// P V of the one before, and the first stage issued before the lengths are compared (no gain).
//
// Weights go to P V in FP16, as in the dense decode. Against the same products in FP32, 8 to 9 % of the BF16 outputs
// are the neighbouring BF16 value, and the root mean square error against 64 bits is 1 % larger (3.05e-4 for 3.02e-4
// over 256 pairs of 2048 tokens): the output's own rounding is nearly all of it.
#pragma once
#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>

#include "decode_kernel.cuh"

namespace cg = cooperative_groups;

namespace nvfp4kv {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxSparsePairs = 65535;  // (sequence, KV head) pairs of a call

// Microseconds of a call, of both ways to cut it, fitted to measurements of 539 calls (head_dim 64 to 256, 1 to 8
// heads a pair, 8 to 1024 pairs of 1 to 128 pages of 64 tokens; profiles/sparse_cut_times.csv has 924 such calls with
// every cut's time, taken again). Runs over all pairs: the stages of an SM, the
// records of the pair that has most, and those that an SM's warps write. Pairs by clusters: rounds of one stage for
// each warp of the longest pair. The cut chosen took over 5 % longer than the soonest in 13 of the 924, 14 % at most.
struct Times {
    float all_base, record;            // runs over all pairs: base, and for each record of a pair
    float own_base, own_round, share;  // pairs by clusters: base, for each round, rounds for each stage
    __host__ __device__ float all(float sm_stages, float records) const {
        return all_base + fminf(9.2f + 0.37f * sm_stages, 13.0f + 0.237f * sm_stages) + record * records;
    }
    __host__ __device__ float own(int stages) const {
        const float rounds = stages * share;
        return own_base + own_round * (0.5f * (rounds + ceilf(rounds)));
    }
};

// B: pairs, H: 1, Hq: query heads of a pair; seq_lens and page_table are those of the pairs.
struct SparseParams : DecodeParams {
    int32_t pool_heads;  // KV heads of a page in the pools
    // pairs by clusters of CTAs, where that is no longer than runs over all pairs: clusters with pairs (0:
    // never) and the stages of a pair that has all its pages
    int32_t clusters, full_each;
    float per_cta;  // 1 / CTAs
    Times times;
};

template <int D>
__global__ void __launch_bounds__(Geo<D>::THREADS, 1) sparse_split_kernel(const SparseParams p) {
    pdl_enter();
    using G_ = Geo<D>;
    constexpr int TOK = G_::TOK;
    constexpr int NW = G_::WARPS;
    constexpr int NT = G_::THREADS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int scan_warp[NW];
    __shared__ int start_bp[NW][3];  // run start of each warp: pair, its first stage, length
    __shared__ int span_pair[2];     // first and last pair the CTA's runs touch
    __shared__ int pend_n;           // pairs whose last piece finished in this CTA ...
    __shared__ int pend[2 * NW][4];  // ... (b, h, first record, records): merged at the end
    __shared__ int most_warp[NW];    // stages of the longest pair of each warp's lengths
    __shared__ int pair_len[NW];     // lengths of the cluster's pairs

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int r = lane >> 2;  // row group of the MMA fragments
    const int c = lane & 3;   // column pair of the MMA fragments
    const int G = p.G, T = p.T;
    const int max_tokens = p.max_pages * T;

    // ------------------------------------------------ lengths
    // Thread t owns pairs [t C, t C + C). The first two lengths stay in registers for the walk below (a second
    // load of the same words would cost another round trip at the start).
    const int C = (p.B + NT - 1) / NT;
    const int b_lo = min(p.B, tid * C), b_hi = min(p.B, b_lo + C);
    const int kept0 = (b_lo < b_hi) ? __ldg(p.seq_lens + b_lo) : 0;
    const int kept1 = (b_lo + 1 < b_hi) ? __ldg(p.seq_lens + b_lo + 1) : 0;
    auto len_of = [&](int b) {
        return b == b_lo ? kept0 : (b == b_lo + 1 ? kept1 : __ldg(p.seq_lens + b));
    };

    // ------------------------------------------------ pairs by clusters, while the lengths are on their way
    // A cluster of CTAs holds pairs of its own, and each of its warps a run of one pair; the runs are merged
    // through shared memory. Every warp starts on that run, with the loads of its pair's length and page ids,
    // and drops it if the lengths ask for runs over all pairs.
    const int num_runs = p.num_runs;
    const int cta0 = blockIdx.x * NW, cta_runs = max(0, min(num_runs - cta0, NW));
    // this CTA's runs of R over all pairs: those k whose place k num_runs / R is one of its warps (fewer runs
    // than warps are spread over the CTAs: 512 stages on 43 of the 152 SMs took 14.8 us, spread over all 11.4)
    auto first_run = [&](int R) { return min(R, (cta0 * R + num_runs - 1) / num_runs); };
    auto end_run = [&](int R) { return min(R, ((cta0 + cta_runs) * R + num_runs - 1) / num_runs); };
    const uint32_t smem_base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const uint32_t qcache = smem_base + G_::Q_OFF;
    auto load_window = [&](int b_, int base) -> int {
        const int i = base + lane;
        return (i < p.max_pages) ? __ldg(p.page_table + static_cast<int64_t>(b_) * p.max_pages + i)
                                 : -1;
    };
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = static_cast<int>(cluster.num_blocks());
    const int rank = static_cast<int>(cluster.block_rank());
    // pairs [c_lo, c_lo + c_pairs), several only in a cluster of one CTA, with c_warps warps each. Warps are dealt
    // to the pairs in turn, counted across the CTAs of a cluster first, so that few runs lie in different CTAs and
    // quarters of an SM (dealt in blocks, 3 or 4 pairs of one page an SM took 7.8 to 8 us, so 6.6 to 7)
    int c_lo = 0, c_pairs = 0, c_warps = 0;
    int e_pair = 0, e_at = 0, e_len = 0;  // the warp's pair, its place there, the pair's length
    int prow = -1, pbase = 0, pwin = 0;   // page-id window loaded ahead, see below
    if (p.clusters > 0) {
        const int cl = blockIdx.x / CS;
        if (cl < p.clusters) {
            c_lo = cl * p.B / p.clusters;
            c_pairs = (cl + 1) * p.B / p.clusters - c_lo;
        }
        if (c_pairs > 0) {
            const int at = warp * CS + rank;
            e_at = at / c_pairs;
            e_pair = c_lo + at - e_at * c_pairs;
            c_warps = CS * NW / c_pairs;
            e_len = __ldg(p.seq_lens + e_pair);
            const int n = min(c_warps, p.full_each);
            if (e_at < n) {
                prow = e_pair;
                pbase = static_cast<int>(__umul64hi(static_cast<uint64_t>(e_at * p.full_each / n) * TOK,
                                                    p.t_magic)) & ~31;
                pwin = load_window(prow, pbase);
            }
        }
        if (tid < c_pairs) pair_len[tid] = __ldg(p.seq_lens + c_lo + tid);
    }

    // ------------------------------------------------ stage prefix over the pairs
    int local = 0, most = 0;  // stages of this thread's pairs, and of the longest
    for (int b = b_lo; b < b_hi; ++b) {
        const int L = len_of(b);
        if (blockIdx.x == 0 && (L < 0 || L > max_tokens))
            flag_status(p.status, NVFP4KV_STATUS_BAD_SEQ_LEN);
        const int n = seq_stages(L, max_tokens, TOK);
        local += n;
        most = max(most, n);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) {
        scan_warp[warp] = incl;
        most_warp[warp] = most;
    }
    if (tid < 2) span_pair[tid] = 0;
    if (tid == 0) pend_n = 0;
    __syncthreads();
    int excl = incl - local, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) excl += scan_warp[w];
        total += scan_warp[w];
        most = max(most, most_warp[w]);
    }
    // pairs by clusters, or runs over all pairs: warp run gw takes [gw W, gw W + W) of the stage list
    const int W = max(1, (total + num_runs - 1) / num_runs);
    const bool own = p.clusters > 0 &&
                     p.times.own(most) <= p.times.all(total * p.per_cta, __fdividef(most, W));
    int gw0 = 0, n_runs_cta = 0;
    int q_first = c_lo, q_pairs = c_pairs;  // pairs of the CTA, whose queries are cached as far as they fit
    if (blockIdx.x == 0) {
        // pairs without stages (length 0 or invalid): output 0, LSE -inf, a warp per pair
        for (int j = 0; j < C; ++j) {
            const int b = b_lo + j;
            const bool none = b < b_hi && seq_stages(len_of(b), max_tokens, TOK) == 0;
            for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, none); todo != 0u; todo &= todo - 1u) {
                const int64_t bz = __shfl_sync(0xFFFFFFFFu, b, __ffs(todo) - 1);
                uint4* ob = reinterpret_cast<uint4*>(p.out + bz * G * D);
                for (int i = lane; i < G * (D / 8); i += 32) ob[i] = make_uint4(0u, 0u, 0u, 0u);
                if (p.lse)
                    for (int i = lane; i < G; i += 32) p.lse[bz * G + i] = -INFINITY;
            }
        }
    }
    if (!own) {
        // One walk over this thread's pairs finds the pair holding each of the CTA's run starts and its two
        // span ends (32-bit arithmetic: the host bounds stages + runs below 2^31).
        const int R = (total + W - 1) / W;
        gw0 = first_run(R);
        n_runs_cta = end_run(R) - gw0;
        const int span_lo = (n_runs_cta > 0 && gw0 < R) ? gw0 * W : total;
        const int span_hi = min(total, (gw0 + n_runs_cta) * W);
        if (local > 0 && span_lo < span_hi && span_lo < excl + local && span_hi > excl) {
            int acc = excl;
            for (int b = b_lo; b < b_hi && acc < span_hi; ++b) {
                const int L = len_of(b);
                const int n = seq_stages(L, max_tokens, TOK);
                if (n > 0 && acc + n > span_lo) {
                    // runs of this CTA starting in [acc, acc + n): w in [w_a, w_b)
                    const int w_a = max(0, (acc - gw0 * W + W - 1) / W);
                    const int w_b = min(n_runs_cta, (acc + n - gw0 * W + W - 1) / W);
                    for (int w = w_a; w < w_b; ++w) {
                        start_bp[w][0] = b;
                        start_bp[w][1] = acc;
                        start_bp[w][2] = L;
                    }
                    if (span_lo >= acc && span_lo < acc + n) span_pair[0] = b;
                    if (span_hi - 1 >= acc && span_hi - 1 < acc + n)
                        span_pair[1] = b;
                }
                acc += n;
            }
        }
        __syncthreads();
        q_first = span_pair[0];
        q_pairs = span_lo < span_hi ? span_pair[1] - span_pair[0] + 1 : 0;
        prow = -1;
    }
    const int q_cached = min(q_pairs, G_::QCACHE / (G * D * 2));
    {
        const uint8_t* qsrc = reinterpret_cast<const uint8_t*>(p.q + static_cast<int64_t>(q_first) * G * D);
        const int nq = q_cached * G * D * 2 / 16;
        for (int ci = tid; ci < nq; ci += NT) cp_async16_plain(qcache + 16 * ci, qsrc + 16 * ci);
        cp_async_commit();
    }

    const int gw = gw0 + warp;
    int ib = 0, ilen = 0, iS = 1, ij = 0;  // pair of the next stage to issue, its length and stages; the stage
    int ips = 0, nlen = 0;                 // flat index of stage 0 of pair ib, length of the next (unless own)
    int n_st = 0;                          // stages of the run
    bool whole = false;                    // the run is its pair
    if (own) {
        const int S = seq_stages(e_len, max_tokens, TOK), n = min(c_warps, S);
        if (e_at < n) {
            ib = e_pair;
            ilen = e_len;
            iS = S;
            ij = e_at * S / n;
            n_st = (e_at + 1) * S / n - ij;
            whole = n == 1;
        }
    } else if (warp < n_runs_cta && static_cast<int64_t>(gw) * W < total) {
        ib = start_bp[warp][0];
        ilen = start_bp[warp][2];
        iS = seq_stages(ilen, max_tokens, TOK);
        ips = start_bp[warp][1];
        ij = gw * W - ips;
        n_st = min(total - gw * W, W);
        nlen = ib + 1 < p.B ? __ldg(p.seq_lens + ib + 1) : 0;
    }

    // ------------------------------------------------ per-lane constants
    const uint32_t ring = smem_base + warp * G_::RING;
    // V chunk j = lane + 32 i of a stage lands XOR-swizzled by its pair row
    uint32_t v_dst[G_::DCH];
#pragma unroll
    for (int i = 0; i < G_::DCH; ++i) {
        const int j = lane + 32 * i;
        const int pr = j / G_::VCH, cj = j - pr * G_::VCH;
        v_dst[i] = G_::V_OFF + pr * D + 16 * (cj ^ (pr & G_::SWZ));
    }
    const int rho = (r >> 1) | ((r & 1) << 2);  // V rows of this lane: chunk rho of a pair row

    // ------------------------------------------------ issue side: the walk over the run
    bool ifirst = true;                     // the next stage to issue starts a piece
    int issued = 0;
    // page-id windows: lane l holds the id of page base + l of a pair's page-table row; the
    // window after the current one (in issue order) is loaded when the current one is taken
    int wrow = -1, wbase = 0, win = 0;
    // make the window holding page pidx of pair ib current (its loads are only issued) and
    // start loading the one after it
    auto set_window = [&](int pidx) {
        const int nbase = pidx & ~31;
        win = (ib == prow && nbase == pbase) ? pwin : load_window(ib, nbase);
        wrow = ib;
        wbase = nbase;
        const int npg = (ilen + T - 1) / T;
        if (nbase + 32 < npg) {
            prow = ib;
            pbase = nbase + 32;
        } else {
            prow = ib + 1;  // an empty next pair makes this a miss
            pbase = 0;
        }
        if (prow < p.B && !(prow == wrow && pbase == wbase))
            pwin = load_window(prow, pbase);
        else
            prow = -1;
    };
    auto page_of = [&](int pidx) -> int {  // warp-uniform pidx of pair ib; every lane calls
        if (ib != wrow || pidx < wbase || pidx >= wbase + 32) set_window(pidx);
        const int pg = __shfl_sync(0xFFFFFFFFu, win, pidx - wbase);
        return (pg >= 0 && pg < p.pool_pages) ? pg : -1;
    };

    const int64_t page_rows = static_cast<int64_t>(p.pool_heads) * T;
    int ih = ib % p.pool_heads;  // KV head of pair ib
    const bool page_aligned = (T % TOK) == 0;
    // issue the next stage of the walk into `slot`, then advance the walk
    auto issue_next = [&](uint32_t slot) {
        const uint64_t kv_pol = l2_policy_evict_first();
        const int t0 = ij * TOK;
        const int nval = min(TOK, ilen - t0);
        const int64_t head_rows = static_cast<int64_t>(ih) * T;
        int64_t row0[G_::SUB];  // token row of each sub-tile in its pool, -1: not real
        if (page_aligned) {
            const int pidx = static_cast<int>(__umul64hi(static_cast<uint64_t>(t0), p.t_magic));
            const int pg = page_of(pidx);
            const int64_t r0 = pg * page_rows + head_rows + (t0 - pidx * T);
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u)
                row0[u] = (pg >= 0 && 16 * u < nval) ? r0 + 16 * u : -1;
        } else {
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int t = t0 + 16 * u;
                const int pidx = static_cast<int>(__umul64hi(static_cast<uint64_t>(t), p.t_magic));
                const int pg = page_of(min(pidx, max(0, (ilen - 1) / T)));
                row0[u] = (pg >= 0 && 16 * u < nval) ? pg * page_rows + head_rows + (t - pidx * T)
                                                      : -1;
            }
        }
        uint32_t okbits = 0;
#pragma unroll
        for (int u = 0; u < G_::SUB; ++u) okbits |= (row0[u] >= 0 ? 1u : 0u) << u;
        const uint32_t want = (1u << ((nval + 15) / 16)) - 1u;
        if (okbits != want && lane == 0) flag_status(p.status, NVFP4KV_STATUS_PAGE_OOB);
        if (page_aligned && okbits == (1u << G_::SUB) - 1) {
            // the whole stage is one run of each pool: offsets are compile-time constants
            const int64_t doff = row0[0] * (D / 2) + 16 * lane;
            const uint8_t* ksrc = p.kd + doff;
            const uint8_t* vsrc = p.vd + doff;
            static_for<G_::DCH>([&](auto I) {
                constexpr int i = decltype(I)::value;
                cp_async16<G_::K_OFF + 512 * i, 512 * i>(slot + 16 * lane, ksrc, kv_pol);
                cp_async16<0, 512 * i>(slot + v_dst[i], vsrc, kv_pol);
            });
            const int64_t soff = row0[0] * G_::NB;
#pragma unroll
            for (int k = 0; k < G_::SC_PER_LANE; ++k) {
                const int jc = lane + 32 * k;
                const bool kpool = jc < G_::SCH;
                const int jj = kpool ? jc : jc - G_::SCH;
                cp_async16<0, 0>(slot + (kpool ? G_::KS_OFF : G_::VS_OFF) + 16 * jj,
                                 (kpool ? p.ks : p.vs) + soff + 16 * jj, kv_pol);
            }
        } else {
#pragma unroll
            for (int i = 0; i < G_::DCH; ++i) {
                const int u = i / G_::SUB_DIV;
                const int jj = lane + 32 * i - u * (D / 2);  // chunk within the sub-tile
                const bool ok = row0[u] >= 0;
                const int64_t off = ok ? row0[u] * (D / 2) + 16 * jj : 0;
                cp_async16_zfill(slot + G_::K_OFF + 16 * (lane + 32 * i), p.kd + off,
                                 ok ? 16u : 0u, kv_pol);
                cp_async16_zfill(slot + v_dst[i], p.vd + off, ok ? 16u : 0u, kv_pol);
            }
#pragma unroll
            for (int k = 0; k < G_::SC_PER_LANE; ++k) {
                const int jc = lane + 32 * k;
                const bool kpool = jc < G_::SCH;
                const int jj = kpool ? jc : jc - G_::SCH;
                const int u = jj / (D / 16);
                int64_t ru = row0[0];  // row0[u] without a dynamically indexed array
#pragma unroll
                for (int uu = 1; uu < G_::SUB; ++uu)
                    if (u == uu) ru = row0[uu];
                const bool ok = ru >= 0;
                const int64_t off = ok ? ru * G_::NB + 16 * (jj - u * (D / 16)) : 0;
                cp_async16_zfill(slot + (kpool ? G_::KS_OFF : G_::VS_OFF) + 16 * jj,
                                 (kpool ? p.ks : p.vs) + off, ok ? 16u : 0u, kv_pol);
            }
        }
        const bool last = (ij == iS - 1) || (issued == n_st - 1);
        const uint32_t flags = (ifirst ? kFirst : 0u) | (last ? kLast : 0u);
        if (lane == 0) {
            sts_v4(slot + G_::HDR_OFF, okbits | (static_cast<uint32_t>(nval) << 8), flags,
                   static_cast<uint32_t>(ib), 0u);
            sts_v4(slot + G_::HDR_OFF + 16, static_cast<uint32_t>(ips), static_cast<uint32_t>(iS), 0u, 0u);
        }
        // advance the walk
        ++issued;
        ifirst = false;
        if (last) {
            ij = 0;
            ips += iS;
            ifirst = true;
            if (issued < n_st) {
                ++ib;
                ilen = nlen;
                iS = seq_stages(ilen, max_tokens, TOK);
                while (iS == 0) {  // pairs without stages are not in the list
                    ++ib;
                    ilen = __ldg(p.seq_lens + ib);
                    iS = seq_stages(ilen, max_tokens, TOK);
                }
                nlen = (ib + 1 < p.B) ? __ldg(p.seq_lens + ib + 1) : 0;
                ih = ib % p.pool_heads;
            }
        } else {
            ++ij;
        }
    };

    // ------------------------------------------------ start: stage 0, then the query cache
    // The first page-id window is loaded while the query cache fills; the first copies go out
    // as soon as the page ids are in, and the queries are waited for behind them.
    if (n_st > 0) issue_next(ring);
    cp_async_commit();
    cp_async_wait<1>();  // this thread's query chunks have landed ...
    __syncthreads();     // ... and every thread's: from here on warps run alone until the merge

    // ------------------------------------------------ compute side
    uint32_t qf[G_::KSTEPS][2];
    float cs0 = 0.0f, cs1 = 0.0f;
    float o[G_::KSTEPS][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    const float gvs = __ldg(p.gv);

#pragma unroll 1
    for (int i = 0; i < n_st; ++i) {
        // the next stage goes into the slot computed at iteration i - 1
        if (i + 1 < n_st) issue_next(ring + ((i + 1) % G_::SLOTS) * G_::SLOT);
        cp_async_commit();
        cp_async_wait<1>();  // this lane's copies of stage i are done ...
        __syncwarp();        // ... and so are the other lanes'
        const uint32_t st = ring + (i % G_::SLOTS) * G_::SLOT;
        uint32_t hdr[4];
        lds_words(hdr, st + G_::HDR_OFF);
        const uint32_t okbits = hdr[0] & 0xFFu;
        const int nval = static_cast<int>(hdr[0] >> 8);
        const uint32_t flags = hdr[1];
        if (flags & kFirst) {
            // ---- Q fragments of the piece: lane (r, c) holds head r of the group; k-step kk
            // covers head dims c*D/4 + 4kk + {0..3} (the same permutation is used for K), as
            // FP16 q * 2^kq. From the query cache, or from global memory for a pair beyond it.
            const int qpair = static_cast<int>(hdr[2]);
            float qv[D / 4];
            float qmax = 0.0f;
            if (r < G) {
                uint32_t qw[D / 8];
                const int qi = qpair - q_first;
                if (qi >= 0 && qi < q_cached) {
                    lds_words(qw, qcache + ((qi * G + r) * D + c * (D / 4)) * 2);
                } else {
                    const uint4* qsrc = reinterpret_cast<const uint4*>(
                        p.q + (static_cast<int64_t>(qpair) * G + r) * D + c * (D / 4));
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        const uint4 v = __ldg(qsrc + k);
                        qw[4 * k] = v.x;
                        qw[4 * k + 1] = v.y;
                        qw[4 * k + 2] = v.z;
                        qw[4 * k + 3] = v.w;
                    }
                }
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    qv[2 * k] = bf16_lo(qw[k]);
                    qv[2 * k + 1] = bf16_hi(qw[k]);
                }
#pragma unroll
                for (int k = 0; k < D / 4; ++k) qmax = fmaxf(qmax, fabsf(qv[k]));
            } else {
#pragma unroll
                for (int k = 0; k < D / 4; ++k) qv[k] = 0.0f;
            }
            qmax = fmaxf(qmax, __shfl_xor_sync(0xFFFFFFFFu, qmax, 1));
            qmax = fmaxf(qmax, __shfl_xor_sync(0xFFFFFFFFu, qmax, 2));
            // qmax * 2^kq in [2^14, 2^15): every BF16 value (8 bits) of the head is exact in FP16,
            // whose last bit is 2^-24, down to 2^-31 of the head maximum.
            int kq = (qmax > 0.0f) ? (14 - ilogbf(qmax)) : 0;
            kq = max(-120, min(kq, 120));
            const float up = ldexpf(1.0f, kq);
#pragma unroll
            for (int kk = 0; kk < G_::KSTEPS; ++kk) {
                qf[kk][0] = pack_f16x2(qv[4 * kk] * up, qv[4 * kk + 1] * up);
                qf[kk][1] = pack_f16x2(qv[4 * kk + 2] * up, qv[4 * kk + 3] * up);
            }
            const float cs_row = (r < G) ? p.sm_scale * __ldg(p.gk) * kLog2e * ldexpf(1.0f, -kq)
                                         : 0.0f;
            // score scale of this lane's two S^T columns (query heads 2c, 2c+1)
            cs0 = __shfl_sync(0xFFFFFFFFu, cs_row, 8 * c);
            cs1 = __shfl_sync(0xFFFFFFFFu, cs_row, 8 * c + 4);
#pragma unroll
            for (int m = 0; m < G_::KSTEPS; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[m][k] = 0.0f;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.0f;
        }

        if (okbits != 0u) {
            const bool full = (okbits == (1u << G_::SUB) - 1) && nval >= TOK;
            // valid-token bits of each sub-tile (only read when !full)
            uint32_t tmask[G_::SUB];
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int nv = min(16, max(0, nval - 16 * u));
                tmask[u] = ((okbits >> u) & 1u) ? ((nv >= 16) ? 0xFFFFu : ((1u << nv) - 1u)) : 0u;
            }

            // ---- S^T = K^ Q^T for the SUB sub-tiles
            float x[G_::SUB][4];
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int row0 = 16 * u + r;
                const int row1 = row0 + 8;
                uint32_t kw0[G_::CW], kw1[G_::CW];
                lds_words(kw0, st + G_::K_OFF + row0 * (D / 2) + c * G_::CHUNK);
                lds_words(kw1, st + G_::K_OFF + row1 * (D / 2) + c * G_::CHUNK);
                // FP16 (s, s) of the lane's D/64 blocks in rows row0 / row1: the scale byte
                // is duplicated by an integer multiply, then converted as an E4M3 pair
                uint32_t ks0[D / 64], ks1[D / 64];
#pragma unroll
                for (int q = 0; q < D / 64; ++q) {
                    ks0[q] = e4m3x2_to_f16x2(
                        lds_u8(st + G_::KS_OFF + row0 * G_::NB + c * (D / 64) + q) * 0x0101u);
                    ks1[q] = e4m3x2_to_f16x2(
                        lds_u8(st + G_::KS_OFF + row1 * G_::NB + c * (D / 64) + q) * 0x0101u);
                }
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int q = 0; q < G_::CW; ++q) {
                    uint32_t c0[4], c1[4];
                    e2m1x8_to_f16x2x4(kw0[q], c0);
                    e2m1x8_to_f16x2x4(kw1[q], c1);
#pragma unroll
                    for (int hk = 0; hk < 2; ++hk) {
                        const int kk = 2 * q + hk;  // k-step: bytes 2kk, 2kk+1 of the chunk
                        const int blk = kk / 4;     // block of the lane's chunk
                        uint32_t a[4];
                        a[0] = h2_mul(c0[2 * hk], ks0[blk]);
                        a[1] = h2_mul(c1[2 * hk], ks1[blk]);
                        a[2] = h2_mul(c0[2 * hk + 1], ks0[blk]);
                        a[3] = h2_mul(c1[2 * hk + 1], ks1[blk]);
                        mma_f16_16816(acc, a, qf[kk][0], qf[kk][1]);
                    }
                }
                x[u][0] = acc[0] * cs0;
                x[u][1] = acc[1] * cs1;
                x[u][2] = acc[2] * cs0;
                x[u][3] = acc[3] * cs1;
            }

            // ---- online softmax over the stage, columns = query heads 2c, 2c+1
            if (!full) {
#pragma unroll
                for (int u = 0; u < G_::SUB; ++u) {
                    if (!((tmask[u] >> r) & 1u)) x[u][0] = x[u][1] = -INFINITY;
                    if (!((tmask[u] >> (r + 8)) & 1u)) x[u][2] = x[u][3] = -INFINITY;
                }
            }
            float lm0 = fmaxf(x[0][0], x[0][2]), lm1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
            for (int u = 1; u < G_::SUB; ++u) {
                lm0 = fmaxf(lm0, fmaxf(x[u][0], x[u][2]));
                lm1 = fmaxf(lm1, fmaxf(x[u][1], x[u][3]));
            }
            float mx0, mx1;
            column_maxima(lm0, lm1, mx0, mx1);
            const bool grow = (mx0 > m0 + kRescaleThreshold) || (mx1 > m1 + kRescaleThreshold);
            if (__any_sync(0xFFFFFFFFu, grow)) {
                const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
                const float a0 = ex2_approx(m0 - n0), a1 = ex2_approx(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int m = 0; m < G_::KSTEPS; ++m) {
                    o[m][0] *= a0;
                    o[m][1] *= a1;
                    o[m][2] *= a0;
                    o[m][3] *= a1;
                }
            }
            uint32_t pb[G_::SUB][2];
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const float p0 = ex2_approx(x[u][0] - m0), p1 = ex2_approx(x[u][1] - m1);
                const float p2 = ex2_approx(x[u][2] - m0), p3 = ex2_approx(x[u][3] - m1);
                l0 += p0 + p2;
                l1 += p1 + p3;
                // P^T (tokens x heads) -> B operand (k = tokens, n = heads), rounded to FP16: 11 bits
                // where the output has 8, and FP16 is what V is exact in; the sum takes p as it is
                pb[u][0] = movmatrix_trans(pack_f16x2(p0, p1));
                pb[u][1] = movmatrix_trans(pack_f16x2(p2, p3));
            }

            // ---- O^T += V^^T P^T. Lane pairs: pr0 (tokens 2c, 2c+1), pr1 (tokens 2c+8, 2c+9)
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int pr0 = 8 * u + c, pr1 = pr0 + 4;
                // the lane's chunk covers head dims rho*D/8 .. +D/8-1: blocks (rho*D/8)/16 ...
                constexpr int kBlkPerChunk = (D / 8 + 15) / 16;
                uint32_t vsc0[kBlkPerChunk], vsc1[kBlkPerChunk];
#pragma unroll
                for (int q = 0; q < kBlkPerChunk; ++q) {
                    const int blk = (rho * (D / 8)) / 16 + q;
                    vsc0[q] = e4m3x2_to_f16x2(lds_u16(st + G_::VS_OFF + pr0 * 2 * G_::NB + 2 * blk));
                    vsc1[q] = e4m3x2_to_f16x2(lds_u16(st + G_::VS_OFF + pr1 * 2 * G_::NB + 2 * blk));
                }
                if (!full && tmask[u] != 0xFFFFu) {
                    // tokens past the pair end in a real page: their V scales may be
                    // anything, so they are zeroed (P is 0 there already)
                    const uint32_t tm = tmask[u];
                    const uint32_t keep0 = (((tm >> (2 * c)) & 1u) ? 0x0000FFFFu : 0u) |
                                           (((tm >> (2 * c + 1)) & 1u) ? 0xFFFF0000u : 0u);
                    const uint32_t keep1 = (((tm >> (2 * c + 8)) & 1u) ? 0x0000FFFFu : 0u) |
                                           (((tm >> (2 * c + 9)) & 1u) ? 0xFFFF0000u : 0u);
#pragma unroll
                    for (int q = 0; q < kBlkPerChunk; ++q) {
                        vsc0[q] &= keep0;
                        vsc1[q] &= keep1;
                    }
                }
                uint32_t vw0[G_::CW], vw1[G_::CW];
#pragma unroll
                for (int q = 0; q < G_::CW; q += (G_::CW >= 4 ? 4 : G_::CW)) {
                    const int xb = rho * G_::CHUNK + 4 * q;  // logical byte of the chunk piece
                    uint32_t t0w[G_::CW >= 4 ? 4 : G_::CW], t1w[G_::CW >= 4 ? 4 : G_::CW];
                    lds_words(t0w, st + G_::V_OFF + v_swz<D>(pr0, xb));
                    lds_words(t1w, st + G_::V_OFF + v_swz<D>(pr1, xb));
#pragma unroll
                    for (int e = 0; e < (G_::CW >= 4 ? 4 : G_::CW); ++e) {
                        vw0[q + e] = t0w[e];
                        vw1[q + e] = t1w[e];
                    }
                }
#pragma unroll
                for (int q = 0; q < G_::CW; ++q) {
                    uint32_t c0[4], c1[4];
                    e2m1x8_to_f16x2x4(vw0[q], c0);
                    e2m1x8_to_f16x2x4(vw1[q], c1);
#pragma unroll
                    for (int hm2 = 0; hm2 < 2; ++hm2) {
                        const int m = 2 * q + hm2;   // M-tile: bytes 2m, 2m+1 of the chunk
                        const int sq = (2 * m) / 16; // block of that byte within the chunk
                        uint32_t a[4];
                        a[0] = h2_mul(c0[2 * hm2], vsc0[sq]);
                        a[1] = h2_mul(c0[2 * hm2 + 1], vsc0[sq]);
                        a[2] = h2_mul(c1[2 * hm2], vsc1[sq]);
                        a[3] = h2_mul(c1[2 * hm2 + 1], vsc1[sq]);
                        mma_f16_16816(o[m], a, pb[u][0], pb[u][1]);
                    }
                }
            }
        }

        if ((flags & kLast) && (!own || whole)) {
            // ---- end of a piece: the whole pair (outputs) or a record
            uint32_t h2[4];
            lds_words(h2, st + G_::HDR_OFF + 16);
            const int pair = static_cast<int>(hdr[2]);
            const int pps = static_cast<int>(h2[0]), pS = static_cast<int>(h2[1]);
            float ls0 = l0, ls1 = l1;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                ls0 += __shfl_xor_sync(0xFFFFFFFFu, ls0, off);
                ls1 += __shfl_xor_sync(0xFFFFFFFFu, ls1, off);
            }
            const int g0 = 2 * c, g1 = 2 * c + 1;
            const int gf = pps / W, gl = (pps + pS - 1) / W;  // the pair's first and last run
            const int64_t bh = pair;
            if (whole || gf == gl) {
                // the whole pair is this piece: normalise and write the output directly
                uint16_t* ob = p.out + bh * G * D;
                const float f0 = ls0 > 0.0f ? gvs / ls0 : 0.0f;
                const float f1 = ls1 > 0.0f ? gvs / ls1 : 0.0f;
#pragma unroll
                for (int m = 0; m < G_::KSTEPS; ++m) {
                    const int d0 = rho * (D / 8) + 2 * m;
                    if (g0 < G)
                        *reinterpret_cast<uint32_t*>(ob + g0 * D + d0) =
                            pack_bf16x2(o[m][0] * f0, o[m][2] * f0);
                    if (g1 < G)
                        *reinterpret_cast<uint32_t*>(ob + g1 * D + d0) =
                            pack_bf16x2(o[m][1] * f1, o[m][3] * f1);
                }
                if (r == 0 && p.lse) {
                    float* lb = p.lse + bh * G;
                    if (g0 < G) lb[g0] = ls0 > 0.0f ? (m0 + log2f(ls0)) * 0.6931471805599453f : -INFINITY;
                    if (g1 < G) lb[g1] = ls1 > 0.0f ? (m1 + log2f(ls1)) * 0.6931471805599453f : -INFINITY;
                }
            } else {
                const int64_t rec = gw + bh;
                float* ro = p.rec_o + rec * G * D;
#pragma unroll
                for (int m = 0; m < G_::KSTEPS; ++m) {
                    const int d0 = rho * (D / 8) + 2 * m;
                    if (g0 < G) *reinterpret_cast<float2*>(ro + g0 * D + d0) = make_float2(o[m][0], o[m][2]);
                    if (g1 < G) *reinterpret_cast<float2*>(ro + g1 * D + d0) = make_float2(o[m][1], o[m][3]);
                }
                if (r == 0) {
                    if (g0 < G) *reinterpret_cast<float2*>(p.rec_ml + (rec * G + g0) * 2) = make_float2(m0, ls0);
                    if (g1 < G) *reinterpret_cast<float2*>(p.rec_ml + (rec * G + g1) * 2) = make_float2(m1, ls1);
                }
                __syncwarp();
                if (lane == 0) {
                    fence_acq_rel_gpu();  // release: the record is visible before the count says so
                    unsigned long long* cnt = p.done + bh;
                    const uint32_t k = tagged_finish(cnt, atomicAdd(cnt, 1ull), p.nonce, 1);
                    if (k == kTagGiveUp) flag_status(p.status, NVFP4KV_STATUS_TIMEOUT);
                    if (k == static_cast<uint32_t>(gl - gf)) {  // every piece is in: merge here
                        // acquire: the other pieces' records are read after their counts (the
                        // CTA barrier before the merge carries this to every thread)
                        fence_acq_rel_gpu();
                        const int slot = atomicAdd(&pend_n, 1);
                        pend[slot][0] = pair;
                        pend[slot][1] = 0;
                        pend[slot][2] = static_cast<int>(gf + bh);
                        pend[slot][3] = gl - gf + 1;
                    }
                }
            }
        }
        __syncwarp();  // every lane is done reading the slot before it refills
    }
    cp_async_wait<0>();
    if (own) {
        // ---- merge of a cluster's pairs. A warp leaves its run in its own ring, as its lanes have it: four outputs
        // (heads 2c, 2c + 1 of two dims) per lane and 16 dims, behind them (max, sum) of heads 2c, 2c + 1. The runs
        // of a pair in this CTA become the output, or, in a cluster of several CTAs, one record like theirs in the
        // second slot of the first ring, joined with those of the other CTAs. (As [G][D] the lanes of a store would
        // share a bank: 8 pairs of 64 pages 10.4 us against 9.2, of 8 heads of 256 24.6 against 14.3.)
        //
        // Runs of the cluster's pair j to be merged: one alone has written the outputs itself, and a pair without
        // any is the first CTA's.
        auto runs_of = [&](int j) {
            const int n = min(c_warps, seq_stages(pair_len[j], max_tokens, TOK));
            return n > 1 ? n : 0;
        };
        int any = 0;
        for (int j = 0; j < c_pairs; ++j) any |= runs_of(j);
        if (any == 0) return;  // (the same in all CTAs of the cluster)
        constexpr int ML = G_::KSTEPS * 32;  // float4 of a record before the maxima and sums
        static_assert(16 * (ML + 4) <= G_::SLOT, "a record in a slot");
        auto record = [&](int w, int slot) {
            return reinterpret_cast<float4*>(smem + w * G_::RING + slot * G_::SLOT);
        };
        if (n_st > 0 && !whole) {
            float ls0 = l0, ls1 = l1;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                ls0 += __shfl_xor_sync(0xFFFFFFFFu, ls0, off);
                ls1 += __shfl_xor_sync(0xFFFFFFFFu, ls1, off);
            }
            float4* rec = record(warp, 0);
#pragma unroll
            for (int m = 0; m < G_::KSTEPS; ++m) rec[32 * m + lane] = make_float4(o[m][0], o[m][1], o[m][2], o[m][3]);
            if (r == 0) rec[ML + c] = make_float4(m0, ls0, m1, ls1);
        }
        __syncthreads();
        // a column: the lane and 16 dims whose four outputs are joined
        struct Column {
            int m, r, c;
            float m0, m1, l0, l1;
            float4 o;
        };
        const int CC = (G + 1) / 2, columns = G_::KSTEPS * 8 * CC;
        auto column = [&](int i) {
            Column k;
            k.m = i / (8 * CC);
            const int at = i - k.m * 8 * CC;
            k.r = at / CC;
            k.c = at - k.r * CC;
            k.m0 = k.m1 = -INFINITY;
            k.l0 = k.l1 = 0.0f;
            k.o = make_float4(0.f, 0.f, 0.f, 0.f);
            return k;
        };
        auto raise = [](Column& k, const float4* rec) {
            k.m0 = fmaxf(k.m0, rec[ML + k.c].x);
            k.m1 = fmaxf(k.m1, rec[ML + k.c].z);
        };
        auto join = [](Column& k, const float4* rec) {
            const float4 ml = rec[ML + k.c], v = rec[32 * k.m + 4 * k.r + k.c];
            const float w0 = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - k.m0);
            const float w1 = ml.z == -INFINITY ? 0.0f : exp2f(ml.z - k.m1);
            k.l0 += w0 * ml.y;
            k.l1 += w1 * ml.w;
            k.o.x += w0 * v.x;
            k.o.y += w1 * v.y;
            k.o.z += w0 * v.z;
            k.o.w += w1 * v.w;
        };
        const float gvs = __ldg(p.gv);
        auto finish = [&](int j, const Column& k) {
            const int64_t row = static_cast<int64_t>(c_lo + j) * G + 2 * k.c;
            const int d0 = ((k.r >> 1) | ((k.r & 1) << 2)) * (D / 8) + 2 * k.m;
            const float f0 = k.l0 > 0.0f ? gvs / k.l0 : 0.0f, f1 = k.l1 > 0.0f ? gvs / k.l1 : 0.0f;
            *reinterpret_cast<uint32_t*>(p.out + row * D + d0) = pack_bf16x2(k.o.x * f0, k.o.z * f0);
            if (2 * k.c + 1 < G)
                *reinterpret_cast<uint32_t*>(p.out + (row + 1) * D + d0) = pack_bf16x2(k.o.y * f1, k.o.w * f1);
            if (p.lse && k.m == 0 && k.r == 0) {
                p.lse[row] = k.l0 > 0.0f ? (k.m0 + log2f(k.l0)) * 0.6931471805599453f : -INFINITY;
                if (2 * k.c + 1 < G)
                    p.lse[row + 1] = k.l1 > 0.0f ? (k.m1 + log2f(k.l1)) * 0.6931471805599453f : -INFINITY;
            }
        };
        for (int it = tid; it < c_pairs * columns; it += NT) {
            const int j = it / columns;
            Column k = column(it - j * columns);
            // in this CTA every (rank + i CS)-th run, of its warps j, j + c_pairs, ..
            const int n = (runs_of(j) - rank + CS - 1) / CS;
            if (n <= 0) continue;
            for (int i = 0; i < n; ++i) raise(k, record(j + i * c_pairs, 0));
            for (int i = 0; i < n; ++i) join(k, record(j + i * c_pairs, 0));
            if (CS == 1) {
                finish(j, k);
            } else {
                record(0, 1)[32 * k.m + 4 * k.r + k.c] = k.o;
                if (k.m == 0 && k.r == 0) record(0, 1)[ML + k.c] = make_float4(k.m0, k.l0, k.m1, k.l1);
            }
        }
        if (CS == 1) return;
        cluster.sync();
        const int n = min(CS, any);  // CTAs with a record of the cluster's one pair
        for (int it = rank * NT + tid; it < columns; it += CS * NT) {
            Column k = column(it);
            for (int q = 0; q < n; ++q) raise(k, cluster.map_shared_rank(record(0, 1), q));
            for (int q = 0; q < n; ++q) join(k, cluster.map_shared_rank(record(0, 1), q));
            finish(0, k);
        }
        cluster.sync();  // the records stay until every CTA has read them
        return;
    }
    __syncthreads();  // every warp's run is done: the rings are free for the merge
    const int n_pend = pend_n;
    for (int k = 0; k < n_pend;) {
        const int m = merge_batch<D>(p, pend, k, n_pend, smem);
        if (m == 0) {  // a pair whose records do not fit at once: by chunks
            merge_pair<D>(p, pend[k][0], pend[k][1], pend[k][2], pend[k][3], smem);
            ++k;
        }
        k += m;
    }
}

// Pairs by clusters (see the kernel): CTAs of a cluster, clusters with pairs, clusters of the grid.
struct ClusterPlan {
    int size, with_pairs, grid;
    Times times;
};

template <int D>
int max_clusters(int size) {  // clusters that run at once
    if (size == 1) return num_sms();
    static std::atomic<int> known[64][3];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::atomic<int>& n = known[dev][size == 2 ? 0 : size == 4 ? 1 : 2];
    if (n.load() == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(num_sms() / size * size));
        cfg.blockDim = dim3(Geo<D>::THREADS);
        cfg.dynamicSmemBytes = Geo<D>::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(size);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int v = 0;
        if (cudaOccupancyMaxActiveClusters(&v, sparse_split_kernel<D>, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            v = -1;
        }
        n.store(v > 0 ? std::min(v, num_sms() / size) : -1);
    }
    return std::max(0, n.load());
}

// The clusters that take the least time when every pair has all its pages; single CTAs where runs over all pairs
// take less, for calls whose pairs turn out shorter. The host does not know the lengths: under a table wider than they
// are, the clusters it chose can cost more than they save, their barriers on short pairs and the SMs that no cluster
// covers on uneven ones. Of 84 calls each (8 to 72 pairs, 16 to 256 pages), that was over 5 % of what single CTAs or
// runs over all SMs take in 50 at a tenth of the width (3.0 us at most, 9.4 for 6.4), 21 at half (2.3), 6 ragged
// (1.4) and 24 with one long pair (1.7); in the mean of the last three kinds clusters save 0.9 to 1.3 us.
// (profiles/sparse_cut_times_short.csv)
template <int D>
ClusterPlan choose_clusters(int64_t pairs, int64_t each, int G) {
    constexpr int NW = Geo<D>::WARPS;
    const int sms = num_sms();
    const float record_kb = G * D * 4 / 1024.0f;
    auto plan = [&](int size, int64_t with_pairs, int grid) {
        const int64_t held = (pairs + with_pairs - 1) / with_pairs, warps = std::max<int64_t>(1, NW * size / held);
        Times t;
        t.all_base = std::max(0.0f, 0.15f * (NW * record_kb - 24.0f));
        t.record = 0.012f + 0.016f * record_kb;
        t.own_base = size == 1 ? 6.5f : size == 2 ? 7.2f : size == 4 ? 7.6f : 7.9f;
        t.own_round = 1.35f + 0.13f * static_cast<float>(warps * held / size);
        t.share = 1.0f / static_cast<float>(warps);
        return ClusterPlan{size, held <= NW ? static_cast<int>(with_pairs) : 0, grid, t};
    };
    ClusterPlan best = plan(1, std::min<int64_t>(pairs, sms), sms);
    if (each * NW * kMaxCluster > INT32_MAX) best.with_pairs = 0;  // (places of stages are 32-bit products)
    if (best.with_pairs == 0) return best;
    const int64_t runs = static_cast<int64_t>(sms) * NW, W = (pairs * each + runs - 1) / runs;
    const float all = best.times.all(static_cast<float>(pairs * each) / sms, static_cast<float>(each) / W);
    float least = std::min(all, best.times.own(static_cast<int>(each)));
    for (int size = 2; size <= kMaxCluster && pairs * size <= sms; size *= 2) {
        ClusterPlan c = plan(size, pairs, 0);
        const float t = c.times.own(static_cast<int>(each));
        if (t >= least) continue;
        c.grid = max_clusters<D>(size);
        if (pairs > c.grid) continue;
        best = c;
        least = t;
    }
    return best;
}

template <int D>
cudaError_t launch_sparse(SparseParams& p, cudaStream_t s) {
    using G_ = Geo<D>;
    const cudaError_t e = cudaFuncSetAttribute(sparse_split_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         G_::SMEM);
    if (e != cudaSuccess) return e;
    const ClusterPlan plan = choose_clusters<D>(p.B, p.full_each, p.G);
    p.clusters = plan.with_pairs;
    p.times = plan.times;
    const int ctas = plan.grid * plan.size;
    p.num_runs = ctas * G_::WARPS;
    p.per_cta = 1.0f / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(G_::THREADS);
    cfg.dynamicSmemBytes = G_::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan.size);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plan.size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sparse_split_kernel<D>, static_cast<const SparseParams&>(p));
}

}  // namespace
}  // namespace nvfp4kv
