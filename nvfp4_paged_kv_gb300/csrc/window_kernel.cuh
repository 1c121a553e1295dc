// Split-KV decode attention with a sliding window, over NVFP4 K/V or over FP8 pages (E4M3, a scale for each page and
// head). The pipeline, the run cut and the join are those of the dense decode (decode_kernel.cuh, whose helpers this
// file uses); what differs is which stages a sequence has, which tokens of a stage count, and what the cache holds. It is
// a kernel of its own because the dense one loses 1 to 3 % to the additional cases (32 sequences of 8192 tokens:
// 123.5 us, so 120.2).
//
// The window. A sequence of L tokens shows token t if t >= L - window or t < sinks. Its stages are those of the first
// tokens, then those from the window's first token on; none between is listed, so the work is the visible tokens' and a
// table entry of a page without a visible token is never read as a page. A token of a stage that is hidden has its score
// set to -inf and, since 0 times anything need not be 0, its V to 0. Without a window
// (FP8 pages alone; WIN = false) what tells hidden tokens is left out: 32 sequences of 8192 tokens 99.5 us, so 101 with a
// window that no length passes.
//
// FP8. An E4M3 value is exact in FP16, so K and V are converted (cvt.rn.f16x2.e4m3x2) and multiplied without scales:
// the page's K scale multiplies the score in FP32, and the page's V scale s becomes log2(s) added to the score, so that
// the weight is already p s for P V, and the row's sum takes it times 1 / s. A slot then needs no scale pools but one
// scale of K and of V for each 16 tokens. Rows have twice the bytes of NVFP4, so a stage has half the tokens: the same
// 8 KB of K and V in flight for each warp. V rows of two tokens are paired byte by byte in registers (__byte_perm).
// Weights go to P V in FP16 (2^-11), as in the dense decode, the sum takes them in FP32. They are relative to the largest
// p s_V, so a page must not raise that for nothing: V of a page without a value has scale 1, whatever the others' scales, and
// beside pages of 2^-20 it would leave them in FP16's subnormals. Before the maximum grows, a tile of scale 1 is therefore looked
// at, and where all of it is 0 it takes part with a scale of 2^-50 (any is right for it).
//
// Measured (head_dim 128, 32 heads on 8): FP8, 32 sequences of 8192 tokens (537 MB) 98 to 101 us, 5.4 TB/s, 0.79 of the copy rate.
// Bound by the latency of a warp's own chain (3 warps a scheduler, an instruction each 7 clocks): 10 % fewer instructions
// gave 1.5 %, three slots instead of two at head_dim 64 and 256, where they fit, nothing; 12 warps instead of 8 at
// head_dim 256 took 93 us for 87. NVFP4 with a window of 4096 and 4 first tokens, 32 sequences (151 MB) 43 us, of which start
// and join are 15; one sequence of 1005 tokens 11.5 us, all latency. FP8, head_dim 256, 19 ragged sequences with a window of
// 2048, pages of 16 (100 MB) 27 to 33 us by their lengths, 34 to 50 with one to six sequences of length 0 among them: a thread of the
// first CTA writes the outputs of each before that CTA's runs begin.
#pragma once
#include <algorithm>

#include "decode_kernel.cuh"

namespace nvfp4kv {
namespace {

// What the cache holds: NVFP4 (packed as above), or FP8 E4M3 rows of D bytes for K and for V.
enum Format { kNvfp4 = 0, kFp8 = 1 };

template <int D, int F>
struct WGeo {
    static constexpr int TOK = ((D == 256) ? 32 : 64) >> F;  // tokens of a stage (8 or 9 KB of K and V)
    static constexpr int ROW = (F == kFp8) ? D : D / 2;      // bytes of a token's K
    static constexpr int SUB = TOK / 16;              // 16-token MMA tiles of a stage
    static constexpr int NB = D / 16;                 // blocks (= scales) per token row
    static constexpr int SK = TOK * ROW;              // packed K rows of a stage
    static constexpr int SV = TOK * ROW;              // V rows of D bytes (NVFP4: TOK / 2, of token pairs)
    static constexpr int SS = (F == kFp8) ? 0 : TOK * NB;  // one scale pool of a stage
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = SK;
    static constexpr int KS_OFF = SK + SV;
    static constexpr int VS_OFF = KS_OFF + SS;
    static constexpr int HDR_OFF = VS_OFF + SS;  // slot header (8 words; FP8: then the sub-tiles' scales of K, of V)
    static constexpr int SLOT = HDR_OFF + 32 + (F == kFp8 ? 16 : 0);
    static constexpr int SLOTS = 2;              // ring slots per warp: one in flight, one computed
    // warps of the one CTA per SM (register budget: 16 x 32 x 128, 12 x 32 x 170, 8 x 32 x 255)
    static constexpr int WARPS = (D == 64) ? 16 : (D == 128 ? 12 : 8);
    static constexpr int THREADS = WARPS * 32;
    static constexpr int RING = SLOTS * SLOT;     // per warp
    static constexpr int QCACHE = (D == 128) ? 8192 : 16384;  // queries of the CTA's pairs
    static constexpr int Q_OFF = WARPS * RING;
    static constexpr int SMEM = Q_OFF + QCACHE;
    static constexpr int KSTEPS = D / 16;       // k-steps of S^T = K Q^T
    static constexpr int CHUNK = ROW / 4;       // bytes of a row one quad lane owns
    static constexpr int CW = CHUNK / 4;        // ... as 32-bit words
    static constexpr int VCH = D / 16;          // 16-byte chunks per V pair row
    static constexpr int SWZ = (VCH < 8 ? VCH : 8) - 1;  // chunk XOR mask
    static constexpr int DCH = SK / (16 * 32);  // 16-byte chunks per lane of one data pool
    static constexpr int SUB_DIV = DCH / SUB;   // data chunk i of a lane lies in sub-tile i / SUB_DIV
    static constexpr int SCH = SS / 16;         // 16-byte chunks of one scale pool
    static constexpr int SC_PER_LANE = 2 * SCH / 32;
    static_assert(DCH * 32 * 16 == SK && DCH == SUB * SUB_DIV, "copy split");
    static_assert(SC_PER_LANE * 32 == 2 * SCH, "scale copy split");
    static_assert(F == kNvfp4 || 2 * SUB * 4 <= 16, "scales in the slot header");
    static_assert(SLOT % 16 == 0 && RING % 16 == 0, "16-byte aligned slots");
    static_assert(SMEM + 1024 + 512 <= kSmemPerSm, "shared memory budget");
};

// With a sliding window: a sequence of L tokens shows those from L - window on and the first `sinks`. FP8 pages have a
// scale for each page and head (null: 1).
struct WindowParams : DecodeParams {
    const float* kbs;  // [pool_pages][H]
    const float* vbs;
    int32_t window, sinks;
};

// FP8 rows in shared memory, 16-byte chunks XOR-swizzled so that the eight lanes of a quarter warp hit distinct banks.
// K: lanes (r, c) of rows r, r + 1 take chunk c D/64 + k; V: lanes of rows 2c take the chunk of dims rho D/8.
template <int D>
__device__ __forceinline__ uint32_t k8_swz(int row, int ch) {
    if constexpr (D == 64) return static_cast<uint32_t>(row * D + 16 * ch);
    else if constexpr (D == 128) return static_cast<uint32_t>(row * D + 16 * (ch ^ (row & 1)));
    else return static_cast<uint32_t>(row * D + 16 * (ch ^ (((ch >> 3) & 1) | ((row & 1) << 1))));
}
template <int D>
__device__ __forceinline__ uint32_t v8_swz(int row, int ch) {
    const int g = (row >> 1) & 3;
    if constexpr (D == 64)  // two rows to a 128-byte line
        return static_cast<uint32_t>((row >> 1) * 128 + 16 * (((row & 1) * 4 + ch) ^ ((g & 1) | ((g & 2) << 1))));
    else if constexpr (D == 128) return static_cast<uint32_t>(row * D + 16 * (ch ^ g));
    else return static_cast<uint32_t>(row * D + 16 * (ch ^ ((g << 1) | ((ch >> 3) & 1))));
}

// Log2 of the scale that V tiles of zeros get in place of 1: below the others', and far from where p s_V leaves FP32's range.
constexpr float kZeroLog = -50.0f, kZeroInv = 1125899906842624.0f;

// All lanes: every code of the 16 tokens of V from `row` on is 0, but for tokens that `seen` leaves out.
template <int D>
__device__ __forceinline__ bool zero_tile(uint32_t v, int row, uint32_t seen, int lane) {
    uint32_t some = 0u;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        const int i = lane + 32 * k, r = i / (D / 16);
        uint32_t w[4];
        lds_words(w, v + v8_swz<D>(row + r, i % (D / 16)));
        if ((seen >> r) & 1u) some |= (w[0] | w[1] | w[2] | w[3]) & 0x7F7F7F7Fu;
    }
    return !__any_sync(0xFFFFFFFFu, some != 0u);
}

// A device scalar that may be left out.
__device__ __forceinline__ float scalar_or_1(const float* p) { return p ? __ldg(p) : 1.0f; }

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The stages of a sequence with a window: those of the first tokens, then those from the window's first token on.
struct WindowStages {
    int lo;     // first token of the window; those between `sinks` and it are hidden
    int sink;   // stages of the first tokens that do not belong to the window's stages
    int first;  // first stage of the window
    int count;  // of both
};
__device__ __forceinline__ WindowStages window_stages(int L, int max_tokens, int tok, int window, int sinks) {
    WindowStages w;
    w.lo = L > window ? L - window : 0;
    w.sink = (min(sinks, w.lo) + tok - 1) / tok;
    w.first = max(w.lo / tok, w.sink);
    w.count = (L > 0 && L <= max_tokens) ? w.sink + (L + tok - 1) / tok - w.first : 0;
    return w;
}

template <int D, int F, bool WIN>
__global__ void __launch_bounds__(WGeo<D, F>::THREADS, 1) window_split_kernel(const WindowParams p) {
    pdl_enter();
    using G_ = WGeo<D, F>;
    constexpr int TOK = G_::TOK;
    constexpr int NW = G_::WARPS;
    constexpr int NT = G_::THREADS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int scan_warp[NW];
    __shared__ int start_bp[NW][3];  // run start of each warp: sequence, its first stage, length
    __shared__ int span_pair[2];     // first and last pair (b H + h) the CTA's runs touch
    __shared__ int pend_n;           // pairs whose last piece finished in this CTA ...
    __shared__ int pend[2 * NW][4];  // ... (b, h, first record, records): merged at the end

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int r = lane >> 2;  // row group of the MMA fragments
    const int c = lane & 3;   // column pair of the MMA fragments
    const int H = p.H, G = p.G, T = p.T;
    const int max_tokens = p.max_pages * T;
    const int window = WIN ? p.window : INT32_MAX, sinks = WIN ? p.sinks : 0;
    auto stages_of = [&](int L) { return window_stages(L, max_tokens, TOK, window, sinks).count; };

    // ------------------------------------------------ stage prefix over the sequences
    // Thread t owns sequences [t C, t C + C); PS_b = H * sum_{b' < b} stages(b').
    // The first two lengths stay in registers for the walk below (a second load of the same
    // words would cost another round trip at the start).
    const int C = (p.B + NT - 1) / NT;
    const int b_lo = min(p.B, tid * C), b_hi = min(p.B, b_lo + C);
    const int kept0 = (b_lo < b_hi) ? __ldg(p.seq_lens + b_lo) : 0;
    const int kept1 = (b_lo + 1 < b_hi) ? __ldg(p.seq_lens + b_lo + 1) : 0;
    auto len_of = [&](int b) {
        return b == b_lo ? kept0 : (b == b_lo + 1 ? kept1 : __ldg(p.seq_lens + b));
    };
    int local = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        const int L = len_of(b);
        if (blockIdx.x == 0 && (L < 0 || L > max_tokens))
            flag_status(p.status, NVFP4KV_STATUS_BAD_SEQ_LEN);
        local += H * stages_of(L);
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan_warp[warp] = incl;
    if (tid < 2) span_pair[tid] = 0;
    if (tid == 0) pend_n = 0;
    __syncthreads();
    int excl = incl - local, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) excl += scan_warp[w];
        total += scan_warp[w];
    }
    // warp run gw takes [gw W, gw W + W) of the stage list
    const int num_runs = p.num_runs;
    const int W = max(1, (total + num_runs - 1) / num_runs);
    if (blockIdx.x == 0) {
        // sequences without stages (length 0 or invalid): output 0, LSE -inf
        for (int b = b_lo; b < b_hi; ++b) {
            if (stages_of(__ldg(p.seq_lens + b)) != 0) continue;
            uint16_t* ob = p.out + static_cast<int64_t>(b) * p.Hq * D;
            for (int i = 0; i < p.Hq * D; ++i) ob[i] = 0;
            if (p.lse)
                for (int i = 0; i < p.Hq; ++i) p.lse[static_cast<int64_t>(b) * p.Hq + i] = -INFINITY;
        }
    }
    // One walk over this thread's sequences finds the sequence holding each of the CTA's run
    // starts and its two span ends (32-bit arithmetic: the host bounds stages + runs below 2^31).
    int gw0 = blockIdx.x * NW;
    int n_runs_cta = max(0, min(num_runs - gw0, NW));
    // Few runs are spread over the CTAs (a window leaves few stages: 136 of them, 8 pairs of 1005 tokens, on 9 of the 152
    // SMs took 14.2 us, spread over all 10.6): run k is at place k num_runs / R of all warps, and a CTA has the runs at
    // its places.
    const int R = (total + W - 1) / W;
    if (R < num_runs) {
        auto first_at = [&](int place) {
            return static_cast<int>((static_cast<int64_t>(place) * R + num_runs - 1) / num_runs);
        };
        const int end = min(R, first_at(gw0 + n_runs_cta));
        gw0 = min(R, first_at(gw0));
        n_runs_cta = max(0, end - gw0);
    }
    const int span_lo = (n_runs_cta > 0 && gw0 < (total + W - 1) / W) ? gw0 * W : total;
    const int span_hi = min(total, (gw0 + n_runs_cta) * W);
    if (local > 0 && span_lo < span_hi && span_lo < excl + local && span_hi > excl) {
        int acc = excl;
        for (int b = b_lo; b < b_hi && acc < span_hi; ++b) {
            const int L = len_of(b);
            const int S = stages_of(L);
            const int n = H * S;
            if (n > 0 && acc + n > span_lo) {
                // runs of this CTA starting in [acc, acc + n): w in [w_a, w_b)
                const int w_a = max(0, (acc - gw0 * W + W - 1) / W);
                const int w_b = min(n_runs_cta, (acc + n - gw0 * W + W - 1) / W);
                for (int w = w_a; w < w_b; ++w) {
                    start_bp[w][0] = b;
                    start_bp[w][1] = acc;
                    start_bp[w][2] = L;
                }
                if (span_lo >= acc && span_lo < acc + n) span_pair[0] = b * H + (span_lo - acc) / S;
                if (span_hi - 1 >= acc && span_hi - 1 < acc + n)
                    span_pair[1] = b * H + (span_hi - 1 - acc) / S;
            }
            acc += n;
        }
    }
    __syncthreads();

    // ------------------------------------------------ queries of the CTA's pairs
    const uint32_t smem_base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const uint32_t qcache = smem_base + G_::Q_OFF;
    const int q_first = span_pair[0];
    const int q_cached = (span_lo < span_hi)
                             ? min(span_pair[1] - span_pair[0] + 1, G_::QCACHE / (G * D * 2))
                             : 0;
    {
        const uint8_t* qsrc = reinterpret_cast<const uint8_t*>(p.q + static_cast<int64_t>(q_first) * G * D);
        const int nq = q_cached * G * D * 2 / 16;
        for (int ci = tid; ci < nq; ci += NT) cp_async16_plain(qcache + 16 * ci, qsrc + 16 * ci);
        cp_async_commit();
    }

    const int gw = gw0 + warp;
    const int64_t s_begin64 = static_cast<int64_t>(gw) * W;
    const bool has_run = warp < n_runs_cta && s_begin64 < total;
    const int s_begin = has_run ? static_cast<int>(s_begin64) : 0;
    const int n_st = has_run ? min(total - s_begin, W) : 0;

    // ------------------------------------------------ per-lane constants
    const uint32_t ring = smem_base + warp * G_::RING;
    // V chunk j = lane + 32 i of a stage lands XOR-swizzled by its pair row
    uint32_t v_dst[G_::DCH];
#pragma unroll
    for (int i = 0; i < G_::DCH; ++i) {
        const int j = lane + 32 * i;
        const int pr = j / G_::VCH, cj = j - pr * G_::VCH;
        if constexpr (F == kFp8) v_dst[i] = G_::V_OFF + v8_swz<D>(pr, cj);
        else v_dst[i] = G_::V_OFF + pr * D + 16 * (cj ^ (pr & G_::SWZ));
    }
    // K chunk lane + 32 i: at 512 i bytes from the lane's first (FP8 rows are swizzled by their parity, the same for all)
    const uint32_t k_dst = F == kFp8 ? G_::K_OFF + k8_swz<D>(lane / G_::VCH, lane % G_::VCH) : G_::K_OFF + 16 * lane;
    const int rho = (r >> 1) | ((r & 1) << 2);  // V rows of this lane: chunk rho of a pair row

    // ------------------------------------------------ issue side: the walk over the run
    int ib = has_run ? start_bp[warp][0] : 0;
    int ilen = has_run ? start_bp[warp][2] : 0;
    int iS = has_run ? stages_of(ilen) : 1;
    int ih = has_run ? (s_begin - start_bp[warp][1]) / iS : 0;
    int ij = has_run ? (s_begin - start_bp[warp][1]) - ih * iS : 0;
    int ips = has_run ? start_bp[warp][1] + ih * iS : 0;  // flat index of stage 0 of (ib, ih)
    bool ifirst = true;                     // the next stage to issue starts a piece
    int issued = 0;
    int nlen = (has_run && ib + 1 < p.B) ? __ldg(p.seq_lens + ib + 1) : 0;  // next sequence
    // page-id windows: lane l holds the id of page base + l of a sequence's page-table row; the
    // window after the current one (in issue order) is loaded when the current one is taken
    int wrow = -1, wbase = 0, win = 0;
    int prow = -1, pbase = 0, pwin = 0;
    auto load_window = [&](int b_, int base) -> int {
        const int i = base + lane;
        return (i < p.max_pages) ? __ldg(p.page_table + static_cast<int64_t>(b_) * p.max_pages + i)
                                 : -1;
    };
    // make the window holding page pidx of sequence ib current (its loads are only issued) and
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
            prow = (ih + 1 < H) ? ib : ib + 1;  // a zero-length next sequence makes this a miss
            pbase = 0;
        }
        if (prow < p.B && !(prow == wrow && pbase == wbase))
            pwin = load_window(prow, pbase);
        else
            prow = -1;
    };
    auto page_of = [&](int pidx) -> int {  // warp-uniform pidx of sequence ib; every lane calls
        if (ib != wrow || pidx < wbase || pidx >= wbase + 32) set_window(pidx);
        const int pg = __shfl_sync(0xFFFFFFFFu, win, pidx - wbase);
        return (pg >= 0 && pg < p.pool_pages) ? pg : -1;
    };

    const int64_t page_rows = static_cast<int64_t>(H) * T;
    const bool page_aligned = (T % TOK) == 0;
    // issue the next stage of the walk into `slot`, then advance the walk
    auto issue_next = [&](uint32_t slot) {
        const uint64_t kv_pol = l2_policy_evict_first();
        const WindowStages w = window_stages(ilen, max_tokens, TOK, window, sinks);
        const int t0 = (ij >= w.sink ? ij - w.sink + w.first : ij) * TOK;
        const int lo = w.lo;  // tokens of the sequence from `sinks` to lo are hidden by the window
        // sub-tile u has tokens of the sequence, and not all of them hidden
        auto seen = [&](int u) {
            return t0 + 16 * u < ilen && (!WIN || t0 + 16 * u + 15 >= lo || t0 + 16 * u < sinks);
        };
        const int nval = min(TOK, ilen - t0);
        const int64_t head_rows = static_cast<int64_t>(ih) * T;
        int64_t row0[G_::SUB];  // token row of each sub-tile in its pool, -1: not real
        [[maybe_unused]] int pgs[G_::SUB];
        if (page_aligned) {
            const int pidx = static_cast<int>(__umul64hi(static_cast<uint64_t>(t0), p.t_magic));
            const int pg = page_of(pidx);
            const int64_t r0 = pg * page_rows + head_rows + (t0 - pidx * T);
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u)
                row0[u] = (pg >= 0 && seen(u)) ? r0 + 16 * u : -1;
            if constexpr (F == kFp8) {
#pragma unroll
                for (int u = 0; u < G_::SUB; ++u) pgs[u] = pg;
            }
        } else {
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int t = t0 + 16 * u;
                const int pidx = static_cast<int>(__umul64hi(static_cast<uint64_t>(t), p.t_magic));
                // (warp-uniform; the page of a hidden sub-tile may have been given back)
                const int pg = seen(u) ? page_of(pidx) : -1;
                row0[u] = pg >= 0 ? pg * page_rows + head_rows + (t - pidx * T) : -1;
                pgs[u] = pg;
            }
        }
        uint32_t okbits = 0, want = 0;
#pragma unroll
        for (int u = 0; u < G_::SUB; ++u) {
            okbits |= (row0[u] >= 0 ? 1u : 0u) << u;
            want |= (seen(u) ? 1u : 0u) << u;
        }
        if (okbits != want && lane == 0) flag_status(p.status, NVFP4KV_STATUS_PAGE_OOB);
        if (page_aligned && okbits == (1u << G_::SUB) - 1) {
            // the whole stage is one run of each pool: offsets are compile-time constants
            const int64_t doff = row0[0] * G_::ROW + 16 * lane;
            const uint8_t* ksrc = p.kd + doff;
            const uint8_t* vsrc = p.vd + doff;
            static_for<G_::DCH>([&](auto I) {
                constexpr int i = decltype(I)::value;
                cp_async16<512 * i, 512 * i>(slot + k_dst, ksrc, kv_pol);
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
                const int jj = lane + 32 * i - u * G_::ROW;  // chunk within the sub-tile
                const bool ok = row0[u] >= 0;
                const int64_t off = ok ? row0[u] * G_::ROW + 16 * jj : 0;
                cp_async16_zfill(slot + k_dst + 512 * i, p.kd + off,
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
        if constexpr (F == kFp8) {
            // scales of the sub-tiles' pages: K's from lanes 0 .. SUB-1, V's from the next
            const int u = lane % G_::SUB;
            const float* pool = lane < G_::SUB ? p.kbs : p.vbs;
            int pg = pgs[0];
#pragma unroll
            for (int uu = 1; uu < G_::SUB; ++uu)
                if (u == uu) pg = pgs[uu];
            if (lane < 2 * G_::SUB && pool && ((okbits >> u) & 1u))
                cp_async4(slot + G_::HDR_OFF + 32 + 4 * lane, pool + static_cast<int64_t>(pg) * H + ih);
        }
        const bool last = (ij == iS - 1) || (issued == n_st - 1);
        const uint32_t flags = (ifirst ? kFirst : 0u) | (last ? kLast : 0u);
        if (lane == 0) {
            sts_v4(slot + G_::HDR_OFF, okbits | (static_cast<uint32_t>(nval) << 8), flags,
                   static_cast<uint32_t>(ib), static_cast<uint32_t>(ih));
            // the stage's tokens from the low half on to the high half are hidden
            const uint32_t hide = !WIN ? 0u
                                       : static_cast<uint32_t>(min(max(sinks - t0, 0), TOK)) |
                                             (static_cast<uint32_t>(min(max(lo - t0, 0), TOK)) << 16);
            sts_v4(slot + G_::HDR_OFF + 16, static_cast<uint32_t>(ips), static_cast<uint32_t>(iS),
                   hide, 0u);
        }
        // advance the walk
        ++issued;
        ifirst = false;
        if (last) {
            ij = 0;
            ips += iS;
            ifirst = true;
            if (issued < n_st && ++ih == H) {
                ih = 0;
                ++ib;
                ilen = nlen;
                iS = stages_of(ilen);
                while (iS == 0) {  // sequences without stages are not in the list
                    ++ib;
                    ilen = __ldg(p.seq_lens + ib);
                    iS = stages_of(ilen);
                }
                nlen = (ib + 1 < p.B) ? __ldg(p.seq_lens + ib + 1) : 0;
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
    const float gvs = F == kFp8 ? scalar_or_1(p.gv) : __ldg(p.gv);

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
            const int qpair = static_cast<int>(hdr[2]) * H + static_cast<int>(hdr[3]);
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
            const float gk = F == kFp8 ? scalar_or_1(p.gk) : __ldg(p.gk);
            const float cs_row = (r < G) ? p.sm_scale * gk * kLog2e * ldexpf(1.0f, -kq)
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
            uint32_t hide[1] = {0u};
            if constexpr (WIN) lds_words(hide, st + G_::HDR_OFF + 24);
            const int hide0 = hide[0] & 0xFFFFu, hide1 = hide[0] >> 16;
            const bool full = (okbits == (1u << G_::SUB) - 1) && nval >= TOK && hide0 >= hide1;
            // valid-token bits of each sub-tile (only read when !full)
            uint32_t tmask[G_::SUB];
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int nv = min(16, max(0, nval - 16 * u));
                tmask[u] = ((okbits >> u) & 1u) ? ((nv >= 16) ? 0xFFFFu : ((1u << nv) - 1u)) : 0u;
                const int a = min(16, max(0, hide0 - 16 * u)), b = min(16, max(0, hide1 - 16 * u));
                if (a < b) tmask[u] &= ~(((1u << b) - 1u) & ~((1u << a) - 1u));
            }
            // FP8 pages: with the page's scales s_K, s_V, a score x s_K + log2(s_V) (log2 units) makes the weight
            // p s_V, which is what the sum over V needs; the sum of the weights takes it times 1 / s_V
            [[maybe_unused]] float ksc[G_::SUB], vlog[G_::SUB], vinv[G_::SUB];
            if constexpr (F == kFp8) {
                uint32_t w[4];
                lds_words(w, st + G_::HDR_OFF + 32);
#pragma unroll
                for (int u = 0; u < G_::SUB; ++u) {
                    const bool ok = (okbits >> u) & 1u;
                    ksc[u] = ok && p.kbs ? __uint_as_float(w[u]) : 1.0f;
                    const float s = ok && p.vbs ? __uint_as_float(w[G_::SUB + u]) : 1.0f;
                    vlog[u] = lg2_approx(s);
                    vinv[u] = __fdividef(1.0f, s);
                }
            }

            // ---- S^T = K^ Q^T for the SUB sub-tiles
            float x[G_::SUB][4];
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                const int row0 = 16 * u + r;
                const int row1 = row0 + 8;
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (F == kFp8) {
                    // (head_dim 256 has one tile a stage: four sums, as a product waits for the one before into the same, take 86.1 us,
                    // so 87.4, for 32 sequences of 4096 tokens; with more tiles a stage two sums gained nothing)
                    constexpr int NS = D == 256 ? 4 : 1;
                    float part[NS][4] = {};
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        uint32_t w0[4], w1[4];
                        lds_words(w0, st + G_::K_OFF + k8_swz<D>(row0, c * (D / 64) + k));
                        lds_words(w1, st + G_::K_OFF + k8_swz<D>(row1, c * (D / 64) + k));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t c0[2], c1[2];
                            e4m3x4_to_f16x2x2(w0[q], c0);
                            e4m3x4_to_f16x2x2(w1[q], c1);
                            const uint32_t a[4] = {c0[0], c1[0], c0[1], c1[1]};
                            mma_f16_16816(part[(4 * k + q) % NS], a, qf[4 * k + q][0], qf[4 * k + q][1]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < NS; ++j) acc[i] += part[j][i];
                } else {
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
                }
                if constexpr (F == kFp8) {
                    const float c0 = cs0 * ksc[u], c1 = cs1 * ksc[u];
                    x[u][0] = fmaf(acc[0], c0, vlog[u]);
                    x[u][1] = fmaf(acc[1], c1, vlog[u]);
                    x[u][2] = fmaf(acc[2], c0, vlog[u]);
                    x[u][3] = fmaf(acc[3], c1, vlog[u]);
                } else {
                    x[u][0] = acc[0] * cs0;
                    x[u][1] = acc[1] * cs1;
                    x[u][2] = acc[2] * cs0;
                    x[u][3] = acc[3] * cs1;
                }
            }

            // ---- online softmax over the stage, columns = query heads 2c, 2c+1
            if (!full) {
#pragma unroll
                for (int u = 0; u < G_::SUB; ++u) {
                    if (!((tmask[u] >> r) & 1u)) x[u][0] = x[u][1] = -INFINITY;
                    if (!((tmask[u] >> (r + 8)) & 1u)) x[u][2] = x[u][3] = -INFINITY;
                }
            }
            float mx0, mx1;
            auto maxima = [&]() {
                float lm0 = fmaxf(x[0][0], x[0][2]), lm1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
                for (int u = 1; u < G_::SUB; ++u) {
                    lm0 = fmaxf(lm0, fmaxf(x[u][0], x[u][2]));
                    lm1 = fmaxf(lm1, fmaxf(x[u][1], x[u][3]));
                }
                column_maxima(lm0, lm1, mx0, mx1);
                return (mx0 > m0 + kRescaleThreshold) || (mx1 > m1 + kRescaleThreshold);
            };
            bool grow = maxima();
            if constexpr (F == kFp8) {
                if (p.vbs && __any_sync(0xFFFFFFFFu, grow)) {
                    bool zeros = false;
                    uint32_t w[4];
                    lds_words(w, st + G_::HDR_OFF + 32);
#pragma unroll
                    for (int u = 0; u < G_::SUB; ++u)
                        if (((okbits >> u) & 1u) && w[G_::SUB + u] == __float_as_uint(1.0f) &&
                            zero_tile<D>(st + G_::V_OFF, 16 * u, tmask[u], lane)) {
                            zeros = true;
                            vinv[u] = kZeroInv;
#pragma unroll
                            for (int k = 0; k < 4; ++k) x[u][k] += kZeroLog;
                        }
                    if (zeros) grow = maxima();
                }
            }
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
                if constexpr (F == kFp8) {
                    l0 = fmaf(p0 + p2, vinv[u], l0);
                    l1 = fmaf(p1 + p3, vinv[u], l1);
                } else {
                    l0 += p0 + p2;
                    l1 += p1 + p3;
                }
                // P^T (tokens x heads) -> B operand (k = tokens, n = heads), rounded to FP16: 11 bits
                // where the output has 8, and FP16 is what V is exact in; the sum takes p as it is
                pb[u][0] = movmatrix_trans(pack_f16x2(p0, p1));
                pb[u][1] = movmatrix_trans(pack_f16x2(p2, p3));
            }

            // ---- O^T += V^^T P^T. Lane pairs: pr0 (tokens 2c, 2c+1), pr1 (tokens 2c+8, 2c+9)
#pragma unroll
            for (int u = 0; u < G_::SUB; ++u) {
                if constexpr (F == kFp8) {
                    // the lane's chunk of tokens 2c, 2c + 1, 2c + 8, 2c + 9; pairs of tokens are made byte by byte
                    constexpr int VW = D / 32;
                    uint32_t vw[4][VW];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int row = 16 * u + 2 * c + (t & 1) + 8 * (t >> 1);
                        if constexpr (D == 64) {
                            lds_words(vw[t], st + G_::V_OFF + v8_swz<D>(row, rho >> 1) + 8 * (rho & 1));
                        } else {
#pragma unroll
                            for (int k = 0; k < D / 128; ++k)
                                lds_words(*reinterpret_cast<uint32_t(*)[4]>(vw[t] + 4 * k),
                                          st + G_::V_OFF + v8_swz<D>(row, rho * (D / 128) + k));
                        }
                        // a hidden token's V may be anything, and 0 times it need not be 0
                        if (!full && !((tmask[u] >> (row - 16 * u)) & 1u))
#pragma unroll
                            for (int k = 0; k < VW; ++k) vw[t][k] = 0u;
                    }
#pragma unroll
                    for (int q = 0; q < VW; ++q) {
#pragma unroll
                        for (int hm2 = 0; hm2 < 2; ++hm2) {
                            uint32_t lo2[2], hi2[2];
                            e4m3x4_to_f16x2x2(__byte_perm(vw[0][q], vw[1][q], hm2 ? 0x7362 : 0x5140), lo2);
                            e4m3x4_to_f16x2x2(__byte_perm(vw[2][q], vw[3][q], hm2 ? 0x7362 : 0x5140), hi2);
                            const uint32_t a[4] = {lo2[0], lo2[1], hi2[0], hi2[1]};
                            mma_f16_16816(o[2 * q + hm2], a, pb[u][0], pb[u][1]);
                        }
                    }
                    continue;
                }
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
                    // tokens past the sequence end in a real page: their V scales may be
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

        if (flags & kLast) {
            // ---- end of a piece: the whole pair (outputs) or a record
            uint32_t h2[4];
            lds_words(h2, st + G_::HDR_OFF + 16);
            const int pb_ = static_cast<int>(hdr[2]), ph = static_cast<int>(hdr[3]);
            const int pps = static_cast<int>(h2[0]), pS = static_cast<int>(h2[1]);
            float ls0 = l0, ls1 = l1;
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                ls0 += __shfl_xor_sync(0xFFFFFFFFu, ls0, off);
                ls1 += __shfl_xor_sync(0xFFFFFFFFu, ls1, off);
            }
            const int g0 = 2 * c, g1 = 2 * c + 1;
            const int gf = pps / W, gl = (pps + pS - 1) / W;
            const int64_t bh = static_cast<int64_t>(pb_) * H + ph;
            if (gf == gl) {
                // the whole pair is this piece: normalise and write the output directly
                uint16_t* ob = p.out + (static_cast<int64_t>(pb_) * p.Hq + ph * G) * D;
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
                    float* lb = p.lse + static_cast<int64_t>(pb_) * p.Hq + ph * G;
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
                        pend[slot][0] = pb_;
                        pend[slot][1] = ph;
                        pend[slot][2] = static_cast<int>(gf + bh);
                        pend[slot][3] = gl - gf + 1;
                    }
                }
            }
        }
        __syncwarp();  // every lane is done reading the slot before it refills
    }
    cp_async_wait<0>();
    __syncthreads();  // every warp's run is done: the rings are free for the merge
    const int n_pend = pend_n;
    for (int k = 0; k < n_pend;) {
        const int m = merge_batch<D, G_, F == kFp8>(p, pend, k, n_pend, smem);
        if (m == 0) {  // a pair whose records do not fit at once: by chunks
            merge_pair<D, G_, F == kFp8>(p, pend[k][0], pend[k][1], pend[k][2], pend[k][3], smem);
            ++k;
        }
        k += m;
    }
}

bool window_size_ok(int batch, int H, int D, int max_pages, int T, int64_t runs, Format format) {
    return stage_list_ok(batch, H, stage_tokens(D) >> format, max_pages, T, runs);
}

template <int D, int F, bool WIN>
cudaError_t launch_window(const WindowParams& p, int64_t runs, cudaStream_t s) {
    using G_ = WGeo<D, F>;
    const cudaError_t e = cudaFuncSetAttribute(window_split_kernel<D, F, WIN>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, G_::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t ctas = (runs + G_::WARPS - 1) / G_::WARPS;
    return launch_pdl(window_split_kernel<D, F, WIN>, static_cast<unsigned>(ctas), G_::THREADS,
                      static_cast<size_t>(G_::SMEM), s, p);
}

}  // namespace
}  // namespace nvfp4kv
