// Attention of an extend step: the rows of each sequence's chunk over its FP8 pages, causal, with an optional sliding
// window and first tokens that stay visible (LMSYS, "Accelerating Long-Context and Agentic Inference with NVFP4 KV
// Cache": "Path 2: Chunked prefill / Extend", whose attention reads the FP8 workspace).
//
// Work. The query heads of a KV head share its keys, so a row tile of M = 128 rows holds floor(128 / G) tokens times the G
// heads of a group. A unit is a block of such rows (two row tiles at head_dim 64 and 128, one at 256) of one sequence and KV
// head; its work is the list of KV tiles (128 tokens, 64 at head_dim 256) that hold a token visible to a row of it. The
// tiles of all units form one list, cut into equal parts, one per SM: a part that begins or ends inside a unit leaves a
// partial result (row maxima, sums, unnormalised output) that a second kernel joins. Cuts close to a unit's border are
// moved onto it. The cuts are made from the lengths, by every CTA for itself.
//
// A CTA per SM, with a role for each warp:
//  * The scout walks over the CTA's part and writes into a ring where each tile lies and what the others need to know of it.
//  * 4 loader warps each for K and V bring the tiles in. FP8 values have to pass through registers to become FP16 (exact), so
//    they are loaded there directly and stored in the 128-byte-swizzled layout that tcgen05.mma reads: K with the head dims
//    contiguous (K-major), V with the same store and read as MN-major.
//  * A warp per row tile issues its S = Q K^T and O += P V (tcgen05.mma, FP16 in, FP32 accumulators in TMEM), in steps of 64
//    tokens. P lies in TMEM over the scores it came from. Each row tile has two slots of scores, so a step's scores are there
//    when its softmax begins.
//  * 4 softmax warps per row tile, one row a thread, so that row maxima and sums need no exchange.
// The running maximum moves only when it grows by more than 2^8, so rescaling O in TMEM is rare.
//
// NaN. A hidden token's score is set to -inf, but its weight 0 times a NaN in V is NaN. A tile that hides a token from one row of its
// unit and not from another (`uneven`: the last tokens of a chunk, a window's begin) is stored with NaN codes of V as 0, and where
// there were any, the join looks for those that each row sees and puts NaN into their dims. A page whose scale is not
// finite (nvfp4_kv_fp8_pages, of a page with NaN) has NaN keys instead, so that the rows that see it are NaN and no others.
//
// Scales. With a page's scales s_K, s_V, a score becomes x = S c s_K + log2(s_V) in log2 units, so that p = 2^(x - m) is the
// weight times s_V, as the sum over V needs it, with one FMA and one 2^x an element; the sum of the weights takes p / s_V. Q is
// brought to [2^14, 2^15) by a power of two a row (exact in FP16 but for elements below 2^-31 of the row's largest); P is rounded
// to FP16 (11 bits, where the output has 8). P is relative to the largest p s_V, so a page must not raise that for nothing: V of a page
// without a value has scale 1, whatever the others' scales, and beside pages of 2^-20 it would leave them in FP16's subnormals. The
// scout looks at groups of scale 1 where the sequence has others, and those that are all 0 take part with a scale of 2^-50 (any is right
// for them).
//
// Measured (one GB300): 16 chunks of 512 rows behind 4096 tokens, 32 heads on 8, head_dim 128 (584 GFLOP): 510 us, 1145 TFLOP/s,
// 0.59 of the bf16 product rate; 2048 rows at 65536 tokens (2.16 TFLOP): 1.66 ms, 1300 TFLOP/s, 0.67; 24 ragged sequences with a
// window at head_dim 64 (15.6 GFLOP): 60 us; 8 chunks of 256 rows behind 4096 tokens at head_dim 256 (284 GFLOP), which has one row
// tile and 64 tokens a KV tile: 406 us, 700 TFLOP/s, 0.36. A few per cent from one GPU to another; further times here are from one each.
// The flags for NaN cost 0.5 % of the long cases, 1 to 2 % of ragged ones, 1.4 of 18 us for a single row at 3000 tokens.
// Bound, at head_dim 128: the tensor core, busy for nine tenths of the time (in the long case, 3600 clocks for 256 x 128 scores),
// with products at less than its rate. A 128 x 64 x 16 product with both operands in shared memory takes 72 clocks, hardly more than
// a 128 x 128 x 16 one (64): its 128 rows of Q have to be read either way. Scores of 128 tokens at once leave no room in TMEM (512
// columns) for two slots beside two outputs, and then the softmax waits for its scores: 640 to 730 us for the 16 chunks, in
// three arrangements.
// Pairs of CTAs (cta_group::2, a row tile in each, half of each KV tile loaded by each, three slots of 128 scores) keep the
// tensor core busy for 42 % alone: the two softmax warps of a scheduler then share their rows and work in step, maxima while the
// other's are taken and powers of two while the other's are; 604 us (1.86 ms the long case). The two row tiles of a CTA
// alternate by themselves.
// What it took, for the 16 chunks: 975 us with one issuing lane and scores read from TMEM twice; 683 a row's scores in registers, packed
// FMAs, pool addresses once a tile; 641 in steps of 64 tokens with two slots; 627 the scout, so that the roles' code fits the
// instruction cache (90 KB of code had warps waiting for instructions 15 % of the time), and products issued by an elected lane
// (the instruction takes its operands from uniform registers; with a lane that the compiler does not know to be one alone, it
// fills them in a loop over lanes); 551 a tile's place read from shared memory while its scores come from TMEM, as shared memory
// is slow beside the tensor core's reads; 529 queries in one pass and no divisions in the walk; 521 the next piece's queries
// before this one's outputs; 509 a tile's barriers waited for at once (the long case 1.69 ms before, 1.98 with cuts moved by up to
// an eighth of a part).
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "host_util.h"

using namespace nvfp4kv;

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kZeroScale = 8.8817841970012523e-16f;  // 2^-50: of V that is all 0, below the others', far from where p s_V leaves FP32's range
constexpr float kTiny = 1.1754943508222875e-38f;  // 2^-126: the least factor of a score (0 would turn a hidden one, -inf, into NaN)
constexpr int kMaxGroup = 8;
constexpr int kRowsM = 128;       // rows of a tile
constexpr int kStep = 64;         // tokens of a step: scores, weights, product with V
constexpr int kLoaderWarps = 4;   // for K, and as many for V
// Tiles that a cut may move to meet a unit's border, and at most an eighth of a part: parts of unequal length against partial results
// (2, 6, 24 tiles: 16 chunks 516, 515, 509 us, 2048 rows at 65536 tokens 1.60, 1.60, 1.62 ms; an eighth alone, 110 tiles there, 1.98).
constexpr int kSlack = 24;
constexpr int kUnitCost = 1;      // of a unit beside its tiles: queries in, outputs out (in tiles)
// A wait gives up after kTries tries of at most about kTryNs, seconds (a defect: no wait depends on another CTA).
constexpr uint32_t kTryNs = 2000, kTries = 2000000;

template <int D>
struct Shape {
    static constexpr int MT = D == 256 ? 1 : 2;      // row tiles of a unit
    static constexpr int TK = D == 256 ? 64 : 128;   // tokens of a KV tile
    static constexpr int GRP = TK / 16;              // 16-token groups, each in one page
    static constexpr int BLOCKS = D / 64;            // 128-byte columns of a 16-bit row
    static constexpr int QB = kRowsM * D * 2;        // bytes of a tile's queries
    static constexpr int KB = TK * D * 2;            // bytes of a tile of K or V
    static constexpr int STAGES = 2;
    static constexpr int K_OFF = MT * QB;
    static constexpr int V_OFF = K_OFF + STAGES * KB;
    static constexpr int SMEM = V_OFF + STAGES * KB + 1024;  // the base is rounded up to 1024
    static constexpr int SOFT_WARPS = 4 * MT;
    static constexpr int WARPS = SOFT_WARPS + 2 * kLoaderWarps + 4;  // (the issuers' warpgroup: they, the scout, one that finds the part's end, and an idle one where MT = 1)
    static constexpr int THREADS = WARPS * 32;
    static constexpr int STEPS = TK / kStep;         // of a KV tile
    // TMEM columns: two slots of scores for each row tile, then the outputs
    static constexpr int O_COL = MT * 2 * kStep;
    static_assert(O_COL + MT * D <= 512, "TMEM");
    static_assert(SMEM <= 232448 - 1024, "shared memory");
};

struct PlanEntry {
    int64_t cut;     // first position of this CTA in the list of units and tiles
    int64_t begin;   // of the unit that holds it: its first position ...
    int64_t end;     // ... and its end
    int32_t b, h, qb, tile;  // the unit, and the first tile
    int32_t nan, unused;     // the CTA met NaN in V of a tile that is not seen evenly
};

struct ExtendParams {
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const float* kbs;
    const float* vbs;
    const float* gk;
    const float* gv;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    uint16_t* out;
    float* lse;
    int32_t* status;
    PlanEntry* plan;    // [ctas + 1]
    float* rec_o;       // [2 ctas][MT * 128][D]
    float2* rec_ml;     // [2 ctas][MT * 128]
    int64_t q_stride, out_stride;
    uint64_t t_magic;
    int32_t B, rows, Hq, H, G, T, pool_pages, max_pages, window, sinks, ctas;
    int32_t per;  // tokens of a row tile, floor(128 / G)
    uint32_t unit_magic;  // ceil(2^32 / tokens of a unit)
    float sm_scale;
};

// ------------------------------------------------------------------------------------------ what a unit is

// A sequence's rows [first, first + n) and length; n = 0 for one without rows or with lengths out of range.
struct Seq {
    int first, n, len;
    bool bad;
};
__device__ __forceinline__ Seq sequence(const ExtendParams& p, int b) {
    const int a = __ldg(p.starts + b), e = __ldg(p.starts + b + 1), len = __ldg(p.lens + b);
    Seq s{a, e - a, len, false};
    if (a < 0 || e < a || e > p.rows) return Seq{0, 0, 0, true};
    if (len < 0 || len > p.max_pages * p.T || s.n > len) {
        s.bad = true;
        s.n = 0;
    }
    return s;
}

// Block qb of a sequence's rows: tokens [t0, t1) of the chunk, and its KV tiles: `sink` tiles of the first tokens, then
// those from `first` on.
struct Unit {
    int t0, t1;    // tokens of the chunk
    int lo, hi;    // tokens [lo, hi) of the sequence, and the first `sinks`, are visible to a row of it
    int sink, first, tiles;
};
template <int D>
__device__ __forceinline__ Unit unit_of(const ExtendParams& p, const Seq& s, int qb) {
    using G_ = Shape<D>;
    const int each = G_::MT * p.per;
    Unit u;
    u.t0 = qb * each;
    u.t1 = min(s.n, u.t0 + each);
    const int p0 = s.len - s.n + u.t0;
    u.hi = s.len - s.n + u.t1;
    u.lo = p0 >= p.window ? p0 - p.window + 1 : 0;
    constexpr unsigned kTk = G_::TK;  // (unsigned: shifts)
    u.sink = static_cast<int>((static_cast<unsigned>(min(p.sinks, u.lo)) + kTk - 1) / kTk);
    u.first = max(static_cast<int>(static_cast<unsigned>(u.lo) / kTk), u.sink);
    u.tiles = u.sink + static_cast<int>((static_cast<unsigned>(u.hi) + kTk - 1) / kTk) - u.first;
    return u;
}
// Tile t0 hides a token from one row of the unit, whose first row has position p0, and not from another.
template <int D>
__device__ __forceinline__ bool uneven(const ExtendParams& p, const Unit& u, int p0, int t0) {
    return p0 + 1 < u.hi && (t0 + Shape<D>::TK - 1 > p0 || (t0 < u.hi - p.window && t0 + Shape<D>::TK > p.sinks));
}
// ceil(n / tokens of a unit): the magic number's quotient may be one too large, where n is large.
template <int D>
__device__ __forceinline__ int blocks_of(const ExtendParams& p, int n) {
    const int each = Shape<D>::MT * p.per;
    int q = static_cast<int>(__umulhi(static_cast<unsigned>(n), p.unit_magic));
    q -= static_cast<int64_t>(q) * each > n;
    return q + (q * each != n);
}
template <int D>
__device__ __forceinline__ int tile_start(const Unit& u, int j) {
    return (j < u.sink ? j : j - u.sink + u.first) * Shape<D>::TK;
}

// ------------------------------------------------------------------------------------------ the cuts

// Positions in the list that one KV head of a sequence takes, summed by a whole warp or by one thread.
template <int D>
__device__ __forceinline__ int64_t cost_of(const ExtendParams& p, const Seq& s, int lane, int lanes) {
    int64_t sum = 0;
    for (int qb = lane, n = blocks_of<D>(p, s.n); qb < n; qb += lanes) sum += unit_of<D>(p, s, qb).tiles + kUnitCost;
    return sum;
}
__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Every CTA makes the list for itself: thread t owns sequences [t C, t C + C), and chunk[t] is where they begin. (A kernel of its
// own that made all cuts took 17 us; this takes about 2, while the CTA sets itself up.) Returns the list's length. All threads.
template <int D>
__device__ __forceinline__ int64_t list_sequences(const ExtendParams& p, int64_t* chunk, int64_t* part) {
    constexpr int NT = Shape<D>::THREADS, kSerial = 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (p.B + NT - 1) / NT;
    int64_t local = 0;
    for (int i = 0; i < each; ++i) {  // (the same for all threads, so that a warp can share its long sequences)
        const int b = tid * each + i;
        Seq s{0, 0, 0, false};
        if (b < p.B) s = sequence(p, b);
        if (s.bad && blockIdx.x == 0) flag_status(p.status, NVFP4KV_STATUS_BAD_SEQ_LEN);
        const bool is_long = blocks_of<D>(p, s.n) > kSerial;
        if (!is_long) local += cost_of<D>(p, s, 0, 1);
        for (uint32_t left = __ballot_sync(0xFFFFFFFFu, is_long); left; left &= left - 1) {
            const int l = __ffs(static_cast<int>(left)) - 1;
            Seq t{0, __shfl_sync(0xFFFFFFFFu, s.n, l), __shfl_sync(0xFFFFFFFFu, s.len, l), false};
            const int64_t c = warp_sum64(cost_of<D>(p, t, lane, 32));
            if (lane == l) local += c;
        }
    }
    local *= p.H;
    const int64_t incl = warp_scan64(local, lane);
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    int64_t at = incl - local, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) at += part[w];
        total += part[w];
    }
    chunk[tid] = at;
    __syncthreads();
    return total;
}

// The unit at position x (below the list's length), found by a warp together.
template <int D>
__device__ __forceinline__ PlanEntry find_unit(const ExtendParams& p, const int64_t* chunk, int64_t x, int lane) {
    constexpr int NT = Shape<D>::THREADS;
    PlanEntry e{};
    int lo = 0, hi = NT;
    while (hi - lo > 1) {  // the last chunk that begins at or before x
        const int mid = (lo + hi) >> 1;
        if (chunk[mid] <= x) lo = mid; else hi = mid;
    }
    int64_t at = chunk[lo], per_head;
    Seq s;
    for (e.b = lo * ((p.B + NT - 1) / NT);; ++e.b) {
        if (e.b >= p.B) {  // (only where lengths change under the call)
            e.begin = e.end = x;
            return e;
        }
        s = sequence(p, e.b);
        per_head = warp_sum64(cost_of<D>(p, s, lane, 32));
        if (x < at + per_head * p.H) break;
        at += per_head * p.H;
    }
    e.h = static_cast<int>((x - at) / per_head);
    at += e.h * per_head;
    const int nqb = blocks_of<D>(p, s.n);
    for (int q0 = 0; q0 < nqb; q0 += 32) {
        const int64_t c = q0 + lane < nqb ? unit_of<D>(p, s, q0 + lane).tiles + kUnitCost : 0;
        const int64_t incl = warp_scan64(c, lane);
        const uint32_t in = __ballot_sync(0xFFFFFFFFu, c > 0 && x < at + incl);
        if (in) {
            const int l = __ffs(static_cast<int>(in)) - 1;
            e.qb = q0 + l;
            e.end = at + __shfl_sync(0xFFFFFFFFu, incl, l);
            e.begin = e.end - __shfl_sync(0xFFFFFFFFu, c, l);
            break;
        }
        at += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    return e;
}

// Where CTA c's part begins: c-th of equal parts, on the border of a unit where that is near.
template <int D>
__device__ __forceinline__ PlanEntry cut_at(const ExtendParams& p, const int64_t* chunk, int64_t total, int c, int lane) {
    const int64_t share = (total + p.ctas - 1) / p.ctas, slack = min(share / 8, static_cast<int64_t>(kSlack));
    int64_t x = min(total, share * c);
    PlanEntry e{};
    e.begin = e.end = x;
#pragma unroll 1
    while (x < total) {
        e = find_unit<D>(p, chunk, x, lane);
        if (x - e.begin <= max(slack, static_cast<int64_t>(kUnitCost))) {
            x = e.begin;
            break;
        }
        if (e.end - x > slack) break;
        x = e.begin = e.end;  // the next unit's begin, if there is one
    }
    e.cut = x;
    e.tile = static_cast<int32_t>(max(static_cast<int64_t>(0), x - e.begin - kUnitCost));
    return e;
}

// The pieces of a CTA's part, in order.
template <int D>
struct Walk {
    int64_t pos, end, unit_begin;
    int b, h, qb, tile0, piece_tiles;
    Seq s;
    Unit u;
    __device__ __forceinline__ void start(const ExtendParams& p, const PlanEntry& e, int64_t part_end) {
        pos = e.cut;
        end = part_end;
        unit_begin = e.begin;
        b = e.b;
        h = e.h;
        qb = e.qb;
        tile0 = e.tile;
        if (b >= p.B) pos = end;
        if (pos < end) {
            s = sequence(p, b);
            measure(p);
        }
    }
    __device__ __forceinline__ void measure(const ExtendParams& p) {
        u = unit_of<D>(p, s, qb);
        const int64_t unit_end = unit_begin + kUnitCost + u.tiles;
        piece_tiles = unit_end <= end ? u.tiles - tile0 : static_cast<int>(end - unit_begin - kUnitCost) - tile0;
    }
    __device__ __forceinline__ bool more() const { return pos < end; }
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && piece_tiles == u.tiles; }
    __device__ __forceinline__ void next(const ExtendParams& p) {
        unit_begin += kUnitCost + u.tiles;
        pos = unit_begin;
        tile0 = 0;
        if (pos >= end) return;
        if (++qb >= blocks_of<D>(p, s.n)) {
            qb = 0;
            if (++h == p.H) {
                h = 0;
                do {
                    if (++b >= p.B) {  // (as above)
                        pos = end;
                        return;
                    }
                    s = sequence(p, b);
                } while (s.n == 0);
            }
        }
        measure(p);
    }
};

// ------------------------------------------------------------------------------------------ PTX

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("{\n\t.reg .b64 s;\n\tmbarrier.arrive.shared::cta.b64 s, [%0];\n\t}" ::"r"(bar) : "memory");
}
// (returns after kTryNs at the latest)
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity), "n"(kTryNs) : "memory");
    return ok != 0;
}
// A warp waits for the phase of this parity. Once a wait of the CTA has given up, `dead`, none waits any more: every role runs
// on over the places that are there until it meets the end of the list, which is what places that were never written say, and what the
// scout makes of all of them as soon as it sees `dead`. A place may then be read while it is written, so each of its words is in
// bounds by itself, with whatever flags it is read: rows of the pool (0 where a group has none), rows of q, heads.
__device__ __forceinline__ void warp_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (uint32_t i = 0; !__all_sync(0xFFFFFFFFu, mbar_try(bar, parity)); ++i) {
        if (i == kTries) *dead = 1;
        if (__any_sync(0xFFFFFFFFu, *dead)) return;
    }
}
// A value that is the same in all lanes, so that the compiler knows it.
__device__ __forceinline__ int uniform(int x) { return static_cast<int>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(x))); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// One lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand of tcgen05.mma: 128-byte swizzle, start address and byte offsets in units of 16. For K-major
// operands `stride` is the distance of 8-row groups; for MN-major ones `lead` that of 64-element columns and `stride`
// that of groups of 8 along K.
struct Operand {
    uint32_t lo, hi;
    // `bytes` further on (a multiple of 16; the address field does not overflow)
    __device__ __forceinline__ uint64_t at(uint32_t bytes) const { return static_cast<uint64_t>(hi) << 32 | (lo + (bytes >> 4)); }
};
__device__ __forceinline__ Operand operand(uint32_t addr, uint32_t lead, uint32_t stride) {
    Operand o{((addr & 0x3FFFFu) >> 4) | (lead >> 4) << 16, (stride >> 4) | 1u << 14 | 2u << 29};
    asm volatile("" : "+r"(o.lo));  // the steps' descriptors are made when they are used, not kept in registers for the whole kernel
    return o;
}
// Instruction descriptor: FP16 operands, FP32 accumulators, M = 128, N; B K-major or MN-major.
__host__ __device__ constexpr uint32_t instruction(int n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n) >> 3) << 17 | (128u >> 4) << 24;
}
// D (+)= A B over 64 values of K: A and B K-major, four steps of 32 bytes. (These are called by the lane that elect_one chose: the
// instruction takes its operands from uniform registers, and with a lane that the compiler cannot know to be one alone it
// moves them there in a loop over lanes.)
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D (+)= A B over 32 values of K: A in TMEM, B MN-major, two steps of 16 rows of 128 bytes.
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.s64 b, %2, 128;\n\tadd.s32 a, %1, 8;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 columns of this warp's lanes (with the wait: nothing may use the registers before it).
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// The scores of a step, of this warp's lanes.
__device__ __forceinline__ void tmem_ld_row(uint32_t (&r)[64], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,"
        "%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr));
}
// (a, b) * c + d and (a, b) + (c, d), each rounded as by the scalar instructions.
__device__ __forceinline__ void fma2(uint32_t& a, uint32_t& b, float c, float d) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+r"(a), "+r"(b) : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& a, float& b, uint32_t c, uint32_t d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b) : "r"(c), "r"(d));
}
__device__ __forceinline__ uint4 ldg16(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float scalar_or_1(const float* p) { return p ? __ldg(p) : 1.0f; }

// ------------------------------------------------------------------------------------------ the attention

constexpr uint32_t kNoRow = 0xFFFFFFFFu;
constexpr uint32_t kRing = 8;

enum PlaceFlags {
    kFirst = 1,   // tile of a piece (the part of a unit that this CTA does)
    kLast = 2,
    kEnd = 4,     // last tile of the CTA's part
    kTwo = 8,     // the unit has its second row tile
    kFull = 16,   // every token of the tile is there and visible to a row
    kWhole = 32,  // the piece is its unit
    kGoesOn = 64, // the piece goes on with a unit that another CTA began
    kNothing = 128, // the CTA's part is empty
    kMissing = 1 << 8,  // times 2^g: group g is not to be read: no page, or no token a row sees
    kNoNumber = 1 << 16, // times 2^g: group g has a scale that is not finite
    kUneven = 1 << 24   // a token of the tile is hidden from one row of the unit and not from another
};
constexpr int kOver = kNothing | kLast | kEnd;  // no tile, and none after it

// What the other roles need of a KV tile: of its 16-token groups the first token's row in the pools (0 where it is not to be
// read) and the scales (s_K, log2 s_V, 1 / s_V); its first token, and its unit: visible are tokens lo .. hi and
// the first ones; rows of tokens c0 .. c1 of the chunk, whose row 0 is `row0` and has position pos0; KV head h.
struct Place {
    float4 scales[8];
    uint32_t row[8];
    int4 head;  // flags, t0, lo, hi
    int4 unit;  // c0, c1, row0, pos0
    int h;
};

struct Shared {
    uint64_t full[2][2], empty[2][2];       // [K, V][stage]
    uint64_t qfull[2], ofull[2];             // [row tile]
    uint64_t sfull[2][2], pfull[2][2];       // [row tile][slot]
    uint64_t drained, ended;
    int64_t part_end;
    int64_t part[Shape<64>::WARPS];  // (as many as any)
    uint64_t placed[kRing];
    Place ring[kRing];
    uint32_t loaded;  // tiles of V that its first loader warp has stored
    uint32_t tmem;
    int dead;   // a wait gave up
    int never;  // (stays 0)
};

// Whether a page among the first ones of sequence b, of `tokens` tokens, has a V scale for head h that is not 1. A whole warp.
__device__ __forceinline__ bool scales_differ(const ExtendParams& p, int b, int h, int tokens, int lane) {
    const int pages = (tokens + p.T - 1) / p.T;
    constexpr int U = 4;
#pragma unroll 1
    for (int j0 = 0; j0 < pages; j0 += 32 * U) {
        int page[U];
        float s[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int j = j0 + 32 * k + lane;
            page[k] = j < pages ? __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + j) : -1;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) s[k] = page[k] >= 0 && page[k] < p.pool_pages ? __ldg(p.vbs + static_cast<int64_t>(page[k]) * p.H + h) : 1.0f;
        if (__any_sync(0xFFFFFFFFu, s[0] != 1.0f || s[1] != 1.0f || s[2] != 1.0f || s[3] != 1.0f)) return true;
    }
    return false;
}

// The groups of a tile (a lane for each; `ones`: those to look at) whose V is 0 in every token that a row of the unit sees. `row` and
// `a`: a group's first row in the pool and its first token. First a token of each group at once, which settles nearly all of them,
// then the rest one by one. A whole warp.
template <int D>
__device__ __forceinline__ uint32_t zero_groups(const ExtendParams& p, const Unit& u, uint32_t ones, uint32_t row, int a, int lane) {
    constexpr int GRP = Shape<D>::GRP, EACH = 32 / GRP;
    auto some = [](const uint4& x) { return ((x.x | x.y | x.z | x.w) & 0x7F7F7F7Fu) != 0u; };
    {
        const int g = lane / EACH, ag = __shfl_sync(0xFFFFFFFFu, a, g);
        const uint32_t rg = __shfl_sync(0xFFFFFFFFu, row, g);
        const bool mine = (ones >> g) & 1u;
        const int t = ag < p.sinks ? 0 : max(0, u.lo - ag);  // a token that a row sees
        const bool any = mine && some(ldg16(p.v + (static_cast<uint64_t>(rg) + t) * D + 16 * (lane % EACH)));
        const uint32_t found = __ballot_sync(0xFFFFFFFFu, any);
#pragma unroll
        for (int k = 0; k < GRP; ++k)
            if ((found >> (k * EACH)) & ((1u << EACH) - 1u)) ones &= ~(1u << k);
    }
    for (uint32_t left = ones; left; left &= left - 1) {
        const int g = __ffs(static_cast<int>(left)) - 1, ag = __shfl_sync(0xFFFFFFFFu, a, g);
        const uint8_t* v = p.v + static_cast<uint64_t>(__shfl_sync(0xFFFFFFFFu, row, g)) * D;
        bool any = false;
        for (int i = lane; i < D; i += 32) {  // 16-byte chunks of 16 tokens
            const int t = ag + i / (D / 16);
            if (t < u.hi && (t >= u.lo || t < p.sinks)) any |= some(ldg16(v + 16 * i));
        }
        if (__any_sync(0xFFFFFFFFu, any)) ones &= ~(1u << g);
    }
    return ones;
}

// The scout: one warp that walks over the CTA's part and looks up where the KV tiles lie, ahead of the others, into a ring of
// places. (With every role walking by itself the kernel had 90 KB of code, and 15 % of the warps' time went into waiting for
// instructions.)
template <int D>
__device__ __forceinline__ void scout_tiles(const ExtendParams& p, Shared& sh, const int64_t* chunk, int64_t total, int lane) {
    using S_ = Shape<D>;
    volatile int* dead = &sh.dead;
    const PlanEntry mine = cut_at<D>(p, chunk, total, blockIdx.x, lane);
    if (lane == 0) p.plan[blockIdx.x] = mine;  // (for the join)
    warp_wait(smem_u32(&sh.ended), 0, dead);
    const int64_t part_end = sh.part_end;
    auto give_up = [&]() {  // (the flags alone: what else a place holds may be in use)
        if (lane < static_cast<int>(kRing)) *static_cast<volatile int*>(&sh.ring[lane].head.x) = kOver;
    };
    if (__any_sync(0xFFFFFFFFu, *dead)) return give_up();
    if (mine.cut >= part_end) {  // nothing to do: the others are told by a place without a tile (all are at first)
        if (lane == 0) mbar_arrive(smem_u32(&sh.placed[0]));
        return;
    }
    uint32_t n = 0;
    Walk<D> w;
    for (w.start(p, mine, part_end); w.more(); w.next(p)) {
        const int unit = (w.whole() ? kWhole : 0) | (w.tile0 > 0 ? kGoesOn : 0) |
                         (S_::MT == 2 && w.u.t1 - w.u.t0 > p.per ? kTwo : 0);
        const bool final = w.unit_begin + kUnitCost + w.u.tiles >= w.end;
        enum { kUnknown, kAllOne, kDiffer } scales = kUnknown;  // of V's pages, of this sequence and head
#pragma unroll 1
        for (int j = 0; j < w.piece_tiles; ++j, ++n) {
            const int t0 = tile_start<D>(w.u, w.tile0 + j), a = t0 + 16 * lane;
            uint32_t row = kNoRow;  // (pools have fewer than 2^32 rows)
            float sk = 1.0f, sv = 1.0f;
            bool no_number = false;
            if (lane < S_::GRP && a < w.u.hi && (a + 15 >= w.u.lo || a < p.sinks)) {
                const int idx = static_cast<int>(__umul64hi(static_cast<uint64_t>(a), p.t_magic));
                const int page = __ldg(p.table + static_cast<int64_t>(w.b) * p.max_pages + idx);
                if (page < 0 || page >= p.pool_pages) {
                    flag_status(p.status, NVFP4KV_STATUS_PAGE_OOB);
                } else {
                    const uint32_t at = static_cast<uint32_t>(page) * p.H + w.h;
                    row = at * static_cast<uint32_t>(p.T) + static_cast<uint32_t>(a - idx * p.T);
                    if (p.kbs) sk = __ldg(p.kbs + at);
                    if (p.vbs) sv = __ldg(p.vbs + at);
                    if (!(fabsf(sk) < INFINITY && fabsf(sv) < INFINITY)) {
                        no_number = true;
                        sk = sv = 1.0f;
                    }
                }
            }
            const uint32_t no_numbers = __ballot_sync(0xFFFFFFFFu, no_number);
            // (where all scales are 1, which a look at the sequence's tells once, V of zeros hides nothing: its loads for every tile
            // made the scout the slowest role, 16 chunks of 512 rows 594 us for 510)
            if (const uint32_t ones = __ballot_sync(0xFFFFFFFFu, p.vbs && row != kNoRow && sv == 1.0f && !no_number)) {
                if (scales == kUnknown) scales = scales_differ(p, w.b, w.h, w.u.hi, lane) ? kDiffer : kAllOne;
                if (scales == kDiffer && (zero_groups<D>(p, w.u, ones, row, a, lane) >> lane) & 1u) sv = kZeroScale;
            }
            const bool seen = t0 + S_::TK <= w.u.hi && (t0 >= w.u.lo || t0 + S_::TK <= p.sinks);
            const bool full = __all_sync(0xFFFFFFFFu, seen && (lane >= S_::GRP || row != kNoRow) && !no_number);
            // V of tile m is stored after the products with V of tile m - 2 are done, hence the weights of that tile made and the
            // places up to it read by all: once V of tile n - 6 is stored, the place of tile n - 8 is free.
            if (n >= kRing) {
                for (uint32_t i = 0; *static_cast<volatile uint32_t*>(&sh.loaded) < n - (kRing - 3) && !*dead; ++i) {
                    __nanosleep(100);
                    if (i == 20 * kTries) *dead = 1;
                }
                __syncwarp();
                if (__any_sync(0xFFFFFFFFu, *dead)) return give_up();
            }
            const uint32_t missing = __ballot_sync(0xFFFFFFFFu, lane < S_::GRP && row == kNoRow);
            Place& d = sh.ring[n % kRing];
            if (lane < S_::GRP) {
                d.row[lane] = row != kNoRow ? row : 0u;
                d.scales[lane] = row != kNoRow ? make_float4(sk, log2f(sv), 1.0f / sv, 0.0f) : make_float4(1.0f, -INFINITY, 0.0f, 0.0f);
            }
            if (lane == 0) {
                const bool last = j + 1 == w.piece_tiles;
                d.head = make_int4(unit | (j == 0 ? kFirst : 0) | (last ? kLast : 0) | (last && final ? kEnd : 0) | (full ? kFull : 0) | static_cast<int>(missing) * kMissing |
                                          static_cast<int>(no_numbers) * kNoNumber | (uneven<D>(p, w.u, w.s.len - w.s.n + w.u.t0, t0) ? kUneven : 0),
                                      t0, w.u.lo, w.u.hi);
                d.unit = make_int4(w.u.t0, w.u.t1, w.s.first, w.s.len - w.s.n);
                d.h = w.h;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.placed[n % kRing]));
        }
    }
}

// Where the CTA's part ends, found by a warp of its own beside the scout (ragged windows 57.4 us, so 58.8).
template <int D>
__device__ __forceinline__ void find_end(const ExtendParams& p, Shared& sh, const int64_t* chunk, int64_t total, int lane) {
    const PlanEntry end = cut_at<D>(p, chunk, total, blockIdx.x + 1, lane);
    if (lane == 0) {
        if (blockIdx.x == gridDim.x - 1) p.plan[gridDim.x] = end;
        sh.part_end = end.cut;
        mbar_arrive(smem_u32(&sh.ended));
    }
}

// What a lane reads for a token that no row sees, or that has no page. (Two branches, one of them without a load, would meet in
// copies of registers, and those wait for the load.)
__device__ uint4 g_zeros[16];
// ... and for K whose scale is not finite: NaN
#define NANS_16 {0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu}
#define NANS_64 NANS_16, NANS_16, NANS_16, NANS_16
__device__ uint4 g_nans[16] = {NANS_64, NANS_64, NANS_64, NANS_64};
#undef NANS_64
#undef NANS_16

// Where bytes of w are E4M3's NaN (0x7F, 0xFF): their highest bits.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nans(uint32_t w) { return w & ~((nan_bytes(w) >> 7) * 0xFFu); }

// The loader's threads: a warp's load covers R rows of 64 or 128 bytes (whole lines of a row), a lane one 16-byte chunk, which
// becomes two in the swizzled layout. The eight lanes of a store phase lie in an even row and the odd one after it, four chunks
// each: the even row's land in even 16-byte columns or in odd ones, the odd row's in the others, so they hit distinct banks.
template <int D>
__device__ __forceinline__ void load_tiles(const ExtendParams& p, Shared& sh, uint32_t smem, int kv, int warp, int lane) {
    using S_ = Shape<D>;
    constexpr int WIDE = D >= 128 ? 2 : 1;               // 64-byte columns of a load
    constexpr int R = 8 / WIDE;                          // its rows
    constexpr int LOADS = S_::TK / R / kLoaderWarps;     // of a column: rows R (warp + 4 g) on
    constexpr int COLS = S_::BLOCKS / WIDE;
    constexpr int N = LOADS * COLS;                      // chunks of a lane
    const int ch = lane & 3, blk = WIDE == 2 ? (lane >> 3) & 1 : 0;
    const int r0 = R * warp + (((lane >> 2) & 1) | (WIDE == 2 ? (lane >> 4) << 1 : (lane >> 3) << 1));  // the lane's first row
    const int g0 = r0 >> 4;                              // its 16-token group; further rows lie in every (R / 4)th group on
    const uint32_t at0 = static_cast<uint32_t>(blk * (S_::TK * 128) + r0 * 128 + (((2 * ch) ^ (r0 & 7)) << 4));
    const uint32_t src0 = static_cast<uint32_t>((r0 & 15) * D + 64 * blk + 16 * ch);
    volatile int* dead = &sh.dead;

    const uint8_t* base = (kv ? p.v : p.k) + src0;
    const uint32_t buf = smem + (kv ? S_::V_OFF : S_::K_OFF) + at0;
    const uint32_t full = smem_u32(&sh.full[kv][0]), empty = smem_u32(&sh.empty[kv][0]);
    uint4 r[N];
    // (tile n's values are loaded as soon as the ones before are stored; K and V have warps of their own, so each waits for its
    // own loads alone)
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
        const Place& t = sh.ring[n % kRing];
        warp_wait(smem_u32(&sh.placed[n % kRing]), (n / kRing) & 1u, dead);
        const int4 head = t.head;
        const int flags = uniform(head.x);
        if (flags & kNothing) return;
#pragma unroll
        for (int g = 0; g < LOADS; ++g) {
            const uint32_t row = t.row[g0 + g * (R * kLoaderWarps / 16)];
            const uint8_t* src = base + static_cast<uint64_t>(row) * D;
            if (!(flags & kFull)) {
                const int tok = head.y + r0 + g * R * kLoaderWarps;
                const int group = flags >> (g0 + g * (R * kLoaderWarps / 16));
                if (group & kMissing || tok >= head.w || (tok < head.z && tok >= p.sinks)) src = reinterpret_cast<const uint8_t*>(g_zeros);
                else if (group & kNoNumber) src = reinterpret_cast<const uint8_t*>(kv ? g_zeros : g_nans);
            }
#pragma unroll
            for (int c = 0; c < COLS; ++c) r[g * COLS + c] = ldg16(src + 64 * WIDE * c);
        }
        uint32_t nans = 0u;
        if (kv && (flags & kUneven))  // (here, where the warp waits anyway)
#pragma unroll
            for (int i = 0; i < N; ++i) nans |= nan_bytes(r[i].x) | nan_bytes(r[i].y) | nan_bytes(r[i].z) | nan_bytes(r[i].w);
        const uint32_t stage = n & 1u;
        warp_wait(empty + 8 * stage, ((n >> 1) & 1u) ^ 1u, dead);
        const uint32_t at = buf + stage * S_::KB, at1 = at ^ 16u;
        auto store = [&](int g, int c, const uint4& x) {
            const uint32_t off = WIDE * c * (S_::TK * 128) + g * (R * kLoaderWarps * 128);
            uint32_t a[2], b[2];
            e4m3x4_to_f16x2x2(x.x, a);
            e4m3x4_to_f16x2x2(x.y, b);
            sts16(at + off, a[0], a[1], b[0], b[1]);
            e4m3x4_to_f16x2x2(x.z, a);
            e4m3x4_to_f16x2x2(x.w, b);
            sts16(at1 + off, a[0], a[1], b[0], b[1]);
        };
#pragma unroll
        for (int g = 0; g < LOADS; ++g)
#pragma unroll
            for (int c = 0; c < COLS; ++c) store(g, c, r[g * COLS + c]);
        if (nans) {
            p.plan[blockIdx.x].nan = 1;  // (the scout wrote 0 before the first place)
#pragma unroll
            for (int g = 0; g < LOADS; ++g)
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    const uint4 x = r[g * COLS + c];
                    store(g, c, make_uint4(without_nans(x.x), without_nans(x.y), without_nans(x.z), without_nans(x.w)));
                }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(full + 8 * stage);
            if (kv == 1 && warp == 0) *static_cast<volatile uint32_t*>(&sh.loaded) = n + 1;
        }
        if (flags & kEnd) return;
    }
}

// The warp that issues the products of row tile x.
template <int D>
__device__ __forceinline__ void issue_products(const ExtendParams& p, Shared& sh, uint32_t qbuf, uint32_t kbuf, uint32_t vbuf, uint32_t tmem, int x, int lane) {
    using S_ = Shape<D>;
    volatile int* dead = &sh.dead;
    constexpr uint32_t qk = instruction(kStep, false), pv = instruction(D, true);
    uint32_t units = 0;  // pieces with this row tile
    // step `part` of KV tile n has slot `part`, or n % 2 where a tile is one step
    auto slot_of = [](uint32_t n, uint32_t part) { return S_::STEPS == 2 ? part : n & 1u; };
    auto phase_of = [](uint32_t n) { return (S_::STEPS == 2 ? n : n >> 1) & 1u; };
    auto scores = [&](uint32_t n, uint32_t part) {
        const uint32_t stage = n & 1u, slot = slot_of(n, part);
        if (part == 0) warp_wait(smem_u32(&sh.full[0][stage]), (n >> 1) & 1u, dead);
        tc_after();
        if (elect_one()) {
            const Operand a = operand(qbuf + x * S_::QB, 16, 1024), b = operand(kbuf + stage * S_::KB + part * (kStep * 128), 16, 1024);
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
                mma4_ss(tmem + (2 * x + slot) * kStep, a.at(k * (kRowsM * 128)), b.at(k * (S_::TK * 128)), qk, k > 0);
            tc_commit(smem_u32(&sh.sfull[x][slot]));
            if (part == S_::STEPS - 1) tc_commit(smem_u32(&sh.empty[0][stage]));
        }
        __syncwarp();
    };
    int flags = 0, next = 0;  // of tiles n and n + 1
    // (Shared memory answers late beside the tensor core's reads, so a tile's barriers are waited for at once, each by lanes of its
    // own, and the next tile's flags are read meanwhile.)
    auto weighted = [&](uint32_t n, uint32_t part, bool first) {
        const uint32_t stage = n & 1u, slot = slot_of(n, part);
        uint32_t bar = smem_u32(&sh.pfull[x][slot]), parity = phase_of(n);
        if (part == 0) {
            if (lane == 1) bar = smem_u32(&sh.full[1][stage]), parity = (n >> 1) & 1u;
            if (lane == 2 && !(flags & kEnd)) bar = smem_u32(&sh.placed[(n + 1) % kRing]), parity = ((n + 1) / kRing) & 1u;
        }
        warp_wait(bar, parity, dead);
        tc_after();
        if (part == 0) next = sh.ring[(n + 1) % kRing].head.x;
        if (elect_one()) {
            const Operand b = operand(vbuf + stage * S_::KB + part * (kStep * 128), S_::TK * 128, 1024);
#pragma unroll
            for (int k = 0; k < kStep; k += 32)
                mma2_ts(tmem + S_::O_COL + x * D, tmem + (2 * x + slot) * kStep + k / 2, b.at(k * 128), pv, k > 0 || !first);
            tc_commit(smem_u32(&sh.ofull[x]));
            if (part == S_::STEPS - 1) tc_commit(smem_u32(&sh.empty[1][stage]));
        }
        __syncwarp();
    };
    warp_wait(smem_u32(&sh.placed[0]), 0, dead);
    next = sh.ring[0].head.x;
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
        flags = uniform(next);
        if (flags & kNothing) return;
        if (S_::MT == 2 && x > 0 && !(flags & kTwo)) {
            // A unit without this row tile: a stage is free as soon as it is full. Its softmax warps are taken along step by
            // step, as ever (a barrier's parity does not tell them two tiles ahead).
            const uint32_t stage = n & 1u;
            warp_wait(smem_u32(&sh.full[0][stage]), (n >> 1) & 1u, dead);
            if (lane == 0) {
                mbar_arrive(smem_u32(&sh.empty[0][stage]));
                mbar_arrive(smem_u32(&sh.sfull[x][0]));
                mbar_arrive(smem_u32(&sh.sfull[x][1]));
            }
            warp_wait(smem_u32(&sh.full[1][stage]), (n >> 1) & 1u, dead);
            warp_wait(smem_u32(&sh.pfull[x][0]), phase_of(n), dead);
            warp_wait(smem_u32(&sh.pfull[x][1]), phase_of(n), dead);
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty[1][stage]));
            if (!(flags & kEnd)) {
                warp_wait(smem_u32(&sh.placed[(n + 1) % kRing]), ((n + 1) / kRing) & 1u, dead);
                next = sh.ring[(n + 1) % kRing].head.x;
            }
        } else {
            // A step's scores are issued two steps ahead (one, where a KV tile is one step), behind the product with V of the
            // step whose weights they overwrite.
            if (flags & kFirst) {
                warp_wait(smem_u32(&sh.qfull[x]), units & 1u, dead);
                ++units;
#pragma unroll 1
                for (uint32_t part = 0; part < S_::STEPS; ++part) scores(n, part);
            }
#pragma unroll 1
            for (uint32_t part = 0; part < S_::STEPS; ++part) {
                if (S_::STEPS == 1 && !(flags & kLast)) scores(n + 1, part);
                weighted(n, part, (flags & kFirst) && part == 0);
                if (S_::STEPS == 2 && !(flags & kLast)) scores(n + 1, part);
            }
        }
        if (flags & kEnd) return;
    }
}

// A softmax warp: 32 rows of row tile x.
template <int D>
__device__ __forceinline__ void softmax_rows(const ExtendParams& p, Shared& sh, uint32_t qbuf, uint32_t tmem, int x, int warp, int lane) {
    using S_ = Shape<D>;
    volatile int* dead = &sh.dead;
    const int row = 32 * (warp & 3) + lane;       // of the tile
    const int per = p.per;                        // tokens of a tile
    const int tok = row / p.G, head = row - tok * p.G;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t o_col = lanes + S_::O_COL + x * D;
    const uint32_t qrow = qbuf + x * S_::QB + row * 128;
    const float scale = p.sm_scale * scalar_or_1(p.gk);
    const float gv = scalar_or_1(p.gv);
    uint32_t on = 0;  // products with V asked for
    // A row's piece: its unit's flags, the row's position, those of the warp's first and last row, its place in q and out, and the
    // factor of its scores.
    struct Piece {
        int flags, pos, first_pos, last_pos, hq;
        int64_t out_row;
        float cs;
        bool real;
    };
    // The piece that begins with KV tile n: this thread's row of the queries, to FP16 by a power of two.
    auto begin_piece = [&](uint32_t n, Piece& u) {
        const Place& begin = sh.ring[n % kRing];
        warp_wait(smem_u32(&sh.placed[n % kRing]), (n / kRing) & 1u, dead);
        u.flags = begin.head.x;
        if ((u.flags & kNothing) || (S_::MT == 2 && x > 0 && !(u.flags & kTwo))) return;
        const int4 unit = begin.unit;
        const int t = unit.x + x * per + tok;  // token of the chunk
        u.real = tok < per && t < unit.y && unit.z + t < p.rows;  // (the last for places read while they are written)
        u.pos = unit.w + (u.real ? t : unit.y - 1);
        // (of the warp's rows, not of the tile's: fewer steps are masked, 16 chunks 508 us, so 513)
        u.first_pos = __reduce_min_sync(0xFFFFFFFFu, u.real ? u.pos : INT32_MAX);
        u.last_pos = __reduce_max_sync(0xFFFFFFFFu, u.real ? u.pos : -1);
        u.out_row = unit.z + t;
        u.hq = begin.h * p.G + head;
        {
            // (all of the row in flight at once; at head_dim 256 half of it, read a second time to be stored)
            const uint16_t* src = p.q + u.out_row * p.q_stride + u.hq * D;
            constexpr int N = D >= 256 ? 16 : D / 8;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            uint4 v[N];
            __nv_bfloat162 most = __float2bfloat162_rn(0.0f);
#pragma unroll 1
            for (int c0 = 0; c0 < D / 8; c0 += N) {
#pragma unroll
                for (int c = 0; c < N; ++c) v[c] = u.real ? ldg16(src + 8 * (c0 + c)) : zero;
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) most = __hmax2(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[k])));
                }
            }
            const float top = fmaxf(__low2float(most), __high2float(most));
            int kq = top > 0.0f ? 14 - ilogbf(top) : 0;
            kq = max(-120, min(kq, 120));
            const float up = copysignf(ldexpf(1.0f, kq), scale);  // a negative scale turns the queries: c is never negative
            u.cs = fabsf(scale) * kLog2e * ldexpf(1.0f, -kq);
#pragma unroll 1
            for (int c0 = D / 8 - N; c0 >= 0; c0 -= N) {
                if (c0 < D / 8 - N)
#pragma unroll
                    for (int c = 0; c < N; ++c) v[c] = u.real ? ldg16(src + 8 * (c0 + c)) : zero;
#pragma unroll
                for (int c = 0; c < N; ++c)
                    sts16(qrow + ((c0 + c) / 8) * (kRowsM * 128) + (((c & 7) ^ (row & 7)) << 4), pack_f16x2(bf16_lo(v[c].x) * up, bf16_hi(v[c].x) * up),
                          pack_f16x2(bf16_lo(v[c].y) * up, bf16_hi(v[c].y) * up), pack_f16x2(bf16_lo(v[c].z) * up, bf16_hi(v[c].z) * up),
                          pack_f16x2(bf16_lo(v[c].w) * up, bf16_hi(v[c].w) * up));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.qfull[x]));
        }
    };
    Piece u;
    begin_piece(0, u);
    if (u.flags & kNothing) return;
#pragma unroll 1
    for (uint32_t n = 0;;) {  // a piece; n: its first KV tile
        int flags = u.flags;
        if (S_::MT == 2 && x > 0 && !(flags & kTwo)) {  // a unit without this row tile
            while (true) {
                for (int slot = 0; slot < 2; ++slot) {
                    warp_wait(smem_u32(&sh.sfull[x][slot]), n & 1u, dead);
                    flags = sh.ring[n % kRing].head.x;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.pfull[x][slot]));
                }
                ++n;
                if (flags & kLast) break;
            }
            if (flags & kEnd) return;
            begin_piece(n, u);
            continue;
        }
        const bool real = u.real;
        const int pos = u.pos, first_pos = u.first_pos, last_pos = u.last_pos, hq = u.hq;
        const int64_t out_row = u.out_row;
        const float cs = u.cs;
        float m = -INFINITY, l = 0.0f;
        bool begins = true;
        int t0 = 0;
#pragma unroll 1
        for (uint32_t part = 0;; begins = false) {
            const uint32_t slot = S_::STEPS == 2 ? part : n & 1u;
            const uint32_t s_col = lanes + (2 * x + slot) * kStep;
            warp_wait(smem_u32(&sh.sfull[x][slot]), (S_::STEPS == 2 ? n : n >> 1) & 1u, dead);
            tc_after();
            // (where the tile's scores are, its place is there: read while the scores come, as shared memory is slow beside the
            // tensor core's reads)
            const Place& at = sh.ring[n % kRing];
            const int4 info = at.head;
            float4 f[kStep / 16];
#pragma unroll
            for (int g = 0; g < kStep / 16; ++g) f[g] = at.scales[4 * part + g];
            uint32_t x_[kStep];  // the row's scores, then its weights
            tmem_ld_row(x_, s_col);
            flags = info.x;
            t0 = info.y + static_cast<int>(part) * kStep;
            const bool ends = (flags & kLast) && part == S_::STEPS - 1;
            // columns [0, hi) of the step are at or before the row, those below lo hidden by the window but for the first `sk`
            const bool edge = t0 + kStep - 1 > first_pos || (t0 < last_pos - p.window + 1 && t0 + kStep > p.sinks);
            if (edge) {
                const int hi = pos - t0 + 1, lo = pos >= p.window ? pos - p.window + 1 - t0 : 0, sk = p.sinks - t0;
                auto below = [](int k) { return k >= 32 ? 0xFFFFFFFFu : (k <= 0 ? 0u : (1u << k) - 1u); };
#pragma unroll
                for (int c = 0; c < kStep; c += 32) {
                    const uint32_t seen = below(hi - c) & (~below(lo - c) | below(sk - c));  // bit i: column c + i is visible
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((seen >> i) & 1u)) x_[c + i] = 0xFF800000u;
                }
            }
            float mt = -INFINITY;
#pragma unroll
            for (int g = 0; g < kStep / 16; ++g) {
                f[g].x = fmaxf(cs * f[g].x, kTiny);
                float a = fmaxf(__uint_as_float(x_[16 * g]), __uint_as_float(x_[16 * g + 1]));
#pragma unroll
                for (int i = 2; i < 16; i += 2) a = fmaxf(a, fmaxf(__uint_as_float(x_[16 * g + i]), __uint_as_float(x_[16 * g + i + 1])));
                mt = fmaxf(mt, fmaf(a, f[g].x, f[g].y));
            }
            if (__any_sync(0xFFFFFFFFu, mt > m + kRescale)) {
                const float mn = fmaxf(m, mt);
                const float a = mn == -INFINITY ? 1.0f : ex2_approx(m - mn);
                m = mn;
                l *= a;
                if (!begins) {
                    warp_wait(smem_u32(&sh.ofull[x]), (on - 1) & 1u, dead);
                    tc_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {  // (16 at a time: the scores are held in registers meanwhile)
                        uint32_t o[16];
                        tmem_ld16(o, o_col + c);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                        tmem_st16(o_col + c, o);
                    }
                }
            }
            const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int g = 0; g < kStep / 16; ++g) {
                const float off = f[g].y - mu;
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    uint32_t &u0 = x_[16 * g + i], &u1 = x_[16 * g + i + 1];
                    fma2(u0, u1, f[g].x, off);
                    u0 = __float_as_uint(ex2_approx(__uint_as_float(u0)));
                    u1 = __float_as_uint(ex2_approx(__uint_as_float(u1)));
                    add2(sum0, sum1, u0, u1);
                }
                l = fmaf(sum0 + sum1, f[g].z, l);
                if (g % 2 == 1) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = pack_f16x2(__uint_as_float(x_[16 * (g - 1) + 2 * i]), __uint_as_float(x_[16 * (g - 1) + 2 * i + 1]));
                    tmem_st16(s_col + 8 * (g - 1), pk);
                }
            }
            tc_wait_st();
            // A parity tells a phase from the one before and the one after alone. The wait for the last product with V, below,
            // must not find the barrier two phases back, and this one, for the last but one, not two ahead: so it stands here,
            // before the last weights are handed over.
            if (ends && !begins) warp_wait(smem_u32(&sh.ofull[x]), (on - 1) & 1u, dead);
            ++on;
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.pfull[x][slot]));
            if (++part == S_::STEPS) {
                part = 0;
                ++n;
                if (flags & kLast) break;
            }
        }
        // the next piece's queries: its first scores come while this one's outputs are written (ragged windows 57.3 us, so 61.2)
        if (!(flags & kEnd)) begin_piece(n, u);
        // ---- the piece's end: outputs, or a partial result
        warp_wait(smem_u32(&sh.ofull[x]), (on - 1) & 1u, dead);
        tc_after();
        const bool whole = flags & kWhole;
        const int64_t rec = (2 * static_cast<int64_t>(blockIdx.x) + (flags & kGoesOn ? 0 : 1)) * (S_::MT * kRowsM) + x * kRowsM + row;
        const float f = l > 0.0f ? gv / l : 0.0f;
        uint16_t* dst = p.out + out_row * p.out_stride + hq * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o, o_col + 32 * c);
            if (real && whole) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 v;
                    v.x = pack_bf16x2(__uint_as_float(o[8 * i]) * f, __uint_as_float(o[8 * i + 1]) * f);
                    v.y = pack_bf16x2(__uint_as_float(o[8 * i + 2]) * f, __uint_as_float(o[8 * i + 3]) * f);
                    v.z = pack_bf16x2(__uint_as_float(o[8 * i + 4]) * f, __uint_as_float(o[8 * i + 5]) * f);
                    v.w = pack_bf16x2(__uint_as_float(o[8 * i + 6]) * f, __uint_as_float(o[8 * i + 7]) * f);
                    *reinterpret_cast<uint4*>(dst + 32 * c + 8 * i) = v;
                }
            } else if (real) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(p.rec_o + rec * D + 32 * c + 4 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            __syncwarp();
        }
        if (real) {
            if (!whole) p.rec_ml[rec] = make_float2(m, l);
            else if (p.lse) p.lse[out_row * p.Hq + hq] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
        tc_before();  // the next unit's products overwrite what was read here
        if (flags & kEnd) return;
    }
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1) extend_kernel(const ExtendParams p) {
    using S_ = Shape<D>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            for (int kv = 0; kv < 2; ++kv) {
                mbar_init(smem_u32(&sh.full[kv][i]), kLoaderWarps);
                mbar_init(smem_u32(&sh.empty[kv][i]), S_::MT);
            }
            mbar_init(smem_u32(&sh.qfull[i]), 4);
            for (int k = 0; k < 2; ++k) {
                mbar_init(smem_u32(&sh.sfull[i][k]), 1);
                mbar_init(smem_u32(&sh.pfull[i][k]), 4);
            }
            mbar_init(smem_u32(&sh.ofull[i]), 1);
        }
        for (uint32_t i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&sh.placed[i]), 1);
            Place& d = sh.ring[i];
            for (int g = 0; g < 8; ++g) d.row[g] = 0u;
            d.head = make_int4(kOver, 0, 0, 0);
            d.unit = make_int4(0, 0, 0, 0);
            d.h = 0;
        }
        sh.part_end = 0;
        mbar_init(smem_u32(&sh.drained), S_::MT);
        mbar_init(smem_u32(&sh.ended), 1);
        sh.dead = sh.never = 0;
        sh.loaded = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    constexpr int kIssuer = S_::WARPS - 4;
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = sh.tmem;
    pdl_enter();
    // (the list's chunks lie where the first tiles of K and V will)
    int64_t* chunk = reinterpret_cast<int64_t*>(raw + (base - smem_u32(raw)) + S_::K_OFF);
    const int64_t total = list_sequences<D>(p, chunk, sh.part);
    // registers: 640 threads start with 96 each; a softmax thread holds a row's scores of a step: 2 x 128 + 2 x 72 + 80 = 5 x 96
    if constexpr (S_::MT == 2) {
        if (warp < S_::SOFT_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        else if (warp < kIssuer) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    }
    if (warp < S_::SOFT_WARPS) {
        softmax_rows<D>(p, sh, base, tmem, warp / 4, warp, lane);
    } else if (warp < kIssuer) {
        const int i = warp - S_::SOFT_WARPS;
        load_tiles<D>(p, sh, base, i / kLoaderWarps, i % kLoaderWarps, lane);
    } else if (warp < kIssuer + S_::MT) {
        issue_products<D>(p, sh, base, base + S_::K_OFF, base + S_::V_OFF, tmem, uniform(warp - kIssuer), lane);
        // all products are done before TMEM is given back
        if (elect_one()) tc_commit(smem_u32(&sh.drained));
        __syncwarp();
        warp_wait(smem_u32(&sh.drained), 0, &sh.never);
    } else if (warp == kIssuer + S_::MT) {
        scout_tiles<D>(p, sh, chunk, total, lane);
    } else if (warp == kIssuer + S_::MT + 1) {
        find_end<D>(p, sh, chunk, total, lane);
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    if (warp == kIssuer) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
    if (threadIdx.x == 0 && sh.dead) flag_status(p.status, NVFP4KV_STATUS_TIMEOUT);
}

// ------------------------------------------------------------------------------------------ the join

// Over N lanes side by side.
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A warp's rows in the join: 32 / kJoinLanes of them from `first` on, and so on in steps of `step`.
template <int D>
constexpr int kJoinLanes = D == 64 ? 16 : 32;
template <int D>
__device__ __forceinline__ void join_rows(int& first, int& step) {
    first = (blockIdx.y * 8 + (threadIdx.x >> 5)) * (32 / kJoinLanes<D>);
    step = gridDim.y * 8 * (32 / kJoinLanes<D>);
}

// NaN into the dims of outputs of unit (b, h, qb) in which V of a token that the row sees is NaN, of the tiles that load_tiles leaves
// NaN out of. (Only where there were any.)
template <int D>
__device__ __forceinline__ void put_nans(const ExtendParams& p, int b, int h, int qb) {
    constexpr int EACH = D / 32;  // dims of a lane
    const Seq s = sequence(p, b);
    const Unit u = unit_of<D>(p, s, qb);
    const int p0 = s.len - s.n, lane = threadIdx.x & 31;
    int first, step;
    join_rows<D>(first, step);
    for (int row0 = first; row0 < Shape<D>::MT * kRowsM; row0 += step)
        for (int row = row0; row < row0 + 32 / kJoinLanes<D>; ++row) {
            const int x = row / kRowsM, r = row - x * kRowsM, t1 = u.t0 + x * p.per + r / p.G, pos = p0 + t1;
            if (r / p.G >= p.per || t1 >= u.t1) continue;
            uint32_t dims = 0u;
            for (int j = 0; j < u.tiles; ++j) {
                const int t0 = tile_start<D>(u, j);
                if (!uneven<D>(p, u, p0 + u.t0, t0)) continue;
                for (int t = t0; t < t0 + Shape<D>::TK && t <= pos; ++t) {
                    if (t <= pos - p.window && t >= p.sinks) continue;
                    const int idx = static_cast<int>(__umul64hi(static_cast<uint64_t>(t), p.t_magic));
                    const int page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + idx);
                    if (page < 0 || page >= p.pool_pages) continue;
                    const uint8_t* v = p.v + ((static_cast<int64_t>(page) * p.H + h) * p.T + (t - idx * p.T)) * D + EACH * lane;
                    for (int k = 0; k < EACH; ++k)
                        if ((__ldg(v + k) & 0x7F) == 0x7F) dims |= 1u << k;
                }
            }
            uint16_t* out = p.out + (s.first + t1) * p.out_stride + (h * p.G + r % p.G) * D + EACH * lane;
            for (int k = 0; k < EACH; ++k)
                if ((dims >> k) & 1u) out[k] = 0x7FC0u;
        }
}
// ... of the units that CTA c begins.
template <int D>
__device__ __forceinline__ void put_nans_of(const ExtendParams& p, int c) {
    Walk<D> w;
    for (w.start(p, p.plan[c], p.plan[c + 1].cut); w.more(); w.next(p))
        if (w.tile0 == 0) put_nans<D>(p, w.b, w.h, w.qb);
}

// Block (c, y): the unit that CTA c begins and others go on with, rows of it for every 8 gridDim.y warps; and the rows of
// sequences with lengths out of range. A row's pieces lie side by side in a warp (maxima, sums) and its values are all loaded at
// once, two rows to a warp at head_dim 64. Bound by latency: 8 blocks for each CTA (with 16 a call of one row took 12.5 us, so 11.3; with 6 a
// chunk of 100 rows at 3000 tokens, ten pieces a unit, 35.5, so 33.4). Returns whether a unit that CTA c begins has met NaN (put_nans).
template <int D>
__device__ __forceinline__ bool join_rows_of(const ExtendParams& p) {
    using S_ = Shape<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = (blockIdx.x * gridDim.y + blockIdx.y) * 8 + warp, workers = gridDim.x * gridDim.y * 8;
    for (int b = worker; b < p.B; b += workers) {
        const Seq s = sequence(p, b);
        if (!s.bad) continue;
        const int a = __ldg(p.starts + b), e = __ldg(p.starts + b + 1);
        if (a < 0 || e < a || e > p.rows) continue;
        for (int64_t r = a; r < e; ++r) {
            for (int i = lane; i < p.Hq * D / 8; i += 32)
                *reinterpret_cast<uint4*>(p.out + r * p.out_stride + 8 * i) = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse)
                for (int i = lane; i < p.Hq; i += 32) p.lse[r * p.Hq + i] = -INFINITY;
        }
    }
    const int c = blockIdx.x;
    constexpr int N = kJoinLanes<D>, V = D / N;  // lanes of a row, values of a lane
    const int64_t cut = p.plan[c].cut;
    bool nan = p.plan[c].nan != 0;
    const PlanEntry next = p.plan[c + 1];
    if (!(next.cut > next.begin && next.cut < next.end) || next.begin < cut) return nan;
    nan |= next.nan != 0;
    int pieces = 2;  // of the unit: CTA c's, c + 1's and those of the ones after that begin before its end
    for (int k = c + 2;; k += 32) {
        const bool mine = k + lane < p.ctas && p.plan[k + lane].cut < next.end;
        nan |= __any_sync(0xFFFFFFFFu, mine && p.plan[k + lane].nan != 0);
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, mine));
        pieces += n;
        if (n < 32) break;
    }
    const Seq s = sequence(p, next.b);
    const Unit u = unit_of<D>(p, s, next.qb);
    const int per = p.per;
    const float gv = scalar_or_1(p.gv);
    struct alignas(16) Values {
        float x[V];
    };
    const int at = lane % N;
    int first, step;
    join_rows<D>(first, step);
    for (int row0 = first; row0 < S_::MT * kRowsM; row0 += step) {
        const int row = row0 + lane / N, x = row / kRowsM, r = row - x * kRowsM, tok = r / p.G, head = r - tok * p.G;
        const int t = u.t0 + x * per + tok;
        const bool real = tok < per && t < u.t1;
        if (!__any_sync(0xFFFFFFFFu, real)) continue;
        auto rec = [&](int k) { return (2 * static_cast<int64_t>(c + k) + (k == 0 ? 1 : 0)) * (S_::MT * kRowsM) + row; };
        // running maximum, sum and outputs, over N pieces at a time: a lane has a piece's maximum and sum
        float m = -INFINITY, l = 0.0f, o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = 0.0f;
        for (int k0 = 0; k0 < pieces; k0 += N) {
            const int n = min(N, pieces - k0);
            const float2 ml = real && at < n ? p.rec_ml[rec(k0 + at)] : make_float2(-INFINITY, 0.0f);
            constexpr int U = 4;
            Values v[U];
            auto load = [&](int k) {
#pragma unroll
                for (int i = 0; i < U; ++i)
                    if (real && k + i < n) v[i] = *reinterpret_cast<const Values*>(p.rec_o + rec(k0 + k + i) * D + V * at);
            };
            load(0);
            const float mn = fmaxf(m, lanes_max<N>(ml.x)), back = m == -INFINITY ? 0.0f : exp2f(m - mn);
            const float w = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - mn);
            m = mn;
            l = l * back + lanes_sum<N>(w * ml.y);
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] *= back;
            for (int k = 0; k < n; k += U) {
                if (k > 0) load(k);
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const float wk = __shfl_sync(0xFFFFFFFFu, w, k + i, N);
                    if (real && k + i < n)
#pragma unroll
                        for (int e = 0; e < V; ++e) o[e] = fmaf(wk, v[i].x[e], o[e]);
                }
            }
        }
        if (!real) continue;
        const float f = l > 0.0f ? gv / l : 0.0f;
        const int64_t out_row = s.first + t;
        const int hq = next.h * p.G + head;
        uint16_t* dst = p.out + out_row * p.out_stride + hq * D + V * at;
        uint32_t b[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) b[i] = pack_bf16x2(o[2 * i] * f, o[2 * i + 1] * f);
        if constexpr (V == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(b[0], b[1]);
        else *reinterpret_cast<uint4*>(dst) = make_uint4(b[0], b[1], b[2], b[3]);
        if (at == 0 && p.lse) p.lse[out_row * p.Hq + hq] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
    return nan;
}
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ ExtendParams p) {
    pdl_enter();
    const bool nan = join_rows_of<D>(p);
    __syncwarp();  // (the rows' outputs are other lanes' stores)
    if (nan) put_nans_of<D>(p, blockIdx.x);
}

// ------------------------------------------------------------------------------------------ host

struct Carve {
    size_t plan, ml, o, total;
};
Carve carve(int D, int ctas) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t records = static_cast<size_t>(2 * ctas) * (D == 256 ? 1 : 2) * kRowsM;
    Carve c;
    c.plan = 0;
    c.ml = up(static_cast<size_t>(ctas + 1) * sizeof(PlanEntry));
    c.o = c.ml + up(records * sizeof(float2));
    c.total = c.o + records * D * sizeof(float);
    return c;
}

bool shape_ok(const nvfp4kv_layout* l, int Hq) {
    const int D = l->head_dim;
    if ((D != 64 && D != 128 && D != 256) || l->page_size % 16 != 0 || Hq % l->num_kv_heads != 0) return false;
    return Hq / l->num_kv_heads <= kMaxGroup;
}

template <int D>
cudaError_t launch_extend(const ExtendParams& p, cudaStream_t s) {
    using S_ = Shape<D>;
    cudaError_t e = cudaFuncSetAttribute(extend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S_::SMEM);
    if (e == cudaSuccess) e = launch_pdl(extend_kernel<D>, dim3(p.ctas), dim3(S_::THREADS), S_::SMEM, s, p);
    if (e == cudaSuccess) e = launch_pdl(join_kernel<D>, dim3(p.ctas, 8), dim3(256), 0, s, p);
    return e;
}

}  // namespace

extern "C" size_t nvfp4_paged_extend_attention_workspace_size(const nvfp4kv_layout* layout, int32_t batch,
                                                              int32_t num_q_heads) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || !shape_ok(layout, num_q_heads)) return 0;
    return carve(layout->head_dim, num_sms()).total;
}

extern "C" nvfp4kv_status nvfp4_paged_extend_attention(
    const nvfp4kv_layout* layout, int32_t batch, int32_t num_rows, int32_t num_q_heads, const void* q,
    int64_t q_row_stride, const int32_t* row_starts, const uint8_t* k_pages, const float* k_block_scales,
    const float* k_scale, const uint8_t* v_pages, const float* v_block_scales, const float* v_scale,
    int32_t pool_pages, const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens,
    int32_t window, int32_t sink_tokens, float sm_scale, void* workspace, size_t workspace_bytes, void* out,
    int64_t out_row_stride, float* lse, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || num_rows < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 ||
        pool_pages <= 0 || window < 0 || sink_tokens < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!shape_ok(layout, num_q_heads)) return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0 || num_rows == 0) return NVFP4KV_OK;
    const int D = layout->head_dim, H = layout->num_kv_heads, T = layout->page_size;
    const int64_t width = static_cast<int64_t>(num_q_heads) * D;
    if (!q || !row_starts || !k_pages || !v_pages || !page_table || !seq_lens || !out || q == out)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out) || q_row_stride % 8 != 0 ||
        out_row_stride % 8 != 0 || q_row_stride < width || out_row_stride < width)
        return NVFP4KV_ERR_INVALID_ARG;
    // token positions and the rows of a pool in 32 bits
    if (batch > 65535 || num_q_heads > 65535 || static_cast<int64_t>(max_pages_per_seq) * T > INT32_MAX - 1024 ||
        static_cast<int64_t>(pool_pages) * H > UINT32_MAX / T)
        return NVFP4KV_ERR_UNSUPPORTED;
    const int ctas = num_sms();
    const Carve c = carve(D, ctas);
    if (!workspace || workspace_bytes < c.total || !aligned16(workspace)) return NVFP4KV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    ExtendParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = k_pages;
    p.v = v_pages;
    p.kbs = k_block_scales;
    p.vbs = v_block_scales;
    p.gk = k_scale;
    p.gv = v_scale;
    p.table = page_table;
    p.lens = seq_lens;
    p.starts = row_starts;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.status = status;
    p.plan = reinterpret_cast<PlanEntry*>(ws + c.plan);
    p.rec_ml = reinterpret_cast<float2*>(ws + c.ml);
    p.rec_o = reinterpret_cast<float*>(ws + c.o);
    p.q_stride = q_row_stride;
    p.out_stride = out_row_stride;
    p.t_magic = UINT64_MAX / static_cast<uint64_t>(T) + 1;
    p.B = batch;
    p.rows = num_rows;
    p.Hq = num_q_heads;
    p.H = H;
    p.G = num_q_heads / H;
    p.per = kRowsM / p.G;
    const unsigned unit = static_cast<unsigned>((D == 256 ? 1 : 2) * p.per);
    p.unit_magic = static_cast<uint32_t>(((uint64_t{1} << 32) + unit - 1) / unit);
    p.T = T;
    p.pool_pages = pool_pages;
    p.max_pages = max_pages_per_seq;
    p.window = window > 0 ? window : INT32_MAX;
    p.sinks = sink_tokens;
    p.ctas = ctas;
    p.sm_scale = sm_scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (D) {
    case 64: return launched(launch_extend<64>(p, s));
    case 128: return launched(launch_extend<128>(p, s));
    default: return launched(launch_extend<256>(p, s));
    }
}
