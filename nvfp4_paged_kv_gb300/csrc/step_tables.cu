// Page tables and token slots of a step, built from the lengths of its requests.
//
// With p_b tokens cached and a_b to add, sequence b needs n_b = ceil((p_b + a_b) / T) - ceil(p_b / T) more pages, and
// all that a step's other calls take follows from prefix sums over the sequences: of a (the rows), of n (which pages of
// the free stack are whose), of the pages given back, and of the pages that become full.
//
// Every CTA makes all the prefix sums for itself, in shared memory (1024 threads, a few sequences each: reading 8 bytes a
// sequence again costs less than passing sums on). Outputs are spread over the threads of all CTAs; each finds its sequence by
// bisection in shared memory, four outputs at a time so that their loads overlap. Nothing is read that the call writes, but for
// lengths and the count of free pages where they are written in place: pages are popped below the old count of the stack and
// pushed from it on, and table entries are read below ceil(p_b / T) and written from it on. In place the CTAs are one cluster (up
// to 8), with its barrier between the last read of those and the first write; otherwise there are as many as the outputs ask for.
//
// A sequence that ended may have given pages back before (a sliding window leaves its first pages and its last): entries
// below 0. How many of its entries are pages is counted first; where none is missing the k-th page is the k-th entry, otherwise it
// is looked for from the nearer end of the row, which finds a window's pages at once.
//
// Bound: latency. A step of 256 requests, 13 of which ended with 1024 pages each, is three dependent round trips to memory, two
// block-wide sums and the launch: 11.1 us, call after call; 16 chunks of 512 rows 11.9 us (the launch's cost), 700 ragged requests, 70 of
// them ended, 18 us. (With one CTA, 64-bit sums and an output at a time the first took 7 us more.)
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "host_util.h"

namespace cg = cooperative_groups;
using namespace nvfp4kv;

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBatch = 8192;      // 28 bytes of shared memory each
constexpr int kMaxCluster = 8;       // CTAs where lengths or the count are written in place (portable cluster size)
constexpr int kMaxCtas = 64;
constexpr int kItemsPerCta = 4096;   // outputs of a CTA before another one is worth it

struct TablesParams {
    const int32_t* past;   // in and out arrays may be the same memory: no __restrict__, no __ldg
    const int32_t* add;
    int32_t* stack;
    const int32_t* count;
    int32_t* table;
    int32_t* lens;
    int32_t* starts;
    int64_t* slots;
    int32_t* positions;
    int32_t* full;
    int32_t* left;
    int32_t* status;
    uint32_t t_magic, t_shift;  // x / T = (x t_magic >> 32) >> t_shift for 0 <= x < 2^31, T > 1
    int32_t B, T, max_pages, capacity, rows, full_cap;
    bool in_place;     // lengths or the count are written where they are read
};

// Sums of counts, held at 2^31 - 1 once there (which is associative).
__device__ __forceinline__ int add_sat(int a, int b) {
    return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), 0x7FFFFFFFu));
}

// Exclusive prefix sums over the CTA's threads of N counts each, and their totals. All threads call.
template <int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (&total)[N], int (*part)[kWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl[N], before[N];
#pragma unroll
    for (int k = 0; k < N; ++k) incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, incl[k], o);
            if (lane >= o) incl[k] = add_sat(incl[k], u);
        }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        before[k] = __shfl_up_sync(0xFFFFFFFFu, incl[k], 1);
        if (lane == 0) before[k] = 0;
        if (lane == 31) part[k][warp] = incl[k];
    }
    __syncthreads();
    if (warp < N) {
        int s = part[warp][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s = add_sat(s, u);
        }
        part[warp][lane] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = warp > 0 ? add_sat(before[k], part[k][warp - 1]) : before[k];
        total[k] = part[k][kWarps - 1];
    }
    __syncthreads();
}

// For each of N elements the last b with first[b] <= i, for first[0] = 0 <= i: the sequence that element i of a list belongs
// to. `half` is the largest power of two below B.
template <int N>
__device__ __forceinline__ void owners(const int* first, int B, int half, const int (&i)[N], int (&b)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) b[k] = 0;
    for (int s = half; s > 0; s >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (b[k] + s < B && first[b[k] + s] <= i[k]) b[k] += s;
}

__global__ void __launch_bounds__(kThreads, 1) step_tables_kernel(const TablesParams p) {
    pdl_enter();
    extern __shared__ __align__(16) int smem[];
    __shared__ int part[3][kWarps], n_ended;
    const int B = p.B, T = p.T;
    // of each sequence: its first row, its first page popped, given back and becoming full, its tokens cached and to
    // add (kUnserved: it keeps what it has), and its full pages
    int *row0 = smem, *need0 = row0 + B, *back0 = need0 + B, *full0 = back0 + B, *past_s = full0 + B, *add_s = past_s + B, *whole_s = add_s + B;
    constexpr int kUnserved = -2;

    const int tid = threadIdx.x;
    const int max_tokens = p.max_pages * T;  // (the host bounds it)
    const int each = (B + kThreads - 1) / kThreads;
    const int b_lo = min(B, tid * each), b_hi = min(B, b_lo + each);
    // 0 <= x < 2^31
    auto whole_pages = [&](int x) { return T == 1 ? x : static_cast<int>(__umulhi(static_cast<unsigned>(x), p.t_magic) >> p.t_shift); };
    auto pages_of = [&](int x) {
        const int n = whole_pages(x);
        return n + (n * T != x);
    };
    struct Seq {
        int past, add, rows, whole, need, back;
        bool ok;
    };
    auto look = [&](int b) {
        Seq s{p.past[b], p.add[b], 0, 0, 0, 0, true};
        s.rows = max(s.add, 0);
        if (s.past < 0 || s.past > max_tokens) {
            s.past = 0;
            s.ok = false;
        } else if (s.add < -1 || s.rows > max_tokens - s.past) {
            s.ok = false;
        } else {
            s.whole = whole_pages(s.past);
            const int have = s.whole + (s.whole * T != s.past);
            if (s.add < 0) s.back = have;
            else s.need = pages_of(s.past + s.add) - have;
        }
        return s;
    };

    // ------------------------------------------------ rows, pages to pop, pages given back
    const int given_count = *p.count;
    if (tid == 0) n_ended = 0;
    int at[3] = {0, 0, 0}, total[3];
    Seq kept{};
    bool ends = false;
    for (int b = b_lo; b < b_hi; ++b) {
        kept = look(b);
        at[0] = add_sat(at[0], kept.rows);
        at[1] = add_sat(at[1], kept.need);
        ends |= kept.back > 0;
    }
    // Sequences that ended: which of their entries are pages. (In a list, so that rows are spread over the warps, several of
    // which share a row where there are few: 70 rows of 280 entries on average take 4 us, 13 of 1024 less than 1. A thread for each of
    // all entries, with its sequence bisected, took 10 and 4.)
    if (__syncthreads_or(ends)) {
        int *list = need0, *missing = back0;
        for (int k = 0; k < each; ++k) {
            const int b = b_lo + k;
            if (each > 1 && b < b_hi) kept = look(b);
            const bool mine = b < b_hi && kept.back > 0;
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, mine), lane = tid & 31;
            int first = 0;
            if (lane == 0 && who) first = atomicAdd(&n_ended, __popc(who));
            first = __shfl_sync(0xFFFFFFFFu, first, 0);
            if (mine) {
                list[first + __popc(who & ((1u << lane) - 1u))] = b;
                past_s[b] = kept.past;
                missing[b] = 0;
            }
        }
        __syncthreads();
        constexpr int U = 16;  // entries of a lane at a time
        const int n = n_ended, share = n < kWarps ? kWarps / n : 1, warp = tid / 32, lane = tid & 31;
        for (int e = warp / share; e < n; e += kWarps / share) {
            const int b = list[e], have = pages_of(past_s[b]);
            const int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages;
            int holes = 0;
            for (int64_t j0 = static_cast<int64_t>(warp % share) * 32 * U + lane; j0 < have; j0 += share * 32 * U) {
                int page[U];
#pragma unroll
                for (int k = 0; k < U; ++k) page[k] = j0 + 32 * k < have ? row[j0 + 32 * k] : 0;
#pragma unroll
                for (int k = 0; k < U; ++k) holes += page[k] < 0;
            }
            holes = __reduce_add_sync(0xFFFFFFFFu, holes);
            if (lane == 0 && holes) atomicAdd(&missing[b], holes);
        }
        __syncthreads();
        for (int b = b_lo; b < b_hi; ++b) {
            if (each > 1) kept = look(b);
            if (kept.back > 0) kept.back -= missing[b];
            at[2] = add_sat(at[2], kept.back);
        }
    }
    block_scan<3>(at, total, part);
    int32_t flags = 0;
    const int count = max(0, min(given_count, p.capacity));
    if (count != given_count) flags |= NVFP4KV_STATUS_PAGE_OOB;
    const int returned = min(total[2], p.capacity - count);
    if (total[2] > returned) flags |= NVFP4KV_STATUS_PAGE_OOB;
    const int top = count + returned;

    // ------------------------------------------------ who is served
    // A sequence that needs pages is served when its needs and those of all before it fit, and one with rows when
    // they fit, so the pages of those that are served are the first of the stack, without gaps. (A sum that was held at
    // 2^31 - 1 is above both bounds.)
    int done[2] = {0, 0}, done_total[2];  // pages that become full, pages popped
    for (int b = b_lo; b < b_hi; ++b) {
        if (each > 1) kept = look(b);
        const Seq& s = kept;
        bool ok = s.ok;
        if (!ok || (s.rows > 0 && add_sat(at[0], s.rows) > p.rows)) {
            flags |= NVFP4KV_STATUS_BAD_SEQ_LEN;
            ok = false;
        } else if (s.need > 0 && add_sat(at[1], s.need) > top) {
            flags |= NVFP4KV_STATUS_NO_PAGES;
            ok = false;
        }
        row0[b] = at[0];
        need0[b] = at[1];
        const int left = s.back > 0 && each > 1 ? s.back - back0[b] : s.back;  // (back0 still counts what is missing)
        back0[b] = at[2];
        past_s[b] = s.past;
        add_s[b] = ok ? s.add : kUnserved;
        whole_s[b] = s.whole;
        if (ok && s.add > 0) {
            done[0] += whole_pages(s.past + s.add) - s.whole;  // (rows fit into 2^30)
            done[1] += s.need;
        }
        at[0] = add_sat(at[0], s.rows);
        at[1] = add_sat(at[1], s.need);
        at[2] = add_sat(at[2], left);
    }
    block_scan<2>(done, done_total, part);
    for (int b = b_lo; b < b_hi; ++b) {
        full0[b] = done[0];
        if (add_s[b] > 0) done[0] += whole_pages(past_s[b] + add_s[b]) - whole_s[b];
    }
    if (flags && blockIdx.x == 0) flag_status(p.status, flags);
    // in place, every CTA's last read comes before any write
    if (p.in_place && gridDim.x > 1) cg::this_cluster().sync();
    else __syncthreads();

    // ------------------------------------------------ outputs
    const int g = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
    const int n_rows = min(total[0], p.rows);
    int half = 1;
    while (half * 2 < B) half *= 2;
    constexpr int U = 4;  // outputs of a thread at a time
    const int nothing = -1;
    auto have_of = [&](int b) { return whole_s[b] + (whole_s[b] * T != past_s[b]); };
    // the entry of page i of those given back, of sequence b
    auto entry_of = [&](int b, int i) -> const int32_t* {
        const int32_t* row = p.table + static_cast<int64_t>(b) * p.max_pages;
        const int have = have_of(b), pages = (b + 1 < B ? back0[b + 1] : total[2]) - back0[b];
        int k = i - back0[b];
        if (pages == have) return row + k;
        if (2 * static_cast<int64_t>(k) < pages) {
            for (int j = 0; j < have; ++j)
                if (row[j] >= 0 && k-- == 0) return row + j;
        } else {
            k = pages - 1 - k;
            for (int j = have - 1; j >= 0; --j)
                if (row[j] >= 0 && k-- == 0) return row + j;
        }
        return row;  // (only where the table changes under the call)
    };
    // where page k of the stack's top lies, counted down: in the stack, or, where this very call gives it back, in its table
    auto given_back = [&](int i) {
        const int ii[1] = {i};
        int b[1];
        owners<1>(back0, B, half, ii, b);
        return entry_of(b[0], i);
    };
    auto popped = [&](int k) -> const int32_t* {
        const int i = top - 1 - k;
        return i < count ? p.stack + i : given_back(i - count);
    };
    // and page j of sequence b, cached or new
    auto page_at = [&](int b, int j) -> const int32_t* {
        const int have = have_of(b);
        return j < have ? p.table + static_cast<int64_t>(b) * p.max_pages + j : popped(need0[b] + j - have);
    };
    for (int b = g; b < B; b += step) {
        const int add = add_s[b];
        p.lens[b] = add == -1 ? 0 : past_s[b] + max(add, 0);
        p.starts[b] = min(row0[b], n_rows);
    }
    if (g == 0) {
        p.starts[B] = n_rows;
        *p.left = top - done_total[1];
    }
    bool no_page = false;
    for (int64_t r0 = g; r0 < p.rows; r0 += int64_t{U} * step) {
        int r[U], b[U], pos[U], j[U], page[U];
        const int32_t* src[U];
#pragma unroll
        for (int k = 0; k < U; ++k) r[k] = static_cast<int>(min(r0 + static_cast<int64_t>(k) * step, static_cast<int64_t>(INT32_MAX)));
        owners<U>(row0, B, half, r, b);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            pos[k] = j[k] = 0;
            src[k] = nullptr;
            if (r[k] < n_rows && add_s[b[k]] > 0) {
                pos[k] = past_s[b[k]] + (r[k] - row0[b[k]]);
                j[k] = whole_pages(pos[k]);
                src[k] = page_at(b[k], j[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) page[k] = src[k] ? *src[k] : nothing;
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (r[k] < p.rows) {
                const bool there = page[k] >= 0;
                no_page |= src[k] && !there;
                p.slots[r[k]] = there ? static_cast<int64_t>(page[k]) * T + (pos[k] - j[k] * T) : -1;
                p.positions[r[k]] = there ? pos[k] : 0;
            }
    }
    if (no_page) flag_status(p.status, NVFP4KV_STATUS_PAGE_OOB);
    // new pages into the tables, full pages into their list, pages given back on the stack: (sequence, page) pairs alike
    auto copy_pages = [&](const int* first, int n, auto from, auto to) {
        for (int64_t i0 = g; i0 < n; i0 += int64_t{U} * step) {
            int i[U], b[U], page[U];
            const int32_t* src[U];
#pragma unroll
            for (int k = 0; k < U; ++k) i[k] = static_cast<int>(min(i0 + static_cast<int64_t>(k) * step, static_cast<int64_t>(INT32_MAX)));
            owners<U>(first, B, half, i, b);
#pragma unroll
            for (int k = 0; k < U; ++k) src[k] = i[k] < n ? from(b[k], i[k]) : nullptr;
#pragma unroll
            for (int k = 0; k < U; ++k) page[k] = src[k] ? *src[k] : nothing;
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i[k] < n) *to(b[k], i[k]) = page[k];
        }
    };
    copy_pages(back0, returned, [&](int b, int i) { return entry_of(b, i); },
               [&](int, int i) { return p.stack + count + i; });
    copy_pages(need0, done_total[1], [&](int, int i) { return popped(i); },
               [&](int b, int i) { return p.table + static_cast<int64_t>(b) * p.max_pages + have_of(b) + (i - need0[b]); });
    if (p.full)
        copy_pages(full0, p.full_cap,
                   [&](int b, int i) -> const int32_t* { return i < done_total[0] ? page_at(b, whole_s[b] + (i - full0[b])) : nullptr; },
                   [&](int, int i) { return p.full + i; });
}

}  // namespace

extern "C" nvfp4kv_status nvfp4_kv_step_tables(
    const nvfp4kv_layout* layout, int32_t batch, const int32_t* past_lens, const int32_t* new_lens,
    int32_t* free_pages, int32_t free_capacity, const int32_t* free_count, int32_t* free_left,
    int32_t* page_table, int32_t max_pages_per_seq, int32_t* seq_lens, int32_t* row_starts,
    int64_t* slots, int32_t* positions, int32_t num_rows, int32_t* full_pages,
    int32_t full_capacity, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || free_capacity < 0 || max_pages_per_seq <= 0 || num_rows < 0 ||
        full_capacity < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (batch == 0) return NVFP4KV_OK;
    const int T = layout->page_size;
    if (!past_lens || !new_lens || !free_count || !free_left || !page_table || !seq_lens || !row_starts ||
        (free_capacity > 0 && !free_pages) || (num_rows > 0 && (!slots || !positions)))
        return NVFP4KV_ERR_INVALID_ARG;
    // every page of the rows may become full, and one more of each sequence
    if (full_pages && full_capacity < static_cast<int64_t>(batch) + num_rows / T) return NVFP4KV_ERR_INVALID_ARG;
    if (batch > kMaxBatch || static_cast<int64_t>(max_pages_per_seq) * T > INT32_MAX ||
        num_rows > (1 << 30) || full_capacity > (1 << 30))
        return NVFP4KV_ERR_UNSUPPORTED;

    TablesParams p{};
    p.past = past_lens;
    p.add = new_lens;
    p.stack = free_pages;
    p.count = free_count;
    p.table = page_table;
    p.lens = seq_lens;
    p.starts = row_starts;
    p.slots = slots;
    p.positions = positions;
    p.full = full_pages;
    p.left = free_left;
    p.status = status;
    p.B = batch;
    p.T = T;
    p.max_pages = max_pages_per_seq;
    p.capacity = free_capacity;
    p.rows = num_rows;
    p.full_cap = full_capacity;
    const size_t smem = static_cast<size_t>(batch) * 7 * sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxBatch * 7 * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return launched(e);
    // 2^l >= T > 2^(l - 1), m = ceil(2^(31 + l) / T) < 2^32: m T = 2^(31 + l) + e with e < T <= 2^l, so x m / 2^(31 + l) exceeds
    // x / T by less than 1 / T for x < 2^31
    int l = 0;
    while ((int64_t{1} << l) < T) ++l;
    p.t_magic = l ? static_cast<uint32_t>(((uint64_t{1} << (31 + l)) + T - 1) / T) : 0u;
    p.t_shift = l ? l - 1 : 0;
    auto apart = [](const int32_t* a, size_t na, const int32_t* b, size_t nb) { return a + na <= b || b + nb <= a; };
    const size_t n = static_cast<size_t>(batch);
    p.in_place = !(apart(seq_lens, n, past_lens, n) && apart(seq_lens, n, new_lens, n) && apart(row_starts, n + 1, past_lens, n) &&
                   apart(row_starts, n + 1, new_lens, n) && free_left != free_count && apart(free_left, 1, past_lens, n) &&
                   apart(free_left, 1, new_lens, n) && apart(seq_lens, n, free_count, 1) && apart(row_starts, n + 1, free_count, 1));
    // outputs, and a share of the pages that may come back (of 256 requests with up to 2048 pages each 13 ended: one CTA
    // took 16.8 us)
    const int64_t back = static_cast<int64_t>(batch) * max_pages_per_seq;
    const int64_t items = static_cast<int64_t>(num_rows) + (full_pages ? full_capacity : 0) + batch +
                          (back < free_capacity ? back : free_capacity) / 16;
    const int most = p.in_place ? kMaxCluster : kMaxCtas;
    int ctas = 1;
    while (ctas < most && items > static_cast<int64_t>(ctas) * kItemsPerCta) ctas *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.in_place && ctas > 1 ? 2 : 1;
    return launched(cudaLaunchKernelEx(&cfg, step_tables_kernel, static_cast<const TablesParams&>(p)));
}
