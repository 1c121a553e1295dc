// Page tables and token slots of a step, built from the lengths of its requests.
//
// With p_b tokens cached and a_b to add, sequence b needs n_b = ceil((p_b + a_b) / T) - ceil(p_b / T) more pages, and
// all that a step's other calls take follows from prefix sums over the sequences: of a (the rows), of n (which pages of
// the free stack are whose), of the pages given back, and of the pages that become full.
//
// One cluster of 1 to 8 CTAs. Every CTA makes all the prefix sums for itself, in shared memory (1024 threads, a few
// sequences each: reading 8 bytes a sequence again costs less than passing sums on), so the CTAs meet only once, at a
// cluster barrier between the last read of what may be written in place (lengths, the count of free pages) and the first
// write. After it nothing is read that is written: pages are popped below the old count of the stack and pushed from it
// on, and table entries are read below ceil(p_b / T) and written from it on. The outputs are spread over all threads;
// each finds its sequence by bisection in shared memory.
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
constexpr int kMaxBatch = 8192;      // 21 bytes of shared memory each
constexpr int kMaxCtas = 8;          // portable cluster size
constexpr int kItemsPerCta = 2048;   // outputs that one CTA writes before a second one is worth its cluster

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
    int32_t B, T, max_pages, capacity, rows, full_cap;
};

__device__ __forceinline__ int clamp_i32(int64_t x) {
    return static_cast<int>(min(x, static_cast<int64_t>(INT32_MAX)));
}

// Exclusive prefix sums over the CTA's threads of N values each, and their totals. All threads call.
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t (&total)[N], int64_t (*part)[kWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        incl[k] = v[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, incl[k], o);
            if (lane >= o) incl[k] += u;
        }
        if (lane == 31) part[k][warp] = incl[k];
    }
    __syncthreads();
    if (warp < N) {
        int64_t s = part[warp][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += u;
        }
        part[warp][lane] = s;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = incl[k] - v[k] + (warp > 0 ? part[k][warp - 1] : 0);
        total[k] = part[k][kWarps - 1];
    }
    __syncthreads();
}

// The last b with first[b] <= i, for first[0] = 0 <= i: the sequence that element i of a list belongs to.
__device__ __forceinline__ int owner(const int* first, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1) step_tables_kernel(const TablesParams p) {
    pdl_enter();
    extern __shared__ __align__(16) int smem[];
    __shared__ int64_t part[3][kWarps];
    const int B = p.B, T = p.T;
    // of each sequence: its first row, its first page popped, given back and becoming full, its tokens cached and to
    // add (kUnserved: it keeps what it has)
    int *row0 = smem, *need0 = row0 + B, *back0 = need0 + B, *full0 = back0 + B, *past_s = full0 + B, *add_s = past_s + B;
    constexpr int kUnserved = -2;

    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
    const int tid = threadIdx.x;
    const int max_tokens = p.max_pages * T;  // (the host bounds it)
    const int each = (B + kThreads - 1) / kThreads;
    const int b_lo = min(B, tid * each), b_hi = min(B, b_lo + each);
    auto pages_of = [&](int tokens) { return tokens / T + (tokens % T != 0); };
    struct Seq {
        int past, add, rows, need, back;
        bool ok;
    };
    auto look = [&](int b) {
        Seq s{p.past[b], p.add[b], 0, 0, 0, true};
        s.rows = max(s.add, 0);
        if (s.past < 0 || s.past > max_tokens) {
            s.past = 0;
            s.ok = false;
        } else if (s.add < -1 || s.rows > max_tokens - s.past) {
            s.ok = false;
        } else if (s.add < 0) {
            s.back = pages_of(s.past);
        } else {
            s.need = pages_of(s.past + s.add) - pages_of(s.past);
        }
        return s;
    };

    // ------------------------------------------------ rows, pages to pop, pages given back
    int64_t at[3] = {0, 0, 0}, total[3];
    for (int b = b_lo; b < b_hi; ++b) {
        const Seq s = look(b);
        at[0] += s.rows;
        at[1] += s.need;
        at[2] += s.back;
    }
    block_scan<3>(at, total, part);
    int count = *p.count;
    int32_t flags = 0;
    if (count < 0 || count > p.capacity) {
        flags |= NVFP4KV_STATUS_PAGE_OOB;
        count = max(0, min(count, p.capacity));
    }
    const int returned = static_cast<int>(min(total[2], static_cast<int64_t>(p.capacity - count)));
    if (total[2] > returned) flags |= NVFP4KV_STATUS_PAGE_OOB;
    const int top = count + returned;

    // ------------------------------------------------ who is served
    // A sequence that needs pages is served when its needs and those of all before it fit, and one with rows when
    // they fit, so the pages of those that are served are the first of the stack, without gaps.
    int64_t done[2] = {0, 0}, done_total[2];  // pages that become full, pages popped
    for (int b = b_lo; b < b_hi; ++b) {
        const Seq s = look(b);
        bool ok = s.ok;
        if (!ok || (s.rows > 0 && at[0] + s.rows > p.rows)) {
            flags |= NVFP4KV_STATUS_BAD_SEQ_LEN;
            ok = false;
        } else if (s.need > 0 && at[1] + s.need > top) {
            flags |= NVFP4KV_STATUS_NO_PAGES;
            ok = false;
        }
        row0[b] = clamp_i32(at[0]);
        need0[b] = clamp_i32(at[1]);
        back0[b] = clamp_i32(at[2]);
        past_s[b] = s.past;
        add_s[b] = ok ? s.add : kUnserved;
        if (ok && s.add > 0) {
            done[0] += (s.past + s.add) / T - s.past / T;
            done[1] += s.need;
        }
        at[0] += s.rows;
        at[1] += s.need;
        at[2] += s.back;
    }
    block_scan<2>(done, done_total, part);
    for (int b = b_lo; b < b_hi; ++b) {
        full0[b] = clamp_i32(done[0]);
        if (add_s[b] > 0) done[0] += (past_s[b] + add_s[b]) / T - past_s[b] / T;
    }
    if (flags && rank == 0) flag_status(p.status, flags);
    // the last read of what may be written in place is behind every CTA
    if (ctas > 1) cluster.sync();
    else __syncthreads();

    // ------------------------------------------------ outputs
    const int g = rank * kThreads + tid, step = ctas * kThreads;
    const int n_rows = static_cast<int>(min(total[0], static_cast<int64_t>(p.rows)));
    auto given_back = [&](int i) {
        const int b = owner(back0, B, i);
        return p.table[static_cast<int64_t>(b) * p.max_pages + (i - back0[b])];
    };
    // page k of the stack's top, counted down: from the stack, or, where this very call gives it back, from its table
    auto pop = [&](int k) {
        const int i = top - 1 - k;
        return i < count ? p.stack[i] : given_back(i - count);
    };
    // page j of sequence b, cached or new
    auto page_at = [&](int b, int j) {
        const int have = pages_of(past_s[b]);
        return j < have ? p.table[static_cast<int64_t>(b) * p.max_pages + j] : pop(need0[b] + j - have);
    };
    for (int b = g; b < B; b += step) {
        const int add = add_s[b];
        p.lens[b] = add == -1 ? 0 : past_s[b] + max(add, 0);
        p.starts[b] = min(row0[b], n_rows);
    }
    if (g == 0) {
        p.starts[B] = n_rows;
        *p.left = top - static_cast<int>(done_total[1]);
    }
    for (int i = g; i < returned; i += step) p.stack[count + i] = given_back(i);
    for (int i = g; i < done_total[1]; i += step) {
        const int b = owner(need0, B, i);
        p.table[static_cast<int64_t>(b) * p.max_pages + pages_of(past_s[b]) + (i - need0[b])] = pop(i);
    }
    for (int r = g; r < p.rows; r += step) {
        int64_t slot = -1;
        int pos = 0;
        if (r < n_rows) {
            const int b = owner(row0, B, r);
            if (add_s[b] > 0) {
                pos = past_s[b] + (r - row0[b]);
                const int j = pos / T;
                slot = static_cast<int64_t>(page_at(b, j)) * T + (pos - j * T);
            }
        }
        p.slots[r] = slot;
        p.positions[r] = pos;
    }
    if (p.full) {
        for (int i = g; i < p.full_cap; i += step) {
            int page = -1;
            if (i < done_total[0]) {
                const int b = owner(full0, B, i);
                page = page_at(b, past_s[b] / T + (i - full0[b]));
            }
            p.full[i] = page;
        }
    }
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
    const size_t smem = static_cast<size_t>(batch) * 6 * sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxBatch * 6 * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return launched(e);
    const int64_t items = static_cast<int64_t>(num_rows) + (full_pages ? full_capacity : 0) + batch;
    int ctas = 1;
    while (ctas < kMaxCtas && items > static_cast<int64_t>(ctas) * kItemsPerCta) ctas *= 2;
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
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return launched(cudaLaunchKernelEx(&cfg, step_tables_kernel, static_cast<const TablesParams&>(p)));
}
