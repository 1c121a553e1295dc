// Append of a step's rows to the NVFP4 paged cache, with the rotary position encoding applied on
// the way, for sm_103a.
//
// What it computes, per row n with token slot s = slots[n] (page s / T, token s % T) and position
// p = positions[n]: the rotated dims of q and k as
//   x1' = fp32(fp32(x1 c) - fp32(x2 s)),  x2' = fp32(fp32(x2 c) + fp32(x1 s))
// (c, s: the FP32 table row of p), then K and V rows encoded to NVFP4 exactly as the page codec
// encodes the same FP32 values (codec_core.cuh), K without a rounding to 16 bits between the
// rotation and the encoder. The rotation rounds each product and each sum (no fused multiply-add),
// so that the stored codes do not depend on how a compiler contracts them.
//
// Bound: HBM for a chunk, latency for a decode step. Every source value is read once and every output
// written once; the table row of a position (at most 4 D bytes) is read once per warp task into registers
// and reused for every head of the task. Measured: 8192 rows of 32 + 8 + 8 heads of 128 with all outputs
// (215 MB) 39.4 us, 5.5 TB/s; 32 such rows 3.4 us.
//
// A warp task is a row's q and K heads, or its V heads, as many head groups of it as make about 32 warps to an
// SM. (q with K, and V, are rounded up to tasks apart, so there can be a few more: 1237 rows of 20 + 4 heads of 256
// are 4948 tasks for 4864 warps, and 21 CTAs wait for a second wave.)
// A thread owns 8 dims of each of two 16-value blocks of one head that rotate with one another (block i
// of the first half with block i of the second, or two neighbouring blocks when adjacent dims pair
// up), so the rotation needs no other thread, and two neighbouring lanes hold the two blocks: they
// share the block maximum by a shuffle and each picks the scale of one block. (With whole blocks in a
// thread the kernel needed 157 registers, and 128 with spills kept 16 warps on an SM: 46.6 us; the halves
// take 64, 32 warps.)
//
// K bytes belong to one token each. A V byte holds two tokens (token pairs): when the next row of
// the call is the second token of the pair, one thread encodes both and stores whole bytes; a token
// whose partner is not its neighbour in the call replaces its nibbles with two 32-bit atomics (and,
// or) that leave the partner's nibbles alone, so no order of rows, calls or streams loses a token.
#include <cstdint>
#include <cuda_runtime.h>

#include "codec_core.cuh"
#include "common.cuh"
#include "host_util.h"

namespace nvfp4kv {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
    const uint8_t* q;
    const uint8_t* k;
    const uint8_t* v;
    int64_t q_stride, k_stride, v_stride;  // bytes between rows
    const int64_t* slots;
    const int32_t* positions;  // null: no rotation
    const float* table;        // [max_pos][32 rot_units]: cosines, then sines
    const float* gk;
    const float* gv;
    uint8_t* kd;
    uint8_t* ks;
    uint8_t* vd;
    uint8_t* vs;
    uint8_t* q_out;
    int64_t q_out_stride;      // bytes between rows
    uint8_t* k_out;
    uint8_t* v_out;
    int32_t* status;
    uint64_t t_magic;          // ceil(2^64 / T)
    int64_t num_slots;         // pool_pages * T
    int32_t rows, Hq, H, T;
    int32_t first_blk;         // first rotated block of a head
    int32_t rot_units;         // rotated dims / 32
    int32_t max_pos;
    int32_t out_f16;           // the 16-bit outputs are FP16 (else BF16)
    int32_t segs_rot, segs_v;  // warp-wide head groups of a row: q and K heads; V heads
    int32_t rot_each, rot_tasks, v_each, v_tasks;  // head groups of a warp's task, tasks of a row
    int64_t rot_total, tasks;  // tasks of q and K, tasks of all
};

// 8 values of a source row as exact fp32.
template <int SRC>
__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = SRC == NVFP4KV_BF16 ? bf16_lo(w[j]) : f16_lo(w[j]);
        x[2 * j + 1] = SRC == NVFP4KV_BF16 ? bf16_hi(w[j]) : f16_hi(w[j]);
    }
}

// 8 values rounded to the 16-bit output type (round to nearest even), stored past L1, which they would
// only fill (8192 rows 42.4 -> 39.4 us), but left in L2 for the attention that reads them next.
__device__ __forceinline__ void store8(uint8_t* a, const float (&x)[8], bool f16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = f16 ? pack_f16x2(x[2 * j], x[2 * j + 1]) : pack_bf16x2(x[2 * j], x[2 * j + 1]);
    asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3])
                 : "memory");
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(x[j]));
    return a;
}

// The scale picks of two blocks whose halves lie in lanes 2j and 2j + 1: a0, a1 are this lane's
// maxima of block 0 and 1; the even lane picks for block 0, the odd one for block 1 (the arithmetic of
// pick_scale), and both get scale bytes and reciprocals of both. Both lanes of a pair call.
__device__ __forceinline__ void pick_two(float a0, float a1, float g, float d, uint32_t& s0, uint32_t& s1,
                                         float& r0, float& r1) {
    const bool odd = (threadIdx.x & 1) != 0;
    const uint32_t lanes = 3u << (threadIdx.x & 30);
    // the other lane's maximum of the block that this lane picks for
    const float other = __shfl_xor_sync(lanes, odd ? a0 : a1, 1);
    const float a = fmaxf(odd ? a1 : a0, other);
    const uint32_t sb = f32x2_to_e4m3x2(__fdiv_rn(a, d), 0.0f) & 0xFFu;
    const float sg = __fmul_rn(e4m3_to_f32(sb), g);
    const float r = (sg == 0.0f) ? 0.0f : __frcp_rn(sg);
    const uint32_t so = __shfl_xor_sync(lanes, sb, 1);
    const float ro = __shfl_xor_sync(lanes, r, 1);
    s0 = odd ? so : sb;
    s1 = odd ? sb : so;
    r0 = odd ? ro : r;
    r1 = odd ? r : ro;
}

// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), every product and sum rounded to fp32.
__device__ __forceinline__ void rotate(float& x1, float& x2, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    x1 = a;
}

// The V heads of groups seg0 .. seg1 - 1 of a row, alone or with the next row as the other token of its
// pair.
template <int SRC, int D>
__device__ __forceinline__ void append_v(const AppendParams& p, int row, int seg0, int seg1, int64_t slot,
                                         int64_t page, int t, float gv, bool f16) {
    constexpr int L = D / 16, HW = 32 / L, NB = D / 16;
    const int lane = threadIdx.x & 31;
    const int i = (lane % L) >> 1, half = lane & 1, hl = lane / L;
    const int half_T = p.T / 2;
    const bool odd = (t & 1) != 0;
    bool both = false;
    {
        const int other = odd ? row - 1 : row + 1;
        if (other >= 0 && other < p.rows && __ldg(p.slots + other) == (odd ? slot - 1 : slot + 1)) {
            const int opos = p.positions ? __ldg(p.positions + other) : 0;
            both = !p.positions || (opos >= 0 && opos < p.max_pos);
        }
    }
    if (both && odd) return;  // written with the row before
    for (int seg = seg0; seg < seg1; ++seg) {
        const int h = seg * HW + hl;
        if (h >= p.H) continue;
        const uint8_t* src = p.v + row * p.v_stride + h * (D * 2) + 64 * i + 16 * half;
        const int64_t vrow = (page * p.H + h) * half_T + (t >> 1);
        const float d = __fmul_rn(6.0f, gv);
        uint4 w0[2], w1[2];  // blocks 2i and 2i + 1 of this row and the next
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w0[u] = ld_stream_16B(src + 32 * u);
            w1[u] = both ? ld_stream_16B(src + p.v_stride + 32 * u) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int b = 2 * i + u;
            float x0[8], x1[8];  // first and second token of the pair
            widen8<SRC>(w0[u], x0);
            widen8<SRC>(w1[u], x1);
            uint32_t s0, s1;
            float r0, r1;
            pick_two(amax8(x0), amax8(x1), gv, d, s0, s1, r0, r1);
            uint32_t w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[e] = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 4 * e + j;
                    w[e] |= f32x2_to_e2m1x2(__fmul_rn(x0[k], r0), __fmul_rn(x1[k], r1)) << (8 * j);
                }
            }
            uint8_t* vd = p.vd + vrow * D + 16 * b + 8 * half;
            uint8_t* vs = p.vs + vrow * (2 * NB) + 2 * b;
            if (both) {
                *reinterpret_cast<uint2*>(vd) = make_uint2(w[0], w[1]);
                if (!half) *reinterpret_cast<uint16_t*>(vs) = static_cast<uint16_t>(s0 | (s1 << 8));
            } else {
                unsigned int* words = reinterpret_cast<unsigned int*>(vd);
                const uint32_t keep = odd ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t code = w[e] & 0x0F0F0F0Fu;
                    atomicAnd(words + e, keep);
                    atomicOr(words + e, odd ? code << 4 : code);
                }
                if (!half) vs[odd ? 1 : 0] = static_cast<uint8_t>(s0);
            }
            if (p.v_out) {
                // a byte's two codes times the two tokens' scales, exact in FP16
                const uint32_t s2 = e4m3x2_to_f16x2(s0 | (s1 << 8));
                float y0[8], y1[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t c[4];
                    e2m1x8_to_f16x2x4(w[e], c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t v2 = hmul2_u32(c[j], s2);
                        y0[4 * e + j] = __fmul_rn(f16_lo(v2), gv);
                        y1[4 * e + j] = __fmul_rn(f16_hi(v2), gv);
                    }
                }
                uint8_t* dst = p.v_out + ((static_cast<int64_t>(row) * p.H + h) * D + 16 * b + 8 * half) * 2;
                store8(dst, y0, f16);
                if (both) store8(dst + static_cast<int64_t>(p.H) * D * 2, y1, f16);
            }
        }
    }
}

template <int SRC, int D, int STYLE>
__global__ void __launch_bounds__(kAppendThreads, 8) append_kernel(const AppendParams p) {
    pdl_enter();
    constexpr int L = D / 16;   // lanes of a head
    constexpr int HW = 32 / L;  // heads of a warp
    constexpr int NB = D / 16;
    const int lane = threadIdx.x & 31;
    const int i = (lane % L) >> 1, half = lane & 1, hl = lane / L;
    const int warps = static_cast<int>(gridDim.x) * (kAppendThreads / 32);
    const float gk = p.gk ? __ldg(p.gk) : 1.0f, gv = p.gv ? __ldg(p.gv) : 1.0f;
    const bool f16 = p.out_f16 != 0;

    // the thread's two blocks: a rotated pair, or two of the blocks outside the rotated dims
    const bool turns = i < p.rot_units;
    int b0, b1;
    if (turns) {
        b0 = p.first_blk + (STYLE == NVFP4KV_ROTARY_HALVES ? i : 2 * i);
        b1 = STYLE == NVFP4KV_ROTARY_HALVES ? b0 + p.rot_units : b0 + 1;
    } else {
        const int e = 2 * (i - p.rot_units);
        b0 = e < p.first_blk ? e : e + 2 * p.rot_units;
        b1 = e + 1 < p.first_blk ? e + 1 : e + 1 + 2 * p.rot_units;
    }
    const int o0 = 32 * b0 + 16 * half, o1 = 32 * b1 + 16 * half;  // bytes of its values within a head

    for (int64_t task = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
         task < p.tasks; task += warps) {
        const bool is_v = task >= p.rot_total;
        const int64_t at = is_v ? task - p.rot_total : task;
        const int row = static_cast<int>(at / (is_v ? p.v_tasks : p.rot_tasks));
        const int part = static_cast<int>(at - static_cast<int64_t>(row) * (is_v ? p.v_tasks : p.rot_tasks));
        const int64_t slot = __ldg(p.slots + row);
        const int pos = p.positions ? __ldg(p.positions + row) : 0;

        if (slot == -1) continue;  // a padding row
        const bool pos_ok = !p.positions || (pos >= 0 && pos < p.max_pos);
        if (slot < 0 || slot >= p.num_slots || !pos_ok) {
            if (lane == 0)
                flag_status(p.status, pos_ok ? NVFP4KV_STATUS_PAGE_OOB : NVFP4KV_STATUS_BAD_POSITION);
            continue;
        }
        const int64_t page = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(slot), p.t_magic));
        const int t = static_cast<int>(slot - page * p.T);

        if (is_v) {
            append_v<SRC, D>(p, row, part * p.v_each, min((part + 1) * p.v_each, p.segs_v), slot, page, t, gv, f16);
            continue;
        }

        // a head group's q and K values are loaded while the one before is worked on (two groups ahead was
        // 5 us slower for 8192 rows, the first group's loads before the slot is known 2 us)
        const int seg0 = part * p.rot_each, rot1 = min(seg0 + p.rot_each, p.segs_rot);
        auto source = [&](int seg) -> const uint8_t* {  // null: no head for this thread
            const int head = seg * HW + hl;
            if (seg >= rot1 || head >= p.Hq + p.H) return nullptr;
            return head < p.Hq ? p.q + row * p.q_stride + head * (D * 2)
                               : p.k + row * p.k_stride + (head - p.Hq) * (D * 2);
        };
        uint4 n0, n1;
        if (const uint8_t* src = source(seg0)) {
            n0 = ld_stream_16B(src + o0);
            n1 = ld_stream_16B(src + o1);
        }
        // halves: the cosines and sines of dims 8 half .. +7 of the block; adjacent pairs: those of the
        // four pairs in each of the two blocks
        float cs[8], sn[8];
        if (turns) {
            const float* row_cs = p.table + static_cast<int64_t>(pos) * 32 * p.rot_units + 16 * i +
                                  (STYLE == NVFP4KV_ROTARY_HALVES ? 8 : 4) * half;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float* at = row_cs + (STYLE == NVFP4KV_ROTARY_HALVES ? 4 : 8) * j;
                const float4 c4 = __ldg(reinterpret_cast<const float4*>(at));
                const float4 s4 = __ldg(reinterpret_cast<const float4*>(at + 16 * p.rot_units));
                cs[4 * j] = c4.x;
                cs[4 * j + 1] = c4.y;
                cs[4 * j + 2] = c4.z;
                cs[4 * j + 3] = c4.w;
                sn[4 * j] = s4.x;
                sn[4 * j + 1] = s4.y;
                sn[4 * j + 2] = s4.z;
                sn[4 * j + 3] = s4.w;
            }
        }
        // ---- q and K heads
        for (int seg = seg0; seg < rot1; ++seg) {
            const int head = seg * HW + hl;
            float x0[8], x1[8];
            widen8<SRC>(n0, x0);
            widen8<SRC>(n1, x1);
            if (const uint8_t* src = source(seg + 1)) {
                n0 = ld_stream_16B(src + o0);
                n1 = ld_stream_16B(src + o1);
            }
            if (head >= p.Hq + p.H) continue;
            if (turns) {
                if constexpr (STYLE == NVFP4KV_ROTARY_HALVES) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) rotate(x0[j], x1[j], cs[j], sn[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        rotate(x0[2 * j], x0[2 * j + 1], cs[j], sn[j]);
                        rotate(x1[2 * j], x1[2 * j + 1], cs[4 + j], sn[4 + j]);
                    }
                }
            }
            if (head < p.Hq) {
                uint8_t* dst = p.q_out + row * p.q_out_stride + head * (D * 2);
                store8(dst + o0, x0, f16);
                store8(dst + o1, x1, f16);
            } else {
                const int kh = head - p.Hq;
                const int64_t krow = (page * p.H + kh) * p.T + t;
                uint32_t s0, s1;
                float r0, r1;
                pick_two(amax8(x0), amax8(x1), gk, __fmul_rn(6.0f, gk), s0, s1, r0, r1);
                auto put = [&](const float(&x)[8], uint32_t sb, float rr, int b) {
                    uint32_t code = 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        code |= f32x2_to_e2m1x2(__fmul_rn(x[2 * j], rr), __fmul_rn(x[2 * j + 1], rr)) << (8 * j);
                    *reinterpret_cast<uint32_t*>(p.kd + krow * (D / 2) + 8 * b + 4 * half) = code;
                    if (p.k_out) {
                        uint32_t v[4];
                        e2m1x8_to_f16x2x4(code, v);
                        const uint32_t s2 = e4m3x2_to_f16x2(sb * 0x0101u);
                        float y[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t e = hmul2_u32(v[j], s2);
                            y[2 * j] = __fmul_rn(f16_lo(e), gk);
                            y[2 * j + 1] = __fmul_rn(f16_hi(e), gk);
                        }
                        store8(p.k_out + ((static_cast<int64_t>(row) * p.H + kh) * D + 16 * b + 8 * half) * 2, y, f16);
                    }
                };
                put(x0, s0, r0, b0);
                put(x1, s1, r1, b1);
                p.ks[krow * NB + (half ? b1 : b0)] = static_cast<uint8_t>(half ? s1 : s0);
            }
        }
    }
}

template <int SRC, int D>
cudaError_t launch_append(const AppendParams& p, int style, int grid, cudaStream_t s) {
    if (style == NVFP4KV_ROTARY_HALVES)
        return launch_pdl(append_kernel<SRC, D, NVFP4KV_ROTARY_HALVES>, grid, kAppendThreads, 0, s, p);
    return launch_pdl(append_kernel<SRC, D, NVFP4KV_ROTARY_PAIRS>, grid, kAppendThreads, 0, s, p);
}

// A 16-bit row tensor: 16-byte aligned, rows at least `elems` values apart in multiples of 8.
bool rows_ok(const void* p, int64_t stride, int64_t elems) {
    return p && aligned16(p) && stride >= elems && stride % 8 == 0;
}

}  // namespace
}  // namespace nvfp4kv

using namespace nvfp4kv;

extern "C" nvfp4kv_status nvfp4_kv_append(
    const nvfp4kv_layout* layout, nvfp4kv_dtype src_dtype, int32_t num_rows, int32_t num_q_heads,
    const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
    int64_t v_row_stride, const int64_t* slots, const nvfp4kv_rotary* rotary,
    const int32_t* positions, const float* k_global_scale, const float* v_global_scale,
    uint8_t* k_data, uint8_t* k_scales, uint8_t* v_data, uint8_t* v_scales, int32_t pool_pages,
    nvfp4kv_dtype out_dtype, void* q_out, int64_t q_out_row_stride, void* k_out, void* v_out,
    int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || !dtype_ok(src_dtype) || !dtype_ok(out_dtype) || num_rows < 0 ||
        num_q_heads < 0 || layout->page_size % 2 != 0)
        return NVFP4KV_ERR_INVALID_ARG;
    const int D = layout->head_dim, H = layout->num_kv_heads;
    if ((D != 64 && D != 128 && D != 256) || src_dtype == NVFP4KV_FP8_E4M3 ||
        out_dtype == NVFP4KV_FP8_E4M3)
        return NVFP4KV_ERR_UNSUPPORTED;
    if (rotary) {
        if ((rotary->style != NVFP4KV_ROTARY_HALVES && rotary->style != NVFP4KV_ROTARY_PAIRS) ||
            rotary->dims <= 0 || rotary->dims > D || rotary->dims % 32 != 0 ||
            rotary->first_dim < 0 || rotary->first_dim > D - rotary->dims ||
            rotary->first_dim % 16 != 0 || rotary->max_positions <= 0)
            return NVFP4KV_ERR_INVALID_ARG;
    }
    if (num_rows == 0) return NVFP4KV_OK;
    if (rotary && (!rotary->cos_sin || !aligned16(rotary->cos_sin) || !positions))
        return NVFP4KV_ERR_INVALID_ARG;
    if (!rows_ok(k, k_row_stride, static_cast<int64_t>(H) * D) ||
        !rows_ok(v, v_row_stride, static_cast<int64_t>(H) * D) || !slots || pool_pages <= 0 ||
        !k_data || !k_scales || !v_data || !v_scales || !aligned16(k_data) ||
        !aligned16(k_scales) || !aligned16(v_data) || !aligned16(v_scales))
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_q_heads > 0 &&
        (!rows_ok(q, q_row_stride, static_cast<int64_t>(num_q_heads) * D) ||
         !rows_ok(q_out, q_out_row_stride, static_cast<int64_t>(num_q_heads) * D) || q == q_out))
        return NVFP4KV_ERR_INVALID_ARG;
    if ((k_out && (!aligned16(k_out) || k_out == k)) || (v_out && (!aligned16(v_out) || v_out == v)))
        return NVFP4KV_ERR_INVALID_ARG;
    if (num_q_heads > 65535 || H > 65535) return NVFP4KV_ERR_UNSUPPORTED;

    AppendParams p{};
    p.q = static_cast<const uint8_t*>(q);
    p.k = static_cast<const uint8_t*>(k);
    p.v = static_cast<const uint8_t*>(v);
    p.q_stride = 2 * q_row_stride;
    p.k_stride = 2 * k_row_stride;
    p.v_stride = 2 * v_row_stride;
    p.slots = slots;
    p.gk = k_global_scale;
    p.gv = v_global_scale;
    p.kd = k_data;
    p.ks = k_scales;
    p.vd = v_data;
    p.vs = v_scales;
    p.q_out = static_cast<uint8_t*>(q_out);
    p.q_out_stride = 2 * q_out_row_stride;
    p.k_out = static_cast<uint8_t*>(k_out);
    p.v_out = static_cast<uint8_t*>(v_out);
    p.status = status;
    p.t_magic = UINT64_MAX / static_cast<uint64_t>(layout->page_size) + 1;
    p.num_slots = static_cast<int64_t>(pool_pages) * layout->page_size;
    p.rows = num_rows;
    p.Hq = num_q_heads;
    p.H = H;
    p.T = layout->page_size;
    int style = NVFP4KV_ROTARY_HALVES;
    if (rotary) {
        style = rotary->style;
        p.positions = positions;
        p.table = rotary->cos_sin;
        p.first_blk = rotary->first_dim / 16;
        p.rot_units = rotary->dims / 32;
        p.max_pos = rotary->max_positions;
    }
    p.out_f16 = out_dtype == NVFP4KV_FP16;
    const int HW = 32 / (D / 16);
    p.segs_rot = (num_q_heads + H + HW - 1) / HW;
    p.segs_v = (H + HW - 1) / HW;
    // few rows are spread over the GPU, and with many rows the position's table row is read once for all
    // heads (1237 rows of 24 + 4 heads of 256: 12.7 us so, 14.9 with 16 warps to an SM)
    const int64_t spread = static_cast<int64_t>(num_rows) * (p.segs_rot + p.segs_v);
    const int64_t each = (spread + num_sms() * 32 - 1) / (num_sms() * 32);
    p.rot_each = static_cast<int>(each < p.segs_rot ? each : p.segs_rot);
    p.rot_tasks = (p.segs_rot + p.rot_each - 1) / p.rot_each;
    p.v_each = static_cast<int>(each < p.segs_v ? each : p.segs_v);
    p.v_tasks = (p.segs_v + p.v_each - 1) / p.v_each;
    p.rot_total = static_cast<int64_t>(num_rows) * p.rot_tasks;
    p.tasks = p.rot_total + static_cast<int64_t>(num_rows) * p.v_tasks;
    const int64_t ctas = (p.tasks + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    const int64_t most = static_cast<int64_t>(num_sms()) * 32;
    const int grid = static_cast<int>(ctas < most ? ctas : most);

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (src_dtype == NVFP4KV_BF16) {
        switch (D) {
        case 64: e = launch_append<NVFP4KV_BF16, 64>(p, style, grid, s); break;
        case 128: e = launch_append<NVFP4KV_BF16, 128>(p, style, grid, s); break;
        default: e = launch_append<NVFP4KV_BF16, 256>(p, style, grid, s); break;
        }
    } else {
        switch (D) {
        case 64: e = launch_append<NVFP4KV_FP16, 64>(p, style, grid, s); break;
        case 128: e = launch_append<NVFP4KV_FP16, 128>(p, style, grid, s); break;
        default: e = launch_append<NVFP4KV_FP16, 256>(p, style, grid, s); break;
        }
    }
    return launched(e);
}
