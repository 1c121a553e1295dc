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
// Bound: HBM. Every source value is read once and every output written once; the table row of a
// position (at most 4 D bytes) is read once per warp task into registers and reused for every head
// of the task.
//
// A thread owns 32 dims of one head: two 16-value blocks that rotate with one another (block i of
// the first half with block i of the second, or two neighbouring blocks when adjacent dims pair
// up), so the rotation, the block maximum and the packing need no other thread. A warp covers
// 32 / (D / 32) heads at a time.
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
    int32_t wide;              // every source row is 32-byte aligned
    int32_t segs_rot, segs;    // warp-wide head groups of a row: q and K heads, then V heads
    int32_t segs_per_task, tasks_per_row;
    int64_t tasks;
};

// 16 values of a source row.
__device__ __forceinline__ U8x32 load_block(const uint8_t* a, bool wide) {
    if (wide) return ld_stream_32B(a);
    const uint4 lo = ld_stream_16B(a), hi = ld_stream_16B(a + 16);
    return U8x32{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

// 16 values rounded to the 16-bit output type (round to nearest even).
__device__ __forceinline__ void store_block(uint8_t* a, const float (&x)[16], bool f16) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        w[j] = f16 ? pack_f16x2(x[2 * j], x[2 * j + 1]) : pack_bf16x2(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<uint4*>(a) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(a + 16) = make_uint4(w[4], w[5], w[6], w[7]);
}

// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), every product and sum rounded to fp32.
__device__ __forceinline__ void rotate(float& x1, float& x2, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
    x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
    x1 = a;
}

template <int SRC, int D, int STYLE>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const AppendParams p) {
    pdl_enter();
    constexpr int U = D / 32;   // threads of a head
    constexpr int HW = 32 / U;  // heads of a warp
    constexpr int NB = D / 16;
    const int lane = threadIdx.x & 31;
    const int i = lane % U, hl = lane / U;
    const int warps = static_cast<int>(gridDim.x) * (kAppendThreads / 32);
    const int half_T = p.T / 2;
    const float gk = p.gk ? __ldg(p.gk) : 1.0f, gv = p.gv ? __ldg(p.gv) : 1.0f;
    const bool wide = p.wide != 0, f16 = p.out_f16 != 0;

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

    for (int64_t task = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
         task < p.tasks; task += warps) {
        const int row = static_cast<int>(task / p.tasks_per_row);
        const int seg0 = static_cast<int>(task - static_cast<int64_t>(row) * p.tasks_per_row) * p.segs_per_task;
        const int seg1 = min(seg0 + p.segs_per_task, p.segs);
        const int64_t slot = __ldg(p.slots + row);
        if (slot == -1) continue;  // a padding row
        const int pos = p.positions ? __ldg(p.positions + row) : 0;
        const bool pos_ok = !p.positions || (pos >= 0 && pos < p.max_pos);
        if (slot < 0 || slot >= p.num_slots || !pos_ok) {
            if (lane == 0)
                flag_status(p.status, pos_ok ? NVFP4KV_STATUS_PAGE_OOB : NVFP4KV_STATUS_BAD_POSITION);
            continue;
        }
        const int64_t page = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(slot), p.t_magic));
        const int t = static_cast<int>(slot - page * p.T);

        float cs[16], sn[16];
        if (seg0 < p.segs_rot && turns) {
            const float* row_cs = p.table + static_cast<int64_t>(pos) * 32 * p.rot_units + 16 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 c4 = __ldg(reinterpret_cast<const float4*>(row_cs) + j);
                const float4 s4 = __ldg(reinterpret_cast<const float4*>(row_cs + 16 * p.rot_units) + j);
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

        // ---- q and K heads; a head group's values are loaded while the one before is worked on
        const int rot1 = min(seg1, p.segs_rot);
        auto source = [&](int seg) -> const uint8_t* {  // null: no head for this thread
            const int head = seg * HW + hl;
            if (seg >= rot1 || head >= p.Hq + p.H) return nullptr;
            return head < p.Hq ? p.q + row * p.q_stride + static_cast<int64_t>(head) * D * 2
                               : p.k + row * p.k_stride + static_cast<int64_t>(head - p.Hq) * D * 2;
        };
        U8x32 n0, n1;
        {
            const uint8_t* src = source(seg0);
            if (src) {
                n0 = load_block(src + 32 * b0, wide);
                n1 = load_block(src + 32 * b1, wide);
            }
        }
        for (int seg = seg0; seg < rot1; ++seg) {
            const int head = seg * HW + hl;
            float x0[16], x1[16];
            widen<SRC>(n0, 1.0f, x0);
            widen<SRC>(n1, 1.0f, x1);
            const uint8_t* src = source(seg + 1);
            if (src) {
                n0 = load_block(src + 32 * b0, wide);
                n1 = load_block(src + 32 * b1, wide);
            }
            if (head >= p.Hq + p.H) continue;
            const bool is_q = head < p.Hq;
            const int kh = head - p.Hq;
            if (turns) {
                if constexpr (STYLE == NVFP4KV_ROTARY_HALVES) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) rotate(x0[j], x1[j], cs[j], sn[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        rotate(x0[2 * j], x0[2 * j + 1], cs[j], sn[j]);
                        rotate(x1[2 * j], x1[2 * j + 1], cs[8 + j], sn[8 + j]);
                    }
                }
            }
            if (is_q) {
                uint8_t* dst = p.q_out + row * p.q_out_stride + static_cast<int64_t>(head) * D * 2;
                store_block(dst + 32 * b0, x0, f16);
                store_block(dst + 32 * b1, x1, f16);
            } else {
                const int64_t krow = (page * p.H + kh) * p.T + t;
                const float d = __fmul_rn(6.0f, gk);
                auto put = [&](const float(&x)[16], int b) {
                    uint32_t sb;
                    float r;
                    pick_scale(x, gk, d, sb, r);
                    const uint2 code = pack_e2m1_block(x, r);
                    *reinterpret_cast<uint2*>(p.kd + krow * (D / 2) + 8 * b) = code;
                    p.ks[krow * NB + b] = static_cast<uint8_t>(sb);
                    if (p.k_out) {
                        float y[16];
                        block_values(code, sb, y);
#pragma unroll
                        for (int j = 0; j < 16; ++j) y[j] = __fmul_rn(y[j], gk);
                        store_block(p.k_out + ((static_cast<int64_t>(row) * p.H + kh) * D + 16 * b) * 2, y, f16);
                    }
                };
                put(x0, b0);
                put(x1, b1);
            }
        }
        if (seg1 <= p.segs_rot) continue;

        // ---- V heads: this row alone, or with the next one as the other token of its pair
        const bool odd = (t & 1) != 0;
        bool both = false;
        {
            const int other = odd ? row - 1 : row + 1;
            if (other >= 0 && other < p.rows && __ldg(p.slots + other) == (odd ? slot - 1 : slot + 1)) {
                const int opos = p.positions ? __ldg(p.positions + other) : 0;
                both = !p.positions || (opos >= 0 && opos < p.max_pos);
            }
        }
        if (both && odd) continue;  // written with the row before
        for (int seg = max(seg0, p.segs_rot); seg < seg1; ++seg) {
            const int h = (seg - p.segs_rot) * HW + hl;
            if (h >= p.H) continue;
            const uint8_t* src = p.v + row * p.v_stride + static_cast<int64_t>(h) * D * 2;
            const int64_t vrow = (page * p.H + h) * half_T + (t >> 1);
            const float d = __fmul_rn(6.0f, gv);
            U8x32 v0[2], v1[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                v0[u] = load_block(src + 32 * (2 * i + u), wide);
                if (both) v1[u] = load_block(src + p.v_stride + 32 * (2 * i + u), wide);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int b = 2 * i + u;
                float x0[16], x1[16];  // first and second token of the pair
                widen<SRC>(v0[u], 1.0f, x0);
                if (both) widen<SRC>(v1[u], 1.0f, x1);
                uint32_t s0, s1 = 0u;
                float r0, r1 = 0.0f;
                pick_scale(x0, gv, d, s0, r0);
                if (both) pick_scale(x1, gv, d, s1, r1);
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float y0 = __fmul_rn(x0[4 * e + j], r0);
                        const float y1 = both ? __fmul_rn(x1[4 * e + j], r1) : 0.0f;
                        w[e] |= f32x2_to_e2m1x2(y0, y1) << (8 * j);
                    }
                }
                uint8_t* vd = p.vd + vrow * D + 16 * b;
                uint8_t* vs = p.vs + vrow * (2 * NB) + 2 * b;
                if (both) {
                    *reinterpret_cast<uint4*>(vd) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint16_t*>(vs) = static_cast<uint16_t>(s0 | (s1 << 8));
                } else {
                    unsigned int* words = reinterpret_cast<unsigned int*>(vd);
                    const uint32_t keep = odd ? 0x0F0F0F0Fu : 0xF0F0F0F0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        atomicAnd(words + e, keep);
                        atomicOr(words + e, odd ? w[e] << 4 : w[e]);
                    }
                    vs[odd ? 1 : 0] = static_cast<uint8_t>(s0);
                }
                if (p.v_out) {
                    // a byte's two codes times the two tokens' scales, exact in FP16
                    const uint32_t s2 = e4m3x2_to_f16x2(s0 | (s1 << 8));
                    float y0[16], y1[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t c[4];
                        e2m1x8_to_f16x2x4(w[e], c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t v2 = hmul2_u32(c[j], s2);
                            y0[4 * e + j] = __fmul_rn(f16_lo(v2), gv);
                            y1[4 * e + j] = __fmul_rn(f16_hi(v2), gv);
                        }
                    }
                    uint8_t* dst = p.v_out + ((static_cast<int64_t>(row) * p.H + h) * D + 16 * b) * 2;
                    store_block(dst, y0, f16);
                    if (both) store_block(dst + static_cast<int64_t>(p.H) * D * 2, y1, f16);
                }
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
    auto wide = [](const void* a, int64_t stride) {
        return reinterpret_cast<uintptr_t>(a) % 32 == 0 && stride % 32 == 0;
    };
    p.wide = wide(k, p.k_stride) && wide(v, p.v_stride) && (num_q_heads == 0 || wide(q, p.q_stride));
    const int HW = 32 / (D / 32);
    p.segs_rot = (num_q_heads + H + HW - 1) / HW;
    p.segs = p.segs_rot + (H + HW - 1) / HW;
    // a warp takes as many head groups of a row as leave 16 warps to an SM: few rows are spread over
    // the GPU, and with many rows the position's table row is read once for all heads
    const int64_t spread = static_cast<int64_t>(num_rows) * p.segs;
    const int64_t each = (spread + num_sms() * 16 - 1) / (num_sms() * 16);
    p.segs_per_task = static_cast<int>(each < p.segs ? each : p.segs);
    p.tasks_per_row = (p.segs + p.segs_per_task - 1) / p.segs_per_task;
    p.tasks = static_cast<int64_t>(num_rows) * p.tasks_per_row;
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
    if (e != cudaSuccess) return NVFP4KV_ERR_CUDA;
    return launch_status();
}
