// C entry point of the paged decode attention over FP8 pages (a scale for each page and head), with or without a sliding
// window; the kernel is in window_kernel.cuh.
#include <cstdint>
#include <cuda_runtime.h>

#include "window_kernel.cuh"

using namespace nvfp4kv;

extern "C" size_t nvfp4_paged_fp8_decode_workspace_size(const nvfp4kv_layout* layout, int32_t batch,
                                                        int32_t num_q_heads, int32_t max_pages_per_seq) {
    if (batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || !decode_shape_ok(layout, num_q_heads)) return 0;
    const int H = layout->num_kv_heads;
    return ws_layout(batch, H, num_q_heads, layout->head_dim, decode_runs(batch, H, layout->head_dim, 0)).total;
}

extern "C" nvfp4kv_status nvfp4_paged_fp8_decode_attention(
    const nvfp4kv_layout* layout, int32_t batch, int32_t num_q_heads, const void* q,
    const uint8_t* k_pages, const float* k_block_scales, const float* k_scale,
    const uint8_t* v_pages, const float* v_block_scales, const float* v_scale, int32_t pool_pages,
    const int32_t* page_table, int32_t max_pages_per_seq, const int32_t* seq_lens, int32_t window,
    int32_t sink_tokens, float sm_scale, void* workspace, size_t workspace_bytes, void* out,
    float* lse, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || pool_pages <= 0 ||
        window < 0 || sink_tokens < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!decode_shape_ok(layout, num_q_heads)) return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0) return NVFP4KV_OK;
    if (!q || !k_pages || !v_pages || !page_table || !seq_lens || !out) return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out)) return NVFP4KV_ERR_INVALID_ARG;
    if (batch > 65535 || num_q_heads > 65535) return NVFP4KV_ERR_UNSUPPORTED;
    const int D = layout->head_dim, H = layout->num_kv_heads, T = layout->page_size;
    const int64_t runs = decode_runs(batch, H, D, 0);
    if (!window_size_ok(batch, H, D, max_pages_per_seq, T, runs, kFp8)) return NVFP4KV_ERR_UNSUPPORTED;
    const WsLayout wl = ws_layout(batch, H, num_q_heads, D, runs);
    if (!workspace || workspace_bytes < wl.total || !aligned16(workspace)) return NVFP4KV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);

    WindowParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.kd = k_pages;
    p.vd = v_pages;
    p.kbs = k_block_scales;
    p.vbs = v_block_scales;
    p.gk = k_scale;
    p.gv = v_scale;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.done = reinterpret_cast<unsigned long long*>(ws + wl.done);
    p.nonce = next_nonce();
    p.rec_ml = reinterpret_cast<float*>(ws + wl.ml);
    p.rec_o = reinterpret_cast<float*>(ws + wl.o);
    p.status = status;
    p.t_magic = UINT64_MAX / static_cast<uint64_t>(T) + 1;
    p.B = batch;
    p.Hq = num_q_heads;
    p.H = H;
    p.G = num_q_heads / H;
    p.T = T;
    p.pool_pages = pool_pages;
    p.max_pages = max_pages_per_seq;
    p.num_runs = static_cast<int32_t>(runs);
    p.sm_scale = sm_scale;
    p.window = window > 0 ? window : INT32_MAX;
    p.sinks = sink_tokens;

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool win = window > 0;
    switch (D) {
    case 64: return launched(win ? launch_window<64, kFp8, true>(p, runs, s) : launch_window<64, kFp8, false>(p, runs, s));
    case 128: return launched(win ? launch_window<128, kFp8, true>(p, runs, s) : launch_window<128, kFp8, false>(p, runs, s));
    default: return launched(win ? launch_window<256, kFp8, true>(p, runs, s) : launch_window<256, kFp8, false>(p, runs, s));
    }
}
