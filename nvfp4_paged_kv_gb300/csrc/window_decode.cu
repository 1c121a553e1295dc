// C entry point of the paged decode attention over NVFP4 K/V with a sliding window and first tokens that stay visible;
// the kernel is in window_kernel.cuh.
#include <cstdint>
#include <cuda_runtime.h>

#include "window_kernel.cuh"

using namespace nvfp4kv;

extern "C" size_t nvfp4_paged_window_decode_workspace_size(const nvfp4kv_layout* layout, int32_t batch,
                                                           int32_t num_q_heads, int32_t max_pages_per_seq) {
    if (batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || !decode_shape_ok(layout, num_q_heads)) return 0;
    const int H = layout->num_kv_heads;
    return ws_layout(batch, H, num_q_heads, layout->head_dim, decode_runs(batch, H, layout->head_dim, 0)).total;
}

extern "C" nvfp4kv_status nvfp4_paged_window_decode_attention(
    const nvfp4kv_layout* layout, int32_t batch, int32_t num_q_heads, const void* q,
    const uint8_t* k_data, const uint8_t* k_scales, const float* k_global_scale,
    const uint8_t* v_data, const uint8_t* v_scales, const float* v_global_scale,
    int32_t pool_pages, const int32_t* page_table, int32_t max_pages_per_seq,
    const int32_t* seq_lens, int32_t window, int32_t sink_tokens, float sm_scale, void* workspace,
    size_t workspace_bytes, void* out, float* lse, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 || pool_pages <= 0 ||
        window <= 0 || sink_tokens < 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!decode_shape_ok(layout, num_q_heads)) return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0) return NVFP4KV_OK;
    if (!q || !k_data || !k_scales || !k_global_scale || !v_data || !v_scales || !v_global_scale || !page_table ||
        !seq_lens || !out)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_data) || !aligned16(k_scales) || !aligned16(v_data) || !aligned16(v_scales) ||
        !aligned16(out))
        return NVFP4KV_ERR_INVALID_ARG;
    if (batch > 65535 || num_q_heads > 65535) return NVFP4KV_ERR_UNSUPPORTED;
    const int D = layout->head_dim, H = layout->num_kv_heads, T = layout->page_size;
    const int64_t runs = decode_runs(batch, H, D, 0);
    if (!window_size_ok(batch, H, D, max_pages_per_seq, T, runs, kNvfp4)) return NVFP4KV_ERR_UNSUPPORTED;
    const WsLayout wl = ws_layout(batch, H, num_q_heads, D, runs);
    if (!workspace || workspace_bytes < wl.total || !aligned16(workspace)) return NVFP4KV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);

    WindowParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.kd = k_data;
    p.ks = k_scales;
    p.vd = v_data;
    p.vs = v_scales;
    p.gk = k_global_scale;
    p.gv = v_global_scale;
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
    p.window = window;
    p.sinks = sink_tokens;

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (D) {
    case 64: return launched(launch_window<64, kNvfp4, true>(p, runs, s));
    case 128: return launched(launch_window<128, kNvfp4, true>(p, runs, s));
    default: return launched(launch_window<256, kNvfp4, true>(p, runs, s));
    }
}
