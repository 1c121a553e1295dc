// C entry points of the paged decode attention; the kernel and its host helpers are in
// decode_kernel.cuh.
#include <cstdint>
#include <cuda_runtime.h>

#include "decode_kernel.cuh"

using namespace nvfp4kv;

extern "C" size_t nvfp4_paged_decode_workspace_size(const nvfp4kv_layout* layout, int32_t batch,
                                                    int32_t num_q_heads,
                                                    int32_t max_pages_per_seq,
                                                    int32_t max_num_splits) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 ||
        max_num_splits < 0 || max_num_splits > kMaxSplits)
        return 0;
    if (num_q_heads % layout->num_kv_heads != 0) return 0;
    const int H = layout->num_kv_heads;
    const int64_t runs = decode_runs(batch, H, layout->head_dim, max_num_splits);
    return ws_layout(batch, H, num_q_heads, layout->head_dim, runs).total;
}

extern "C" nvfp4kv_status nvfp4_paged_decode_attention(
    const nvfp4kv_layout* layout, int32_t batch, int32_t num_q_heads, const void* q,
    const uint8_t* k_data, const uint8_t* k_scales, const float* k_global_scale,
    const uint8_t* v_data, const uint8_t* v_scales, const float* v_global_scale,
    int32_t pool_pages, const int32_t* page_table, int32_t max_pages_per_seq,
    const int32_t* seq_lens, float sm_scale, int32_t max_num_splits, void* workspace,
    size_t workspace_bytes, void* out, float* lse, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_pages_per_seq <= 0 ||
        pool_pages <= 0 || max_num_splits < 0 || max_num_splits > kMaxSplits)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!decode_shape_ok(layout, num_q_heads)) return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0) return NVFP4KV_OK;
    if (!q || !k_data || !k_scales || !k_global_scale || !v_data || !v_scales ||
        !v_global_scale || !page_table || !seq_lens || !out)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_data) || !aligned16(k_scales) || !aligned16(v_data) ||
        !aligned16(v_scales) || !aligned16(out))
        return NVFP4KV_ERR_INVALID_ARG;
    if (batch > 65535 || num_q_heads > 65535) return NVFP4KV_ERR_UNSUPPORTED;
    const int D = layout->head_dim;
    const int H = layout->num_kv_heads;
    const int T = layout->page_size;
    const int64_t runs = decode_runs(batch, H, D, max_num_splits);
    if (!decode_size_ok(batch, H, D, max_pages_per_seq, T, runs)) return NVFP4KV_ERR_UNSUPPORTED;
    const WsLayout wl = ws_layout(batch, H, num_q_heads, D, runs);
    if (!workspace || workspace_bytes < wl.total || !aligned16(workspace))
        return NVFP4KV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);

    DecodeParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.kd = k_data;
    p.ks = k_scales;
    p.vd = v_data;
    p.vs = v_scales;
    p.gk = k_global_scale;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.gv = v_global_scale;
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

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
    case 64: e = launch_decode<64>(p, runs, s); break;
    case 128: e = launch_decode<128>(p, runs, s); break;
    default: e = launch_decode<256>(p, runs, s); break;
    }
    return launched(e);
}
