// C entry points of the paged decode attention over selected pages; the kernel is in sparse_kernel.cuh.
#include <cstdint>
#include <cuda_runtime.h>

#include "sparse_kernel.cuh"

using namespace nvfp4kv;

extern "C" size_t nvfp4_paged_sparse_decode_workspace_size(const nvfp4kv_layout* layout,
                                                           int32_t batch, int32_t num_q_heads,
                                                           int32_t max_sel_pages) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_sel_pages <= 0) return 0;
    if (num_q_heads % layout->num_kv_heads != 0) return 0;
    const int H = layout->num_kv_heads;
    const int64_t pairs = static_cast<int64_t>(batch) * H;
    if (pairs > kMaxSparsePairs) return 0;
    const int64_t runs = decode_runs(static_cast<int>(pairs), 1, layout->head_dim, 0);
    return ws_layout(static_cast<int>(pairs), 1, num_q_heads / H, layout->head_dim, runs).total;
}

extern "C" nvfp4kv_status nvfp4_paged_sparse_decode_attention(
    const nvfp4kv_layout* layout, int32_t batch, int32_t num_q_heads, const void* q,
    const uint8_t* k_data, const uint8_t* k_scales, const float* k_global_scale,
    const uint8_t* v_data, const uint8_t* v_scales, const float* v_global_scale,
    int32_t pool_pages, const int32_t* sel_page_table, int32_t max_sel_pages,
    const int32_t* sel_lens, float sm_scale, void* workspace, size_t workspace_bytes, void* out,
    float* lse, int32_t* status, nvfp4kv_stream_t stream) {
    if (!layout_ok(layout) || batch < 0 || num_q_heads <= 0 || max_sel_pages <= 0 ||
        pool_pages <= 0)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!decode_shape_ok(layout, num_q_heads)) return NVFP4KV_ERR_UNSUPPORTED;
    if (batch == 0) return NVFP4KV_OK;
    if (!q || !k_data || !k_scales || !k_global_scale || !v_data || !v_scales ||
        !v_global_scale || !sel_page_table || !sel_lens || !out)
        return NVFP4KV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_data) || !aligned16(k_scales) || !aligned16(v_data) ||
        !aligned16(v_scales) || !aligned16(out))
        return NVFP4KV_ERR_INVALID_ARG;
    const int D = layout->head_dim;
    const int H = layout->num_kv_heads;
    const int T = layout->page_size;
    const int64_t pairs = static_cast<int64_t>(batch) * H;
    if (pairs > kMaxSparsePairs) return NVFP4KV_ERR_UNSUPPORTED;
    const int B = static_cast<int>(pairs), G = num_q_heads / H;
    const int64_t runs = decode_runs(B, 1, D, 0);
    if (!decode_size_ok(B, 1, D, max_sel_pages, T, runs)) return NVFP4KV_ERR_UNSUPPORTED;
    const WsLayout wl = ws_layout(B, 1, G, D, runs);
    if (!workspace || workspace_bytes < wl.total || !aligned16(workspace))
        return NVFP4KV_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);

    SparseParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.kd = k_data;
    p.ks = k_scales;
    p.vd = v_data;
    p.vs = v_scales;
    p.gk = k_global_scale;
    p.page_table = sel_page_table;
    p.seq_lens = sel_lens;
    p.gv = v_global_scale;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.done = reinterpret_cast<unsigned long long*>(ws + wl.done);
    p.nonce = next_nonce();
    p.rec_ml = reinterpret_cast<float*>(ws + wl.ml);
    p.rec_o = reinterpret_cast<float*>(ws + wl.o);
    p.status = status;
    p.t_magic = UINT64_MAX / static_cast<uint64_t>(T) + 1;
    p.B = B;
    p.Hq = G;
    p.H = 1;
    p.G = G;
    p.T = T;
    p.pool_pages = pool_pages;
    p.max_pages = max_sel_pages;
    p.pool_heads = H;
    const int64_t each = (static_cast<int64_t>(max_sel_pages) * T + stage_tokens(D) - 1) / stage_tokens(D);
    p.full_each = static_cast<int32_t>(each);  // (pairs * each is bounded by decode_size_ok)
    p.sm_scale = sm_scale;

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
    case 64: e = launch_sparse<64>(p, s); break;
    case 128: e = launch_sparse<128>(p, s); break;
    default: e = launch_sparse<256>(p, s); break;
    }
    return launched(e);
}
