"""The library shares the CUDA runtime with its caller. An error that someone else's call left as the runtime's last one
is not reported as a failure of a call whose work is enqueued. (Whether it is still there afterwards is the runtime's
affair: cudaFuncSetAttribute resets it.)"""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kv(cuda):
    from nvfp4_paged_kv_gb300 import build
    build.build()
    import nvfp4_paged_kv_gb300 as m
    m.load()
    return m


def calls(kv, dev):
    """name -> (call, tensor that it has to change)."""
    B, H, G, D, T, P = 2, 2, 2, 64, 16, 6
    lay = kv.Layout(H, D, T)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    i32 = lambda fill, *s: torch.full(s, fill, dtype=torch.int32, device=dev)  # noqa: E731
    kd, ks, vd, vs = u8(P, H, T, D // 2), u8(P, H, T, D // 16), u8(P, H, T // 2, D), u8(P, H, T // 2, D // 16, 2)
    pages = torch.randn((P, H, T, D), device=dev).to(torch.bfloat16)
    rows = torch.randn((B, H, D), device=dev).to(torch.bfloat16)
    q = torch.randn((B, H * G, D), device=dev).to(torch.bfloat16)
    g = torch.ones(1, device=dev)
    ws = u8(8 << 20)
    new = lambda t: torch.full_like(t, 7)  # noqa: E731
    qd, qs, ad, vd2 = new(kd), new(ks), new(kd), new(vd)
    ad2, ks2, vs2 = new(vd), new(ks), new(vs)
    back, scale, out, out2 = new(pages), new(g), new(q), new(q)
    bounds = torch.full((P, H, 2, D), 7, dtype=torch.int8, device=dev)
    bscales = torch.full((P, H), 7.0, device=dev)
    sel, sl = i32(7, B, H, 3), i32(7, B, H)
    x, e2m1, fp8, slots = torch.randn(100, device=dev), new(u8(100)), new(pages.to(torch.uint8)), torch.arange(B, device=dev)
    bl = kv.nvfp4_kv_cold_block_layout(lay)
    cold, table, lens = new(u8(P, bl.bytes)), i32(0, B, 4), i32(40, B)
    sel_in, sl_in = i32(1, B, H, 4), i32(40, B, H)
    hot = [new(pages), new(pages)]
    return {
        "append": (lambda: kv.nvfp4_kv_append(lay, rows, rows, slots, ad, ks2, vd2, vs2), ad),
        "bounds": (lambda: kv.nvfp4_kv_page_bounds(lay, kd, ks, bounds, bscales), bscales),
        "select": (lambda: kv.nvfp4_kv_select_pages(lay, q, bounds, bscales, table, lens, sel, sl), sl),
        "attention over selected pages": (lambda: kv.nvfp4_paged_sparse_decode_attention(
            lay, q, kd, ks, g, vd, vs, g, sel_in, sl_in, 0.1, out, workspace=ws), out),
        "attention": (lambda: kv.nvfp4_paged_decode_attention(
            lay, q, kd, ks, g, vd, vs, g, table, lens, 0.1, out2, workspace=ws), out2),
        "global scale": (lambda: kv.nvfp4_kv_compute_global_scale(lay, pages, scale, workspace=ws), scale),
        "quantize": (lambda: kv.nvfp4_kv_quantize_pages(lay, pages, g, qd, qs), qd),
        "dequantize": (lambda: kv.nvfp4_kv_dequantize_pages(lay, kd, ks, g, back), back),
        "extend write": (lambda: kv.nvfp4_kv_extend_write(lay, pages, g, qd, qs, fp8), fp8),
        "round": (lambda: kv.nvfp4_kv_round_f32(x, 0, e2m1), e2m1),
        "offload": (lambda: kv.nvfp4_kv_offload_pages(lay, pages, pages, cold), cold),
        "onboard": (lambda: kv.nvfp4_kv_onboard_pages(lay, cold, *hot), hot[0]),
    }


def test_an_error_from_before_the_call_is_not_the_calls(kv, cuda):
    runtime = ctypes.CDLL("libcudart.so.13")
    for name, (call, changed) in calls(kv, cuda).items():
        before = changed.clone()
        torch.cuda.synchronize()
        # an error that changes nothing: there is no device 1000 (cudaErrorInvalidDevice, 101)
        assert runtime.cudaSetDevice(1000) == 101
        try:
            call()
        finally:
            runtime.cudaGetLastError()   # nor is it for torch's next check
        torch.cuda.synchronize()
        assert not torch.equal(changed, before), name
