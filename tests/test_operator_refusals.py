"""Calls of the routing and microscaled-4-bit entry points that their documentation refuses, beyond single bad arguments:
launches that no grid holds, buffers that the call itself would overwrite, tensors that do not fit.  No GPU needed: each
is refused before any device work."""

import ctypes

import pytest
import torch

import int4_quantized_expert_amd as M

BIG = 1 << 46      # an address that nothing here reads


def experts_call(d, T, n=1 << 60):
    """mx_experts_forward on far-apart addresses: it must be refused before it reads one."""
    at = [BIG + (i << 50) for i in range(1, 9)]
    return M.lib().mx_experts_forward(ctypes.byref(d), T, at[0], None, at[1], None, at[2], at[3], at[4], at[5], n, None)


@pytest.mark.parametrize("n,T,k", [(1 << 20, 1024, 1), (1 << 20, 512, 16), (1000000, 2048, 4)])
def test_a_launch_of_grouped_tiles_that_no_grid_holds(n, T, k):
    """Gated: 64 outputs in a block of 256 threads, for each of 1024 experts and every 128 pairs."""
    d = M.mx_product_desc(n, 32, act="swiglu", n_experts=1024, top_k=k, scales_off=1 << 30, pool_bytes=1 << 40)
    assert (1024 + T * k // 128) * (n // 64) * 256 >= 1 << 32      # with the highest tiles
    assert M.lib().mx_workspace_bytes(ctypes.byref(d), T) == 0
    assert "too many" in M.last_error()
    assert experts_call(d, T) == -1
    assert M.lib().mx_workspace_bytes(ctypes.byref(d), 512 // k) > 0      # fewer pairs, fewer experts that have any


def test_tiles_grow_rather_than_refuse():
    """23 pairs an expert would take tiles of 32 rows, which need more threads than a launch holds; tiles of 64 rows fit.
    Fewer pairs than a permitted number are permitted too."""
    d = M.mx_product_desc(640000, 32, act="swiglu", n_experts=1024, top_k=23, scales_off=1 << 30, pool_bytes=1 << 40)
    assert (1025 + 23552 // 64) * 10000 * 256 < 1 << 32 < (1025 + 23552 // 32) * 10000 * 256
    sizes = [M.lib().mx_workspace_bytes(ctypes.byref(d), T) for T in (1, 64, 500, 1024, 1025, 1100, 1500, 3000, 6000)]
    refused = [s == 0 for s in sizes]
    assert refused == sorted(refused) and not refused[3] and refused[-1]


@pytest.mark.parametrize("a", ["f32", "bf16"])
def test_a_dense_quantisation_that_no_grid_holds(a):
    d = M.mx_product_desc(16, 1 << 20, a=a)
    assert M.lib().mx_workspace_bytes(ctypes.byref(d), 1 << 17) == 0
    assert M.lib().mx_workspace_bytes(ctypes.byref(d), 1 << 16) > 0
    mx = M.mx_product_desc(16, 1 << 20, a="mx")
    assert M.lib().mx_workspace_bytes(ctypes.byref(mx), 1 << 17) > 0


def u8(n, step=1):
    return torch.zeros(n * step, dtype=torch.uint8)[::step]


def test_router_route_checks_its_tensors():
    """x and router_w of too few values, another floating-point type or strided rows; the same as raw bytes pass on to the
    next check (tensors that are not on a GPU)."""
    d = M.desc_for(256, 16, 2, 128, 128, 4, "bf16", "f32", "f32", pool_bytes=1 << 20)
    r = M.route_desc(16, 2)
    ids, w, ws = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), u8(M.workspace_bytes(d, 3))

    def refused(x=None, router=None, ws=ws):
        x = torch.zeros(3, 256, dtype=torch.bfloat16) if x is None else x
        router = torch.zeros(16, 256, dtype=torch.bfloat16) if router is None else router
        with pytest.raises(M.MoeError) as err:
            M.router_route(d, r, 3, x, router, None, ids, w, ws)
        return str(err.value)
    assert "not on a GPU" in refused()
    assert "not on a GPU" in refused(x=u8(3 * 512), router=u8(16 * 512))
    assert "x has" in refused(x=torch.zeros(2, 256, dtype=torch.bfloat16)) and "x has" in refused(x=u8(3 * 512 - 1))
    assert "x is torch.float32" in refused(x=torch.zeros(3, 256)) and "x is torch.float16" in refused(x=torch.zeros(3, 256, dtype=torch.float16))
    assert "not contiguous" in refused(x=torch.zeros(3, 512, dtype=torch.bfloat16)[:, :256])
    assert "router_w has" in refused(router=torch.zeros(15, 256, dtype=torch.bfloat16))
    assert "router_w is" in refused(router=torch.zeros(16, 256))
    assert "not contiguous" in refused(router=torch.zeros(256, 16, dtype=torch.bfloat16).t())
    assert "workspace" in refused(ws=BIG) and "workspace" in refused(ws=None) and "not contiguous" in refused(ws=u8(ws.numel(), 2))


def test_products_check_their_pool_and_workspace():
    d = M.mx_product_desc(32, 64, n_experts=4, top_k=2, scales_off=4096, pool_bytes=65536)
    a, ids, slots = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    out, need = torch.zeros(8, 32, dtype=torch.bfloat16), M.mx_workspace_bytes(d, 4)

    def refused(pool=u8(65536), ws=u8(need)):
        with pytest.raises(M.MoeError) as err:
            M.mx_experts(d, 4, a, None, ids, None, slots, pool, out, ws)
        return str(err.value)
    assert "not on a GPU" in refused() and "not on a GPU" in refused(pool=torch.zeros(16384))
    assert "pool has" in refused(pool=u8(65535)) and "not contiguous" in refused(pool=u8(65536, 2))
    assert "workspace" in refused(ws=BIG) and "workspace" in refused(ws=None) and "not contiguous" in refused(ws=u8(need, 2))
    d = M.mx_product_desc(32, 64)
    need = M.mx_workspace_bytes(d, 4)
    for ws in (BIG, None, u8(need, 2)):
        with pytest.raises(M.MoeError) as err:
            M.mx_linear(d, 4, a, None, u8(32 * 128), u8(32 * 8), out, ws)
        assert "workspace" in str(err.value)


def test_quantisation_takes_tensors():
    for call in (lambda: M.mx_quantize(BIG, BIG, BIG), lambda: M.mx_dequantize(BIG, BIG, BIG), lambda: M.mx_quantize(None, BIG, BIG)):
        with pytest.raises(M.MoeError) as err:
            call()
        assert "has to be a tensor" in str(err.value)


def test_router_route_refuses_buffers_that_the_call_would_overwrite():
    d = M.desc_for(256, 16, 2, 128, 128, 4, "f32", "f32", "f32", pool_bytes=1 << 20)
    r, need = M.route_desc(16, 2), M.workspace_bytes(d, 3)
    buf = ctypes.create_string_buffer(need + (1 << 18))
    p = ctypes.addressof(buf) // 256 * 256 + 256
    x, router, bias, ids, w, ws = p, p + 4096, p + 32768, p + 36864, p + 40960, p + 65536

    def call(x=x, router=router, bias=bias, ids=ids, w=w, T=3):
        return M.lib().moe_router_route(ctypes.byref(d), ctypes.byref(r), T, x, router, bias, ids, w, ws, need, None)
    end = ws + need // 256 * 256
    # the logits would be written over them, or read in their place
    assert call(bias=ws + 1024) == -1 and call(x=ws + 4096) == -1 and call(router=ws + 4096) == -1 and call(bias=end - 4) == -1
    assert call(x=ws - 3 * 1024 + 16) == -1 and call(bias=ws - 60) == -1
    # the outputs over an input
    assert call(ids=x + 3 * 1024 - 4) == -1 and call(w=x) == -1 and call(ids=router + 16 * 1024 - 4) == -1 and call(w=router - 20) == -1
    assert call(ids=bias + 60) == -1
    # T = 0 reads and writes nothing
    assert call(T=0) == 0


def test_rows_whose_last_place_does_not_fit_64_bits():
    """2^30 rows a stride of 2^33 apart and more: their extent is no 64-bit number of bytes, so that nothing could be said
    about what they overlap."""
    L = M.lib()
    for rows, stride in ((1 << 30, 1 << 33), ((1 << 31) - 1, 1 << 40), (1 << 20, 1 << 37)):
        assert L.mx_quantize(0, rows, 4, BIG, stride, BIG << 1, BIG << 2, None) == -1
        assert L.mx_dequantize(0, rows, 4, BIG << 1, BIG << 2, BIG, stride, None) == -1
        assert "stride" in M.last_error()
