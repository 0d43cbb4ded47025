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
