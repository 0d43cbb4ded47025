"""Checks of the routing and microscaled-4-bit entry points that need no GPU: every declared symbol is exported, sizes,
and refusals before any device call."""

import ctypes
import os
import re

import pytest
import torch

import int4_quantized_expert_amd as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Host:
    """Host memory standing in for device buffers: every call here is refused, or does nothing, before any device work."""

    def __init__(self, n=1 << 20):
        self.buf = ctypes.create_string_buffer(n + 512)
        self.p = ctypes.addressof(self.buf) // 256 * 256 + 256


def test_declared_symbols_are_exported():
    names = []
    for f in ("moe_route.h", "mxfp4.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", f)).read(), flags=re.S)
        names += re.findall(r"^[A-Za-z_][\w\s\*]*?\b((?:moe|mx)_\w+)\s*\(", text, flags=re.M)
    assert len(set(names)) == 9
    for n in names:
        assert hasattr(M.lib(), n), n


def test_mx_sizes():
    L = M.lib()
    assert L.mx_codes_bytes(3, 300) == 3 * 256 and L.mx_scales_bytes(3, 300) == 3 * 16
    assert L.mx_codes_bytes(0, 5) == 0 and L.mx_codes_bytes(2, 256) == 256
    assert L.mx_codes_bytes(-1, 5) == -1 and L.mx_codes_bytes(1 << 31, 5) == -1 and L.mx_scales_bytes(1, (1 << 20) + 1) == -1
    assert M.mx_shapes(3, 300) == ((3, 256), (3, 16))
    with pytest.raises(M.MoeError):
        M.mx_shapes(1, -1)


@pytest.mark.parametrize("field,value", [
    ("n_experts", 0), ("n_experts", 1025), ("top_k", 0), ("top_k", 65), ("top_k", 33), ("score", 2), ("n_groups", 0),
    ("n_groups", 7), ("n_groups", 128), ("top_groups", 0), ("top_groups", 9), ("group_top", 0), ("group_top", 3),
    ("renormalize", 2), ("logit_dtype", 2), ("scale", float("nan")), ("scale", float("inf")),
])
def test_route_bad_descriptor(field, value):
    h = Host()
    r = M.route_desc(128, 8, "sigmoid", 8, 2, 2)      # 32 experts stay
    setattr(r, field, value)
    assert M.lib().moe_route_forward(ctypes.byref(r), 1, h.p, 128, None, h.p + 4096, h.p + 8192, None) == -1
    assert M.last_error()


def test_route_bad_arguments():
    h, L = Host(), M.lib()
    r = M.route_desc(128, 8)

    def call(T=2, logits=h.p, stride=128, bias=h.p + 2048, ids=h.p + 4096, w=h.p + 8192, d=r):
        return L.moe_route_forward(ctypes.byref(d) if d else None, T, logits, stride, bias, ids, w, None)
    assert call(d=None) == -1 and call(T=-1) == -1 and call(T=(1 << 20) + 1) == -1 and call(stride=127) == -1
    assert call(logits=None) == -1 and call(ids=None) == -1 and call(w=None) == -1
    assert call(logits=h.p + 2) == -1 and call(ids=h.p + 4097) == -1 and call(bias=h.p + 2050) == -1
    assert call(ids=h.p + 1020) == -1            # inside the second row of logits
    assert call(w=h.p + 4096 + 60) == -1         # over the ids
    assert call(ids=h.p + 2048 + 508) == -1      # over the end of the bias
    assert call(T=0) == 0
    with pytest.raises(M.MoeError):
        M.route(r, 2, torch.zeros(2, 127), None, h.p, h.p)
    with pytest.raises(M.MoeError):
        M.route(r, 2, torch.zeros(2, 128, dtype=torch.bfloat16), None, h.p, h.p)
    with pytest.raises(M.MoeError):
        M.route(r, 2, torch.zeros(2, 128), None, torch.zeros(15, dtype=torch.int32), h.p)
    with pytest.raises(M.MoeError):              # tensors that are not on a GPU
        M.route(r, 2, torch.zeros(2, 128), None, h.p, h.p)


def test_router_route_refusals():
    h, L = Host(), M.lib()
    d = M.desc_for(256, 16, 2, 128, 128, 4, "f32", "f32", "f32", pool_bytes=1 << 20)
    need = M.workspace_bytes(d, 1)
    r = M.route_desc(16, 2)

    def call(r=r, x=h.p, bias=None, ids=h.p + 4096, w=h.p + 8192, ws=h.p + 65536, n=need, T=1):
        return L.moe_router_route(ctypes.byref(d), ctypes.byref(r), T, x, h.p, bias, ids, w, ws, n, None)
    assert call(r=M.route_desc(15, 2)) == -1 and call(r=M.route_desc(16, 3)) == -1
    assert call(r=M.route_desc(16, 2, logits="bf16")) == -1
    assert call(x=None) == -1 and call(ids=None) == -1 and call(n=need - 1) == -4 and call(T=-1) == -1
    assert call(ids=h.p + 65536 + 64) == -1      # inside the workspace
    assert call(T=0) == 0


def test_mx_quantize_refusals():
    h, L = Host(), M.lib()

    def call(fn=L.mx_quantize, dt=0, rows=4, cols=64, x=h.p, stride=64, codes=h.p + 65536, scales=h.p + 131072):
        args = (dt, rows, cols, x, stride, codes, scales) if fn is L.mx_quantize else (dt, rows, cols, codes, scales, x, stride)
        return fn(*args, None)
    for fn in (L.mx_quantize, L.mx_dequantize):
        assert call(fn, dt=2) == -1 and call(fn, rows=-1) == -1 and call(fn, cols=-1) == -1 and call(fn, cols=(1 << 20) + 1) == -1
        assert call(fn, stride=63) == -1 and call(fn, x=None) == -1 and call(fn, codes=None) == -1 and call(fn, scales=None) == -1
        assert call(fn, x=h.p + 2) == -1 and call(fn, codes=h.p + 65544) == -1 and call(fn, scales=h.p + 131080) == -1
        assert call(fn, codes=h.p + 512) == -1 and call(fn, scales=h.p + 65536 + 256) == -1
        assert call(fn, rows=0) == 0 and call(fn, cols=0) == 0
    far = 1 << 46                               # 2^37 values: more threads than a launch holds
    for fn in (L.mx_quantize, L.mx_dequantize):
        assert call(fn, rows=1 << 17, cols=1 << 20, stride=1 << 20, codes=far, scales=far << 1) == -1
    with pytest.raises(M.MoeError):
        M.mx_quantize(torch.zeros(2, 64, dtype=torch.float16), h.p, h.p)
    with pytest.raises(M.MoeError):
        M.mx_quantize(torch.zeros(64, 2).t(), h.p, h.p)          # rows of strided values
    with pytest.raises(M.MoeError):
        M.mx_quantize(torch.zeros(2, 64), torch.zeros(255, dtype=torch.uint8), h.p)
    with pytest.raises(M.MoeError):                              # not on a GPU
        M.mx_quantize(torch.zeros(2, 64), torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.uint8))


@pytest.mark.parametrize("field,value", [
    ("n", 0), ("n", (1 << 20) + 1), ("k", 0), ("a_dtype", 3), ("out_dtype", 2), ("act", 2), ("n_experts", 1), ("top_k", 1),
    ("pair_rows", 1), ("codes_off", 16), ("pool_bytes", 1),
])
def test_mx_linear_bad_descriptor(field, value):
    h = Host()
    d = M.mx_product_desc(32, 64)
    setattr(d, field, value)
    assert M.lib().mx_linear_forward(ctypes.byref(d), 1, h.p, None, h.p, h.p, h.p, h.p, 1 << 30, None) == -1


def test_mx_linear_bad_arguments():
    h, L = Host(1 << 23), M.lib()
    d = M.mx_product_desc(32, 64)
    need = M.mx_workspace_bytes(d, 4)
    a, wc, wsc, out, ws = h.p, h.p + 8192, h.p + 32768, h.p + 65536, h.p + 131072

    def call(d=d, M_=4, a=a, a_s=None, wc=wc, wsc=wsc, out=out, ws=ws, n=need):
        return L.mx_linear_forward(ctypes.byref(d), M_, a, a_s, wc, wsc, out, ws, n, None)
    assert call(M_=-1) == -1 and call(M_=(1 << 20) + 1) == -1 and call(a=None) == -1 and call(wc=None) == -1 and call(wsc=None) == -1
    assert call(out=None) == -1 and call(ws=None) == -1 and call(ws=ws + 8) == -1 and call(n=need - 1) == -4
    assert call(a=a + 1) == -1 and call(wc=wc + 8) == -1 and call(out=out + 1) == -1 and call(a_s=h.p) == -1
    assert call(out=a + 128) == -1 and call(out=wc + 64) == -1 and call(out=ws + 64) == -1 and call(ws=wc) == -1
    assert call(d=M.mx_product_desc(32, 64, a="mx")) == -1       # no scales
    assert call(M_=0) == 0
    assert M.lib().mx_workspace_bytes(ctypes.byref(d), -1) == 0
    with pytest.raises(M.MoeError):
        M.mx_workspace_bytes(M.mx_product_desc(0, 64), 4)
    big = M.mx_product_desc(1 << 20, 64)
    assert call(d=big, M_=1 << 20, n=1 << 62) == -1              # more blocks than a launch holds


@pytest.mark.parametrize("field,value", [
    ("n_experts", -1), ("n_experts", 1025), ("top_k", 0), ("top_k", 65), ("pair_rows", 2), ("codes_off", 8), ("codes_off", -16),
    ("scales_off", 16), ("pool_bytes", 4096), ("pool_bytes", 0),
])
def test_mx_experts_bad_descriptor(field, value):
    h = Host()
    d = M.mx_product_desc(32, 64, n_experts=4, top_k=2, scales_off=4096, pool_bytes=65536)
    setattr(d, field, value)
    assert M.lib().mx_experts_forward(ctypes.byref(d), 1, h.p, None, h.p, None, h.p, h.p, h.p, h.p, 1 << 30, None) == -1


def test_mx_experts_bad_arguments():
    h, L = Host(1 << 23), M.lib()
    d = M.mx_product_desc(32, 64, n_experts=4, top_k=2, scales_off=4096, pool_bytes=65536)
    need = M.mx_workspace_bytes(d, 4)
    base = dict(T=4, a=h.p, ids=h.p + 8192, w=None, slots=h.p + 16384, pool=h.p + 65536, out=h.p + 32768, ws=h.p + 262144, n=need)

    def call(**over):
        c = {**base, **over}
        return L.mx_experts_forward(ctypes.byref(d), c["T"], c["a"], None, c["ids"], c["w"], c["slots"], c["pool"], c["out"],
                                    c["ws"], c["n"], None)
    assert call(T=-1) == -1 and call(T=65537) == -1 and call(n=need - 1) == -4
    for k in ("a", "ids", "slots", "pool", "out", "ws"):
        assert call(**{k: None}) == -1, k
    assert call(pool=h.p + 65536 + 128) == -1 and call(slots=h.p + 16388) == -1 and call(ids=h.p + 8194) == -1
    assert call(w=h.p + 8193) == -1
    assert call(out=h.p + 65536 + 512) == -1 and call(out=h.p + 8192) == -1 and call(ws=h.p + 65536) == -1
    assert call(T=0) == 0
    # launches of 2^32 threads: the sum over experts, the quantisation, pairs by few rows (A beyond 4 GiB)
    for n, k, a_dtype, top_k, T in ((1 << 16, 64, "bf16", 1, 1 << 16), (64, 1 << 19, "bf16", 1, 1 << 16),
                                    (1 << 17, 1 << 20, "mx", 1, 1 << 14)):
        big = M.mx_product_desc(n, k, a=a_dtype, n_experts=4, top_k=top_k, scales_off=1 << 38, pool_bytes=1 << 39)
        assert L.mx_workspace_bytes(ctypes.byref(big), T) == 0, (n, k)
        assert L.mx_workspace_bytes(ctypes.byref(big), T // 8) > 0, (n, k)
    with pytest.raises(M.MoeError):
        M.mx_experts(d, 4, torch.zeros(4, 64, dtype=torch.bfloat16), None, torch.zeros(4, 2, dtype=torch.int64), None, h.p, h.p,
                     h.p, torch.zeros(need, dtype=torch.uint8))
    with pytest.raises(M.MoeError):
        M.mx_experts(d, 4, h.p, None, h.p, None, h.p, torch.zeros(100, dtype=torch.uint8), h.p,
                     torch.zeros(need, dtype=torch.uint8))
