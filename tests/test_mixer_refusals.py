"""Checks of the chunked delta rule and of attention over a paged cache that need no GPU: exported symbols, sizes, refusals before
any device call, and the attention oracle against its own formulas."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
from oracle import attn_oracle as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Host:
    """Host memory standing in for device buffers: every call here is refused, or does nothing, before any device work."""

    def __init__(self, n=1 << 22):
        self.buf = ctypes.create_string_buffer(n + 512)
        self.p = ctypes.addressof(self.buf) // 256 * 256 + 256


def test_declared_symbols_are_exported():
    names = []
    for f in ("gdn_chunk.h", "attention.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", f)).read(), flags=re.S)
        names += re.findall(r"^[A-Za-z_][\w\s\*]*?\b((?:gdn|attn)_\w+)\s*\(", text, flags=re.M)
    assert len(set(names)) == 5
    for n in names:
        assert hasattr(M.lib(), n), n


MB = 1 << 16


def gdn_call(h, d=None, B=2, N=10, T=8, ws_n=None, **over):
    d = M.gdn_desc(1, 2, 64, 16, act="f32") if d is None else d
    need = M.lib().gdn_chunk_workspace_bytes(ctypes.byref(d), B, N) if ws_n is None else ws_n
    at = dict(cu=h.p, q=h.p + MB, k=h.p + 2 * MB, v=h.p + 3 * MB, alpha=h.p + 4 * MB, beta=h.p + 5 * MB, state_in=h.p + 6 * MB,
              state_out=h.p + 8 * MB, out=h.p + 10 * MB, ws=h.p + 16 * MB)
    at.update(over)
    return M.lib().gdn_chunk_forward(ctypes.byref(d), B, N, T, at["cu"], at["q"], at["k"], at["v"], at["alpha"], at["beta"],
                                     at["state_in"], at["state_out"], at["out"], at["ws"], need, None)


@pytest.mark.parametrize("field,value", [("n_k_heads", 0), ("n_v_heads", 3), ("n_v_heads", 2048), ("d_k", 96), ("d_v", 8), ("d_v", 272),
                                         ("act_dtype", 2), ("out_dtype", 5), ("scale", float("nan")), ("eps", -1.0)])
def test_gdn_bad_descriptor(field, value):
    d = M.gdn_desc(2, 4, 64, 16)
    setattr(d, field, value)
    assert gdn_call(Host(), d, ws_n=1 << 20) == -1 and M.last_error()
    assert M.lib().gdn_chunk_workspace_bytes(ctypes.byref(d), 1, 64) == ctypes.c_size_t(-1).value
    with pytest.raises(M.MoeError):
        M.gdn_chunk_workspace_bytes(d, 1, 64)


def test_gdn_refusals():
    h = Host()
    assert M.lib().gdn_chunk_forward(None, 1, 1, 1, *[h.p] * 10, 1 << 20, None) == -1
    assert gdn_call(h, B=-1) == -1 and gdn_call(h, B=(1 << 16) + 1) == -1 and gdn_call(h, N=-1) == -1 and gdn_call(h, T=-1) == -1
    assert gdn_call(h, N=(1 << 24) + 1) == -1
    for name in ("cu", "q", "k", "v", "alpha", "beta", "state_out", "out", "ws"):
        assert gdn_call(h, **{name: None}) == -1, name
    for name in ("q", "k", "v", "state_in", "state_out", "out", "ws"):
        assert gdn_call(h, **{name: h.p + 12 * MB + 8}) == -1, name
    for name in ("cu", "alpha", "beta"):
        assert gdn_call(h, **{name: h.p + 12 * MB + 2}) == -1, name
    for out in ("state_out", "out", "ws"):
        for name, at in (("cu", 0), ("q", 1), ("k", 2), ("v", 3), ("alpha", 4), ("beta", 5), ("state_in", 6)):
            if (out, name) != ("state_out", "state_in"):
                assert gdn_call(h, **{out: h.p + at * MB}) == -1, (out, name)
    assert gdn_call(h, state_out=h.p + 6 * MB + 256) == -1           # half over the incoming state
    assert gdn_call(h, out=h.p + 8 * MB) == -1 and gdn_call(h, ws=h.p + 8 * MB) == -1 and gdn_call(h, ws=h.p + 10 * MB) == -1
    assert gdn_call(h, ws_n=100) == -4
    assert gdn_call(h, B=0) == 0
    d = M.gdn_desc(1, 1024, 64, 256)
    assert gdn_call(h, d, B=1 << 16, N=0) == -1                      # more blocks than a launch takes


def test_gdn_workspace_is_bounded():
    d = M.gdn_desc(16, 32, 128, 128)
    assert M.gdn_chunk_workspace_bytes(d, 0, 10) == 0 and M.gdn_chunk_workspace_bytes(d, 3, 0) == 0
    assert 0 < M.gdn_chunk_workspace_bytes(d, 1, 64) < M.gdn_chunk_workspace_bytes(d, 1, 4096)
    assert M.gdn_chunk_workspace_bytes(d, 1, 1 << 24) <= 512 << 20


def test_gdn_binding_refusals():
    d = M.gdn_desc(1, 2, 64, 16, act="f32")
    f = torch.zeros
    ok = dict(cu=f(2, dtype=torch.int32), q=f(4, 1, 64), k=f(4, 1, 64), v=f(4, 2, 16), alpha=f(4, 2), beta=f(4, 2), state_in=None,
              state_out=f(1, 2, 16, 64), out=f(4, 2, 16), ws=f(8, dtype=torch.uint8))
    for name, bad in (("cu", f(2, dtype=torch.int64)), ("cu", f(1, dtype=torch.int32)), ("q", f(3, 1, 64)), ("k", f(4, 1, 64).bfloat16()),
                      ("v", f(2, 4, 16).transpose(0, 1)), ("alpha", f(4, 2).double()), ("state_out", f(1, 2, 16, 32)), ("out", f(4, 2, 8)),
                      ("ws", None), ("ws", 4096)):
        with pytest.raises(M.MoeError):
            M.gdn_chunk_forward(d, 1, 4, 4, **{**ok, name: bad})
    with pytest.raises(M.MoeError, match="not on a GPU"):
        M.gdn_chunk_forward(d, 1, 4, 4, **ok)


def attn(**kw):
    d = M.attn_desc(4, 2, 64, 16, 8, 4, dtype="f32", rotary_dim=32)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD = [("n_q_heads", 0), ("n_q_heads", 5), ("n_q_heads", 512), ("n_kv_heads", 0), ("head_dim", 96), ("dtype", 2), ("page_size", 0),
       ("page_size", 24), ("page_size", 2048), ("max_pages", 0), ("max_pages", (1 << 24) + 1), ("rotary_dim", 65), ("rotary_dim", 31),
       ("rotary_dim", -2), ("rotary_pairs", 2), ("n_pages", 0), ("n_pages", 1 << 31), ("scale", float("inf")), ("eps", -1e-6),
       ("eps", float("nan")), ("norm_offset", float("nan"))]


def append_call(h, d=None, B=2, N=10, **over):
    d = attn() if d is None else d
    at = dict(cu=h.p, lens=h.p + 1024, table=h.p + 2048, positions=h.p + 4096, q=h.p + MB, qs=256, k=h.p + 2 * MB, ks=128,
              v=h.p + 3 * MB, vs=128, q_norm=h.p + 8192, k_norm=h.p + 9216, inv_freq=h.p + 10240, q_out=h.p + 4 * MB, pages=h.p + 8 * MB)
    at.update(over)
    return M.lib().attn_append(ctypes.byref(d), B, N, *at.values(), None)


def forward_call(h, d=None, B=2, N=10, new=6, length=60, ws_n=None, **over):
    d = attn() if d is None else d
    at = dict(cu=h.p, lens=h.p + 1024, table=h.p + 2048, tree=h.p + 4096, q=h.p + MB, pages=h.p + 8 * MB, out=h.p + 4 * MB,
              ws=h.p + 24 * MB)
    at.update(over)
    need = M.lib().attn_workspace_bytes(ctypes.byref(d), B, N, new, length) if ws_n is None else ws_n
    return M.lib().attn_forward(ctypes.byref(d), B, N, new, length, *at.values(), need, None)


@pytest.mark.parametrize("field,value", BAD)
def test_attn_bad_descriptor(field, value):
    h, d = Host(), attn(**{field: value})
    assert append_call(h, d) == -1 and M.last_error()
    assert forward_call(h, d, ws_n=1 << 20) == -1
    with pytest.raises(M.MoeError):
        M.attn_workspace_bytes(d, 1, 1, 1, 1)


def test_append_refusals():
    h = Host()
    assert M.lib().attn_append(None, 1, 1, *[h.p] * 4, h.p, 256, h.p, 128, h.p, 128, *[h.p] * 5, None) == -1
    assert append_call(h, B=-1) == -1 and append_call(h, B=(1 << 16) + 1) == -1 and append_call(h, N=-1) == -1
    assert append_call(h, N=(1 << 20) + 1) == -1
    for name in ("cu", "lens", "table", "positions", "q", "k", "v", "inv_freq", "q_out", "pages"):
        assert append_call(h, **{name: None}) == -1, name
    for name in ("q", "k", "v", "q_out", "pages"):
        assert append_call(h, **{name: h.p + 40 * MB + 8}) == -1, name
    for name in ("cu", "lens", "table", "positions", "q_norm", "k_norm", "inv_freq"):
        assert append_call(h, **{name: h.p + 40 * MB + 2}) == -1, name
    assert append_call(h, qs=255) == -1 and append_call(h, ks=127) == -1 and append_call(h, vs=64) == -1 and append_call(h, qs=258) == -1
    for out in ("q_out", "pages"):
        for at in (0, 1024, 2048, 4096, 8192, 9216, 10240, MB, 2 * MB, 3 * MB):
            assert append_call(h, **{out: h.p + at}) == -1, (out, at)
    assert append_call(h, q_out=h.p + 8 * MB) == -1
    assert append_call(h, B=0) == 0 and append_call(h, N=0) == 0


def test_forward_refusals():
    h = Host()
    assert M.lib().attn_forward(None, 1, 1, 1, 1, *[h.p] * 8, 1 << 20, None) == -1
    assert forward_call(h, B=-1) == -1 and forward_call(h, N=(1 << 20) + 1) == -1 and forward_call(h, new=-1) == -1
    assert forward_call(h, length=-1) == -1 and forward_call(h, length=0x7fffffff) == -1
    assert forward_call(h, N=200, new=65) == -1                       # a tree of more than 64 tokens
    for name in ("cu", "lens", "table", "q", "pages", "out"):
        assert forward_call(h, **{name: None}) == -1, name
    for name in ("q", "pages", "out"):
        assert forward_call(h, **{name: h.p + 40 * MB + 8}) == -1, name
    for name in ("cu", "lens", "table", "tree"):
        assert forward_call(h, **{name: h.p + 40 * MB + 2}) == -1, name
    for at in (0, 1024, 2048, 4096, MB, 8 * MB):
        assert forward_call(h, out=h.p + at) == -1, at
    long = dict(new=1, length=4000)
    d = attn()
    assert M.attn_workspace_bytes(d, 2, 10, 1, 4000) > 0
    assert forward_call(h, **long, ws=None) == -1 and forward_call(h, **long, ws=h.p + 40 * MB + 16) == -1
    assert forward_call(h, **long, ws_n=16) == -4 and forward_call(h, **long, ws=h.p + 4 * MB) == -1 and forward_call(h, **long, ws=h.p + MB) == -1
    assert forward_call(h, B=0) == 0 and forward_call(h, N=0) == 0 and forward_call(h, new=0) == 0
    many = M.attn_desc(256, 256, 64, 16, 8, 4)
    assert forward_call(h, many, B=1 << 16, N=1 << 20, new=1 << 20, ws_n=1 << 20) == -1     # more blocks than a launch takes


def test_attn_binding_refusals():
    d = M.attn_desc(4, 2, 64, 16, 3, 2, dtype="f32", rotary_dim=32)
    f, i32 = torch.zeros, torch.int32
    batch = dict(cu=f(2, dtype=i32), lens=f(1, dtype=i32), table=f(1, 2, dtype=i32))
    ap = dict(batch, positions=f(5, dtype=i32), q=f(5, 4, 64), k=f(5, 2, 64), v=f(5, 2, 64), q_norm=None, k_norm=None, inv_freq=f(16),
              q_out=f(5, 4, 64), pages=f(3, 2, 2, 16, 64))
    for name, bad in (("cu", f(1, dtype=i32)), ("lens", f(1)), ("table", f(1, dtype=i32)), ("q", f(5, 3, 64)), ("q", f(4, 4, 64)),
                      ("k", f(5, 64, 2).transpose(1, 2)), ("v", f(5, 2, 64).bfloat16()), ("inv_freq", f(8)), ("q_out", f(5, 4, 32)),
                      ("pages", f(2, 2, 2, 16, 64)), ("positions", f(5, dtype=torch.int64)), ("k_norm", f(32))):
        with pytest.raises(M.MoeError):
            M.attn_append(d, 1, 5, **{**ap, name: bad})
    with pytest.raises(M.MoeError, match="not on a GPU"):
        M.attn_append(d, 1, 5, **ap)
    fw = dict(batch, tree=None, q=f(5, 4, 64), pages=f(3, 2, 2, 16, 64), out=f(5, 4, 64))
    for name, bad in (("tree", f(5, dtype=i32)), ("tree", f(4, dtype=torch.int64)), ("q", f(4, 4, 64)), ("out", f(5, 4, 64).double()),
                      ("pages", f(2, 2, 2, 16, 64))):
        with pytest.raises(M.MoeError):
            M.attn_forward(d, 1, 5, 5, 20, **{**fw, name: bad})
    with pytest.raises(M.MoeError, match="not on a GPU"):
        M.attn_forward(d, 1, 5, 5, 20, **fw)
    with pytest.raises(KeyError):
        M.attn_desc(4, 2, 64, 16, 3, 2, dtype="f16")


def test_oracle_rotation_and_norm():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 2, 8))
    for style in ("half", "adjacent"):
        y = A.rotate(x, [0, 1, 7], [1.0, 0.1], 4, style)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 4:], x[..., 4:])
        a, b = A.pair_indices(4, style)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * np.array([0, 1, 7])[:, None, None] * np.array([1.0, 0.1]))
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
    n = A.head_norm(x, np.zeros(8), 0.0, 1.0)
    assert np.allclose(np.mean(n * n, axis=-1), 1)


def test_oracle_attention_by_hand():
    """Two tokens cached, one new: weights 1/2, 1/4, 1/4; a tree bit that is not set takes the new token out."""
    pages = np.zeros((2, 2, 1, 2, 2))
    pages[1, 0, 0, 0, 0] = np.log(2)
    pages[1, 1, 0, 0], pages[1, 1, 0, 1], pages[0, 1, 0, 0] = [1, 0], [0, 1], [4, 4]
    q = np.array([[[1.0, 0.0]]])
    out, mag, _ = A.attend(q, pages, [0, 1], [3], [[1, 0]], 1.0, 1, 3)
    assert np.allclose(out[0, 0], [1.5, 1.25]) and np.allclose(mag, out)
    out, _, _ = A.attend(q, pages, [0, 1], [3], [[1, 0]], 1.0, 1, 3, tree=[0])
    assert np.allclose(out[0, 0], [2 / 3, 1 / 3])
    out, _, _ = A.attend(q, pages, [0, 1], [1], [[1, 0]], 1.0, 1, 3, tree=[0])
    assert np.all(out == 0)
