"""Norms, rotation and append on the GPU (attn_append through the C ABI) against the float64 oracle, within the bound derived in
attn_util; and a layer's steps in a row."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
from attn_util import DEV, HALF, TYPES, U, Batch, g, held, ints, put
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


class Append:
    def __init__(self, batch, R, style="half", norm=True, offset=1.0, seed=0, far=0, fused=True, eps=1e-6):
        b, rng = batch, np.random.default_rng(seed + 100)
        self.b, self.R, self.style, self.offset, self.eps = b, R, style, offset, eps
        size = rng.choice([0.01, 1.0, 30.0], size=(b.N, 1, 1))
        self.q, self.k, self.v = (held(size * rng.normal(size=(b.N, h, b.D)), b.dtype) for h in (b.nq, b.nkv, b.nkv))
        self.positions = rng.integers(0, 5000, size=b.N) + far
        self.inv_freq = (1e6 ** (-np.arange(R // 2) / max(R // 2, 1))).astype(np.float32)
        self.qw, self.kw = ((0.3 * rng.normal(size=b.D)).astype(np.float32) if norm else None for _ in range(2))
        self.fused = fused

    def call(self, pages, stream=None, with_q=True):
        b, dt = self.b, TYPES[self.b.dtype]
        if self.fused:      # parts of one product's rows, with room between them
            row = (b.nq + 2 * b.nkv) * b.D + 16
            qkv = torch.full((b.N, row), float("nan"), dtype=dt, device=DEV)
            parts, at = [], 0
            for x, h in ((self.q, b.nq), (self.k, b.nkv), (self.v, b.nkv)):
                parts.append(qkv[:, at:at + h * b.D].unflatten(1, (h, b.D)))
                parts[-1].copy_(put(x, b.dtype))
                at += h * b.D
            q, k, v = parts
        else:
            q, k, v = (put(x, b.dtype) for x in (self.q, self.k, self.v))
        f32 = lambda x: None if x is None else torch.from_numpy(x).to(DEV)
        out = torch.full((b.N, b.nq, b.D), 7.0, dtype=dt, device=DEV) if with_q else None
        d = b.desc(rotary_dim=self.R, rotary=self.style, norm_offset=self.offset, eps=self.eps)
        M.attn_append(d, b.B, b.N, ints(b.cu), ints(b.lens), ints(b.table), ints(self.positions) if self.R else None,
                      q if with_q else None, k, v, f32(self.qw), f32(self.kw), f32(self.inv_freq) if self.R else None, out, pages,
                      stream=stream)
        return out

    def turned(self, x, w):
        """(value, bound)"""
        b = self.b
        n = x if w is None else A.head_norm(x, w, self.eps, self.offset)
        mag = np.abs(n)
        e = (g(b.D / 2 + 11) if w is not None else 0.0) * np.ones_like(mag)
        y = n
        if self.R:
            y = A.rotate(n, self.positions, self.inv_freq, self.R, self.style)
            i, j = A.pair_indices(self.R, self.style)
            mag = mag.copy()
            mag[..., i] = mag[..., j] = np.abs(n[..., i]) + np.abs(n[..., j])
            e[..., :self.R] += 10 * U
        return y, e * mag + HALF[b.dtype] * np.abs(y)

    def check(self, with_q=True):
        b = self.b
        pages = put(b.pages, b.dtype)
        out = self.call(pages, with_q=with_q)
        got = pages.double().cpu().numpy()
        want, bound = b.pages.copy(), np.zeros_like(b.pages)
        k, kb = self.turned(self.k, self.kw)
        for s in range(b.B):
            n = b.news[s]
            for i in range(n):
                at = A.place_of(b.table[s], b.lens[s] - n + i, b.page, b.n_pages)
                if at is not None:
                    row = b.cu[s] + i
                    want[at[0], 0, :, at[1]], bound[at[0], 0, :, at[1]] = k[row], kb[row]
                    want[at[0], 1, :, at[1]] = self.v[row]
        assert np.all(np.abs(got - want) <= bound)
        if with_q:
            y, yb = self.turned(self.q, self.qw)
            o = out.double().cpu().numpy()
            inside = np.zeros(b.N, dtype=bool)
            inside[b.cu[0]:b.cu[-1]] = True
            assert np.all(o[~inside] == 7.0)
            assert np.all(np.abs(o - y)[inside] <= yb[inside])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 0), (64, 6), (128, 126), (128, 32), (256, 64), (256, 2)])
@pytest.mark.parametrize("style", ["half", "adjacent"])
@pytest.mark.parametrize("norm", [True, False])
def test_append(dtype, D, R, style, norm):
    print("append", dtype, D, R, style, norm, flush=True)
    b = Batch([1, 0, 5, 33], [40, 17, 5, 70], 6, 2, D, 16, dtype, seed=R, first=2, behind=3)
    Append(b, R, style, norm, seed=D, fused=norm).check()


@pytest.mark.parametrize("nq,nkv,page", [(1, 1, 1), (16, 2, 64), (3, 3, 1024), (64, 1, 8)])
def test_layouts(nq, nkv, page):
    print("layouts", nq, nkv, page, flush=True)
    for dtype in ("bf16", "f32"):
        Append(Batch([1, 2], [9, 77], nq, nkv, 64, page, dtype, seed=nq), 32).check()


def test_far_positions_keep_their_angles():
    print("far", flush=True)
    b = Batch([40], [40], 2, 1, 64, 16, "f32", seed=3)
    Append(b, 64, norm=False, far=(1 << 30)).check()


def test_many_sequences_and_keys_only():
    print("many", flush=True)
    rng = np.random.default_rng(1)
    news = rng.integers(0, 4, size=300).tolist()
    b = Batch(news, [n + int(rng.integers(0, 20)) for n in news], 2, 1, 64, 16, "bf16", seed=4)
    Append(b, 64).check()
    Append(b, 64).check(with_q=False)


def test_places_that_are_not_there():
    print("places", flush=True)
    b = Batch([5, 4, 3], [20, 4, 2], 2, 1, 64, 4, "f32", seed=6)
    b.table[0, 4], b.table[1, 0] = -1, b.n_pages          # nothing is appended there
    b.lens[2] = 1                                          # two of its three tokens have no number
    Append(b, 64).check()
    b.lens[0] = 400                                        # behind its table
    Append(b, 64).check()


def test_tiny_and_zero_heads():
    print("zero", flush=True)
    b = Batch([4], [4], 2, 1, 128, 16, "f32", seed=7)
    a = Append(b, 64, eps=1e-6)
    a.q[0] = 0
    a.k[1] = 1e-30
    a.check()


def test_stream_and_graph():
    print("graph", flush=True)
    b = Batch([3, 1], [40, 20], 4, 2, 128, 16, "bf16", seed=8)
    a = Append(b, 64, fused=False)
    pages = put(b.pages, "bf16")
    want = a.call(pages)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = put(b.pages, "bf16")
        out = a.call(again)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(pages, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_layer_step_by_step(dtype):
    """Append and attention as a program runs them: a prompt in two parts, then token by token, against everything at once."""
    print("layer", dtype, flush=True)
    T = 75
    whole = Batch([T], [T], 4, 2, 64, 16, dtype, seed=31)
    a = Append(whole, 32, fused=False, seed=5)
    a.positions = np.arange(T)
    pages = put(whole.pages, dtype)
    q = a.call(pages)
    d = whole.desc()
    ws = torch.empty(M.attn_workspace_bytes(d, 1, T, T, T), dtype=torch.uint8, device=DEV)
    full = torch.empty_like(q)
    M.attn_forward(d, 1, T, T, T, ints([0, T]), ints([T]), ints(whole.table), None, q, pages, full, ws)
    step_pages, at = put(whole.pages, dtype), 0
    for n in (40, 30, 1, 1, 1, 1, 1):
        part = Batch([n], [at + n], 4, 2, 64, 16, dtype, seed=31)
        part.table, part.cols, part.n_pages = whole.table, whole.cols, whole.n_pages
        s = Append(part, 32, fused=False, seed=5)
        s.q, s.k, s.v, s.qw, s.kw = a.q[at:at + n], a.k[at:at + n], a.v[at:at + n], a.qw, a.kw
        s.positions = np.arange(at, at + n)
        sq = s.call(step_pages)
        assert torch.equal(sq, q[at:at + n])
        out = torch.empty_like(sq)
        dd = part.desc()
        w = torch.empty(M.attn_workspace_bytes(dd, 1, n, n, at + n), dtype=torch.uint8, device=DEV)
        M.attn_forward(dd, 1, n, n, at + n, ints([0, n]), ints([at + n]), ints(whole.table), None, sq, step_pages, out, w)
        # both are within their bound of the exact result; here relative to the largest value
        far = (out.double() - full[at:at + n].double()).abs().max().item()
        assert far <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -16) * full.double().abs().max().item()
        at += n
    assert torch.equal(step_pages, pages)
