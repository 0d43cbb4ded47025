"""Helpers of the attention GPU tests: seeded batches over a paged cache, the calls, and bounds on their rounding.

u = 2^-24, g(n) = n u / (1 - n u).

Append.  A norm's factor r has a relative error of at most g(D / 2 + 8) (a sum of squares under a square root, a product,
a sum, a division); x r (offset + w) gains 3 u more.  An angle is formed in double precision and reduced to
half a turn before it becomes fp32 (2^-24 of half a turn: pi u), sincospi is within 4 u: cos and sin are off by at most 8 u.  The
rotated value a c - b s is then off by at most (g(D / 2 + 11) + 10 u) (|a| + |b|).  Half a step of the output's type on top.

Attention.  A score's product sum is off by at most 2 g(D + 4) scale sum |q k| (twice: the matrix unit's adder is not
specified as round-to-nearest), its scaling to base 2 and the difference to the maximum by 3 u of the score's size, the
exponential by 4 u: relative error of a weight at most d = 2 g(D + 4) S + 6 u S + 8 u with S the largest scale sum |q k| of the
row, numerator and denominator together 2 d.  For bf16 the weights enter the second product in bf16, a relative
error of at most 2^-9 each, in numerator and denominator 2^-8; sums over the n keys 2 g(n + 64) and as much for the
denominator.  Together (2 d + 2^-8 + 4 g(n + 64)) sum w |v| and half a step of the output's type."""

import numpy as np
import torch

import int4_quantized_expert_amd as M
from oracle import attn_oracle as A

DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def g(n):
    return n * U / (1 - n * U)


def held(x, dtype):
    """The values that x has once stored in dtype, as float64."""
    t = torch.from_numpy(np.ascontiguousarray(x)).float()
    return (t.to(torch.bfloat16) if dtype == "bf16" else t).double().numpy()


def put(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(TYPES[dtype]).to(DEV)


def ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x).tolist(), dtype=dtype, device=DEV)


class Batch:
    """Sequences with `news` new tokens each, `lens` long with them, over a shuffled cache full of other values."""

    def __init__(self, news, lens, nq, nkv, D, page, dtype, seed=0, first=0, behind=0, spare=2, spread=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.news, self.lens, self.nq, self.nkv, self.D, self.page, self.dtype = list(news), list(lens), nq, nkv, D, page, dtype
        self.B = len(self.news)
        self.cu = np.concatenate(([0], np.cumsum(self.news))) + first
        self.N = int(self.cu[-1]) + behind
        pages_of = [max(0, -(-t // page)) for t in self.lens]
        self.cols = max(1, max(pages_of))
        self.n_pages = sum(pages_of) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.zeros((self.B, self.cols), dtype=np.int64)
        at = 0
        for b, n in enumerate(pages_of):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.pages = held(rng.normal(size=(self.n_pages, 2, nkv, page, D)), dtype)
        self.q = held(spread * rng.normal(size=(self.N, nq, D)), dtype)
        self.tree = None
        self.scale = D ** -0.5

    def desc(self, **kw):
        return M.attn_desc(self.nq, self.nkv, self.D, self.page, self.n_pages, self.cols, dtype=self.dtype, scale=self.scale, **kw)

    def forward(self, new_max=None, len_max=None, ws=None, stream=None):
        """The call; rows of no sequence start as 7."""
        d = self.desc()
        new_max = max(self.news) if new_max is None else new_max
        len_max = max(0, max(self.lens)) if len_max is None else len_max
        if ws is None:
            ws = torch.full((M.attn_workspace_bytes(d, self.B, self.N, new_max, len_max),), 0xff, dtype=torch.uint8, device=DEV)
        out = torch.full((self.N, self.nq, self.D), 7.0, dtype=TYPES[self.dtype], device=DEV)
        tree = None if self.tree is None else torch.from_numpy(self.tree.view(np.int64)).to(DEV)
        M.attn_forward(d, self.B, self.N, new_max, len_max, ints(self.cu), ints(self.lens), ints(self.table), tree,
                       put(self.q, self.dtype), put(self.pages, self.dtype), out, ws, stream=stream)
        return out.double().cpu().numpy()

    def expected(self, new_max=None, len_max=None):
        new_max = max(self.news) if new_max is None else new_max
        len_max = max(0, max(self.lens)) if len_max is None else len_max
        return A.attend(self.q, self.pages, self.cu, self.lens, self.table, float(np.float32(self.scale)), new_max, len_max, self.tree)

    def check(self, new_max=None, len_max=None):
        got = self.forward(new_max, len_max)
        want, mag, spread = self.expected(new_max, len_max)
        assert_close(got, want, mag, spread, self.D, max(self.lens), self.dtype)
        return got


def assert_close(got, want, mag, spread, D, keys, dtype):
    outside = np.isnan(want) & (mag == 0)                       # rows of no sequence
    assert np.all(got[outside] == 7.0)
    d = 2 * g(D + 4) * spread + 6 * U * spread + 8 * U
    bound = (2 * d + (2.0 ** -8 if dtype == "bf16" else 0.0) + 4 * g(keys + 64))[..., None] * mag + HALF[dtype] * np.abs(want) + 1e-37
    ok = outside | (np.isnan(want) & np.isnan(got)) | (got == want)
    with np.errstate(invalid="ignore"):
        ok |= np.abs(got - want) <= bound
    assert np.all(ok), f"{np.sum(~ok)} of {ok.size} values, first at {np.argwhere(~ok)[0]}: {got[~ok][0]} for {want[~ok][0]}"


def random_tree(rng, n):
    """A mask for each of n drafted tokens: itself and the tokens that it follows."""
    mask = np.zeros(n, dtype=np.uint64)
    for i in range(n):
        parent = int(rng.integers(-1, i)) if i else -1
        mask[i] = np.uint64(1 << i) | (mask[parent] if parent >= 0 else np.uint64(0))
    return mask
