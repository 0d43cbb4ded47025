"""Products of microscaled 4-bit matrices on the GPU, dense and by routed expert, against the float64 oracle within the
bounds that mx_util derives, and a whole routed layer run as a program runs it."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
import synth
from gpu_util import check_close, make_layer, oracle_shape, upload
from mx_util import DEV, TYPES, close, expected, g, held, matrix, rows, to_gpu, workspace
from oracle import moe_oracle as O
from oracle import mx_oracle as X
from oracle import route_oracle as R

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def a_side(rng, n, k, dtype):
    """(held values, tensor, scales tensor or None) of the left operand."""
    if dtype == "mx":
        c, s, v = matrix(rng, n, k)
        return v, dev(c), dev(s)
    x = rows(rng, n, k, dtype)
    return held(x)[0], to_gpu(x, dtype), None


def linear(Mr, N, K, a="bf16", out="f32", act="none", seed=0):
    rng = np.random.default_rng(seed + Mr + 7 * N + 13 * K)
    av, at, a_s = a_side(rng, Mr, K, a)
    wc, ws, wv = matrix(rng, N * (2 if act == "swiglu" else 1), K)
    d = M.mx_product_desc(N, K, a=a, out=out, act=act)
    o = torch.full((Mr + 1, N), float("nan"), dtype=TYPES[out], device=DEV)
    o[Mr] = 9.0
    M.mx_linear(d, Mr, at, a_s, dev(wc), dev(ws), o[:Mr], workspace(d, Mr))
    torch.cuda.synchronize()
    assert (o[Mr] == 9.0).all()
    y, bound = expected(av, wv, act, K)
    close(o[:Mr], y, bound, out, f"M={Mr} N={N} K={K} {a} {out} {act}")
    return o[:Mr]


SHAPES = [(1, 1, 1), (1, 16, 256), (2, 17, 31), (3, 100, 300), (15, 33, 257), (16, 128, 512), (17, 130, 1000), (33, 64, 2048),
          (64, 96, 700), (100, 200, 90), (129, 257, 513), (300, 520, 260)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("a", ["f32", "bf16", "mx"])
def test_linear_shapes(shape, a):
    linear(*shape, a=a, out="f32")


@pytest.mark.parametrize("shape", [(1, 20, 300), (5, 64, 256), (16, 48, 1111), (40, 70, 100), (200, 140, 600)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_act_and_output(shape, act, out):
    for a in ("f32", "bf16", "mx"):
        linear(*shape, a=a, out=out, act=act, seed=3)


@pytest.mark.parametrize("Mr", [1, 2, 16, 17, 48, 64, 65, 128, 255, 256, 257, 700])
def test_linear_row_counts(Mr):
    """Every side of the rules that choose a kernel by the number of rows."""
    linear(Mr, 320, 768, a="bf16", out="bf16", seed=5)
    linear(Mr, 80, 300, a="bf16", out="f32", act="swiglu", seed=6)


@pytest.mark.parametrize("Mr,N,K", [(16, 40, 2000), (16, 40, 4200), (3, 33, 9000), (17, 50, 500), (32, 33, 1000), (32, 33, 2100),
                                    (25, 20, 4500), (16, 16500, 700), (32, 6600, 1000)])
@pytest.mark.parametrize("a", ["f32", "bf16", "mx"])
def test_linear_few_rows_quantised_in_the_product_or_before(Mr, N, K, a):
    linear(Mr, N, K, a=a)
    linear(Mr, N // 3, K, a=a, out="bf16", act="swiglu")


@pytest.mark.parametrize("N", [129, 130, 131, 132, 515])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_rows_of_any_alignment(N, out):
    """Four outputs a store wherever a row starts, and the columns past the last four."""
    linear(150, N, 300, out=out)
    linear(150, N, 300, out=out, act="swiglu")


def test_linear_long_and_wide():
    linear(3, 40, 20000, seed=7)
    linear(70, 24, 9000, seed=8, act="swiglu")
    linear(2, 5000, 256, seed=9)
    linear(600, 1100, 512, seed=10, out="bf16")
    linear(100, 150, 5000, seed=11, act="swiglu", out="bf16")      # two groups of chunks, the last pair half empty
    linear(150, 300, 4100, seed=12)
    linear(65, 130, 4096 + 256, seed=13, a="mx")
    linear(3500, 3600, 300, seed=14, out="bf16")                   # the largest tiles, ragged in every direction
    linear(2000, 1000, 700, seed=15, act="swiglu")
    linear(3500, 1800, 260, seed=16, act="swiglu", out="bf16")


def test_linear_nan_blocks_stay_in_their_rows():
    rng = np.random.default_rng(1)
    x = rows(rng, 40, 300)
    x[7, 280] = np.nan
    x[33, 3] = np.inf
    wc, ws, _ = matrix(rng, 50, 300)
    d = M.mx_product_desc(50, 300, a="f32", out="f32")
    for m in (10, 40):
        o = torch.zeros(m, 50, device=DEV)
        M.mx_linear(d, m, to_gpu(x[:m], "f32"), None, dev(wc), dev(ws), o, workspace(d, m))
        torch.cuda.synchronize()
        bad = torch.isnan(o).any(1).nonzero().flatten().tolist()
        assert bad == [i for i in (7, 33) if i < m] and torch.isnan(o[bad]).all()


def test_linear_rows_that_start_anywhere():
    """Unaligned operands and outputs: bf16 rows of odd length at an odd place."""
    rng = np.random.default_rng(2)
    for m in (5, 90):
        x = rows(rng, m, 301, "bf16")
        buf = torch.zeros(m * 301 + 3, dtype=torch.bfloat16, device=DEV)
        buf[3:] = to_gpu(x, "bf16").flatten()
        wc, ws, wv = matrix(rng, 37, 301)
        d = M.mx_product_desc(37, 301, a="bf16", out="bf16")
        out = torch.zeros(m * 37 + 1, dtype=torch.bfloat16, device=DEV)
        M.mx_linear(d, m, buf[3:], None, dev(wc), dev(ws), out[1:], workspace(d, m))
        torch.cuda.synchronize()
        assert out[0] == 0
        y, bound = expected(held(x)[0], wv, "none", 301)
        close(out[1:].view(m, 37), y, bound, "bf16")


class Experts:
    """Experts' blobs in a pool, in shuffled slots, behind a gap."""

    def __init__(self, rng, E, N, K, act="none", gap=0):
        self.E, self.N, self.K, self.act = E, N, K, act
        n = N * (2 if act == "swiglu" else 1)
        kp = X.padded(K)
        nc, ns = n * kp // 2, n * kp // 32
        self.scales_off = -(-nc // 16) * 16 + gap
        stride = -(-(self.scales_off + ns) // 256) * 256
        order = rng.permutation(E)
        pool = rng.integers(0, 256, size=(E + 1) * stride, dtype=np.uint8)
        self.values = []
        slots = np.zeros(E, dtype=np.int64)
        for e in range(E):
            c, s, v = matrix(rng, n, K)
            at = stride * (order[e] + 1)
            pool[at:at + nc] = c.reshape(-1)
            pool[at + self.scales_off:at + self.scales_off + ns] = s.reshape(-1)
            slots[e] = at
            self.values.append(v)
        self.pool, self.slots = dev(pool), dev(slots)

    def desc(self, k, a="bf16", out="f32", pair_rows=False):
        return M.mx_product_desc(self.N, self.K, a=a, out=out, act=self.act, n_experts=self.E, top_k=k, pair_rows=pair_rows,
                                 codes_off=0, scales_off=self.scales_off, pool_bytes=self.pool.numel())

    def expect(self, av, ids, pair_rows, lost=()):
        T, k = ids.shape
        y, b = np.zeros((T, k, self.N)), np.zeros((T, k, self.N))
        for e in np.unique(ids):
            if e < 0 or e >= self.E or e in lost:
                continue
            t, i = np.nonzero(ids == e)
            y[t, i], b[t, i] = expected(av[t * k + i] if pair_rows else av[t], self.values[e], self.act, self.K)
        return y, b

    def expect_sum(self, av, ids, w, pair_rows, lost=()):
        """The weighted sums and their bound: the products' own, and the sum's additions over the terms' magnitudes."""
        T, k = ids.shape
        y, b = self.expect(av, ids, pair_rows, lost)
        mag = np.zeros_like(y)
        for e in np.unique(ids):
            if 0 <= e < self.E and e not in lost:
                t, i = np.nonzero(ids == e)
                r = av[t * k + i] if pair_rows else av[t]
                mag[t, i] = np.abs(y[t, i]) if self.act == "swiglu" else np.abs(r) @ np.abs(self.values[e]).T
        return (w[..., None] * y).sum(1), (w[..., None] * b).sum(1) + 2 * g(k + 32) * (w[..., None] * mag).sum(1)


def routing(rng, T, E, k, hot=0.0):
    ids = np.stack([rng.choice(E, size=k, replace=False) for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < hot] = E // 2          # an expert twice in a token, and a full one
    w = rng.random((T, k)).astype(np.float32).astype(np.float64)
    return ids, w


def run_experts(x: Experts, T, k, a="bf16", out="f32", pair_rows=False, combine=False, seed=0, ids=None, hot=0.0, lost=()):
    rng = np.random.default_rng(seed + T * 31 + k)
    made, w = routing(rng, T, x.E, k, hot)
    ids = made if ids is None else ids
    av, at, a_s = a_side(rng, T * k if pair_rows else T, x.K, a)
    d = x.desc(k, a, out, pair_rows)
    n_out = T if combine else T * k
    o = torch.full((n_out + 1, x.N), float("nan"), dtype=TYPES[out], device=DEV)
    o[n_out] = 9.0
    ws = workspace(d, T)
    M.mx_experts(d, T, at, a_s, dev(ids), dev(w.astype(np.float32)) if combine else None, x.slots, x.pool, o[:n_out], ws)
    torch.cuda.synchronize()
    assert (o[n_out] == 9.0).all()
    if combine:
        y, b = x.expect_sum(av, ids, w, pair_rows, lost)
    else:
        y, b = (v.reshape(T * k, -1) for v in x.expect(av, ids, pair_rows, lost))
    close(o[:n_out], y, b, out, f"T={T} k={k} {a} {out} pair_rows={pair_rows} combine={combine}")
    return ws, o[:n_out]


@pytest.mark.parametrize("T,k", [(1, 1), (1, 10), (2, 4), (8, 4), (8, 8), (8, 10), (9, 3), (11, 3), (13, 10), (27, 3), (33, 4), (64, 10), (200, 6)])
@pytest.mark.parametrize("pair_rows", [False, True])
def test_experts_shapes(T, k, pair_rows):
    x = Experts(np.random.default_rng(1), 12, 70, 300)
    for combine in (False, True):
        run_experts(x, T, k, "bf16", "f32", pair_rows, combine)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("a", ["f32", "bf16", "mx"])
def test_experts_types(act, a):
    x = Experts(np.random.default_rng(2), 9, 48, 520, act, gap=48)
    for T in (3, 50, 120):
        for out in ("f32", "bf16"):
            run_experts(x, T, 5, a, out, False, False, seed=4)
            run_experts(x, T, 5, a, out, True, True, seed=5)


@pytest.mark.parametrize("a", ["f32", "bf16", "mx"])
@pytest.mark.parametrize("T,k,N,K,act,combine", [
    (1, 8, 40, 500, "none", True), (1, 8, 40, 1100, "none", True), (9, 8, 40, 600, "none", True),      # sums in one block
    (2, 8, 40, 2000, "none", False), (2, 8, 40, 8300, "none", False), (8, 4, 1500, 300, "swiglu", False),
    (16, 4, 50, 300, "none", False), (16, 4, 50, 300, "swiglu", True), (13, 5, 50, 300, "none", False), # 64 and 65 pairs
    (128, 8, 40, 300, "none", True), (205, 5, 40, 300, "none", True),                                    # 1024 and 1025
    (16, 2, 4096, 1024, "none", False), (16, 2, 4096, 1024, "none", True)])                              # much of W: tiles
def test_experts_few_pairs_on_every_path(T, k, N, K, act, combine, a):
    x = Experts(np.random.default_rng(17), 9, N, K, act)
    run_experts(x, T, k, a=a, combine=combine)
    if combine:
        run_experts(x, T, k, a=a, combine=True, pair_rows=True)


@pytest.mark.parametrize("T", [4, 16, 60, 300])
def test_experts_hot_and_repeated(T):
    """Half of all pairs go to one expert, some tokens name it twice or more."""
    x = Experts(np.random.default_rng(3), 16, 40, 256)
    for combine in (False, True):
        run_experts(x, T, 7, hot=0.5, combine=combine)
    one = Experts(np.random.default_rng(4), 1, 40, 256)
    run_experts(one, T, 1)


def test_experts_many():
    x = Experts(np.random.default_rng(5), 1024, 16, 32)
    run_experts(x, 300, 8)
    run_experts(x, 1, 64, combine=True, pair_rows=True)


@pytest.mark.parametrize("T,k", [(900, 7), (2500, 9), (3100, 9)])
def test_experts_more_pairs_than_a_grouping_step_holds(T, k):
    """Every way of grouping: 4096 pairs a step in registers, two, six, and more pairs than those; some ids unusable."""
    x = Experts(np.random.default_rng(14), 40, 20, 40)
    ids, _ = routing(np.random.default_rng(T), T, 40, k)
    ids[::17, 0] = -1
    ids[5, :] = 40
    ws, _ = run_experts(x, T, k, ids=ids)
    with pytest.raises(M.MoeError):
        M.status_check(ws)
    run_experts(x, T, k, combine=True, pair_rows=True)


def test_rows_of_a_beyond_four_gib():
    """65536 rows of 131072 codes: whole numbers, so that every order of summing gives the same bits."""
    K, rows_, N = 131072, 65536, 16
    gen = torch.Generator(device=DEV).manual_seed(1)
    pick = torch.tensor([0x22, 0xA2, 0x2A, 0xAA], dtype=torch.uint8, device=DEV)      # pairs of +-1
    codes = torch.empty(rows_, K // 2, dtype=torch.uint8, device=DEV)
    for i in range(0, rows_, 4096):
        codes[i:i + 4096] = pick[torch.randint(0, 4, (4096, K // 2), generator=gen, device=DEV, dtype=torch.int32)]
    scales = torch.full((rows_, K // 32), 127, dtype=torch.uint8, device=DEV)
    w = pick[torch.randint(0, 4, (N, K // 2), generator=gen, device=DEV, dtype=torch.int32)]
    ws_ = scales[:N].contiguous()

    def signs(c):
        return torch.stack((1 - 2 * ((c >> 3) & 1).double(), 1 - 2 * (c >> 7).double()), -1).flatten(1)
    at = [0, 1, 40000, 65534, 65535]
    want = (signs(codes[at]) @ signs(w).T).float()
    d = M.mx_product_desc(N, K, a="mx", out="f32")
    out = torch.empty(rows_, N, device=DEV)
    M.mx_linear(d, rows_, codes, scales, w, ws_, out, workspace(d, rows_))
    assert torch.equal(out[at], want)
    nc = N * K // 2
    pool = torch.cat((w.flatten(), ws_.flatten()))
    d = M.mx_product_desc(N, K, a="mx", out="f32", n_experts=1, top_k=1, pair_rows=True, scales_off=nc, pool_bytes=pool.numel())
    out.zero_()
    M.mx_experts(d, rows_, codes, scales, torch.zeros(rows_, 1, dtype=torch.int32, device=DEV), None,
                 torch.zeros(1, dtype=torch.int64, device=DEV), pool, out, workspace(d, rows_))
    assert torch.equal(out[at], want)


@pytest.mark.parametrize("T", [2, 5, 40, 90])
@pytest.mark.parametrize("combine", [False, True])
def test_experts_unusable_ids_and_slots(T, combine):
    """Ids outside the table and slots outside the pool: zero rows, MOE_ERANGE, everything else as it is."""
    rng = np.random.default_rng(6)
    x = Experts(rng, 8, 40, 300)
    ids, _ = routing(rng, T, 8, 4)
    ids[0, 0], ids[1, 1], ids[T - 1, 3] = -1, 8, 2 ** 30
    x.slots[3] = x.pool.numel() - 256
    x.slots[5] = 128
    ws, _ = run_experts(x, T, 4, combine=combine, ids=ids, lost=(3, 5))
    with pytest.raises(M.MoeError) as err:
        M.status_check(ws)
    assert err.value.code == -5
    M.status_check(ws)                                  # cleared
    ws, _ = run_experts(x, T, 4, combine=combine, ids=np.full((T, 4), 2, dtype=np.int32), lost=(3, 5))
    M.status_check(ws)
    run_experts(x, T, 4, combine=combine, ids=np.full((T, 4), -3, dtype=np.int32), lost=(3, 5))


@pytest.mark.parametrize("T", [2, 30, 60])
@pytest.mark.parametrize("combine", [False, True])
def test_an_unusable_pair_is_zero_whatever_its_row_holds(T, combine):
    """A NaN in the input row of a pair without an expert reaches no output."""
    rng = np.random.default_rng(15)
    x = Experts(rng, 6, 40, 300)
    ids, w = routing(rng, T, 6, 3)
    ids[1, 2] = 6
    av, at, _ = a_side(rng, T * 3, 300, "bf16")
    at[1 * 3 + 2, 7] = float("nan")
    d = x.desc(3, pair_rows=True)
    o = torch.full((T if combine else T * 3, 40), float("nan"), device=DEV)
    M.mx_experts(d, T, at, None, dev(ids), dev(w.astype(np.float32)) if combine else None, x.slots, x.pool, o, workspace(d, T))
    torch.cuda.synchronize()
    assert torch.isfinite(o).all()
    if combine:
        close(o, *x.expect_sum(av, ids, w, True), "f32")
    else:
        close(o, *(v.reshape(-1, 40) for v in x.expect(av, ids, True)), "f32")
        assert not o[1 * 3 + 2].any()


@pytest.mark.parametrize("T", [2, 8, 30, 60])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("weight", [float("nan"), float("inf"), -2.0])
def test_the_weight_of_an_unusable_pair_may_be_anything(T, act, weight):
    """A padded batch: the last token has ids of no expert, and one pair of another token is lost; their weights are
    not numbers.  The padded token's sum is zero, everything else as without them.  More experts than a step of the sum."""
    rng = np.random.default_rng(16)
    x = Experts(rng, 16, 40, 300, act=act)
    ids, w = routing(rng, T, 16, 10)
    ids[T - 1], ids[0, 9] = -1, 16
    given = w.astype(np.float32)
    given[T - 1], given[0, 9] = weight, weight
    av, at, _ = a_side(rng, T, 300, "bf16")
    o = torch.full((T, 40), float("nan"), device=DEV)
    d = x.desc(10)
    M.mx_experts(d, T, at, None, dev(ids), dev(given), x.slots, x.pool, o, workspace(d, T))
    torch.cuda.synchronize()
    assert not o[T - 1].any()
    close(o, *x.expect_sum(av, ids, w, False), "f32")


def test_experts_no_tokens():
    x = Experts(np.random.default_rng(7), 4, 16, 32)
    d = x.desc(2)
    o = torch.full((1, 16), 3.0, device=DEV)
    M.mx_experts(d, 0, torch.zeros(0, 32, dtype=torch.bfloat16, device=DEV), None, torch.zeros(0, 2, dtype=torch.int32, device=DEV),
                 None, x.slots, x.pool, o, workspace(d, 1))
    M.mx_linear(M.mx_product_desc(16, 32), 0, torch.zeros(0, 32, dtype=torch.bfloat16, device=DEV), None,
                torch.zeros(16, 128, dtype=torch.uint8, device=DEV), torch.zeros(16, 8, dtype=torch.uint8, device=DEV),
                o.to(torch.bfloat16), workspace(d, 1))
    torch.cuda.synchronize()
    assert (o == 3.0).all()


def test_blobs_beyond_four_gib():
    """A slot offset above 2^32 bytes."""
    rng = np.random.default_rng(8)
    x = Experts(rng, 4, 32, 256)
    n = x.pool.numel()
    far = torch.empty((1 << 32) + 4096 + n, dtype=torch.uint8, device=DEV)
    far[(1 << 32) + 4096:] = x.pool
    x.pool = far
    x.slots += (1 << 32) + 4096
    for T in (2, 80):
        run_experts(x, T, 3)
        run_experts(x, T, 3, combine=True)


def test_one_workspace_serves_calls_of_every_kind():
    """Products of several shapes and the layer of moe_layer.h take turns on one workspace; each gives what it gives on
    a workspace of its own."""
    geo = synth.PRESETS["tiny"]
    data = make_layer(geo, 3, 0, 4)
    dl = upload(data)
    rng = np.random.default_rng(9)
    x = Experts(rng, 6, 40, 300)
    ids, w = routing(rng, 70, 6, 3)
    a = to_gpu(rows(rng, 70, 300, "bf16"), "bf16")
    d = x.desc(3)
    n = max(M.mx_workspace_bytes(d, 70), M.workspace_bytes(dl.desc, 4))
    shared = torch.zeros(n, dtype=torch.uint8, device=DEV)
    M.workspace_init(shared)

    def layer(ws):
        out = torch.empty(4, geo.hidden, device=DEV)
        M.layer_forward(dl.desc, 4, dl.x, dl.R, dl.slots, dl.pool, dl.shared, out, ws)
        return out

    def experts(ws, T, combine):
        out = torch.empty(T if combine else T * 3, 40, device=DEV)
        M.mx_experts(d, T, a, None, dev(ids), dev(w.astype(np.float32)) if combine else None, x.slots, x.pool, out, ws)
        return out
    own = torch.zeros(n, dtype=torch.uint8, device=DEV)
    M.workspace_init(own)
    want = [layer(own)]
    for T, c in ((70, True), (2, False), (70, False)):
        want.append(experts(workspace(d, 70), T, c))
    for _ in range(3):
        got = [layer(shared), experts(shared, 70, True), experts(shared, 2, False), experts(shared, 70, False)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    M.status_check(shared)


@pytest.mark.parametrize("T", [1, 6, 90])
def test_captured_and_replayed(T):
    """A graph of routing and both products, replayed with new inputs between eager calls of the same program."""
    rng = np.random.default_rng(10)
    up, down = Experts(rng, 16, 64, 128, "swiglu"), Experts(rng, 16, 128, 64)
    r = M.route_desc(16, 4, "sigmoid", 4, 2, 2)
    du, dd = up.desc(4, "bf16", "bf16"), down.desc(4, "bf16", "bf16", pair_rows=True)
    x = torch.randn(T, 128, device=DEV).to(torch.bfloat16)
    logits = torch.randn(T, 16, device=DEV)
    bias = torch.randn(16, device=DEV) * 0.1

    def program(b):
        M.route(r, T, logits, bias, b["ids"], b["w"])
        M.mx_experts(du, T, x, None, b["ids"], None, up.slots, up.pool, b["h"], b["ws"])
        M.mx_experts(dd, T, b["h"], None, b["ids"], b["w"], down.slots, down.pool, b["y"], b["ws"])

    def bufs():
        n = max(M.mx_workspace_bytes(du, T), M.mx_workspace_bytes(dd, T))
        return dict(ids=torch.zeros(T, 4, dtype=torch.int32, device=DEV), w=torch.zeros(T, 4, device=DEV),
                    h=torch.zeros(T * 4, 64, dtype=torch.bfloat16, device=DEV), y=torch.zeros(T, 128, dtype=torch.bfloat16, device=DEV),
                    ws=torch.zeros(n, dtype=torch.uint8, device=DEV))
    a, b = bufs(), bufs()
    program(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        program(a)
    for i in range(4):
        x.copy_(torch.randn(T, 128, device=DEV))
        logits.copy_(torch.randn(T, 16, device=DEV))
        graph.replay()
        program(b)
        torch.cuda.synchronize()
        for n in ("ids", "w", "h", "y"):
            assert torch.equal(a[n], b[n]), n
        M.status_check(a["ws"])


def test_launch_timer_counts_the_kernels():
    x = Experts(np.random.default_rng(16), 8, 40, 300)
    ids, w = routing(np.random.default_rng(1), 60, 8, 3)
    d = x.desc(3)
    a, it, wt = torch.randn(60, 300, device=DEV).to(torch.bfloat16), dev(ids), dev(w.astype(np.float32))
    out, ws = torch.zeros(60, 40, device=DEV), workspace(d, 60)
    timer = M.LaunchTimer(8)
    timer.arm()
    M.mx_experts(d, 60, a, None, it, wt, x.slots, x.pool, out, ws)      # the weighted sums in one kernel
    torch.cuda.synchronize()
    assert timer.n_recorded == 2 and all(0 < t < 1e5 for t in timer.kernel_us())
    x = Experts(np.random.default_rng(16), 8, 40, 300, "swiglu")
    timer.arm()
    M.mx_experts(x.desc(3), 60, a, None, it, wt, x.slots, x.pool, out, ws)   # grouping, gated product, weighted sum
    torch.cuda.synchronize()
    assert timer.n_recorded == 6 and all(0 < t < 1e5 for t in timer.kernel_us())
    M.mx_experts(d, 60, a, None, it, wt, x.slots, x.pool, out, ws)      # not armed again
    assert timer.n_recorded == 6
    timer.arm()
    M.route(M.route_desc(8, 2), 60, torch.randn(60, 8, device=DEV), None, torch.zeros(60, 2, dtype=torch.int32, device=DEV),
            torch.zeros(60, 2, device=DEV))
    torch.cuda.synchronize()
    assert timer.n_recorded == 2


def test_two_streams_with_their_own_workspaces():
    rng = np.random.default_rng(11)
    x = Experts(rng, 8, 64, 512)
    d = x.desc(4)
    ids, _ = routing(rng, 100, 8, 4)
    a = to_gpu(rows(rng, 100, 512, "bf16"), "bf16")
    it = dev(ids)
    want = torch.empty(400, 64, device=DEV)
    M.mx_experts(d, 100, a, None, it, None, x.slots, x.pool, want, workspace(d, 100))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [workspace(d, 100) for _ in range(2)]
    outs = [torch.zeros(400, 64, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, ws, o in zip(streams, wss, outs):
            M.mx_experts(d, 100, a, None, it, None, x.slots, x.pool, o, ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("T", [1, 8, 40])
def test_routed_layer_of_microscaled_experts(T):
    """Router, routing, quantised weights and both products as a program runs them; every step against the oracle on the
    step's own input."""
    H, I, E, k = 256, 128, 16, 3
    rng = np.random.default_rng(12)
    wg, wd = rng.normal(size=(E, 2 * I, H)) / 16, rng.normal(size=(E, H, I)) / 11
    (_, cg), (_, sg) = M.mx_shapes(2 * I, H)
    (_, cd), (_, sd) = M.mx_shapes(H, I)
    off = np.cumsum([0, 2 * I * cg, 2 * I * sg, H * cd, H * sd])
    stride = -(-off[4] // 4096) * 4096
    pool = torch.zeros(E * stride, dtype=torch.uint8, device=DEV)
    for e in range(E):                       # weights quantised straight into the experts' blobs
        blob = pool[e * stride:(e + 1) * stride]
        M.mx_quantize(to_gpu(wg[e], "f32"), blob[off[0]:off[1]].view(2 * I, cg), blob[off[1]:off[2]].view(2 * I, sg))
        M.mx_quantize(to_gpu(wd[e], "f32"), blob[off[2]:off[3]].view(H, cd), blob[off[3]:off[4]].view(H, sd))
    slots = torch.arange(E, device=DEV) * stride
    x = rows(rng, T, H, "bf16")
    logits = (rng.normal(size=(T, E))).astype(np.float32)
    bias = (rng.normal(size=E) * 0.2).astype(np.float32)
    sh = R.RouteShape(E, k, "sigmoid", 4, 2, 2, True, 1.5)
    r = M.route_desc(E, k, "sigmoid", 4, 2, 2, True, 1.5)
    ids, w = torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.zeros(T, k, device=DEV)
    M.route(r, T, dev(logits), dev(bias), ids, w)
    d1 = M.mx_product_desc(I, H, out="bf16", act="swiglu", n_experts=E, top_k=k, codes_off=int(off[0]), scales_off=int(off[1]),
                           pool_bytes=pool.numel())
    d2 = M.mx_product_desc(H, I, out="f32", n_experts=E, top_k=k, pair_rows=True, codes_off=int(off[2]), scales_off=int(off[3]),
                           pool_bytes=pool.numel())
    ws = torch.zeros(max(M.mx_workspace_bytes(d1, T), M.mx_workspace_bytes(d2, T)), dtype=torch.uint8, device=DEV)
    h = torch.zeros(T * k, I, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(T, H, device=DEV)
    M.mx_experts(d1, T, to_gpu(x, "bf16"), None, ids, None, slots, pool, h, ws)
    M.mx_experts(d2, T, h, None, ids, w, slots, pool, y, ws)
    M.status_check(ws)
    ids_ref, w_ref = R.route(sh, logits, bias.astype(np.float64))
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    assert np.allclose(w.double().cpu().numpy(), w_ref, rtol=2.0 ** -23, atol=0)
    xv = held(x)[0]
    hv = h.double().cpu().numpy()
    hq = held(hv)[0]
    wt = w.double().cpu().numpy()
    out = np.zeros((T, H))
    bound = np.zeros((T, H))
    for t in range(T):
        for i in range(k):
            e = ids_ref[t, i]
            y1, b1 = expected(xv[t:t + 1], held(wg[e].astype(np.float32).astype(np.float64))[0], "swiglu", H)
            close(h[t * k + i:t * k + i + 1], y1, b1, "bf16", "gate/up")
            wv = held(wd[e].astype(np.float32).astype(np.float64))[0]
            y2, b2 = expected(hq[t * k + i:t * k + i + 1], wv, "none", I)
            out[t] += wt[t, i] * y2[0]
            bound[t] += wt[t, i] * (b2[0] + 2 * g(k + 32) * (np.abs(hq[t * k + i]) @ np.abs(wv).T))
    close(y, out, bound, "f32", "down")


@pytest.mark.parametrize("T", [1, 4, 20])
def test_router_route_feeds_the_int4_experts(T):
    """moe_router_route in place of moe_router_topk before moe_experts_forward: with the plain softmax rule the same
    routing, and with a biased sigmoid the layer of the oracle's routing."""
    geo = synth.PRESETS["tiny"]
    data = make_layer(geo, 21, 0, T)
    dl = upload(data)
    E, k, H = geo.n_experts, geo.top_k, geo.hidden
    ws = torch.zeros(M.workspace_bytes(dl.desc, T), dtype=torch.uint8, device=DEV)
    M.workspace_init(ws)
    new = lambda: (torch.zeros(T, k, dtype=torch.int32, device=DEV), torch.zeros(T, k, device=DEV))
    ids0, w0 = new()
    M.router_topk(dl.desc, T, dl.x, dl.R, ids0, w0, ws)
    ids1, w1 = new()
    M.router_route(dl.desc, M.route_desc(E, k), T, dl.x, dl.R, None, ids1, w1, ws)
    torch.cuda.synchronize()
    assert torch.equal(ids0, ids1) and torch.allclose(w0, w1, rtol=2.0 ** -20, atol=0)   # expf of rounded differences
    bias = (np.random.default_rng(22).normal(size=E) * 0.3).astype(np.float32)
    M.router_route(dl.desc, M.route_desc(E, k, "sigmoid", scale=1.25), T, dl.x, dl.R, dev(bias), ids1, w1, ws)
    y = torch.zeros(T, H, device=DEV)
    M.experts_forward(dl.desc, T, dl.x, ids1, w1, dl.slots, dl.pool, dl.shared, y, ws)
    M.status_check(ws)
    sh = oracle_shape(geo)
    xs, rw, gv = O.load_inputs(sh, T, data.x, data.R, data.shared)
    ids_ref, w_ref = R.route(R.RouteShape(E, k, "sigmoid", scale=1.25), O.router_logits(xs, rw), bias.astype(np.float64))
    assert np.array_equal(ids1.cpu().numpy(), ids_ref)
    out = np.zeros((T, H))
    blob = np.ascontiguousarray(data.shared).view(np.uint8)[:O.blob_bytes(H, sh.shared_inter, sh.bits, sh.sb_dtype)]
    for t in range(T):
        for i, e in enumerate(ids_ref[t]):
            out[t] += w_ref[t, i] * O.expert_forward(*O.parse_blob(O.expert_blob(sh, data.pool, data.slots, int(e)), H, sh.inter,
                                                                   sh.bits, sh.sb_dtype), xs[t])
        out[t] += O.sigmoid(float(gv @ xs[t])) * O.expert_forward(*O.parse_blob(blob, H, sh.shared_inter, sh.bits, sh.sb_dtype), xs[t])
    check_close(y, out, geo.act)


def test_experts_stream_through_the_slot_cache():
    """Blobs of microscaled experts in a pool of fewer slots, filled by the residency manager."""
    rng = np.random.default_rng(13)
    E, N, K, k = 8, 40, 300, 2
    x = Experts(rng, E, N, K)
    stride = -(-(x.scales_off + N * X.padded(K) // 32) // 4096) * 4096
    host = torch.zeros(E, stride, dtype=torch.uint8, pin_memory=True)
    slots, pool = x.slots.cpu().numpy(), x.pool.cpu()
    n = x.scales_off + N * X.padded(K) // 32
    for e in range(E):
        host[e, :n] = pool[slots[e]:slots[e] + n]
    small = torch.zeros(4 * stride, dtype=torch.uint8, device=DEV)
    cache = M.ExpertCache(4, stride, small, host, 1, E)
    copy = torch.cuda.Stream()
    events = []                              # the cache waits for a slot's last reader later on: they live as long as it
    for step in range(4):
        ids = np.stack([rng.choice(E, 2, replace=False)] * 3).astype(np.int32)
        table = np.full(E, -1, dtype=np.int64)
        ready, done = torch.cuda.Event(), torch.cuda.Event()
        events += [ready, done]
        cache.acquire(0, ids, table, copy, ready)
        torch.cuda.current_stream().wait_event(ready)
        x.slots, x.pool = dev(table), small
        x.pool = small
        run_experts(x, 3, k, ids=ids, seed=step)
        done.record()
        cache.release(0, done)
    cache.close()
