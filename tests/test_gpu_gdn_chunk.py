"""The gated delta rule over prompts on the GPU (gdn_chunk_forward through the C ABI) against the fp64 oracle, every output and
every state element, within a bound derived from the arithmetic in chunks; against the recurrence; token by token where
the rule asks for it.

Error bound.  u = 2^-24, g(m) = m u / (1 - m u), n = d_k; |M| is the matrix of magnitudes, S the state before a chunk of at most
64 tokens, E a bound on the 2-norm of each row's error in it.
  factors   rows of K', Q' carry e_k = g(n / 2 + 8) (norms, square root, division, products by g_i and beta); the ratios D_ij
            come from logarithms, each within 4 u of itself and summed in double precision: relative e_D = 8 u (x 2^-x <= 1)
  A         dA = (2 e_k + e_D + 2 g(n + 4)) Abar, Abar_ij = beta_i D_ij sum |k'_i k'_j|
  T         substitution of 64 rows: dT = |T| (dA + 2 g(128) (I + |A|)) |T|
  X         dX = 2 u beta |v| + (2 e_k + e_D + 2 g(n + 4)) beta g |K'| |S|^T + beta g |K'| rows times E (norms of k' are <= 1)
  U = T X   dU = |T| dX + dT |X| + 2 g(64) |T| |X|
  P         dP = (2 e_k + e_D + 2 g(n + 4)) Pbar
  O         dO = (2 e_k + e_D + 2 g(n + 4)) g |Q'| |S|^T + |P| dU + dP |T| |X| + 4 g(64) |P| |T| |X| + g_i ||q'_i|| E
  S         dS = 4 u g_C |S| + sum_j D_Cj (dU_j + (e_k + e_D + 2 g(68)) |T X|_j) |k'_j|
E itself is carried through the exact map of the chunk, g_C (I - ...) products whose rows do not grow for 0 <= beta <= 2, so the
part of dX and dU that comes from E is left out of dS: E <- g_C E + ||dS||.  (The doubled g(.) allow for a matrix unit that
truncates.)  Token by token the bound is the one of test_gpu_gdn, with E <- |alpha| max(1, |1 - beta|) E + d.  The
tests assert twice these first-order bounds, half a step of the output's type on top."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
import synth
from oracle import gdn_oracle as G
from synth.gdn import gdn_inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
EPS = 1e-6


def g(m):
    return m * U / (1 - m * U)


class Case:
    """Sequences of the given lengths, packed; `first` rows in front and `behind` behind them belong to none."""

    def __init__(self, lens, nk=2, nv=4, dk=64, dv=32, act="bf16", out="f32", seed=0, state=True, first=0, behind=0, alpha=None,
                 beta=None, near_one=True):
        self.lens, self.nk, self.nv, self.dk, self.dv, self.act, self.out = list(lens), nk, nv, dk, dv, act, out
        self.cu = np.concatenate(([0], np.cumsum(self.lens))) + first
        self.N = int(self.cu[-1]) + behind
        q, k, v, al, be, st = gdn_inputs(nk, nv, dk, dv, 1, max(self.N, 1), seed, act)
        self.q, self.k, self.v, self.alpha, self.beta = q[0], k[0], v[0], al[0].copy(), be[0].copy()
        if near_one:                                     # gates as layers have them: decay over tens to thousands of tokens
            self.alpha[:] = np.float32(1) - (np.float32(1) - self.alpha) * np.float32(0.06)
        if alpha is not None:
            self.alpha[...] = alpha
        if beta is not None:
            self.beta[...] = beta
        rng = np.random.default_rng(seed)
        self.state = (0.5 * rng.standard_normal((len(self.lens), nv, dv, dk))).astype(np.float32) if state else None
        self.scale = dk ** -0.5

    @property
    def desc(self):
        return M.gdn_desc(self.nk, self.nv, self.dk, self.dv, act=self.act, out=self.out, scale=self.scale, eps=EPS)

    def run(self, T_max=None, ws=None, in_place=False, stream=None):
        put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        if self.act == "bf16":
            act = lambda a: put(a.view(np.int16)).view(torch.bfloat16)
        else:
            act = put
        d, B = self.desc, len(self.lens)
        out = torch.full((self.N, self.nv, self.dv), 7.0, dtype=torch.float32 if self.out == "f32" else torch.bfloat16, device=DEV)
        st = None if self.state is None else put(self.state)
        so = st if in_place else torch.full((B, self.nv, self.dv, self.dk), float("nan"), device=DEV)
        if ws is None:
            ws = torch.full((M.gdn_chunk_workspace_bytes(d, B, self.N),), 0xff, dtype=torch.uint8, device=DEV)
        M.gdn_chunk_forward(d, B, self.N, max(self.lens) if T_max is None else T_max, put(self.cu.astype(np.int32)), act(self.q),
                            act(self.k), act(self.v), put(self.alpha), put(self.beta), st, so, out, ws, stream=stream)
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), so.double().cpu().numpy()

    def values(self):
        return [synth.act_values(x, self.act).astype(np.float64) for x in (self.q, self.k, self.v)]

    def check(self, **kw):
        out, state = self.run(**kw)
        T_max = kw.get("T_max")
        q, k, v = self.values()
        for b, n in enumerate(self.lens):
            rows = slice(self.cu[b], self.cu[b] + (n if T_max is None else min(n, T_max)))
            for h in range(self.nv):
                kh = h // (self.nv // self.nk)
                S0 = np.zeros((self.dv, self.dk)) if self.state is None else self.state[b, h].astype(np.float64)
                o, S, ob, E = head(self, q[rows, kh], k[rows, kh], v[rows, h], self.alpha[rows, h].astype(np.float64),
                                   self.beta[rows, h].astype(np.float64), S0)
                if self.out == "bf16":
                    ob = ob + 2.0 ** -9 * np.abs(o)       # doubled below
                close(out[rows, h], o, 2 * ob, (b, h, "out"))
                close(state[b, h], S, 2 * E[:, None], (b, h, "state"))
        outside = np.ones(self.N, dtype=bool)
        for b, n in enumerate(self.lens):
            outside[self.cu[b]:self.cu[b] + (n if T_max is None else min(n, T_max))] = False
        assert np.all(out[outside] == 7.0)
        return out, state


def close(got, want, bound, what):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= bound + 1e-37)
    assert np.all(ok), f"{what}: {np.sum(~ok)} of {ok.size}; {got[~ok][0]} for {want[~ok][0]}, bound {np.broadcast_to(bound, ok.shape)[~ok][0]}"


def head(c, q, k, v, al, be, S):
    """One head of one sequence: outputs, final state, and their bounds (rows of the state: 2-norms)."""
    n, dk = v.shape[0], c.dk
    e_k, e_q, gn = g(dk / 2 + 8), g(dk / 2 + 8), g(dk + 4)
    scale = float(np.float32(c.scale))
    out, bound = np.zeros((n, c.dv)), np.zeros((n, c.dv))
    S, E = S.copy(), np.zeros(c.dv)
    with np.errstate(all="ignore"):
        kn = k / np.sqrt(np.sum(k * k, axis=1, keepdims=True) + EPS)
        qn = scale * q / np.sqrt(np.sum(q * q, axis=1, keepdims=True) + EPS)
        for t0 in range(0, n, 64):
            s = slice(t0, min(t0 + 64, n))
            K, Q, V, a, b = kn[s], qn[s], v[s], al[s], be[s]
            fine = all(np.all(np.isfinite(x)) for x in (K, Q, a, b))
            whole = fine and np.all((a >= 2.0 ** -20) & (a <= 1)) and np.all((b >= 0) & (b <= 2))
            Sin, Ein = S.copy(), E.copy()
            for t in range(s.start, s.stop):             # the rule itself, and its bound token by token
                w = S @ kn[t]
                A = np.abs(S) @ np.abs(kn[t])
                u = be[t] * (v[t] - al[t] * w)
                dw = (2 * gn + e_k) * A
                du = np.abs(be[t]) * np.abs(al[t]) * dw + g(3) * np.abs(be[t]) * (np.abs(v[t]) + np.abs(al[t]) * (np.abs(w) + dw))
                d = du + np.abs(u) * e_k + g(2) * (np.abs(al[t]) * np.linalg.norm(S, axis=1) + np.abs(u))
                E = np.abs(al[t]) * max(1.0, abs(1 - be[t])) * E + d
                S, out[t] = G.delta_rule_step(S, qn[t], kn[t], v[t], al[t], be[t])
                bound[t] = E * np.linalg.norm(qn[t]) + (2 * gn + e_q) * (np.abs(S) @ np.abs(qn[t]))
            if not whole:
                continue
            eD = 8 * U
            e = 2 * e_k + eD + 2 * gn
            L = np.cumsum(np.log(a))
            D = np.tril(np.exp(np.minimum(L[:, None] - L[None, :], 0)))
            gi = np.exp(L)[:, None]
            m = len(a)
            Ab = b[:, None] * np.tril(D, -1) * (np.abs(K) @ np.abs(K).T)
            Am = b[:, None] * np.tril(D, -1) * (K @ K.T)
            T = np.linalg.inv(np.eye(m) + Am)
            X = b[:, None] * (V - gi * (K @ Sin.T))
            Pm, Pb = D * (Q @ K.T), D * (np.abs(Q) @ np.abs(K).T)
            aT = np.abs(T)
            dT = aT @ (e * Ab + 2 * g(128) * (np.eye(m) + np.abs(Am))) @ aT
            dX0 = b[:, None] * (2 * U * np.abs(V) + e * gi * (np.abs(K) @ np.abs(Sin).T))
            dU = aT @ dX0 + dT @ np.abs(X) + 2 * g(64) * (aT @ np.abs(X))
            TX = aT @ np.abs(X)
            by_token, E_token = bound[s].copy(), E
            bound[s] = (e * gi * (np.abs(Q) @ np.abs(Sin).T) + np.abs(Pm) @ dU + e * (Pb @ TX) + 4 * g(64) * (np.abs(Pm) @ TX)
                        + gi * np.linalg.norm(Q, axis=1)[:, None] * Ein)
            w = D[-1][:, None]
            dS = 4 * U * gi[-1] * np.abs(Sin) + (w * (dU + (e_k + eD + 2 * g(68)) * TX)).T @ np.abs(K)
            E = gi[-1, 0] * Ein + np.linalg.norm(dS, axis=1)
            if not np.all(np.abs(X) <= 2.0 ** 96):       # such rows, and those in their block, run token by token
                bound[s], E = np.fmax(bound[s], by_token), np.fmax(E, E_token)
    return out, S, bound, E


def show(*a):
    print("chunks", *a, flush=True)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2, 1, 63], [64], [65, 0, 128], [17, 200]])
@pytest.mark.parametrize("dk,dv", [(64, 16), (128, 32)])
def test_lengths(act, lens, dk, dv):
    show(act, lens, dk, dv)
    Case(lens, 2, 4, dk, dv, act, seed=len(lens) + dk).check()


@pytest.mark.parametrize("nk,nv,dk,dv", [(1, 1, 128, 256), (1, 3, 64, 48), (4, 4, 128, 128), (2, 16, 64, 64)])
@pytest.mark.parametrize("act,out", [("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
def test_layouts(nk, nv, dk, dv, act, out):
    show(nk, nv, dk, dv, act, out)
    Case([70, 5], nk, nv, dk, dv, act, out, seed=nv).check()


def test_more_sequences_than_a_wave():
    show("many")
    rng = np.random.default_rng(3)
    Case(rng.integers(0, 90, size=150).tolist(), 1, 1, 64, 16, "bf16", seed=4).check()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_zeros_as_first_state_and_in_place(act):
    show("states", act)
    Case([100, 30], act=act, state=False, seed=5).check()
    c = Case([100, 0, 30], act=act, seed=6)
    a, b = c.run(), c.run(in_place=True)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert np.array_equal(a[1][1], c.state[1].astype(np.float64))     # no tokens: the state itself


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_padding_and_bound_on_tokens(act):
    show("padding", act)
    c = Case([100, 0, 30, 64], act=act, seed=7, first=5, behind=40)
    c.check()
    c.check(T_max=65)
    c.check(T_max=1)


@pytest.mark.parametrize("alpha,beta", [(1.0, 1.0), (1.0, 2.0), (0.25, 0.5), (2.0 ** -19, 1.0), (0.999, 0.0), (1.0, 0.01)])
def test_gates_at_their_limits(alpha, beta):
    show("gates", alpha, beta)
    Case([150], alpha=alpha, beta=beta, seed=8, act="f32").check()


def test_repeated_and_zero_keys():
    """The same key at every token (every row of the triangular system full), keys of zeros, tiny and large ones."""
    show("keys")
    c = Case([130], seed=9, act="f32", beta=1.0)
    c.k[:] = c.k[0]
    c.check()
    c = Case([130], seed=10, act="f32")
    c.k[5:20] = 0
    c.q[3] = 0
    c.k[30] *= 1e-4
    c.k[31] *= 1e6
    c.q[70:] *= 1e5
    c.check()


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_gates_outside_the_chunks_range(act):
    """Gates of zero, negative, above one, a write strength above two or below zero: those chunks run token by token."""
    show("odd gates", act)
    c = Case([200, 64], act=act, seed=11)
    c.alpha[10, 0], c.alpha[70, 1], c.alpha[140, 2], c.alpha[210, 3] = 0.0, -0.5, 1.25, 2.0 ** -30
    c.beta[20, 1], c.beta[90, 0] = 2.5, -0.25
    c.check()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["k", "q", "v", "alpha", "beta"])
def test_values_that_are_not_finite_reach_no_earlier_token(act, what):
    show("not finite", act, what)
    c = Case([100, 40], act=act, seed=12)
    clean = c.run()
    x = getattr(c, what)
    bad = np.float32(np.nan)
    if x.dtype != np.float32:
        x[80, 1, 3] = 0x7fc0
    elif x.ndim == 3:
        x[80, 1, 3] = bad
    else:
        x[80, 1] = bad
    out, state = c.run()
    close(out[:80], clean[0][:80], 1e-4 * np.abs(clean[0]).max(), "earlier")
    assert np.array_equal(out[100:], clean[0][100:]) and np.array_equal(state[1], clean[1][1])
    assert np.isnan(out[80:100]).any()
    c.check()


# Sequences enough for blocks of 64 and of 128 state rows (where that many fit) by 32 heads.
SOME = [130, 64, 7, 0, 90, 33, 65, 20]
MANY = [64 + 5 * i for i in range(16)]


@pytest.mark.parametrize("lens,dk,dv,out", [(SOME, 128, 128, "bf16"), (SOME, 128, 64, "f32"), (SOME, 64, 48, "bf16"), (MANY, 64, 128, "f32"),
                                            (MANY, 128, 112, "bf16"), (MANY, 128, 128, "f32")])
def test_many_heads(lens, dk, dv, out):
    show("heads", len(lens), dk, dv, out)
    Case(lens, 8, 32, dk, dv, "bf16", out, seed=dk + dv, first=3, behind=70).check()


@pytest.mark.parametrize("lens,dk,dv", [([130, 64, 7], 128, 32), (SOME, 128, 64), (MANY, 64, 128)])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_values_and_states_out_of_range(lens, dk, dv, act):
    """One row each of three heads: a value that is NaN, one too large for a chunk's products, and an infinite state; and a gate
    of a fourth head.  No other row is touched."""
    show("rows", len(lens), dk, dv, act)
    nv = 4 if len(lens) == 3 else 32
    c = Case(lens, nv // 4, nv, dk, dv, act, seed=15)
    clean, clean_state = c.run()
    set_v = lambda t, h, r, x: c.v.__setitem__((t, h, r), np.float32(x) if act == "f32" else np.float32(x).view(np.uint32) >> 16)
    set_v(70, 0, 5, np.nan)
    set_v(3, 1, 30, 2.0 ** 100)
    c.state[1, 2, 17, 9] = np.inf
    c.alpha[100, 3] = 0.0
    out, state = c.check()
    assert np.isnan(out[70:130, 0, 5]).all() and np.isfinite(out[:70, 0, 5]).all()
    others = np.ones(dv, dtype=bool)
    others[[5, 30, 17]] = False
    assert np.isfinite(out[:, :3][..., others]).all() and np.isfinite(state[:, :3][:, :, others]).all()
    assert np.array_equal(out[:, 4:], clean[:, 4:]) and np.array_equal(state[:, 4:], clean_state[:, 4:])


def test_against_the_recurrence():
    show("recurrence")
    c = Case([90, 90, 90], 2, 4, 128, 64, "bf16", "f32", seed=13)
    out, state = c.run()
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    act = lambda a: put(a.view(np.int16)).view(torch.bfloat16)
    st, o = put(c.state), torch.empty((3, 90, 4, 64), device=DEV)
    M.gdn_forward(c.desc, 3, 90, act(c.q), act(c.k), act(c.v), put(c.alpha), put(c.beta), st, o)
    assert np.abs(o.double().cpu().numpy().reshape(out.shape) - out).max() <= 2.0 ** -16 * np.abs(out).max()
    assert np.abs(st.double().cpu().numpy() - state).max() <= 2.0 ** -16 * np.abs(state).max()


def test_prompt_in_parts_and_tokens_after_it():
    """A prompt in two calls, the state handed on, then single tokens by the recurrence: the same as everything at once."""
    show("parts")
    whole = Case([150], seed=14, act="f32")
    out, state = whole.run()
    st, at = whole.state, 0
    for n in (70, 77, 1, 1, 1):
        part = Case([n], seed=14, act="f32")
        for x in ("q", "k", "v", "alpha", "beta"):
            setattr(part, x, getattr(whole, x)[at:at + n])
        part.state = st
        if n > 1:
            o, s = part.run()
        else:
            put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
            s, o = put(st), torch.empty((1, 4, 32), device=DEV)
            M.gdn_forward(part.desc, 1, 1, *(put(getattr(part, x)) for x in ("q", "k", "v", "alpha", "beta")), s, o)
            s, o = s.double().cpu().numpy(), o.double().cpu().numpy()
        st = s.astype(np.float32)
        assert np.abs(o - out[at:at + n]).max() <= 2.0 ** -15 * np.abs(out).max()
        at += n
    assert np.abs(st - state).max() <= 2.0 ** -15 * np.abs(state).max()


def test_several_passes():
    """More chunks than the workspace holds at once: passes over parts of every sequence, the state carried between them.  The
    same chunks by themselves give the same bits."""
    show("passes")
    lens = [4000, 0, 6000, 64, 70]
    c = Case(lens, 16, 256, 64, 16, "bf16", "bf16", seed=15)
    d = c.desc
    full = M.gdn_chunk_workspace_bytes(d, 1, 64)
    assert M.gdn_chunk_workspace_bytes(d, len(lens), c.N) < full * (c.N // 64) / 3
    out, state = c.run()
    for b in (0, 3, 4):
        one = Case([lens[b]], 16, 256, 64, 16, "bf16", "bf16", seed=15)
        rows = slice(c.cu[b], c.cu[b + 1])
        for x in ("q", "k", "v", "alpha", "beta"):
            setattr(one, x, np.ascontiguousarray(getattr(c, x)[rows]))
        one.state = c.state[b:b + 1]
        o, s = one.run()
        assert np.array_equal(o, out[rows]) and np.array_equal(s[0], state[b])
    assert np.array_equal(state[1], c.state[1].astype(np.float64))


def test_streams_and_graphs():
    show("graphs")
    c = Case([100, 37], seed=16)
    want = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.run()
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    act = lambda a: put(a.view(np.int16)).view(torch.bfloat16)
    d = c.desc
    args = [act(c.q), act(c.k), act(c.v), put(c.alpha), put(c.beta)]
    cu, st = put(c.cu.astype(np.int32)), put(c.state)
    so, out = torch.empty_like(st), torch.empty((c.N, 4, 32), device=DEV)
    ws = torch.empty(M.gdn_chunk_workspace_bytes(d, 2, c.N), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.gdn_chunk_forward(d, 2, c.N, 100, cu, *args, st, so, out, ws)
    for step, lens in enumerate(([100, 37], [64, 73], [0, 1], [100, 37])):
        cu.copy_(torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32))
        out.fill_(7.0)
        ws.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        c.lens, c.cu = lens, np.array([0, lens[0], sum(lens)])
        want = c.run(T_max=100)
        assert np.array_equal(out.double().cpu().numpy(), want[0]) and np.array_equal(so.double().cpu().numpy(), want[1])


def test_launch_timer_counts_the_kernels():
    timer = M.LaunchTimer()
    timer.arm()
    Case([100]).run()
    assert timer.n_recorded == 4 and all(t > 0 for t in timer.kernel_us())
