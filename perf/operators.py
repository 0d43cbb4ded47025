"""Operators around a mixture-of-experts layer: routing from scores, microscaled 4-bit quantisation, and the products of
microscaled matrices, dense and by routed expert.

Routing.  Per token with logits l[E] and an optional bias b[E]:
    s_e = exp(l_e - max l) / sum exp(l - max l)   (softmax)   or   1 / (1 + exp(-l_e))   (sigmoid)
    key_e = s_e + b_e with a bias, else l_e;  -inf where l_e = -inf (an expert that is masked out)
    with G groups: a group's score is the sum of its `group_top` largest values of s_e + b_e (of s_e without a bias),
    masked experts left out; experts outside the `top_groups` best groups are out (ties: the lower group)
    ids = the k first experts by (-key, id);  w_i = s_{ids_i}, divided by their sum if renormalised, times `scale`
    a masked expert has weight 0, and so has every expert of a row that the mask leaves empty.

Microscaled 4-bit values.  32 consecutive values of a row share a power of two: with m = max |x| over the block,
    e = max(floor(log2 m) - 2, -127) (m = 0: -127),   q = x / 2^e rounded to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 with either
    sign (ties to the even code, larger values to 6);   the value held is q 2^e.
Codes take four bits, the first value of a pair in the low half of a byte; the power is held as one byte, e + 127.  Rows are
padded with zeros to a multiple of 256 values (a cache line of codes).

Products.  y = A W^T with A [M, K] and W [N, K] both held as above (A quantised within the call), sums in 32 bits.
By expert: row (t, i) of the product takes the matrix of expert ids[t, i]; its input is row t, or row t k + i.  The output
is one row for each pair, or sum_i w[t, i] y[t, i].  With "swiglu" W holds n gate rows, then n up rows, and the
output is silu(gate) * up.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one token of a served sequence: groups of experts, a bias that balances them
        dict(name="route one token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, scale=2.5, dtype="f32", masked=False),
        # a prompt through a wide router, softmax over all experts, chosen weights renormalised
        dict(name="route prompt softmax", op="route", T=2048, E=512, k=10, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, dtype="f32", masked=False),
        # a large batch with some experts taken out (not resident), some rows without any
        dict(name="route batch masked groups", op="route", T=32768, E=512, k=10, score="sigmoid", bias=True, groups=8, top_groups=3,
             group_top=2, renorm=True, scale=1.0, dtype="bf16", masked=True),
        # the activations of eight decoded tokens
        dict(name="quantise decode rows", op="quantise", rows=8, cols=2048, dtype="bf16"),
        # float32 weights of an odd width
        dict(name="quantise odd float32", op="quantise", rows=1000, cols=1111, dtype="f32"),
        # weights of many experts, laid out once when a model is loaded
        dict(name="quantise weights", op="quantise", rows=131072, cols=2048, dtype="bf16"),
        # one token through a projection
        dict(name="linear one token", op="linear", M=1, N=4096, K=2048, act="none", dtype="bf16", out="bf16"),
        # a ragged batch through a gated projection, nothing a multiple of a tile
        dict(name="linear ragged swiglu", op="linear", M=333, N=1000, K=1111, act="swiglu", dtype="f32", out="f32"),
        # a long prompt through a large projection
        dict(name="linear prompt", op="linear", M=8192, N=8192, K=8192, act="none", dtype="bf16", out="bf16"),
        # one token through the gate and up matrices of its ten experts
        dict(name="experts one token gate up", op="experts", T=1, E=512, k=10, N=512, K=2048, act="swiglu", combine=False,
             dtype="bf16", out="bf16", skew=1.1),
        # a batch of decoded tokens through the down matrices of their experts, the weighted sum of each token's
        dict(name="experts batch down", op="experts", T=64, E=256, k=8, N=2048, K=512, act="none", combine=True,
             dtype="bf16", out="f32", skew=1.1),
        # a prompt through the gate and up matrices of all experts
        dict(name="experts prompt gate up", op="experts", T=2048, E=512, k=10, N=512, K=2048, act="swiglu", combine=False,
             dtype="bf16", out="bf16", skew=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "quantise", "linear", "experts"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        each = _log(rng, 4, 1024 // groups)
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16384), E=groups * each, k=rng.randint(1, min(16, top_groups * each)),
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_top=rng.randint(1, 2), renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                    dtype=rng.choice(("f32", "bf16")), masked=rng.random() < 0.3)
    if op == "quantise":
        cols = _log(rng, 20, 8192)
        return dict(op=op, rows=_log(rng, 1, min(131072, (1 << 28) // cols)), cols=cols, dtype=rng.choice(("f32", "bf16")))
    act = rng.choice(("none", "swiglu"))
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 33, 4096), K=_log(rng, 33, 8192), act=act,
                    dtype=rng.choice(("f32", "bf16")), out=rng.choice(("f32", "bf16")))
    E = rng.choice((16, 64, 128, 256))
    return dict(op=op, T=_log(rng, 1, 2048), E=E, k=rng.randint(1, 10), N=_log(rng, 64, 1024), K=_log(rng, 64, 2048), act=act,
                combine=rng.random() < 0.5, dtype=rng.choice(("f32", "bf16")), out=rng.choice(("f32", "bf16")),
                skew=rng.choice((0.0, 1.1)))


# Sizes of what is held in four bits.

def _padded(cols):
    return -(-cols // 256) * 256


def _blob(c):
    """Bytes of one expert's codes and scales, and the stride from one expert to the next."""
    rows = c["N"] * (2 if c["act"] == "swiglu" else 1)
    codes, scales = rows * _padded(c["K"]) // 2, rows * _padded(c["K"]) // 32
    return rows, codes, scales, -(-(codes + scales) // 4096) * 4096


def work(c):
    if c["op"] == "route":
        item = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * (c["E"] * item + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0), "flops": 4 * c["T"] * c["E"]}
    if c["op"] == "quantise":  # the values in, the codes and scales out and in again, the values that they stand for out
        item = 4 if c["dtype"] == "f32" else 2
        held = c["rows"] * (_padded(c["cols"]) // 2 + _padded(c["cols"]) // 32)
        return {"bytes": 2 * c["rows"] * c["cols"] * item + 2 * held, "flops": 3 * c["rows"] * c["cols"]}
    two = 2 if c["act"] == "swiglu" else 1
    a, o = (4 if c[x] == "f32" else 2 for x in ("dtype", "out"))
    if c["op"] == "linear":
        return {"bytes": c["M"] * c["K"] * a + two * c["N"] * c["K"] * 17 // 32 + c["M"] * c["N"] * o,
                "flops": 2 * two * c["M"] * c["N"] * c["K"]}
    pairs = c["T"] * c["k"]
    p = np.arange(1, c["E"] + 1, dtype=np.float64) ** -c["skew"]
    p = np.minimum(1.0, c["k"] * p / p.sum())
    used = float((1 - (1 - p) ** c["T"]).sum())  # about how many experts the tokens choose
    rows_in = pairs if c["combine"] else c["T"]
    rows_out = c["T"] if c["combine"] else pairs
    return {"bytes": rows_in * c["K"] * a + used * two * c["N"] * c["K"] * 17 / 32 + rows_out * c["N"] * o,
            "flops": 2 * two * pairs * c["N"] * c["K"]}


# Inputs.

def _codes(gen, shape):
    """Four-bit codes as a quantiser leaves them for normal values: about 2.4 steps of one in the middle of a block."""
    q = (torch.arange(256, dtype=torch.float64, device=DEV) + 0.5) / 256
    x = 2.4 * math.sqrt(2) * torch.erfinv(2 * q - 1)
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)
    table = (x.abs()[:, None] - levels).abs().argmin(1).to(torch.uint8) + 8 * (x < 0).to(torch.uint8)
    lo, hi = (table[torch.randint(0, 256, shape, generator=gen, device=DEV, dtype=torch.int32)] for _ in range(2))
    return lo | (hi << 4)


def _matrix(gen, rows, K):
    """Codes and scales of `rows` rows of K values, the padding zero."""
    Kp = _padded(K)
    codes = _codes(gen, (rows, Kp // 2))
    scales = torch.randint(117, 121, (rows, Kp // 32), generator=gen, device=DEV, dtype=torch.uint8)
    codes[:, (K + 1) // 2:] = 0
    if K % 2:
        codes[:, K // 2] &= 15
    scales[:, -(-K // 32):] = 0
    return codes, scales


def _rows(gen, rows, cols, dtype):
    """Activations: normal values, each row with a size of its own, a few columns much larger."""
    x = torch.randn((rows, cols), generator=gen, device=DEV)
    x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=DEV))
    x[:, :: max(1, cols // 5)] *= 8
    return x.to(TYPES[dtype])


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "route":
        x = torch.randn((c["T"], c["E"]), generator=gen, device=DEV) * 1.5
        if c["masked"]:
            x[torch.rand((c["T"], c["E"]), generator=gen, device=DEV) < 0.15] = float("-inf")
            x[torch.rand((c["T"],), generator=gen, device=DEV) < 0.02] = float("-inf")
        s["logits"] = x.to(TYPES[c["dtype"]])
        s["bias"] = torch.randn((c["E"],), generator=gen, device=DEV) * 0.1 if c["bias"] else None
        s["ids"] = torch.empty((c["T"], c["k"]), dtype=torch.int32, device=DEV)
        s["w"] = torch.empty((c["T"], c["k"]), dtype=torch.float32, device=DEV)
        return s
    if c["op"] == "quantise":
        s["x"] = _rows(gen, c["rows"], c["cols"], c["dtype"])
        Kp = _padded(c["cols"])
        s["codes"] = torch.empty((c["rows"], Kp // 2), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((c["rows"], Kp // 32), dtype=torch.uint8, device=DEV)
        s["values"] = torch.empty_like(s["x"])
        return s
    if c["op"] == "linear":
        s["a"] = _rows(gen, c["M"], c["K"], c["dtype"])
        s["codes"], s["scales"] = _matrix(gen, c["N"] * (2 if c["act"] == "swiglu" else 1), c["K"])
        s["out"] = torch.empty((c["M"], c["N"]), dtype=TYPES[c["out"]], device=DEV)
        s["ws"] = torch.zeros(_workspace(c), dtype=torch.uint8, device=DEV)
        return s
    T, E, k = c["T"], c["E"], c["k"]
    pairs = T * k
    rank = torch.randperm(E, generator=gen, device=DEV).double() + 1
    u = torch.rand((T, E), generator=gen, device=DEV, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    key = -c["skew"] * torch.log(rank) - torch.log(-torch.log(u))
    top = torch.sort(key, dim=1, descending=True)
    s["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
    s["w"] = torch.softmax(top.values[:, :k], dim=1).float().contiguous()
    s["a"] = _rows(gen, pairs if c["combine"] else T, c["K"], c["dtype"])
    rows, codes, scales, stride = _blob(c)
    pool = torch.zeros((E, stride), dtype=torch.uint8, device=DEV)
    held = _matrix(gen, E * rows, c["K"])
    pool[:, :codes] = held[0].view(E, codes)
    pool[:, codes:codes + scales] = held[1].view(E, scales)
    s["pool"] = pool.view(-1)
    s["slots"] = torch.randperm(E, generator=gen, device=DEV) * stride
    s["out"] = torch.empty((T if c["combine"] else pairs, c["N"]), dtype=TYPES[c["out"]], device=DEV)
    s["ws"] = torch.zeros(_workspace(c), dtype=torch.uint8, device=DEV)
    s["most"] = int(torch.bincount(s["ids"].view(-1).long(), minlength=E).max())  # the plain form's batch: rows of the fullest expert
    return s


def _workspace(c):
    """A generous bound on the bytes that a product needs beside its operands: its rows quantised, its pairs listed by
    expert, one float32 row of the output for each pair."""
    pairs = c["T"] * c["k"] if c["op"] == "experts" else c["M"]
    return (8 << 20) + pairs * (_padded(c["K"]) + 4 * c["N"] + 256)


# What is computed: by the framework's operators, or in plain steps.

def run(s):
    c = s["case"]
    if own:
        return _own(c, s)
    if c["op"] == "route":
        return _route(c, s["logits"], s["bias"])
    if c["op"] == "quantise":
        return {"values": _values(*_quantise(s["x"].float()), c["cols"]).to(s["x"].dtype)}
    if c["op"] == "linear":
        y = _held(s["a"], c["K"]) @ _values(s["codes"], s["scales"], c["K"]).T
        return {"out": _gated(c, y).to(TYPES[c["out"]])}
    return {"out": _experts(c, s).to(TYPES[c["out"]])}


def _own(c, s):
    import int4_quantized_expert_amd as M
    if c["op"] == "quantise":
        M.mx_quantize(s["x"], s["codes"], s["scales"])
        M.mx_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"]}
    d = s.get("descriptor") or s.setdefault("descriptor", _descriptor(M, c, s))  # a program makes it once
    if c["op"] == "route":
        M.route(d, c["T"], s["logits"], s["bias"], s["ids"], s["w"])
        return {"ids": s["ids"], "w": s["w"]}
    if c["op"] == "linear":
        M.mx_linear(d, c["M"], s["a"], None, s["codes"], s["scales"], s["out"], s["ws"])
    else:
        M.mx_experts(d, c["T"], s["a"], None, s["ids"], s["w"] if c["combine"] else None, s["slots"], s["pool"], s["out"], s["ws"])
    return {"out": s["out"]}


def _descriptor(M, c, s):
    if c["op"] == "route":
        return M.route_desc(c["E"], c["k"], score=c["score"], n_groups=c["groups"], top_groups=c["top_groups"],
                            group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"], logits=c["dtype"])
    if c["op"] == "linear":
        return M.mx_product_desc(c["N"], c["K"], a=c["dtype"], out=c["out"], act=c["act"])
    return M.mx_product_desc(c["N"], c["K"], a=c["dtype"], out=c["out"], act=c["act"], n_experts=c["E"], top_k=c["k"],
                             pair_rows=c["combine"], codes_off=0, scales_off=_blob(c)[1], pool_bytes=s["pool"].numel())


def _route(c, logits, bias):
    x = logits.double()
    masked = x == float("-inf")
    empty = masked.all(1, keepdim=True)
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True).masked_fill(empty, 0.0))
        score = e / e.sum(1, keepdim=True).masked_fill(empty, 1.0)
    shifted = score if bias is None else score + bias.double()
    key = x if bias is None else shifted.masked_fill(masked, float("-inf"))
    if c["groups"] > 1:
        T, G = x.shape[0], c["groups"]
        best = shifted.masked_fill(masked, float("-inf")).view(T, G, -1).topk(min(c["group_top"], c["E"] // G), dim=2).values
        total = torch.where(torch.isinf(best[..., :1]), best[..., :1], best.masked_fill(torch.isinf(best), 0.0).sum(2, keepdim=True))
        order = torch.sort(total[..., 0], dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, order, True)
        out = ~keep.repeat_interleave(c["E"] // G, dim=1)
        # experts outside the chosen groups come after every other one, those that are masked included
        first = torch.sort(out.to(torch.uint8), dim=1, stable=True).indices
        inner = torch.sort(key.gather(1, first).masked_fill(out.gather(1, first), float("-inf")), dim=1, descending=True, stable=True)
        ids = first.gather(1, inner.indices)[:, :c["k"]]
    else:
        ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / total.masked_fill(total == 0, 1.0)
    return {"ids": ids.int(), "w": (w * c["scale"]).float()}


def _quantise(x):
    """Codes and scales of float32 rows."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, _padded(cols) - cols)).view(rows, -1, 32)
    field = (b.abs().amax(2).view(torch.int32) >> 23) - 2  # the exponent of the largest value, less that of 4
    scale = field.clamp_min(0)
    y = b.abs() * _power(254 - scale)[..., None]
    q = torch.where(y < 2, torch.round(2 * y), torch.where(y < 4, 2 + torch.round(y), 4 + torch.round(y / 2))).clamp_max(7)
    codes = (q + 8 * torch.signbit(b)).to(torch.uint8).view(rows, -1, 2)
    return codes[..., 0] | (codes[..., 1] << 4), scale.to(torch.uint8)


def _power(field):
    """2^(field - 127) for whole numbers from 0."""
    return torch.where(field > 0, field << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _values(codes, scales, cols):
    level = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    two = torch.stack((level.repeat(16), level.repeat_interleave(16)), 1)
    v = two[codes.int()].view(*scales.shape, 32) * _power(scales.int())[..., None]
    return v.flatten(-2)[..., :cols]


def _held(a, cols):
    """The values that rows stand for once they are quantised."""
    return _values(*_quantise(a.float()), cols)


def _gated(c, y):
    if c["act"] == "none":
        return y
    g, u = y[..., :c["N"]], y[..., c["N"]:]
    return g / (1 + torch.exp(-g)) * u


def _experts(c, s):
    E, k, pairs = c["E"], c["k"], c["T"] * c["k"]
    e = s["ids"].view(-1).long()
    rows, codes, scales, stride = _blob(c)
    a = _held(s["a"], c["K"])
    few = pairs <= E  # few pairs: the matrix of each pair's expert; many: all matrices, each with a batch of its rows
    at = s["slots"][e] if few else s["slots"]
    blob = s["pool"].view(E, stride)[at // stride]
    weights = _values(blob[:, :codes].reshape(-1, rows, codes // rows), blob[:, codes:codes + scales].reshape(-1, rows, scales // rows), c["K"])
    pair = torch.arange(pairs, device=e.device)
    if few:
        x = a[pair if c["combine"] else pair // k][:, None]
        batch, place = pair, torch.zeros_like(pair)
    else:
        order = torch.sort(e, stable=True).indices
        place = torch.empty_like(pair)
        place[order] = pair - torch.searchsorted(e[order], e[order])
        batch = e
        x = torch.zeros((E, s["most"], c["K"]), dtype=a.dtype, device=a.device)
        x[batch, place] = a[pair if c["combine"] else pair // k]
    y = _gated(c, torch.matmul(x, weights.transpose(1, 2).contiguous())[batch, place])
    return (y.view(c["T"], k, -1) * s["w"][..., None]).sum(1) if c["combine"] else y


# The definition in 64 bits.

def _exact_values(codes, scales, cols):
    level = torch.tensor(LEVELS, dtype=torch.float64, device=codes.device)
    n = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)[..., :cols]
    v = level[(n & 7).int()]
    v[n > 7] *= -1
    e = scales.to(torch.float64) - 127
    return v * torch.exp2(e).repeat_interleave(32, dim=-1)[..., :cols]


def _exact_held(x):
    """What rows stand for once quantised, in 64 bits: the nearest level by distance, ties to the even code."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -cols % 32)).view(rows, -1, 32)
    e = torch.frexp(x.abs().amax(2)).exponent - 3  # frexp's fraction is in [1/2, 1)
    p = torch.exp2(e.double().clamp_min(-127))[..., None]
    y = (x / p).abs()
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    middle = (level[1:] + level[:-1]) / 2
    upper = torch.arange(1, 8, device=x.device) % 2 == 0  # on the middle of two levels: the one of even index
    held = level[((y[..., None] > middle) | ((y[..., None] == middle) & upper)).sum(-1, dtype=torch.int32)]
    return (torch.copysign(held, x) * p).view(rows, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        return _exact_route(c, s["logits"].double().cpu().numpy(), None if s["bias"] is None else s["bias"].double().cpu().numpy())
    if c["op"] == "quantise":
        return {"values": _exact_held(s["x"])}
    a = _exact_held(s["a"])
    if c["op"] == "linear":
        return {"out": _exact_gated(c, a @ _exact_values(s["codes"], s["scales"], c["K"]).T)}
    rows, codes, scales, stride = _blob(c)
    pool, slots, ids = s["pool"], s["slots"].tolist(), s["ids"].long()
    out = torch.zeros((c["T"], c["k"], c["N"]), dtype=torch.float64, device=a.device)
    for e in range(c["E"]):
        at = (ids == e).nonzero()
        if at.shape[0]:
            blob = pool[slots[e]:slots[e] + stride]
            w = _exact_values(blob[:codes].view(rows, -1), blob[codes:codes + scales].view(rows, -1), c["K"])
            row = at[:, 0] * c["k"] + at[:, 1] if c["combine"] else at[:, 0]
            out[at[:, 0], at[:, 1]] = _exact_gated(c, a[row] @ w.T)
    return {"out": (s["w"].double()[..., None] * out).sum(1) if c["combine"] else out.view(-1, c["N"])}


def _exact_gated(c, y):
    return y if c["act"] == "none" else torch.sigmoid(y[..., :c["N"]]) * y[..., :c["N"]] * y[..., c["N"]:]


def _exact_route(c, x, bias):
    T, E = x.shape
    masked = np.isneginf(x)
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            score = np.where(x >= 0, 1 / (1 + np.exp(-x)), np.exp(x) / (1 + np.exp(x)))
        else:
            score = np.exp(x - x.max(1, keepdims=True))
            score = score / score.sum(1, keepdims=True)
    score[masked] = 0
    value = score if bias is None else score + bias
    key = np.where(masked, -np.inf, x if bias is None else value)
    kept = np.ones((T, E), dtype=bool)
    if c["groups"] > 1:
        each = E // c["groups"]
        v = -np.sort(-np.where(masked, -np.inf, value).reshape(T, c["groups"], each), axis=2)[:, :, :c["group_top"]]
        total = np.where(np.isneginf(v[:, :, 0]), -np.inf, np.where(np.isneginf(v), 0, v).sum(2))
        chosen = np.argsort(-total, axis=1, kind="stable")[:, :c["top_groups"]]
        group = np.zeros((T, c["groups"]), dtype=bool)
        np.put_along_axis(group, chosen, True, axis=1)
        kept = np.repeat(group, each, axis=1)
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -key, ~kept), axis=1)[:, :c["k"]]
    w = np.take_along_axis(score, ids, 1)
    if c["renorm"]:
        total = w.sum(1, keepdims=True)
        w = w / np.where(total == 0, 1, total)
    return {"ids": ids.astype(np.int32), "w": w * c["scale"]}
