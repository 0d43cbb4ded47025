"""Token mixers of a hybrid stack: the gated delta rule over prompts, and attention over a paged cache with the norms,
rotation and append that come before it.

Gated delta rule over sequences of any length, packed one after the other (sequence b holds tokens cu[b] .. cu[b + 1]).
Per value head h, with the key head h // (nv / nk), state S [dv, dk]:
    k' = k / sqrt(sum k^2 + eps),  q' = q / sqrt(sum q^2 + eps) / sqrt(dk)
    S <- alpha S + beta (v - alpha S k') k'^T,   out = S q'
The states go in and come out in float32.

Append.  Per token, each head of q and k:
    x <- x / sqrt(mean x^2 + eps) * (offset + weight)     where the model normalises its heads
    the first R values rotated: pairs (i, i + R/2) ("half") or (2 i, 2 i + 1) ("adjacent") by the angle position * inv_freq[i]
q goes to its own tensor, k and v to the cache: pages [2, n_kv, page, D] (k, then v); token i of sequence b's n new ones is
number len[b] - n + i of the sequence, and number t of a sequence lies in page table[b, t // page] at t % page.

Attention.  New token i of sequence b sees the len[b] - n tokens before the new ones, and of the new ones those up to itself,
or with a tree those whose bit is set in its mask.  out = sum_j softmax_j(q k_j / sqrt(D)) v_j, query head h with the
key head h // (nq / nkv).
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a few new tokens of one conversation, longer than a handful: the shortest call
        dict(name="delta short turn", op="delta", nk=16, nv=32, dk=128, dv=128, B=1, least=24, most=24, state=True, dtype="bf16"),
        # one prompt
        dict(name="delta one prompt", op="delta", nk=16, nv=32, dk=128, dv=128, B=1, least=2048, most=2048, state=False, dtype="bf16"),
        # a narrow float32 layer, nothing a multiple of a tile, sequences of one token among longer ones
        dict(name="delta ragged float32", op="delta", nk=2, nv=4, dk=64, dv=48, B=7, least=1, most=701, state=True, dtype="f32"),
        # prompts of many users in one batch, some of them going on from a state
        dict(name="delta batch of prompts", op="delta", nk=16, nv=32, dk=128, dv=128, B=16, least=60, most=4000, state=True, dtype="bf16"),
        # one decoded token
        dict(name="append one token", op="append", nq=16, nkv=2, D=256, R=64, style="half", norm=True, page=64, B=1, new=1,
             least=4000, most=4000, fused=True, dtype="bf16"),
        # drafted tokens of a ragged batch in float32, whole heads rotated, adjacent pairs
        dict(name="append drafts float32", op="append", nq=32, nkv=8, D=128, R=128, style="adjacent", norm=False, page=16, B=33, new=7,
             least=10, most=5000, fused=False, dtype="f32"),
        # a long prompt
        dict(name="append prompt", op="append", nq=16, nkv=2, D=256, R=64, style="half", norm=True, page=64, B=1, new=16384,
             least=16384, most=16384, fused=True, dtype="bf16"),
        # one token of one conversation
        dict(name="attend one token", op="attend", nq=16, nkv=2, D=256, page=64, B=1, new=1, least=4000, most=4000, tree=False, dtype="bf16"),
        # a served batch, contexts from short to long
        dict(name="attend batch of tokens", op="attend", nq=16, nkv=2, D=256, page=64, B=64, new=1, least=100, most=32768, tree=False,
             dtype="bf16"),
        # trees of drafted tokens
        dict(name="attend drafted trees", op="attend", nq=32, nkv=8, D=128, page=16, B=8, new=31, least=500, most=9000, tree=True,
             dtype="bf16"),
        # a few new tokens of a small float32 model
        dict(name="attend ragged float32", op="attend", nq=12, nkv=4, D=64, page=32, B=5, new=77, least=77, most=1500, tree=False,
             dtype="f32"),
        # a prompt behind what is cached of it
        dict(name="attend prompt", op="attend", nq=16, nkv=2, D=256, page=64, B=1, new=8192, least=9001, most=9001, tree=False,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("delta", "append", "attend"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    B = _log(rng, 1, 32)
    if op == "delta":
        nk = rng.choice((1, 2, 4, 8, 16))
        most = _log(rng, 1, 2500)
        return dict(op=op, nk=nk, nv=nk * rng.choice((1, 2, 3)), dk=rng.choice((64, 128)), dv=16 * rng.randint(1, 12),
                    B=min(B, 16), least=_log(rng, 1, most), most=most, state=rng.random() < 0.6, dtype=dtype)
    nkv = rng.choice((1, 2, 4, 8))
    D = rng.choice((64, 128, 256))
    heads = dict(nq=nkv * rng.choice((1, 2, 3, 4, 6, 8)), nkv=nkv, D=D)
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        new = _log(rng, 1, 4096 // B)
        least = new + rng.choice((0, _log(rng, 1, 2000)))
        return dict(op=op, **heads, R=rng.choice((0, D // 4, D // 2, D - 2, D)), style=rng.choice(("half", "adjacent")),
                    norm=rng.random() < 0.6, page=page, B=B, new=new, least=least, most=least + rng.choice((0, _log(rng, 1, 3000))),
                    fused=rng.random() < 0.5, dtype=dtype)
    tree = rng.random() < 0.3
    new = _log(rng, 1, 64) if tree else rng.choice((1, _log(rng, 1, 2048)))
    B = min(B, max(1, 4096 // new))
    least = new + rng.choice((0, _log(rng, 1, 4000)))
    return dict(op=op, **heads, page=page, B=B, new=new, least=least, most=least + rng.choice((0, _log(rng, 1, 8000))), tree=tree,
                dtype=dtype)


def _lengths(c):
    """Tokens of each sequence, spread over the logarithm between the case's least and most, in an order of no meaning."""
    B, lo, hi = c["B"], c["least"], c["most"]
    at = [((7 * b + 3) % B) / max(B - 1, 1) if math.gcd(7, B) == 1 else b / max(B - 1, 1) for b in range(B)]
    return [int(round(lo * (hi / lo) ** a)) for a in at]


def work(c):
    lens = _lengths(c)
    item = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "delta":
        n, state = sum(lens), c["B"] * c["nv"] * c["dv"] * c["dk"] * 4
        return {"bytes": n * (2 * c["nk"] * c["dk"] + 2 * c["nv"] * c["dv"]) * item + 8 * n * c["nv"] + state * (2 if c["state"] else 1),
                "flops": 6 * n * c["nv"] * c["dv"] * c["dk"]}
    n = c["B"] * c["new"]
    if c["op"] == "append":
        return {"bytes": 2 * n * (c["nq"] + 2 * c["nkv"]) * c["D"] * item, "flops": 7 * n * (c["nq"] + c["nkv"]) * c["D"]}
    seen = sum(c["new"] * (t - c["new"]) + (c["new"] * (c["new"] + 1) // 2) for t in lens)
    return {"bytes": 2 * sum(lens) * c["nkv"] * c["D"] * item + 2 * n * c["nq"] * c["D"] * item, "flops": 4 * seen * c["nq"] * c["D"]}


# Inputs.

def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    dtype = TYPES[c["dtype"]]
    lens = _lengths(c)
    B = c["B"]
    s = {"case": c, "lens": lens}
    if c["op"] == "delta":
        n = sum(lens)
        s["cu"] = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device=DEV)
        s["q"], s["k"] = (normal(n, c["nk"], c["dk"]).to(dtype) for _ in range(2))
        # neighbouring keys of a text resemble one another
        s["k"][1:] = (0.8 * s["k"][1:].float() + 0.6 * s["k"][:-1].float()).to(dtype)
        s["v"] = normal(n, c["nv"], c["dv"]).to(dtype)
        # gates as exp(-rate softplus(x)), each head with a rate of its own; write strengths as sigmoids
        rate = torch.exp(2 * torch.rand((c["nv"],), generator=gen, device=DEV) - 3)
        s["alpha"] = torch.exp(-rate * torch.log1p(torch.exp(normal(n, c["nv"]))))
        s["beta"] = torch.sigmoid(normal(n, c["nv"]))
        shape = (B, c["nv"], c["dv"], c["dk"])
        s["state_in"] = 0.3 * normal(*shape) if c["state"] else None
        s["state_out"] = torch.empty(shape, dtype=torch.float32, device=DEV)
        s["out"] = torch.empty_like(s["v"])
        return s
    new, nq, nkv, D, page = c["new"], c["nq"], c["nkv"], c["D"], c["page"]
    n = B * new
    held = [-(-t // page) for t in lens]
    s["columns"] = max(held)
    s["n_pages"] = sum(held) + 3  # the pool has room for more
    order = torch.randperm(s["n_pages"], generator=gen, device=DEV).to(torch.int32)
    s["table"] = torch.zeros((B, s["columns"]), dtype=torch.int32, device=DEV)
    at = 0
    for b, h in enumerate(held):
        s["table"][b, :h] = order[at:at + h]
        at += h
    s["cu"] = torch.arange(B + 1, dtype=torch.int32, device=DEV) * new
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    # what is cached, and behind a sequence's last token what an earlier one left there
    s["pages"] = normal(s["n_pages"], 2, nkv, page, D).to(dtype)
    if c["op"] == "append":
        if c["fused"]:  # one product made q, k and v
            qkv = normal(n, (nq + 2 * nkv) * D).to(dtype)
            s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split((nq * D, nkv * D, nkv * D), dim=1))
        else:
            s["q"], s["k"], s["v"] = (normal(n, h, D).to(dtype) for h in (nq, nkv, nkv))
        s["q_norm"], s["k_norm"] = (0.2 * normal(D) if c["norm"] else None for _ in range(2))
        i = torch.arange(c["R"] // 2, dtype=torch.float64, device=DEV)
        s["inv_freq"] = (1e6 ** (-2 * i / c["R"])).float() if c["R"] else None
        s["positions"] = torch.cat([torch.arange(t - new, t, dtype=torch.int32, device=DEV) for t in lens])
        s["q_out"] = torch.empty((n, nq, D), dtype=dtype, device=DEV)
        return s
    s["q"] = (2 * normal(n, nq, D)).to(dtype)
    s["out"] = torch.empty_like(s["q"])
    s["tree"] = None
    if c["tree"]:  # every drafted token follows an earlier one, or the last token of the sequence
        rng = np.random.default_rng(int(seed))
        masks = np.zeros((B, new), dtype=np.uint64)
        for b in range(B):
            for i in range(new):
                parent = int(rng.integers(-1, i)) if i else -1
                masks[b, i] = np.uint64(1 << i) | (masks[b, parent] if parent >= 0 else np.uint64(0))
        s["tree"] = torch.from_numpy(masks.view(np.int64).reshape(-1)).to(DEV)
    return s


# What is computed: by the framework's operators, or in plain steps.

def run(s):
    c = s["case"]
    if own:
        return _own(c, s)
    return {"delta": _delta, "append": _append, "attend": _attend}[c["op"]](c, s)


def _own(c, s):
    import int4_quantized_expert_amd as M
    d = s.get("descriptor")
    if d is None:  # a program makes its descriptor and its workspace once
        d = s["descriptor"] = _descriptor(M, c, s)
        if c["op"] == "delta":
            size = M.gdn_chunk_workspace_bytes(d, c["B"], s["q"].shape[0])
        elif c["op"] == "attend":
            size = M.attn_workspace_bytes(d, c["B"], s["q"].shape[0], c["new"], max(s["lens"]))
        else:
            size = 0
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    if c["op"] == "delta":
        M.gdn_chunk_forward(d, c["B"], s["q"].shape[0], max(s["lens"]), s["cu"], s["q"], s["k"], s["v"], s["alpha"], s["beta"],
                            s["state_in"], s["state_out"], s["out"], s["ws"])
        return {"out": s["out"], "state": s["state_out"]}
    if c["op"] == "append":
        M.attn_append(d, c["B"], s["q"].shape[0], s["cu"], s["len"], s["table"], s["positions"], s["q"], s["k"], s["v"], s["q_norm"],
                      s["k_norm"], s["inv_freq"], s["q_out"], s["pages"])
        return {"q": s["q_out"], "pages": s["pages"]}
    M.attn_forward(d, c["B"], s["q"].shape[0], c["new"], max(s["lens"]), s["cu"], s["len"], s["table"], s["tree"], s["q"], s["pages"],
                   s["out"], s["ws"])
    return {"out": s["out"]}


def _descriptor(M, c, s):
    if c["op"] == "delta":
        return M.gdn_desc(c["nk"], c["nv"], c["dk"], c["dv"], act=c["dtype"], out=c["dtype"])
    more = dict(rotary_dim=c["R"], rotary=c["style"], norm_offset=1.0) if c["op"] == "append" else {}
    return M.attn_desc(c["nq"], c["nkv"], c["D"], page_size=c["page"], n_pages=s["n_pages"], max_pages=s["columns"], dtype=c["dtype"],
                       **more)


def _delta(c, s):
    """Token by token, all sequences at once; those that have ended keep their state."""
    B, T, each = c["B"], max(s["lens"]), c["nv"] // c["nk"]
    long = torch.arange(T, device=DEV)
    begin, end = s["cu"][:-1].long(), s["cu"][1:].long()
    at = (begin[:, None] + long).clamp_max(s["q"].shape[0] - 1)
    live = begin[:, None] + long < end[:, None]

    def unit(x):
        x = x.float()
        return (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(each, dim=1)

    q = unit(s["q"])[at] / math.sqrt(c["dk"])
    k = unit(s["k"])[at]
    v = s["v"].float()[at]
    alpha = torch.where(live[..., None], s["alpha"][at], 1.0)
    beta = torch.where(live[..., None], s["beta"][at], 0.0)
    shape = (B, c["nv"], c["dv"], c["dk"])
    S = torch.zeros(shape, device=DEV) if s["state_in"] is None else s["state_in"].clone()
    out = torch.empty((B, T, c["nv"], c["dv"]), device=DEV)
    for t in range(T):
        kt = k[:, t]
        S *= alpha[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.matmul(S, kt[..., None])[..., 0])
        S += u[..., None] * kt[..., None, :]
        out[:, t] = torch.matmul(S, q[:, t, :, :, None])[..., 0]
    return {"out": out[live].to(s["out"].dtype), "state": S}


def _places(c, s):
    """Page and place in it of every new token."""
    new = torch.arange(c["new"], device=DEV)
    t = s["len"].long()[:, None] - c["new"] + new
    return s["table"].long().gather(1, t // c["page"]).view(-1), (t % c["page"]).view(-1)


def _rotate(c, s, x, weight):
    x = x.float()
    if c["norm"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (1 + weight)
    R = c["R"]
    if R == 0:
        return x
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()  # far positions: 32 bits lose the angle
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.clone()
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if c["style"] == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    first, second = a * cos - b * sin, b * cos + a * sin
    if c["style"] == "half":
        y[..., :R // 2], y[..., R // 2:R] = first, second
    else:
        y[..., 0:R:2], y[..., 1:R:2] = first, second
    return y


def _append(c, s):
    dtype = s["pages"].dtype
    page, place = _places(c, s)
    s["pages"][page, 0, :, place] = _rotate(c, s, s["k"], s["k_norm"]).to(dtype)
    s["pages"][page, 1, :, place] = s["v"]
    return {"q": _rotate(c, s, s["q"], s["q_norm"]).to(dtype), "pages": s["pages"]}


def _attend(c, s):
    new, nkv, D, each = c["new"], c["nkv"], c["D"], c["nq"] // c["nkv"]
    out = torch.empty(s["q"].shape, device=DEV)
    for b, t in enumerate(s["lens"]):
        held = s["pages"][s["table"][b, :-(-t // c["page"])].long()].float()
        k, v = (held[:, x].transpose(0, 1).reshape(nkv, -1, D)[:, :t] for x in (0, 1))
        k = k.transpose(1, 2).contiguous()
        v = v.contiguous()
        key = torch.arange(t, device=DEV) - (t - new)
        for i in range(0, new, 1024):
            rows = min(1024, new - i)
            q = s["q"][b * new + i:b * new + i + rows].float().view(rows, nkv, each, D).permute(1, 2, 0, 3).reshape(nkv, each * rows, D)
            if s["tree"] is None:
                sees = key <= torch.arange(i, i + rows, device=DEV)[:, None]
            else:
                mask = s["tree"][b * new + i:b * new + i + rows, None]
                sees = (key < 0) | ((mask >> key.clamp_min(0)) & 1).bool()
            x = torch.matmul(q, k).view(nkv, each, rows, t) / math.sqrt(D)
            x = x.masked_fill(~sees, float("-inf"))
            e = torch.exp(x - x.amax(-1, keepdim=True))
            y = torch.matmul(e.view(nkv, each * rows, t), v).view(nkv, each, rows, D) / e.sum(-1, keepdim=True)
            out[b * new + i:b * new + i + rows] = y.permute(2, 0, 1, 3).reshape(rows, -1, D)
    return {"out": out.to(s["out"].dtype)}


# The definition in 64 bits.

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"delta": _exact_delta, "append": _exact_append, "attend": _exact_attend}[c["op"]](c, s)


def _exact_delta(c, s):
    """The tokens of 32 at a time as one triangular system: with u_i = beta_i (v_i - alpha_i S_{i-1} k_i), every state within them is
    the first one, decayed, plus sum_j u_j k_j^T, each decayed since its token."""
    each = c["nv"] // c["nk"]
    q, k, v, alpha, beta = (s[x].double() for x in ("q", "k", "v", "alpha", "beta"))
    q, k = (torch.nn.functional.normalize(torch.cat((x, torch.full_like(x[..., :1], 1e-3)), -1), dim=-1, eps=0.0)[..., :-1] for x in (q, k))
    q, k = (x.repeat_interleave(each, dim=1).transpose(0, 1) for x in (q / c["dk"] ** 0.5, k))  # [heads, tokens, dk]
    v, alpha, beta = v.transpose(0, 1), alpha.T, beta.T
    out = torch.empty_like(v)
    states = []
    at = 0
    for b, n in enumerate(s["lens"]):
        S = torch.zeros(c["nv"], c["dk"], c["dv"], dtype=torch.float64, device=v.device)
        if s["state_in"] is not None:
            S += s["state_in"][b].double().transpose(1, 2)
        for i in range(at, at + n, 32):
            j = min(i + 32, at + n)
            ki, qi, bi = k[:, i:j], q[:, i:j], beta[:, i:j, None]
            since = torch.cumsum(torch.log(alpha[:, i:j]), dim=1)
            decay = torch.exp((since[:, :, None] - since[:, None, :]).tril())
            first = torch.exp(since)[..., None]
            near = torch.matmul(ki, ki.transpose(1, 2).contiguous()) * decay
            system = torch.eye(j - i, dtype=torch.float64, device=v.device) + bi * near.tril(-1)
            u = torch.linalg.solve_triangular(system, bi * (v[:, i:j] - first * torch.matmul(ki, S)), upper=False, unitriangular=True)
            seen = (torch.matmul(qi, ki.transpose(1, 2).contiguous()) * decay).tril()
            out[:, i:j] = first * torch.matmul(qi, S) + torch.matmul(seen, u)
            S = first[:, -1:] * S + torch.matmul(ki.transpose(1, 2).contiguous(), decay[:, -1, :, None] * u)
        states.append(S.transpose(1, 2))
        at += n
    return {"out": out.transpose(0, 1), "state": torch.stack(states)}


def _exact_append(c, s):
    n, D, R = s["q"].shape[0], c["D"], c["R"]
    pos = s["positions"].double()

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * (weight.double() + 1)
        if R == 0:
            return x
        turn = torch.polar(torch.ones((n, R // 2), dtype=torch.float64, device=x.device), pos[:, None] * s["inv_freq"].double())[:, None]
        pairs = x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["style"] == "half" else x[..., :R].unflatten(-1, (R // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2) if c["style"] == "half" else z
        return torch.cat((z.flatten(-2), x[..., R:]), -1)

    pages = s["pages"].double()
    k, v = turned(s["k"], s["k_norm"]), s["v"].double()
    table = s["table"].tolist()
    page, place = [], []
    for b, t in enumerate(s["lens"]):
        for number in range(t - c["new"], t):
            page.append(table[b][number // c["page"]])
            place.append(number % c["page"])
    page, place = torch.tensor(page, device=DEV), torch.tensor(place, device=DEV)
    pages[page, 0, :, place] = k
    pages[page, 1, :, place] = v
    return {"q": turned(s["q"], s["q_norm"]), "pages": pages}


def _exact_attend(c, s):
    new, each = c["new"], c["nq"] // c["nkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, t in enumerate(s["lens"]):
        number = torch.arange(t, device=DEV)
        page, place = s["table"][b].long()[number // c["page"]], number % c["page"]
        before = t - new
        sees = torch.ones((new, t), dtype=torch.bool, device=DEV)
        if s["tree"] is None:
            sees[:, before:] = torch.ones((new, new), dtype=torch.bool, device=DEV).tril()
        else:
            masks = [int(m) for m in s["tree"][b * new:(b + 1) * new].tolist()]
            sees[:, before:] = torch.tensor([[(m >> j) & 1 == 1 for j in range(new)] for m in masks], device=DEV)
        for h in range(c["nq"]):
            k, v = (s["pages"][page, x, h // each, place].double() for x in (0, 1))
            w = (s["q"][b * new:(b + 1) * new, h].double() @ k.T) * c["D"] ** -0.5
            w = torch.softmax(torch.where(sees, w, -torch.inf), dim=-1)
            out[b * new:(b + 1) * new, h] = w @ v
    return {"out": out}
