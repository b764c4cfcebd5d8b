"""Measured cases of what stands between the projections and W_O in a block whose heads are normalised and rotated and
whose attention is windowed: the norm of each head of Q and K with the rotation by position (one or several axes), and
packed causal attention over a sliding window and each document's first tokens, both with their backward passes.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes a case's inputs from a
seed, ``run()`` is one pass: the operators' plain form in elementary torch operations, or (``own``) the calls a user
makes of the library.  ``exact()`` is the same from the definitions in 64 bits, ``work()`` what a pass cannot do without.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
DTYPES = {"bf16": BF16, "fp32": F32}
AXES = {"grid2": 2, "grid3": 3}            # of positions; else one


# ---------------------------------------------------------------------------------------------- cases

def _rotate(name, op, t, T, n_q, n_kv, d, rot=None, norm="bf16", place="docs", batch=1, pad=0, split=0,
            interleaved=False):
    """norm: the type of the heads' weights, or "none"; place: where positions come from -- "docs" (a token's place in
    its document), "far" (a stretch of one long text), "grid2" and "grid3" (text and images, an axis a coordinate)."""
    return {"name": name, "op": op, "t": t, "T": T, "n_q": n_q, "n_kv": n_kv, "d": d, "rot": d if rot is None else rot,
            "norm": norm, "place": place, "batch": batch, "pad": pad, "split": split, "interleaved": interleaved}


def _attn(name, op, t, T, n_q, n_kv, d, window, sinks, batch, pad=0, split=0):
    return {"name": name, "op": op, "t": t, "T": T, "n_q": n_q, "n_kv": n_kv, "d": d, "window": window, "sinks": sinks,
            "batch": batch, "pad": pad, "split": split}


def listed():
    return [
        # The toy block's heads (128 tokens, two shards, four short documents): launch latency.
        _rotate("rotate_fwd_small", "rotate_fwd", 2, 128, 4, 2, 64, batch=4, split=3),
        # The 8-shard block's heads over a pack of 12 documents: norm and rotation behind the projection.
        _rotate("rotate_fwd", "rotate_fwd", 8, 8192, 32, 8, 128, batch=12, split=1),
        # The backward pass of the same, with the gradients of the heads' weights.
        _rotate("rotate_bwd", "rotate_bwd", 8, 8192, 32, 8, 128, batch=12, split=1),
        # Image patches beside text, heads of 80, two axes, no norm: the rotation alone.
        _rotate("rotate_fwd_grid", "rotate_fwd", 4, 8192, 16, 16, 80, norm="none", place="grid2"),
        # A stretch far into one long text, an odd number of tokens, half of each head's columns rotated by
        # neighbouring pairs, weights in fp32.
        _rotate("rotate_bwd_far", "rotate_bwd", 1, 4099, 5, 5, 128, rot=64, norm="fp32", place="far", interleaved=True),
        # A few short documents, among them one of a single token, 64-wide heads: launch latency.
        _attn("window_fwd_small", "window_fwd", 2, 128, 4, 2, 64, 32, 4, 4, split=3),
        # The 8-shard block's heads over a pack of documents of uneven lengths, most longer than the window or near it.
        _attn("window_fwd_packed", "window_fwd", 8, 8192, 32, 8, 128, 1024, 4, 12, split=1),
        # The backward pass of the same.
        _attn("window_bwd_packed", "window_bwd", 8, 8192, 32, 8, 128, 1024, 4, 12, split=1),
        # Narrow layers of a model that alternates them with wide ones: one document, no sinks, 64-wide heads.
        _attn("window_fwd_narrow", "window_fwd", 4, 16384, 16, 4, 64, 128, 0, 1),
        # Their backward pass, with a window that no tile divides and a tail of no document.
        _attn("window_bwd_narrow", "window_bwd", 4, 8192, 16, 4, 64, 200, 16, 3, pad=100, split=5),
        # One shard's heads over one long document.
        _attn("window_fwd_long", "window_fwd", 1, 32768, 4, 1, 128, 4096, 4, 1),
        # The backward pass over half of its length, with a whole tile of sinks.
        _attn("window_bwd_long", "window_bwd", 1, 16384, 4, 1, 128, 2048, 128, 1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotate_fwd", "rotate_bwd", "window_fwd", "window_bwd"])
    t = rng.choice([1, 2, 4, 8])
    n_kv = t * rng.choice([1, 2]) if t < 8 else 8
    n_q = n_kv * rng.choice([1, 2, 3, 4, 8])
    n_q = n_q if n_q <= 32 else n_kv * 4
    if op.startswith("rotate"):
        d = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 256])
        T = _log(rng, 1, min(32768, 8192 * 40 * 128 // ((n_q + n_kv) * d)))
        place = rng.choice(["docs", "docs", "far", "grid2", "grid3"])
        return {"op": op, "t": t, "T": T, "n_q": n_q, "n_kv": n_kv, "d": d,
                "rot": rng.choice([d, d, d // 32 * 16, 16]), "norm": rng.choice(["none", "bf16", "bf16", "fp32"]),
                "place": place, "batch": _log(rng, 1, min(256, T)) if place == "docs" else 1,
                "pad": rng.choice([0, T // 7]) if place == "docs" else 0, "split": rng.randrange(1 << 20),
                "interleaved": rng.random() < 0.3}
    # (the gradients of documents of one token alone are zero: they say nothing about a backward pass)
    T = _log(rng, 1 if op == "window_fwd" else 16, 8192)
    batch = _log(rng, 1, max(1, min(256, T if op == "window_fwd" else T // 8)))
    return {"op": op, "t": t, "T": T, "n_q": n_q, "n_kv": n_kv, "d": rng.choice([64, 128]),
            "window": _log(rng, 1 if op == "window_fwd" else 2, 4096), "sinks": rng.choice([0, 0, 1, 4, 16, 64, 150]),
            "batch": batch, "pad": rng.choice([0, 0, T // 7]), "split": rng.randrange(1 << 20)}


def _lengths(case):
    """The documents' lengths: the used tokens cut at random places (empty documents occur)."""
    used = case["T"] - case["pad"]
    r = random.Random(case["split"])
    cuts = sorted(r.randint(0, used) for _ in range(case["batch"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [used])]


def _frequencies(case):
    """Radians a position for each pair of columns, and its axis: whole stretches of pairs an axis."""
    n = case["rot"] // 2
    axes = AXES.get(case["place"], 1)
    return [10000.0 ** (-i / n) for i in range(n)], [i * axes // n for i in range(n)]


def _grid(T, axes, seed):
    """Positions of text with images in it: a text token counts up on every axis; an image of height x width patches
    holds the time still and counts rows and columns from there."""
    r = random.Random(seed)
    out, at = [], 0
    while len(out) < T:
        for _ in range(r.randint(1, 200)):
            out.append((at,) * 3)
            at += 1
        height, width = r.randint(4, 32), r.randint(4, 32)
        out += [(at, at + i // width, at + i % width) for i in range(height * width)]
        at += max(height, width)
    return np.array(out[:T], dtype=np.int32).T[3 - axes:]


# ---------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))

    def randn(*shape, std=1.0, mean=0.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    t, T, d = case["t"], case["T"], case["d"]
    qc, kc = case["n_q"] // t * d, case["n_kv"] // t * d
    state = {"case": case}
    docs = torch.tensor(np.concatenate([[0], np.cumsum(_lengths(case))]), device="cuda", dtype=torch.int32)
    if case["op"].startswith("rotate"):
        # projections whose columns differ in size, as trained ones do
        column = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))

        def heads(cols):
            return [(randn(T, cols, dtype=F32) * column.repeat(cols // d)).to(BF16) for _ in range(t)]

        state["Q"], state["K"] = heads(qc), heads(kc)
        w = DTYPES.get(case["norm"])
        state["gamma_q"] = None if w is None else randn(d, std=0.1, mean=1.0, dtype=w)
        state["gamma_k"] = None if w is None else randn(d, std=0.1, mean=1.0, dtype=w)
        state["cu_seqlens"] = docs if case["place"] == "docs" else None
        state["positions"] = None
        if case["place"] == "far":
            start = random.Random(int(seed)).randrange(1 << 19, 1 << 20)
            state["positions"] = torch.arange(start, start + T, device="cuda", dtype=torch.int32)[None]
        elif case["place"] != "docs":
            state["positions"] = torch.from_numpy(_grid(T, AXES[case["place"]], int(seed)).copy()).cuda()
        if case["op"] == "rotate_bwd":
            state["dQ"] = [randn(T, qc, std=0.02) for _ in range(t)]
            state["dK"] = [randn(T, kc, std=0.02) for _ in range(t)]
        if own:
            import tensor_transformer_layer_way_gb300 as ttl
            freqs, axes = _frequencies(case)
            state["rotary"] = ttl.Rotary(freqs, axes=axes, interleaved=case["interleaved"])
        return state
    state["Q"] = [randn(T, qc) for _ in range(t)]
    state["K"] = [randn(T, kc) for _ in range(t)]
    state["V"] = [randn(T, kc) for _ in range(t)]
    state["cu_seqlens"] = docs
    if case["op"] == "window_bwd":
        state["dO"] = [randn(T, qc) for _ in range(t)]
        state["fwd"] = _window_fwd(state)
    return state


# ---------------------------------------------------------------------------------------------- plain forms

def _split(shards, d):
    """t shards [T, heads/t d] as [t, T, heads/t, d] in fp32."""
    return torch.stack(shards).float().unflatten(2, (-1, d))


def _join(x):
    return [s.flatten(1).to(BF16) for s in x]


def _angles(state):
    """cos and sin [T, rot/2] of each token's angles, which are taken in 64 bits, and the tokens that count."""
    case, T = state["case"], state["Q"][0].shape[0]
    freqs, axes = _frequencies(case)
    at = torch.arange(T, device="cuda")
    inside = torch.ones(T, device="cuda", dtype=torch.bool)
    if state["positions"] is not None:
        pos = state["positions"].long()
    else:
        cu = state["cu_seqlens"].long()
        doc = torch.searchsorted(cu, at, right=True)
        inside = at < cu[-1]
        pos = torch.where(inside, at - cu[doc - 1], 0)[None]
    angle = pos[axes].T.double() * torch.tensor(freqs, device="cuda", dtype=F64)
    return angle.cos().float(), angle.sin().float(), inside


def _turn(case, x, cos, sin):
    """The pairs of x's first rot columns turned by their angles."""
    rot, cos, sin = case["rot"], cos[:, None], sin[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rotate_fwd(state):
    case = state["case"]
    cos, sin, inside = _angles(state)
    out = {}
    for name in ("Q", "K"):
        x, gamma = _split(state[name], case["d"]), state["gamma_" + name.lower()]
        if gamma is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()
        out[name] = _join(_turn(case, x, cos, sin).masked_fill(~inside[:, None, None], 0.0))
    return out


def _rotate_bwd(state):
    case = state["case"]
    cos, sin, inside = _angles(state)
    out = {}
    for name in ("Q", "K"):
        gamma = state["gamma_" + name.lower()]
        dy = _split(state["d" + name], case["d"]).masked_fill(~inside[:, None, None], 0.0)
        dy = _turn(case, dy, cos, -sin)
        if gamma is not None:
            x = _split(state[name], case["d"])
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            n = x * r
            out["dgamma_" + name.lower()] = (dy * n).sum((0, 1, 2))
            dy = dy * gamma.float()
            dy = r * (dy - n * (dy * n).mean(-1, keepdim=True))
        out["d" + name] = _join(dy)
    return out


def _mask(state, T):
    """True where the query (row) sees the key (column), and the documents' tokens."""
    case, cu = state["case"], state["cu_seqlens"].long()
    at = torch.arange(T, device="cuda")
    doc = torch.searchsorted(cu, at, right=True)      # empty documents are passed over
    inside = at < cu[-1]
    first = cu[doc - 1]
    back = at[:, None] - at[None, :]
    seen = (back >= 0) & ((back < case["window"]) | (at - first < case["sinks"])[None, :])
    return seen & (doc[:, None] == doc[None, :]) & inside[:, None] & inside[None, :], inside


def _heads(shards, d):
    """t shards [T, heads/t d] as [heads, T, d] in fp32."""
    return _split(shards, d).transpose(1, 2).flatten(0, 1)


def _shards(x, t):
    """[heads, T, d] as t shards [T, heads/t d]."""
    return [s.transpose(0, 1).flatten(1).to(BF16) for s in x.chunk(t)]


def _window_fwd(state):
    case, T = state["case"], state["Q"][0].shape[0]
    t, d, grp = case["t"], case["d"], case["n_q"] // case["n_kv"]
    q, k, v = _heads(state["Q"], d), _heads(state["K"], d), _heads(state["V"], d)
    k, v = k.repeat_interleave(grp, 0), v.repeat_interleave(grp, 0)
    seen, inside = _mask(state, T)
    s = (q @ k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    m = s.amax(2, keepdim=True).masked_fill_(~inside[None, :, None], 0.0)
    p = s.sub_(m).exp_()
    l = p.sum(2, keepdim=True)
    o = (p @ v) / l.masked_fill(~inside[None, :, None], 1.0)
    lse = (m + l.log()).squeeze(2)                    # -inf for a token of no document
    return {"O": _shards(o, t), "lse": list(lse.chunk(t))}


def _window_bwd(state):
    case, T = state["case"], state["Q"][0].shape[0]
    t, d, grp = case["t"], case["d"], case["n_q"] // case["n_kv"]
    scale = 1.0 / math.sqrt(d)
    q, k, v = _heads(state["Q"], d), _heads(state["K"], d), _heads(state["V"], d)
    k, v = k.repeat_interleave(grp, 0), v.repeat_interleave(grp, 0)
    do, o = _heads(state["dO"], d), _heads(state["fwd"]["O"], d)
    seen, inside = _mask(state, T)
    lse = torch.cat(list(state["fwd"]["lse"])).masked_fill(~inside, 0.0)
    p = (q @ k.transpose(1, 2)).mul_(scale).sub_(lse[:, :, None]).exp_().masked_fill_(~seen, 0.0)
    dv = p.transpose(1, 2) @ do
    ds = (do @ v.transpose(1, 2)).sub_((do * o).sum(2, keepdim=True)).mul_(p).mul_(scale)
    dq, dk = ds @ k, ds.transpose(1, 2) @ q
    dk, dv = dk.unflatten(0, (-1, grp)).sum(1), dv.unflatten(0, (-1, grp)).sum(1)
    return {"dQ": _shards(dq, t), "dK": _shards(dk, t), "dV": _shards(dv, t)}


PLAIN = {"rotate_fwd": _rotate_fwd, "rotate_bwd": _rotate_bwd, "window_fwd": _window_fwd, "window_bwd": _window_bwd}


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return PLAIN[case["op"]](state)
    import tensor_transformer_layer_way_gb300 as ttl
    op, kept = case["op"], state.get("kept")           # the output and workspace buffers of an earlier pass
    shape = dict(n_q=case["n_q"], n_kv=case["n_kv"], d=case["d"])
    if op.startswith("rotate"):
        shape.update(gamma_q=state["gamma_q"], gamma_k=state["gamma_k"], eps=EPS, positions=state["positions"],
                     cu_seqlens=state["cu_seqlens"])
        if op == "rotate_fwd":
            out = ttl.head_norm_rotary_fwd(state["Q"], state["K"], state["rotary"], out=kept, **shape)
            names = ("Q", "K")
        else:
            normed = state["gamma_q"] is not None
            x = (state["Q"], state["K"]) if normed else (None, None)
            out = ttl.head_norm_rotary_bwd(state["dQ"], state["dK"], state["rotary"], Q=x[0], K=x[1], out=kept, **shape)
            names = ("dQ", "dK", "dgamma_q", "dgamma_k") if normed else ("dQ", "dK")
    else:
        shape.update(window=case["window"], sinks=case["sinks"])
        if op == "window_fwd":
            out = ttl.packed_window_attn_fwd(state["Q"], state["K"], state["V"], state["cu_seqlens"], out=kept, **shape)
            names = ("O", "lse")
        else:
            out = ttl.packed_window_attn_bwd(state["dO"], state["Q"], state["K"], state["V"], state["fwd"],
                                             state["cu_seqlens"], out=kept, **shape)
            names = ("dQ", "dK", "dV")
    state["kept"] = out
    return {n: out[n] for n in names}


def _pairs(case):
    """Pairs of a query and a key it sees, over all documents."""
    total = 0
    for n in _lengths(case):
        i = np.arange(1, n + 1, dtype=np.int64)        # keys up to the query
        near = np.minimum(i, case["window"])
        total += int((near + np.minimum(i - near, case["sinks"])).sum())
    return total


def work(case):
    T, n_q, n_kv, d = case["T"], case["n_q"], case["n_kv"], case["d"]
    if case["op"].startswith("rotate"):
        normed, size = case["norm"] != "none", T * (n_q + n_kv) * d
        where = 4 * (case["batch"] + 1) if case["place"] == "docs" else 4 * T * AXES.get(case["place"], 1)
        weights = 2 * d * (4 if case["norm"] == "fp32" else 2) if normed else 0
        if case["op"] == "rotate_fwd":
            return {"bytes": 4 * size + where + weights, "flops": size * (7 if normed else 3)}
        return {"bytes": size * (6 if normed else 4) + where + weights + (8 * d if normed else 0),
                "flops": size * (15 if normed else 3)}
    if case["op"] == "window_fwd":
        return {"bytes": 2 * T * d * (2 * n_q + 2 * n_kv) + 4 * T * n_q, "flops": 4 * d * n_q * _pairs(case)}
    return {"bytes": 2 * T * d * (4 * n_q + 4 * n_kv) + 4 * T * n_q, "flops": 10 * d * n_q * _pairs(case)}


# ---------------------------------------------------------------------------------------------- 64 bits

def _exact_rotate(case, state):
    T, d, rot = case["T"], case["d"], case["rot"]
    freqs, axes = _frequencies(case)
    if case["place"] == "docs":
        lengths = _lengths(case)
        place = [i for n in lengths for i in range(n)]
        counts = torch.tensor([1.0] * len(place) + [0.0] * (T - len(place)), device="cuda", dtype=F64)
        pos = torch.tensor([place + [0] * (T - len(place))], device="cuda", dtype=F64)
    else:
        counts, pos = torch.ones(T, device="cuda", dtype=F64), state["positions"].double()
    angle = torch.stack([pos[a] * f for a, f in zip(axes, freqs)], 1)
    turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)       # [T, 1, rot/2]
    lead = torch.arange(rot // 2, device="cuda")
    lead, second = (2 * lead, 2 * lead + 1) if case["interleaved"] else (lead, lead + rot // 2)

    def turned(x, by):
        z = torch.complex(x[..., lead], x[..., second]) * by
        y = x.clone()
        y[..., lead], y[..., second] = z.real, z.imag
        return y

    res = {}
    for name in ("Q", "K"):
        gamma = state["gamma_" + name.lower()]
        gamma = None if gamma is None else gamma.to(F64)
        outs, dgamma = [], 0.0
        for i in range(case["t"]):
            x = state[name][i].to(F64).view(T, -1, d)
            rms = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
            if case["op"] == "rotate_fwd":
                y = x if gamma is None else x / rms * gamma
                outs.append((turned(y, turn) * counts[:, None, None]).flatten(1))
                continue
            dy = turned(state["d" + name][i].to(F64).view(T, -1, d), turn.conj()) * counts[:, None, None]
            if gamma is not None:
                dgamma = dgamma + torch.einsum("thd,thd->d", dy, x / rms)
                dn = dy * gamma
                dy = dn / rms - x * (dn * x).sum(-1, keepdim=True) / (d * rms.pow(3))
            outs.append(dy.flatten(1))
        if case["op"] == "rotate_fwd":
            res[name] = outs
        else:
            res["d" + name] = outs
            if gamma is not None:
                res["dgamma_" + name.lower()] = dgamma
    return res


def exact(case, seed):
    state, t, T = prepare(case, seed), case["t"], case["T"]
    if case["op"].startswith("rotate"):
        return _exact_rotate(case, state)
    d, nql, grp = case["d"], case["n_q"] // t, case["n_q"] // case["n_kv"]
    W, S, rows = case["window"], case["sinks"], 2048
    scale = d ** -0.5
    res = {k: [] for k in ("O", "lse", "dQ", "dK", "dV")}
    for i in range(t):
        Q, K, V = (state[n][i].to(F64).view(T, -1, d) for n in ("Q", "K", "V"))
        O, lse = torch.zeros_like(Q), torch.full((nql, T), -math.inf, device="cuda", dtype=F64)
        dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
        dO = state["dO"][i].to(F64).view(T, -1, d) if case["op"] == "window_bwd" else None
        start = 0
        for n in _lengths(case):
            # rows [a, b) of the document against the keys that any of them sees
            for a in range(0, n, rows):
                b = min(n, a + rows)
                near = max(0, a - W + 1)
                key = torch.cat([torch.arange(min(S, near)), torch.arange(near, b)]).cuda()
                query = torch.arange(a, b, device="cuda")
                back = query[:, None] - key[None, :]
                hidden = (back < 0) | ((back >= W) & (key >= S)[None, :])
                key, query = key + start, query + start
                for g in range(K.shape[1]):
                    k, v = K[key, g], V[key, g]
                    for c in range(g * grp, (g + 1) * grp):
                        s = (Q[query, c] @ k.T * scale).masked_fill_(hidden, -math.inf)
                        lse[c, query] = torch.logsumexp(s, 1)
                        p = torch.softmax(s, 1)
                        if dO is None:
                            O[query, c] = p @ v
                            continue
                        go = dO[query, c]
                        dp = go @ v.T
                        ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                        dQ[query, c] = ds @ k
                        dV[key, g] += p.T @ go
                        dK[key, g] += ds.T @ Q[query, c]
            start += n
        for name, x in (("O", O), ("dQ", dQ), ("dK", dK), ("dV", dV)):
            res[name].append(x.flatten(1))
        res["lse"].append(lse)
    return {k: res[k] for k in (("O", "lse") if case["op"] == "window_fwd" else ("dQ", "dK", "dV"))}
