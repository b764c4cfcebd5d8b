"""Measured cases of the operators of one training step on packed documents: the layer norm over token slabs, the
scaled vocab-parallel embedding with its gradient by sorted tokens, and packed causal attention with grouped heads.

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

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
DTYPES = {"bf16": BF16, "fp32": F32}


# ---------------------------------------------------------------------------------------------- cases

def _norm(name, op, t, T, h, dtype="bf16", wdtype="bf16", residual=True):
    return {"name": name, "op": op, "t": t, "T": T, "h": h, "dtype": dtype, "wdtype": wdtype, "residual": residual}


def _embed(name, op, t, T, h, V, ids="zipf"):
    return {"name": name, "op": op, "t": t, "T": T, "h": h, "V": V, "ids": ids}


def _attn(name, op, t, T, n_q, n_kv, d, batch, pad=0, split=0):
    return {"name": name, "op": op, "t": t, "T": T, "n_q": n_q, "n_kv": n_kv, "d": d, "batch": batch, "pad": pad,
            "split": split}


def listed():
    return [
        # The norm in front of the toy block (h = 256, 128 tokens, two slabs): launch latency.
        _norm("norm_fwd_small", "norm_fwd", 2, 128, 256, residual=False),
        # The norm between attention and MLP of the 8-shard block: residual sum and norm in one pass.
        _norm("norm_fwd_residual", "norm_fwd", 8, 8192, 4096),
        # Its backward: the gradient that passes the block is added, the weight gradients are reduced over all slabs.
        _norm("norm_bwd_residual", "norm_bwd", 8, 8192, 4096),
        # A model kept in fp32 with sizes that fit no vector width.
        _norm("norm_bwd_odd_fp32", "norm_bwd", 1, 4099, 1001, "fp32", "fp32", False),
        # The lookup in front of the 8-shard model: every shard gets all tokens' scaled rows.
        _embed("embed_fwd", "embed_fwd", 8, 8192, 4096, 151936),
        # The toy model's gradient: few tokens, small table, launch latency.
        _embed("embed_bwd_small", "embed_bwd", 2, 128, 256, 2048, "uniform"),
        # A fresh table gradient of the 8-shard model: every row is written once.
        _embed("embed_bwd", "embed_bwd", 8, 8192, 4096, 151936),
        # One shard's table with half of the tokens the same padding id: one long sum.
        _embed("embed_bwd_padded", "embed_bwd", 1, 8192, 4096, 18992, "padded"),
        # A few short documents, among them one of a single token, 64-wide heads: launch latency.
        _attn("attn_fwd_small", "attn_fwd", 2, 128, 4, 2, 64, 4, split=3),
        # The 8-shard block's heads over a pack of documents of uneven lengths.
        _attn("attn_fwd_packed", "attn_fwd", 8, 8192, 32, 8, 128, 12, split=1),
        # The backward pass of the same.
        _attn("attn_bwd_packed", "attn_bwd", 8, 8192, 32, 8, 128, 12, split=1),
        # One shard's heads over one document four times as long.
        _attn("attn_fwd_long", "attn_fwd", 1, 32768, 4, 1, 128, 1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd", "attn_fwd", "attn_bwd"])
    t = rng.choice([1, 2, 4, 8])
    if op.startswith("norm"):
        h = _log(rng, 64, 12288)
        if rng.random() < 0.6:
            h = max(64, h // 8 * 8)
        T = _log(rng, 1, min(32768, 8192 * 4096 // h) // t) * t
        return {"op": op, "t": t, "T": T, "h": h, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "wdtype": rng.choice(["bf16", "fp32"]), "residual": rng.random() < 0.5}
    if op.startswith("embed"):
        h = _log(rng, 64, 8192) // 8 * 8
        V = _log(rng, 100, min(200000, 151936 * 4096 // h) // t) * t
        T = _log(rng, 1, min(32768, 8192 * 4096 // h))
        return {"op": op, "t": t, "T": T, "h": h, "V": V, "ids": rng.choice(["zipf", "uniform", "padded"])}
    n_kv = t * rng.choice([1, 2]) if t < 8 else 8
    n_q = n_kv * rng.choice([1, 2, 3, 4, 8])
    n_q = n_q if n_q <= 32 else n_kv * 4
    # (the gradients of documents of one token alone are zero: they say nothing about a backward pass)
    T = _log(rng, 1 if op == "attn_fwd" else 16, 8192)
    batch = _log(rng, 1, max(1, min(256, T if op == "attn_fwd" else T // 8)))
    return {"op": op, "t": t, "T": T, "n_q": n_q, "n_kv": n_kv, "d": rng.choice([64, 128]), "batch": batch,
            "pad": rng.choice([0, 0, T // 7]), "split": rng.randrange(1 << 20)}


def _lengths(case):
    """The documents' lengths: the used tokens cut at random places (empty documents occur)."""
    used = case["T"] - case["pad"]
    r = random.Random(case["split"])
    cuts = sorted(r.randint(0, used) for _ in range(case["batch"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [used])]


# ---------------------------------------------------------------------------------------------- inputs

def _probabilities(case):
    V = case["V"]
    if case["ids"] == "uniform":
        return np.full(V, 1.0 / V)
    p = 1.0 / (np.arange(V) + 1.0)     # words by rank
    p /= p.sum()
    if case["ids"] == "padded":
        p *= 0.5
        p[0] += 0.5
    return p


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))

    def randn(*shape, std=1.0, mean=0.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    t, T = case["t"], case["T"]
    state = {"case": case}
    if case["op"].startswith("norm"):
        h, dt, wt, slab = case["h"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]], T // t
        # a residual stream: some channels are much larger than the others
        channel = torch.where(torch.rand(h, generator=g, device="cuda") < 0.01, 16.0, 1.0)
        state["X"] = [(randn(slab, h, dtype=F32) * channel + 0.1).to(dt) for _ in range(t)]
        state["gamma"] = randn(h, std=0.1, mean=1.0, dtype=wt)
        if case["op"] == "norm_fwd":
            state["beta"] = randn(h, std=0.1, dtype=wt)
            state["residual"] = [randn(slab, h, dtype=dt) for _ in range(t)] if case["residual"] else None
        else:
            state["dY"] = [randn(slab, h, std=0.02, dtype=dt) for _ in range(t)]
            state["dS"] = [randn(slab, h, std=0.02, dtype=dt) for _ in range(t)] if case["residual"] else None
            x = [x.float() for x in state["X"]]
            mean = [v.mean(1) for v in x]
            rstd = [torch.rsqrt((v - m[:, None]).square().mean(1) + EPS) for v, m in zip(x, mean)]
            state["fwd"] = {"mean": mean, "rstd": rstd}
    elif case["op"].startswith("embed"):
        h, V = case["h"], case["V"]
        r = np.random.RandomState(int(seed) % (1 << 32))
        rank = np.searchsorted(np.cumsum(_probabilities(case)), r.random_sample(T)).clip(0, V - 1)
        state["ids"] = torch.from_numpy(r.permutation(V)[rank]).to("cuda", torch.int64)
        if case["op"] == "embed_fwd":
            state["E"] = [randn(V // t, h, std=0.02) for _ in range(t)]
        else:
            state["dY"] = randn(T, h, std=0.02)
            state["dE"] = [torch.empty(V // t, h, device="cuda", dtype=F32) for _ in range(t)]
        state["scale"] = math.sqrt(h)
    else:
        d, qc, kc = case["d"], case["n_q"] // t * case["d"], case["n_kv"] // t * case["d"]
        state["Q"] = [randn(T, qc) for _ in range(t)]
        state["K"] = [randn(T, kc) for _ in range(t)]
        state["V"] = [randn(T, kc) for _ in range(t)]
        state["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(_lengths(case))]), device="cuda",
                                           dtype=torch.int32)
        if case["op"] == "attn_bwd":
            state["dO"] = [randn(T, qc) for _ in range(t)]
            state["fwd"] = _attn_fwd(state)
    return state


# ---------------------------------------------------------------------------------------------- plain forms

def _norm_fwd(state):
    dt, slab = state["X"][0].dtype, state["X"][0].shape[0]
    x = torch.cat(state["X"]).float()
    if state["residual"] is not None:
        x = (x + torch.cat(state["residual"]).float()).to(dt).float()   # the sum is kept in the stream's type
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS)
    y = (c * rstd[:, None] * state["gamma"].float() + state["beta"].float()).to(dt)
    out = {"Y": y.split(slab), "mean": mean.split(slab), "rstd": rstd.split(slab)}
    if state["residual"] is not None:
        out["S"] = x.to(dt).split(slab)
    return out


def _norm_bwd(state):
    dt, slab = state["X"][0].dtype, state["X"][0].shape[0]
    x, dy = torch.cat(state["X"]).float(), torch.cat(state["dY"]).float()
    mean, rstd = torch.cat(state["fwd"]["mean"]), torch.cat(state["fwd"]["rstd"])
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * state["gamma"].float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    if state["dS"] is not None:
        dx = dx + torch.cat(state["dS"]).float()
    return {"dX": dx.to(dt).split(slab), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _embed_fwd(state):
    ids, E = state["ids"], state["E"]
    Vs, t = E[0].shape[0], len(E)
    local = [ids - i * Vs for i in range(t)]
    rows = [torch.where(((k >= 0) & (k < Vs))[:, None], e[k.clamp(0, Vs - 1)], torch.zeros((), device="cuda", dtype=BF16))
            for k, e in zip(local, E)]
    y = (sum(r.float() for r in rows) * state["scale"]).to(BF16)
    return {"out": [y.clone() for _ in range(t)]}


def _embed_bwd(state):
    ids, dE = state["ids"], state["dE"]
    Vs, t = dE[0].shape[0], len(dE)
    g = state["dY"].float() * state["scale"]
    full = torch.zeros(Vs * t, g.shape[1], device="cuda").index_add_(0, ids, g)
    return {"dE": full.split(Vs)}


def _mask(state, T):
    """True where the key (column) belongs to the query's document and is not after it; and the documents' tokens."""
    cu = state["cu_seqlens"].long()
    at = torch.arange(T, device="cuda")
    doc = torch.searchsorted(cu, at, right=True)      # empty documents are passed over
    inside = at < cu[-1]
    return (doc[:, None] == doc[None, :]) & (at[:, None] >= at[None, :]) & inside[:, None] & inside[None, :], inside


def _heads(shards, d):
    """t shards [T, heads/t d] as [heads, T, d] in fp32."""
    x = torch.stack(shards).float()
    return x.unflatten(2, (-1, d)).transpose(1, 2).flatten(0, 1)


def _shards(x, t, dtype=BF16):
    """[heads, T, d] as t shards [T, heads/t d]."""
    return [s.transpose(0, 1).flatten(1).to(dtype) for s in x.chunk(t)]


def _attn_fwd(state):
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


def _attn_bwd(state):
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


PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd,
         "attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd}


# ---------------------------------------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if not own:
        return PLAIN[case["op"]](state)
    import tensor_transformer_layer_way_gb300 as ttl
    op, kept = case["op"], state.get("kept")           # the output and workspace buffers of an earlier pass
    if op == "norm_fwd":
        out = ttl.layer_norm_fwd(state["X"], state["gamma"], state["beta"], eps=EPS, residual=state["residual"],
                                 out=kept)
        names = ("Y", "S", "mean", "rstd") if case["residual"] else ("Y", "mean", "rstd")
    elif op == "norm_bwd":
        out = ttl.layer_norm_bwd(state["X"], state["dY"], state["gamma"], state["fwd"], dS=state["dS"], out=kept)
        names = ("dX", "dgamma", "dbeta")
    elif op == "embed_fwd":
        out = {"out": ttl.vocab_parallel_embedding_scaled_fwd(state["ids"], state["E"], state["scale"],
                                                              out=kept["out"] if kept else None)}
        names = ("out",)
    elif op == "embed_bwd":
        out = kept or {"dE": state["dE"], "ws": ttl.embedding_sorted_bwd_workspace(
            case["t"], case["T"], case["h"], case["V"])}
        ttl.vocab_parallel_embedding_sorted_bwd(state["ids"], state["dY"], state["scale"], out["dE"], ws=out["ws"])
        names = ("dE",)
    else:
        shape = dict(n_q=case["n_q"], n_kv=case["n_kv"], d=case["d"])
        if op == "attn_fwd":
            out = ttl.packed_attn_fwd(state["Q"], state["K"], state["V"], state["cu_seqlens"], out=kept, **shape)
            names = ("O", "lse")
        else:
            out = ttl.packed_attn_bwd(state["dO"], state["Q"], state["K"], state["V"], state["fwd"],
                                      state["cu_seqlens"], out=kept, **shape)
            names = ("dQ", "dK", "dV")
    state["kept"] = out
    return {n: out[n] for n in names}


def work(case):
    T, t = case["T"], case["t"]
    if case["op"].startswith("norm"):
        h, b, w = case["h"], 2 if case["dtype"] == "bf16" else 4, 2 if case["wdtype"] == "bf16" else 4
        if case["op"] == "norm_fwd":
            return {"bytes": T * h * b * (4 if case["residual"] else 2) + 8 * T + 2 * h * w, "flops": 8 * T * h}
        return {"bytes": T * h * b * (4 if case["residual"] else 3) + 8 * T + h * w + 8 * h, "flops": 14 * T * h}
    if case["op"].startswith("embed"):
        h, V = case["h"], case["V"]
        if case["op"] == "embed_fwd":
            rows = float((1.0 - (1.0 - _probabilities(case)) ** T).sum())     # distinct rows expected
            return {"bytes": 8 * T + 2 * h * (rows + t * T), "flops": T * h}
        return {"bytes": 8 * T + 2 * T * h + 4 * V * h, "flops": 2 * T * h}
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
    if case["op"] == "attn_fwd":
        return {"bytes": 2 * T * d * (2 * n_q + 2 * n_kv) + 4 * T * n_q, "flops": 4 * d * n_q * pairs}
    return {"bytes": 2 * T * d * (4 * n_q + 4 * n_kv) + 4 * T * n_q, "flops": 10 * d * n_q * pairs}


# ---------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    state, t, T = prepare(case, seed), case["t"], case["T"]
    f8 = torch.float64
    if case["op"].startswith("norm"):
        res = {"Y": [], "S": [], "mean": [], "rstd": [], "dX": []}
        gamma = state["gamma"].to(f8)
        dgamma, dbeta = torch.zeros_like(gamma), torch.zeros_like(gamma)
        for i in range(t):
            x = state["X"][i].to(f8)
            if case["op"] == "norm_fwd" and case["residual"]:
                x = (x + state["residual"][i].to(f8)).to(state["X"][i].dtype).to(f8)
                res["S"].append(x)
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = (var + EPS) ** -0.5
            n = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
            if case["op"] == "norm_fwd":
                res["Y"].append(n * gamma + state["beta"].to(f8))
                res["mean"].append(mean)
                res["rstd"].append(rstd)
                continue
            dy = state["dY"][i].to(f8)
            dn = dy * gamma
            dx = (dn - dn.mean(1, True) - n * (dn * n).mean(1, True)) * rstd.unsqueeze(1)
            res["dX"].append(dx if state["dS"] is None else dx + state["dS"][i].to(f8))
            dgamma += torch.einsum("th,th->h", dy, n)
            dbeta += dy.sum(0)
        if case["op"] == "norm_bwd":
            return {"dX": res["dX"], "dgamma": dgamma, "dbeta": dbeta}
        return {k: v for k, v in res.items() if v}
    if case["op"] == "embed_fwd":
        y = torch.cat(state["E"]).index_select(0, state["ids"]).to(f8) * state["scale"]
        return {"out": [y] * t}
    if case["op"] == "embed_bwd":
        # rows sorted by id, prefix sums of a run's rows
        ids, order = torch.sort(state["ids"], stable=True)
        rows = state["dY"].to(f8)[order] * state["scale"]
        which, counts = torch.unique_consecutive(ids, return_counts=True)
        ends = torch.cumsum(counts, 0)
        total = torch.cat([torch.zeros_like(rows[:1]), torch.cumsum(rows, 0)])
        dE = torch.zeros(case["V"], case["h"], device="cuda", dtype=f8)
        dE[which] = total[ends] - total[ends - counts]
        return {"dE": list(dE.chunk(t))}
    d, nql, nkl, grp = case["d"], case["n_q"] // t, case["n_kv"] // t, case["n_q"] // case["n_kv"]
    scale = d ** -0.5
    res = {k: [] for k in ("O", "lse", "dQ", "dK", "dV")}
    for i in range(t):
        Q, K, V = (state[n][i].to(f8).view(T, -1, d) for n in ("Q", "K", "V"))
        O, lse = torch.zeros_like(Q), torch.full((nql, T), -math.inf, device="cuda", dtype=f8)
        dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
        dO = state["dO"][i].to(f8).view(T, -1, d) if case["op"] == "attn_bwd" else None
        at = 0
        for n in _lengths(case):
            if n == 0:
                continue
            r = slice(at, at + n)
            at += n
            after = torch.ones(n, n, device="cuda", dtype=torch.bool).triu_(1)
            for c in range(nql):
                g = c // grp
                s = (Q[r, c] @ K[r, g].T * scale).masked_fill_(after, -math.inf)
                lse[c, r] = torch.logsumexp(s, 1)
                p = torch.softmax(s, 1)
                if dO is None:
                    O[r, c] = p @ V[r, g]
                    continue
                dp = dO[r, c] @ V[r, g].T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                dV[r, g] += p.T @ dO[r, c]
                dQ[r, c] = ds @ K[r, g]
                dK[r, g] += ds.T @ Q[r, c]
        for k, x in (("O", O), ("dQ", dQ), ("dK", dK), ("dV", dV)):
            res[k].append(x.flatten(1))
        res["lse"].append(lse)
    return {k: res[k] for k in (("O", "lse") if case["op"] == "attn_fwd" else ("dQ", "dK", "dV"))}
