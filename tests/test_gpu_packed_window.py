"""Packed causal attention over a sliding window and each document's first tokens vs a plain 64-bit implementation (GPU).

Bounds, per element.  The probabilities and the score gradients are rounded to bf16 once before their product (half
a step, 2^-8, of each term), the result once more; scores and statistics are fp32.  Hence
  |O - o|    <= 2^-8 (sum p |v| + |o|),         |dV - dv| <= 2^-8 (sum p |do| + |dv|)
  |dQ - dq|  <= 2^-8 (sum |ds k| + |dq|),       |dK - dk| <= 2^-8 (sum |ds q| + |dk|)
plus the fp32 part: a score is off by at most 2 d u sum |q k| (u = 2^-24) and a few u of the exponential, which moves
every probability, and p (dp - D), by that factor.  The backward reference takes the kernels' O and lse.
"""
import math
import random

import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
F8, BF16 = torch.float64, torch.bfloat16


def _inputs(t, T, n_q, n_kv, d, lens, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)

    def mats(cols, s=1.0):
        return [(torch.randn(T, cols, generator=g) * s).to(BF16).cuda() for _ in range(t)]

    qc, kc = n_q // t * d, n_kv // t * d
    x = {"Q": mats(qc, std), "K": mats(kc, std), "V": mats(kc), "dO": mats(qc)}
    x["cu"] = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()
    return x


def _see(n, W, S):
    """What each query of a document of n tokens sees."""
    i = torch.arange(n, device="cuda")
    back = i[:, None] - i[None, :]
    return (back >= 0) & ((back < W) | (i < S)[None, :])


def _reference(x, t, n_q, n_kv, d, lens, W, S, scale, fwd=None):
    """Per shard: O, lse and (with fwd) dQ, dK, dV, each with its bound."""
    grp, nql, nkl = n_q // n_kv, n_q // t, n_kv // t
    out = []
    for i in range(t):
        T = x["Q"][i].shape[0]
        q, k, v, do = (x[n][i].to(F8).view(T, -1, d) for n in ("Q", "K", "V", "dO"))
        z = lambda h: torch.zeros(T, h, d, dtype=F8, device="cuda")   # noqa: E731
        r = {"O": z(nql), "dO": z(nql), "lse": torch.full((nql, T), -math.inf, dtype=F8, device="cuda"),
             "dlse": torch.zeros(nql, T, dtype=F8, device="cuda"), "dQ": z(nql), "eQ": z(nql), "dK": z(nkl),
             "eK": z(nkl), "dV": z(nkl), "eV": z(nkl)}
        a = 0
        for n in lens:
            s_ = slice(a, a + n)
            a += n
            if n == 0:
                continue
            hide = ~_see(n, W, S)
            for c in range(nql):
                g = c // grp
                qq, kk, vv, gg = q[s_, c], k[s_, g], v[s_, g], do[s_, c]
                s = (scale * qq @ kk.T).masked_fill(hide, -math.inf)
                e = (scale * 2 * d * U * qq.abs() @ kk.abs().T + 16 * U * (1 + s.abs())).masked_fill(hide, 0.0)
                lse = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[:, None])
                es = e.amax(1, keepdim=True) * 2 + n * U           # factor on the row's probabilities
                r["lse"][c, s_] = lse
                r["dlse"][c, s_] = es[:, 0] + 4 * U * lse.abs()
                o, mag = p @ vv, p @ vv.abs()
                r["O"][s_, c] = o
                r["dO"][s_, c] = HALF * (mag + o.abs()) * 1.02 + es * mag * 2
                if fwd is None:
                    continue
                oo = fwd["O"][i].to(F8).view(T, -1, d)[s_, c]
                ll = fwd["lse"][i][c, s_].to(F8)
                p = torch.exp(s - ll[:, None])
                ep = (e + 8 * U * (1 + ll.abs()[:, None])).masked_fill(hide, 0.0)
                dp, D = gg @ vv.T, (gg * oo).sum(1, keepdim=True)
                ds = scale * p * (dp - D)
                eds = scale * p * (ep * (dp - D).abs() + 2 * d * U * (gg.abs() @ vv.abs().T + (gg * oo).abs().sum(1, keepdim=True)))
                r["dQ"][s_, c] = ds @ kk
                r["eQ"][s_, c] = HALF * 1.02 * (ds.abs() @ kk.abs()) + 1.02 * eds @ kk.abs() + n * U * ds.abs() @ kk.abs()
                r["dK"][s_, g] += ds.T @ qq
                r["eK"][s_, g] += (HALF * 1.02 + n * grp * U) * (ds.abs().T @ qq.abs()) + 1.02 * eds.T @ qq.abs()
                r["dV"][s_, g] += p.T @ gg
                r["eV"][s_, g] += (HALF * 1.02 + n * grp * U) * (p.T @ gg.abs()) + 1.02 * (p * ep).T @ gg.abs()
        for n_, e_ in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
            r[e_] = r[e_] * (1 + HALF) + HALF * r[n_].abs()
        out.append(r)
    return out


GRADS = (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV"))


def _near(got, ref, bound, name):
    got = got.to(F8)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - bound - 1e-30
    assert (over <= 0).all(), f"{name}: {over.max().item():.3e} beyond the bound at {over.argmax().item()}"


def _run(x, n_q, n_kv, d, W, S, scale=None, out_f=None, out_b=None, status=0):
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, window=W, sinks=S, scale=scale)
    fwd = ttl.packed_window_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=out_f, **kw)
    assert ttl.device_status() == status
    bwd = ttl.packed_window_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, x["cu"], out=out_b, **kw)
    assert ttl.device_status() == status
    return fwd, bwd


def _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, W, S, scale=None):
    used = sum(lens)
    ref = _reference(x, t, n_q, n_kv, d, lens, W, S, d ** -0.5 if scale is None else scale, fwd)
    for i, r in enumerate(ref):
        _near(fwd["O"][i].view(T, -1, d), r["O"], r["dO"], f"O[{i}]")
        lse = fwd["lse"][i]
        assert torch.isinf(lse[:, used:]).all() and (lse[:, used:] < 0).all()
        _near(lse[:, :used], r["lse"][:, :used], r["dlse"][:, :used], f"lse[{i}]")
        for n, e in GRADS:
            _near(bwd[n][i].view(T, -1, d), r[n], r[e], f"{n}[{i}]")
            assert torch.count_nonzero(bwd[n][i][used:]) == 0
        assert torch.count_nonzero(fwd["O"][i][used:]) == 0


def _ragged(total, n, seed):
    """n lengths of any size, empty ones among them, `total` tokens together."""
    cuts = torch.randint(0, total + 1, (n - 1,), generator=torch.Generator().manual_seed(seed)).sort()[0].tolist()
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


# t, T, query heads, KV heads, d, documents, window, sinks.  Heads paired (even groups) and token tiles paired (odd
# groups); windows of one key, below, at and above whole tiles; sinks that touch the window, lie tiles before it, cross a
# tile's end or fill several tiles; ranges of key tiles with a gap and without.
CASES = [
    (1, 1, 1, 1, 64, [1], 1, 0), (1, 5, 2, 1, 128, [5], 1, 0), (1, 5, 2, 1, 128, [5], 2, 1), (1, 130, 1, 1, 64, [130], 1, 1),
    (1, 400, 2, 2, 64, [400], 1, 0), (1, 700, 4, 1, 128, [700], 128, 0), (1, 700, 4, 1, 128, [700], 128, 4),
    (1, 700, 3, 1, 128, [700], 127, 1), (1, 901, 1, 1, 64, [901], 129, 128), (2, 640, 4, 2, 64, [100, 500, 40], 130, 3),
    (1, 1000, 2, 1, 128, [77, 900], 64, 90), (1, 1000, 3, 3, 64, [120, 880], 50, 20), (1, 1200, 2, 1, 128, [60, 1140], 200, 300),
    (1, 1200, 5, 1, 64, [60, 1140], 10, 300), (1, 800, 1, 1, 128, [256, 256, 256], 256, 256), (1, 500, 2, 1, 128, [3] * 100 + [150, 40], 2, 1),
    (8, 640, 16, 8, 128, [600], 33, 2), (1, 333, 2, 1, 64, [], 5, 5), (1, 400, 4, 4, 128, [1] * 400, 1, 0),
    (2, 300, 6, 2, 128, [0, 17, 0, 200, 83, 0], 40, 0), (1, 1500, 6, 2, 64, [1500], 300, 4), (1, 1025, 2, 2, 128, [1025], 1024, 0),
    (1, 1025, 1, 1, 128, [1025], 1, 1023), (16, 300, 16, 16, 64, [140, 160], 100, 7),
]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens,W,S", CASES)
def test_forward_and_backward(t, T, n_q, n_kv, d, lens, W, S):
    x = _inputs(t, T, n_q, n_kv, d, lens, T)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, W, S)


# More items than SMs (taken by work), key tiles that several items share because sinks are seen from everywhere.
MANY_ITEMS = [
    (1, 3000, 16, 4, 128, [2100] + _ragged(800, 9, 1), 200, 4), (1, 4000, 10, 10, 64, _ragged(3990, 7, 2), 128, 0),
    (1, 4000, 10, 10, 128, [4000], 100, 130), (2, 3333, 24, 8, 64, _ragged(3300, 300, 3), 17, 2),
    (1, 4100, 16, 2, 64, [4097], 1000, 1), (1, 5000, 24, 24, 64, [5000], 64, 4), (1, 2500, 20, 4, 128, _ragged(2500, 700, 4), 3, 0),
    (1, 6000, 32, 32, 64, [200, 5800], 64, 70), (1, 3000, 6, 2, 128, [2990], 300, 200),
]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens,W,S", MANY_ITEMS)
def test_more_items_than_sms(t, T, n_q, n_kv, d, lens, W, S):
    x = _inputs(t, T, n_q, n_kv, d, lens, T)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, W, S)


# Wide windows over few heads: heads and token tiles paired, documents that begin late, sinks of several tiles, rows behind
# the documents, key tiles in shares of more items than blocks and of fewer.
WIDE = [
    (1, 5000, 2, 1, 128, [4990], 1500, 4), (1, 5000, 3, 1, 64, [700, 4200], 1300, 300), (1, 9000, 1, 1, 64, [9000], 2000, 0),
    (2, 4500, 8, 2, 64, [50, 4400], 1100, 1), (1, 4100, 20, 20, 64, [4100], 2000, 2), (1, 4300, 16, 8, 128, [4290], 1100, 0),
    (1, 3000, 5, 5, 128, [60] * 10 + [2300], 1900, 130),
]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens,W,S", WIDE)
def test_wide_windows_over_few_heads(t, T, n_q, n_kv, d, lens, W, S):
    x = _inputs(t, T, n_q, n_kv, d, lens, T)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, W, S)
    f2, b2 = _run(x, n_q, n_kv, d, W, S)
    for a, b in ((fwd, f2), (bwd, b2)):
        assert all(torch.equal(p, q) for n in a if n != "ws" for p, q in zip(a[n], b[n]))


@pytest.mark.parametrize("W,S", [(500, 0), (10 ** 12, 0), (1, 499), (400, 10 ** 12), (200, 300)])
def test_a_window_that_hides_nothing(W, S):
    """Window and sinks together hold every document: the bits of packed_attn."""
    t, T, n_q, n_kv, d, lens = 2, 500, 4, 2, 64, [300, 190]
    x = _inputs(t, T, n_q, n_kv, d, lens, 1)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    f = ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], n_q=n_q, n_kv=n_kv, d=d)
    b = ttl.packed_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], f, x["cu"], n_q=n_q, n_kv=n_kv, d=d)
    for i in range(t):
        assert torch.equal(f["O"][i], fwd["O"][i]) and torch.equal(f["lse"][i], fwd["lse"][i])
        assert all(torch.equal(b[n][i], bwd[n][i]) for n in ("dQ", "dK", "dV"))


@pytest.mark.parametrize("std,scale", [(6.0, None), (1.0, 1.0), (0.01, 0.2), (3.0, 3.0)])
def test_peaked_and_flat_scores(std, scale):
    t, T, n_q, n_kv, d, lens, W, S = 1, 700, 4, 2, 128, [300, 400], 150, 5
    x = _inputs(t, T, n_q, n_kv, d, lens, 9, std)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S, scale)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, W, S, scale)


def test_growing_and_falling_scores():
    """The running maximum moves at every tile, or is the sinks'."""
    t, T, n_q, n_kv, d, lens, W, S = 1, 900, 2, 1, 64, [900], 200, 3
    for sign in (1, -1):
        x = _inputs(t, T, n_q, n_kv, d, lens, 1)
        x["Q"][0][:] = 1.0
        noise = 0.01 * torch.randn(T, d, generator=torch.Generator().manual_seed(2))
        x["K"][0][:] = (torch.linspace(-4, 4, T)[:, None] * sign + noise).to(BF16).cuda()
        fwd, bwd = _run(x, n_q, n_kv, d, W, S)
        _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, W, S)


BESIDE = [(1, 700, 2, 1, 64, [100, 530, 60], 90, 4), (1, 2600, 16, 4, 128, [130, 2100, 300], 300, 0),
          (1, 2600, 6, 2, 64, [2, 2500, 60], 128, 140), (1, 3000, 16, 1, 128, [2800, 150], 100, 2), (1, 700, 1, 1, 128, [690], 40, 1),
          (1, 3200, 2, 1, 128, [100, 3000], 1200, 4), (1, 3200, 3, 1, 64, [3000, 100], 1300, 200)]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens,W,S", BESIDE)
@pytest.mark.parametrize("which", ["V", "K", "Q", "dO"])
def test_a_value_that_is_not_finite_reaches_what_sees_it_and_nothing_else(t, T, n_q, n_kv, d, lens, W, S, which):
    """One NaN inside the longest document: what sees it is NaN, all else is as near as without it."""
    first = lens.index(max(lens))
    a, b = sum(lens[:first]), sum(lens[:first + 1])
    see = torch.zeros(T, T, dtype=torch.bool, device="cuda")
    see[a:b, a:b] = _see(b - a, W, S)
    grp = n_q // n_kv
    for at in (a, a + 3, (a + b) // 2 + 5, b - 2):
        x = _inputs(1, T, n_q, n_kv, d, lens, T + at)
        y = {k: [v.clone() for v in m] if k != "cu" else m for k, m in x.items()}
        y[which][0][at, 3] = float("nan")
        fwd, bwd = _run(x, n_q, n_kv, d, W, S)
        f2, b2 = _run(y, n_q, n_kv, d, W, S)
        # (the backward reference takes this run's O and lse, where a row's are numbers)
        own = {n: [torch.where(torch.isnan(f2[n][0]), fwd[n][0], f2[n][0])] for n in ("O", "lse")}
        ref = _reference(x, t, n_q, n_kv, d, lens, W, S, d ** -0.5, own)[0]
        hit = {n: torch.zeros(T, h, d, dtype=torch.bool, device="cuda") for n, h in
               (("O", n_q), ("dQ", n_q), ("dK", n_kv), ("dV", n_kv))}
        lse = torch.zeros(n_q, T, dtype=torch.bool, device="cuda")
        rows = see[:, at] if which in ("V", "K") else torch.arange(T, device="cuda") == at
        keys = see[rows].any(0)
        heads = slice(0, grp) if which in ("V", "K") else slice(0, 1)
        if which == "V":        # column 3 of o; through dp and D: dq of those rows, dk of the keys that they see
            hit["O"][rows, :grp, 3] = True
            hit["dQ"][rows, :grp] = True
            hit["dK"][keys, 0] = True
        elif which == "K":      # the scores of the rows that see it
            hit["O"][rows, :grp] = True
            lse[:grp, rows] = True
            hit["dQ"][rows, :grp] = True
            hit["dK"][keys, 0] = True
            hit["dV"][keys, 0] = True
        elif which == "Q":      # its own row's scores
            hit["O"][at, heads] = True
            lse[heads, at] = True
            hit["dQ"][at, heads] = True
            hit["dK"][keys, 0] = True
            hit["dV"][keys, 0] = True
        else:                   # its own row's D and dp, and column 3 of what it adds to dv
            hit["dQ"][at, heads] = True
            hit["dK"][keys, 0] = True
            hit["dV"][keys, 0, 3] = True
        got = {"O": f2["O"][0], "dQ": b2["dQ"][0], "dK": b2["dK"][0], "dV": b2["dV"][0]}
        for n, e in (("O", "dO"),) + GRADS:
            g = got[n].view(T, -1, d)
            assert torch.isnan(g[hit[n]]).all(), f"{n} at {at}"
            _near(g[~hit[n]], ref[n][~hit[n]], 2 * ref[e][~hit[n]], f"{n} at {at}")
        assert torch.isnan(f2["lse"][0][lse]).all()
        rest = ~lse
        rest[:, sum(lens):] = False
        _near(f2["lse"][0][rest], ref["lse"][rest], ref["dlse"][rest], "lse")


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens,W,S,left", [(1, 2000, 16, 4, 128, [900, 700], 200, 4, 150),
                                                          (2, 1000, 4, 2, 64, [500, 300], 60, 0, 77), (1, 3000, 4, 1, 64, [2500], 128, 130, 201),
                                                          (1, 3000, 2, 1, 128, [2600], 1200, 5, 130)])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf"), -3.3e38])
def test_rows_of_no_document_hold_anything(t, T, n_q, n_kv, d, lens, W, S, left, bad):
    """Uninitialised rows before and behind the documents."""
    x = _inputs(t, T, n_q, n_kv, d, lens, T)
    used = left + sum(lens)
    x["cu"] += left
    for n in ("Q", "K", "V", "dO"):
        for m in x[n]:
            m[:left] = bad
            m[used:] = bad
    f2, b2 = _run(x, n_q, n_kv, d, W, S)
    part = {k: [v[left:used].contiguous() for v in m] if k != "cu" else m for k, m in x.items()}
    f = {"O": [o[left:used] for o in f2["O"]], "lse": [l[:, left:used] for l in f2["lse"]]}
    n_ = used - left
    for i, r in enumerate(_reference(part, t, n_q, n_kv, d, lens, W, S, d ** -0.5, f)):
        _near(f["O"][i].reshape(n_, -1, d), r["O"], r["dO"], "O")
        _near(f["lse"][i], r["lse"], r["dlse"], "lse")
        for n, e in GRADS:
            _near(b2[n][i][left:used].reshape(n_, -1, d), r[n], r[e], n)
            assert torch.count_nonzero(b2[n][i][:left]) == 0 and torch.count_nonzero(b2[n][i][used:]) == 0


@pytest.mark.parametrize("T,n_q,n_kv,W", [(200, 2, 1, 30), (3000, 16, 4, 30), (3000, 9, 3, 30), (3000, 3, 1, 1300), (3000, 2, 1, 1300)])
@pytest.mark.parametrize("S", [0, 4, 140])
def test_bad_document_bounds_are_reported(T, n_q, n_kv, W, S):
    d = 64
    x = _inputs(1, T, n_q, n_kv, d, [T], 0)
    for cu in ([0, T * 3 // 4, T // 2, T], [-5, T // 3, T * 2 // 3], [0, T // 3, 25 * T], [T + 100, T + 200], [T, 0],
               [0, T // 4, 7, T // 2, 3, T]):
        y = dict(x, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        _run(y, n_q, n_kv, d, W, S, status=ttl.TTL_ERR_DEVICE)
    _run(x, n_q, n_kv, d, W, S)


def test_fused_projection_strides_and_wider_results():
    """Q, K, V as column ranges of one matrix, the gradients and O into others: the same bits, and what lies beside
    them stays."""
    t, T, n_q, n_kv, d, lens, W, S = 2, 333, 8, 4, 64, [200, 130], 60, 4
    x = _inputs(t, T, n_q, n_kv, d, lens, 6)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    qc, kc = n_q // t * d, n_kv // t * d
    fused = [torch.cat([x["Q"][i], x["K"][i], x["V"][i]], 1) for i in range(t)]
    grads = [torch.full((T + 60, qc + 2 * kc + 8), 7.0, dtype=BF16, device="cuda") for _ in fused]
    cut = lambda m: ([f[:T, :qc] for f in m], [f[:T, qc:qc + kc] for f in m], [f[:T, qc + kc:qc + 2 * kc] for f in m])   # noqa: E731
    y = dict(x)
    y["Q"], y["K"], y["V"] = cut(fused)
    big = [torch.full((T + 70, qc + 24), 7.0, dtype=BF16, device="cuda") for _ in range(t)]
    out_f = ttl.packed_window_attn_fwd_buffers(t, T, n_q, n_kv, d, len(lens), W, S)
    out_f["O"] = [m[:T, 16:16 + qc] for m in big]
    out_b = ttl.packed_window_attn_bwd_buffers(t, T, n_q, n_kv, d, len(lens), W, S)
    out_b["dQ"], out_b["dK"], out_b["dV"] = cut(grads)
    f2, b2 = _run(y, n_q, n_kv, d, W, S, out_f=out_f, out_b=out_b)
    for i in range(t):
        assert torch.equal(f2["O"][i], fwd["O"][i]) and torch.equal(f2["lse"][i], fwd["lse"][i])
        assert all(torch.equal(b2[n][i], bwd[n][i]) for n in ("dQ", "dK", "dV"))
        assert (big[i][T:] == 7).all() and (big[i][:, :16] == 7).all() and (big[i][:, 16 + qc:] == 7).all()
        assert (grads[i][T:] == 7).all() and (grads[i][:, qc + 2 * kc:] == 7).all()


def test_same_bits_again_and_from_a_graph_on_a_side_stream():
    t, T, n_q, n_kv, d, lens, W, S = 2, 3000, 8, 2, 128, [500, 2400], 256, 4
    x = _inputs(t, T, n_q, n_kv, d, lens, 2)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    for _ in range(3):
        f2, b2 = _run(x, n_q, n_kv, d, W, S)
        for a, b in ((fwd, f2), (bwd, b2)):
            assert all(torch.equal(p, q) for n in a if n != "ws" for p, q in zip(a[n], b[n]))
    f3 = ttl.packed_window_attn_fwd_buffers(t, T, n_q, n_kv, d, 2, W, S)
    b3 = ttl.packed_window_attn_bwd_buffers(t, T, n_q, n_kv, d, 2, W, S)
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, window=W, sinks=S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        ttl.packed_window_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=f3, **kw)
        ttl.packed_window_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], f3, x["cu"], out=b3, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert ttl.device_status() == 0
    for a, b in ((fwd, f3), (bwd, b3)):
        assert all(torch.equal(p, q) for n in a if n != "ws" for p, q in zip(a[n], b[n]))


def test_gradient_against_differences():
    """The directional derivative of the 64-bit forward against the kernels' gradients."""
    t, T, n_q, n_kv, d, lens, W, S = 1, 150, 4, 2, 64, [60, 90], 20, 3
    x = _inputs(t, T, n_q, n_kv, d, lens, 21)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    gen = torch.Generator("cuda").manual_seed(5)
    dirs = {n: torch.randn(x[n][0].shape, generator=gen, device="cuda", dtype=F8) for n in ("Q", "K", "V")}

    def loss(e):
        y = {n: [x[n][0].to(F8) + e * dirs[n]] for n in ("Q", "K", "V")}
        y["dO"] = x["dO"]
        o = _reference(y, t, n_q, n_kv, d, lens, W, S, d ** -0.5)[0]["O"]
        return (o * x["dO"][0].to(F8).view(T, -1, d)).sum()

    want = (loss(1e-4) - loss(-1e-4)) / 2e-4
    got = sum((bwd["d" + n][0].to(F8) * dirs[n]).sum() for n in ("Q", "K", "V"))
    # Independent roundings of at most half a step in P or dS, O (through D) and the result: their
    # 2-norm is at most 3 half steps of the gradient's, and a random direction sees 4 sigma of it.
    size = sum((bwd["d" + n][0].to(F8).square().sum()) for n in ("Q", "K", "V")).sqrt()
    assert (got - want).abs() <= 4 * 3 * HALF * size


def test_two_graphs_that_share_buffers_and_a_workspace():
    """Replayed in turn they give what each gives alone: nothing of the other's plan is left."""
    T, n_q, n_kv, d, W, S = 4000, 8, 8, 64, 300, 5
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, window=W, sinks=S)
    packs = [_inputs(1, T, n_q, n_kv, d, lens, 40 + len(lens)) for lens in ([4000], [100, 900, 2500])]
    out_f = ttl.packed_window_attn_fwd_buffers(1, T, n_q, n_kv, d, 3, W, S)
    out_b = ttl.packed_window_attn_bwd_buffers(1, T, n_q, n_kv, d, 3, W, S)
    want, graphs = [], []
    for x in packs:
        f = ttl.packed_window_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], **kw)
        want.append((f, ttl.packed_window_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], f, x["cu"], **kw)))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            ttl.packed_window_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=out_f, **kw)
            ttl.packed_window_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], out_f, x["cu"], out=out_b, **kw)
        graphs.append(graph)
    for i in (0, 1, 0, 0, 1):
        graphs[i].replay()
        torch.cuda.synchronize()
        f, b = want[i]
        assert torch.equal(out_f["O"][0], f["O"][0]) and torch.equal(out_f["lse"][0], f["lse"][0])
        assert all(torch.equal(out_b[n][0], b[n][0]) for n in ("dQ", "dK", "dV"))
    assert ttl.device_status() == 0


def test_calls_on_two_streams_at_once():
    T, n_q, n_kv, d, W, S = 3000, 16, 4, 128, 500, 4
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, window=W, sinks=S)
    x, y = (_inputs(1, T, n_q, n_kv, d, lens, 50 + len(lens)) for lens in ([3000], [1200, 1700]))
    want = [_run(v, n_q, n_kv, d, W, S) for v in (x, y)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (v, s) in enumerate(zip((x, y), streams)):
            f = ttl.packed_window_attn_fwd(v["Q"], v["K"], v["V"], v["cu"], stream=s, **kw)
            got[i].append((f, ttl.packed_window_attn_bwd(v["dO"], v["Q"], v["K"], v["V"], f, v["cu"], stream=s, **kw)))
    torch.cuda.synchronize()
    assert ttl.device_status() == 0
    for (f, b), runs in zip(want, got):
        for f2, b2 in runs:
            assert torch.equal(f["O"][0], f2["O"][0]) and all(torch.equal(b[n][0], b2[n][0]) for n in ("dQ", "dK", "dV"))


# Packs of more than a thousand key tiles of one head, where the choice between whole tiles and even shares hangs on which of
# several lengths stands at one place of the work list: T, documents, KV heads, query heads each, window, seed.
NEAR_TIES = [(140000, 2000, 2, 8, 756, 322067657), (140000, 1300, 1, 2, 1299, 330331263), (131072, 1300, 3, 2, 514, 384181818),
             (200000, 1100, 2, 4, 298, 506041774)]


@pytest.mark.parametrize("T,docs,n_kv,grp,W,seed", NEAR_TIES)
def test_long_packs_give_the_same_bits_again(T, docs, n_kv, grp, W, seed):
    rng = random.Random(seed)
    cu = [0] + sorted(rng.randint(0, T) for _ in range(docs - 1)) + [T]
    x = _inputs(1, T, n_kv * grp, n_kv, 64, [b - a for a, b in zip(cu, cu[1:])], 3)
    kw = dict(n_q=n_kv * grp, n_kv=n_kv, d=64, window=W)
    fwd = ttl.packed_window_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], **kw)
    first = ttl.packed_window_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, x["cu"], **kw)
    out = ttl.packed_window_attn_bwd_buffers(1, T, n_kv * grp, n_kv, 64, docs, W)
    same = []
    for _ in range(40):
        again = ttl.packed_window_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, x["cu"], out=out, **kw)
        same += [(first[n][0] == again[n][0]).all() for n in ("dQ", "dK", "dV")]
    assert torch.stack(same).all()
    assert ttl.device_status() == 0


@pytest.mark.parametrize("S", [0, 4])
def test_a_value_that_is_not_finite_beside_a_border_costs_a_window(S):
    """Rows of two documents are computed again together: what they read goes with the window, not with the first document."""
    T, d, W, border = 33000, 64, 64, 32007
    x = _inputs(1, T, 1, 1, d, [border, 900], 77)
    kw = dict(n_q=1, n_kv=1, d=d, window=W, sinks=S)

    def times(at):
        y = {k: [v.clone() for v in m] if k != "cu" else m for k, m in x.items()}
        for n in ("K", "V"):
            y[n][0][at, 3] = float("nan")
        out_f = ttl.packed_window_attn_fwd_buffers(1, T, 1, 1, d, 2, W, S)
        out_b = ttl.packed_window_attn_bwd_buffers(1, T, 1, 1, d, 2, W, S)
        best = [math.inf, math.inf]
        for _ in range(6):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
            e[0].record()
            ttl.packed_window_attn_fwd(y["Q"], y["K"], y["V"], y["cu"], out=out_f, **kw)
            e[1].record()
            ttl.packed_window_attn_bwd(y["dO"], y["Q"], y["K"], y["V"], out_f, y["cu"], out=out_b, **kw)
            e[2].record()
            torch.cuda.synchronize()
            best = [min(best[0], e[0].elapsed_time(e[1])), min(best[1], e[1].elapsed_time(e[2]))]
        return best

    inside, beside = times(20005), times(border - 2)
    assert ttl.device_status() == 0
    assert all(b <= 4 * a for a, b in zip(inside, beside)), (inside, beside)


def _with_empty(total, n, seed):
    """n lengths, `total` tokens together: some fifty of any size, the rest empty, in any order."""
    lens = _ragged(total, 50, seed) + [0] * (n - 50)
    return [lens[i] for i in torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()]


@pytest.mark.parametrize("n", [1024, 1025, 1500])
@pytest.mark.parametrize("T,n_q,n_kv,d,W,S", [(4000, 10, 10, 64, 70, 3), (3000, 16, 4, 128, 200, 0)])
def test_many_documents_and_more_items_than_sms(n, T, n_q, n_kv, d, W, S):
    """As many documents as the plan keeps in shared memory, one more, and far more: empty ones among them."""
    lens = _with_empty(T - 77, n, n + T)
    x = _inputs(1, T, n_q, n_kv, d, lens, n)
    fwd, bwd = _run(x, n_q, n_kv, d, W, S)
    _check(x, fwd, bwd, 1, T, n_q, n_kv, d, lens, W, S)
