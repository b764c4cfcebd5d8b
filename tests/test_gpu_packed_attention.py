"""Causal attention over packed documents vs a plain 64-bit implementation (GPU).

Bounds, per element.  The probabilities and the score gradients are rounded to bf16 once before their
product (half a step, 2^-8, of each term), the result once more; scores and statistics are fp32.  Hence
  |O - o|    <= 2^-8 (sum p |v| + |o|),         |dV - dv| <= 2^-8 (sum p |do| + |dv|)
  |dQ - dq|  <= 2^-8 (sum |ds k| + |dq|),       |dK - dk| <= 2^-8 (sum |ds q| + |dk|)
plus the fp32 part: a score is off by at most 2 d u sum |q k| (u = 2^-24) and a few u of the exponential,
which moves every probability, and p (dp - D), by that factor.  The backward reference takes the
same O and lse as the kernels.
"""
import math

import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8
F8 = torch.float64
BF16 = torch.bfloat16


def _inputs(t, T, n_q, n_kv, d, lens, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)

    def mats(cols, s=1.0):
        return [(torch.randn(T, cols, generator=g) * s).to(BF16).cuda() for _ in range(t)]

    qc, kc = n_q // t * d, n_kv // t * d
    x = {"Q": mats(qc, std), "K": mats(kc, std), "V": mats(kc), "dO": mats(qc)}
    x["cu"] = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32).cuda()
    return x


def _reference(x, t, n_q, n_kv, d, lens, scale, fwd=None):
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
            hide = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
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


def _near(got, ref, bound, name):
    got = got.to(F8)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - bound - 1e-30
    assert (over <= 0).all(), f"{name}: {over.max().item():.3e} beyond the bound at {over.argmax().item()}"


def _run(t, T, n_q, n_kv, d, lens, seed=0, std=1.0, scale=None, x=None, out_f=None, out_b=None):
    x = _inputs(t, T, n_q, n_kv, d, lens, seed, std) if x is None else x
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, scale=scale)
    fwd = ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=out_f, **kw)
    bwd = ttl.packed_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, x["cu"], out=out_b, **kw)
    assert ttl.device_status() == 0
    return x, fwd, bwd


def _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, scale=None):
    used = sum(lens)
    ref = _reference(x, t, n_q, n_kv, d, lens, d ** -0.5 if scale is None else scale, fwd)
    for i, r in enumerate(ref):
        _near(fwd["O"][i].view(T, -1, d), r["O"], r["dO"], f"O[{i}]")
        lse = fwd["lse"][i]
        assert torch.isinf(lse[:, used:]).all() and (lse[:, used:] < 0).all()
        _near(lse[:, :used], r["lse"][:, :used], r["dlse"][:, :used], f"lse[{i}]")
        for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
            _near(bwd[n][i].view(T, -1, d), r[n], r[e], f"{n}[{i}]")
            assert torch.count_nonzero(bwd[n][i][used:]) == 0
        assert torch.count_nonzero(fwd["O"][i][used:]) == 0


CASES = [
    (1, 1, 1, 1, 64, [1]), (1, 5, 2, 1, 128, [5]), (1, 127, 2, 2, 64, [127]), (1, 128, 4, 1, 128, [128]),
    (1, 129, 3, 1, 128, [129]), (2, 130, 4, 2, 64, [1, 64, 65]), (1, 256, 2, 1, 128, [100, 28, 128]),
    (1, 257, 1, 1, 128, [257]), (2, 300, 6, 2, 128, [0, 17, 0, 200, 83, 0]), (1, 384, 5, 1, 64, [383, 1]),
    (1, 400, 4, 4, 128, [1] * 400), (1, 500, 2, 1, 128, [3] * 100 + [150, 40]), (4, 513, 8, 4, 64, [256, 257]),
    (1, 700, 8, 1, 128, [130, 570]), (8, 640, 16, 8, 128, [600]), (1, 333, 2, 1, 64, []), (1, 1025, 2, 1, 128, [1025]),
    (1, 1500, 4, 2, 128, [700, 1, 2, 515, 100]), (1, 2100, 1, 1, 64, [2100]), (16, 200, 16, 16, 64, [99, 101]),
]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens", CASES)
def test_forward_and_backward(t, T, n_q, n_kv, d, lens):
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=T)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens)


@pytest.mark.parametrize("std,scale", [(6.0, None), (1.0, 1.0), (0.01, 0.2), (3.0, 3.0)])
def test_peaked_and_flat_scores(std, scale):
    t, T, n_q, n_kv, d, lens = 1, 700, 4, 2, 128, [300, 400]
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=9, std=std, scale=scale)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens, scale)


def test_growing_scores():
    """Each key scores above all before it (the running maximum moves at every tile), and the reverse."""
    t, T, n_q, n_kv, d, lens = 1, 900, 2, 1, 64, [900]
    for sign in (1, -1):
        x = _inputs(t, T, n_q, n_kv, d, lens, 1)
        ramp = torch.linspace(-4, 4, T)[:, None] * sign
        x["Q"][0][:] = 1.0
        x["K"][0][:] = (ramp + 0.01 * torch.randn(T, d, generator=torch.Generator().manual_seed(2))).to(BF16).cuda()
        x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, x=x)
        _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3e38])
def test_masked_places_do_not_reach_a_row(bad):
    """Tokens of no document, another document's and later tokens hold values that would spread."""
    t, T, n_q, n_kv, d, lens = 1, 600, 4, 2, 128, [150, 230, 100]
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=4)
    y = {k: [v.clone() for v in a] if k != "cu" else a for k, a in x.items()}
    for n in ("Q", "K", "V", "dO"):
        y[n][0][480:] = bad                # of no document
        y[n][0][150:380] = bad             # the second document
    _, f2, b2 = _run(t, T, n_q, n_kv, d, lens, x=y)
    keep = torch.zeros(T, dtype=torch.bool, device="cuda")
    keep[:150] = True
    keep[380:480] = True
    ref = _reference(x, t, n_q, n_kv, d, lens, d ** -0.5, fwd)[0]
    _near(f2["O"][0].view(T, -1, d)[keep], ref["O"][keep], ref["dO"][keep], "O")
    _near(f2["lse"][0][:, keep], ref["lse"][:, keep], ref["dlse"][:, keep], "lse")
    # the backward reference takes this run's O (the other document's rows of it are not looked at)
    own = _reference(x, t, n_q, n_kv, d, lens, d ** -0.5, f2)[0]
    for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
        _near(b2[n][0].view(T, -1, d)[keep], own[n][keep], own[e][keep], n)
        assert torch.count_nonzero(b2[n][0][480:]) == 0
    # a later key and value does not reach the queries before it
    z = {k: [v.clone() for v in a] if k != "cu" else a for k, a in x.items()}
    z["K"][0][140] = bad
    z["V"][0][140] = bad
    f3 = ttl.packed_attn_fwd(z["Q"], z["K"], z["V"], z["cu"], n_q=n_q, n_kv=n_kv, d=d)
    _near(f3["O"][0].view(T, -1, d)[:140], ref["O"][:140], ref["dO"][:140], "O before")
    _near(f3["O"][0].view(T, -1, d)[150:480], ref["O"][150:480], ref["dO"][150:480], "O of other documents")


def test_bad_document_bounds_are_reported():
    t, T, n_q, n_kv, d = 1, 200, 2, 1, 64
    x = _inputs(t, T, n_q, n_kv, d, [200], 0)
    for cu in ([0, 150, 100, 200], [-5, 100, 200], [0, 100, 5000], [300, 400], [200, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fwd = ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], cu, n_q=n_q, n_kv=n_kv, d=d)
        assert ttl.device_status() == ttl.TTL_ERR_DEVICE
        ttl.packed_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, cu, n_q=n_q, n_kv=n_kv, d=d)
        assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    _run(t, T, n_q, n_kv, d, [200])


def test_documents_that_begin_late():
    """cu_seqlens[0] > 0: the tokens before belong to no document."""
    t, T, n_q, n_kv, d = 1, 300, 2, 1, 128
    x = _inputs(t, T, n_q, n_kv, d, [300], 3)
    x["cu"] = torch.tensor([40, 90, 250], dtype=torch.int32, device="cuda")
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, [], x=x)
    part = {k: [v[40:250] for v in a] if k != "cu" else a for k, a in x.items()}
    f = {"O": [fwd["O"][0][40:250]], "lse": [fwd["lse"][0][:, 40:250]]}
    r = _reference(part, t, n_q, n_kv, d, [50, 160], d ** -0.5, f)[0]
    _near(f["O"][0].view(210, -1, d), r["O"], r["dO"], "O")
    for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
        _near(bwd[n][0][40:250].view(210, -1, d), r[n], r[e], n)
        assert torch.count_nonzero(bwd[n][0][:40]) == 0 and torch.count_nonzero(bwd[n][0][250:]) == 0
    assert torch.isinf(fwd["lse"][0][:, :40]).all()


def test_fused_projection_strides():
    """Q, K, V as column ranges of one matrix, the gradients into another: the same bits."""
    t, T, n_q, n_kv, d, lens = 2, 333, 8, 4, 64, [200, 133]
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=6)
    qc, kc = n_q // t * d, n_kv // t * d
    fused = [torch.cat([x["Q"][i], x["K"][i], x["V"][i]], 1) for i in range(t)]
    grads = [torch.full_like(f, float("nan")) for f in fused]
    cut = lambda m: ([f[:, :qc] for f in m], [f[:, qc:qc + kc] for f in m], [f[:, qc + kc:] for f in m])   # noqa: E731
    q, k, v = cut(fused)
    y = {"Q": q, "K": k, "V": v, "dO": x["dO"], "cu": x["cu"]}
    out_b = ttl.packed_attn_bwd_buffers(t, T, n_q, n_kv, d, len(lens))
    out_b["dQ"], out_b["dK"], out_b["dV"] = cut(grads)
    _, f2, b2 = _run(t, T, n_q, n_kv, d, lens, x=y, out_b=out_b)
    for i in range(t):
        assert torch.equal(f2["O"][i], fwd["O"][i]) and torch.equal(f2["lse"][i], fwd["lse"][i])
        for n in ("dQ", "dK", "dV"):
            assert torch.equal(b2[n][i], bwd[n][i])


def test_documents_do_not_see_their_place_in_the_pack():
    """A document alone and the same document behind others give the same result (to the bounds)."""
    t, n_q, n_kv, d = 1, 4, 1, 128
    x, fwd, bwd = _run(t, 700, n_q, n_kv, d, [77, 310, 313], seed=12)
    part = {k: [v[77:387].contiguous() for v in a] if k != "cu" else None for k, a in x.items()}
    part["cu"] = torch.tensor([0, 310], dtype=torch.int32, device="cuda")
    _, f2, b2 = _run(t, 310, n_q, n_kv, d, [310], x=part)
    _check(part, f2, b2, t, 310, n_q, n_kv, d, [310])
    f = {"O": [fwd["O"][0][77:387]], "lse": [fwd["lse"][0][:, 77:387]]}
    r = _reference(part, t, n_q, n_kv, d, [310], d ** -0.5, f)[0]
    for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
        _near(bwd[n][0][77:387].view(310, -1, d), r[n], r[e], n)


def test_same_inputs_same_bits():
    t, T, n_q, n_kv, d, lens = 2, 1200, 8, 2, 128, [500, 700]
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=2)
    for _ in range(4):
        _, f2, b2 = _run(t, T, n_q, n_kv, d, lens, x=x)
        for a, b in ((fwd, f2), (bwd, b2)):
            for n in a:
                if n != "ws":
                    assert all(torch.equal(p, q) for p, q in zip(a[n], b[n])), n


def test_gradient_against_differences():
    """The directional derivative of the 64-bit forward against the kernels' gradients."""
    t, T, n_q, n_kv, d, lens = 1, 150, 4, 2, 64, [60, 90]
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=21)
    gen = torch.Generator("cuda").manual_seed(5)
    dirs = {n: torch.randn(x[n][0].shape, generator=gen, device="cuda", dtype=F8) for n in ("Q", "K", "V")}

    def loss(e):
        y = {n: [x[n][0].to(F8) + e * dirs[n]] for n in ("Q", "K", "V")}
        y["dO"] = x["dO"]
        o = _reference(y, t, n_q, n_kv, d, lens, d ** -0.5)[0]["O"]
        return (o * x["dO"][0].to(F8).view(T, -1, d)).sum()

    step = 1e-4
    want = (loss(step) - loss(-step)) / (2 * step)
    got = sum((bwd["d" + n][0].to(F8) * dirs[n]).sum() for n in ("Q", "K", "V"))
    # Independent roundings of at most half a step in P or dS, O (through D) and the result: their
    # 2-norm is at most 3 half steps of the gradient's, and a random direction sees 4 sigma of it.
    size = sum((bwd["d" + n][0].to(F8).square().sum()) for n in ("Q", "K", "V")).sqrt()
    assert (got - want).abs() <= 4 * 3 * HALF * size


def test_graph_replay_on_a_side_stream():
    t, T, n_q, n_kv, d, lens = 2, 400, 4, 2, 128, [150, 250]
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=30)
    f2 = ttl.packed_attn_fwd_buffers(t, T, n_q, n_kv, d, 2)
    b2 = ttl.packed_attn_bwd_buffers(t, T, n_q, n_kv, d, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    kw = dict(n_q=n_q, n_kv=n_kv, d=d)
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=f2, **kw)
        ttl.packed_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], f2, x["cu"], out=b2, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert ttl.device_status() == 0
    for i in range(t):
        assert torch.equal(f2["O"][i], fwd["O"][i])
        for n in ("dQ", "dK", "dV"):
            assert torch.equal(b2[n][i], bwd[n][i])


def _ragged(total, n, seed):
    """n lengths of any size, empty ones among them, `total` tokens together."""
    cuts = torch.randint(0, total + 1, (n - 1,), generator=torch.Generator().manual_seed(seed)).sort()[0].tolist()
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


# More items than SMs (they are then taken by work): heads paired (even groups) and token tiles paired (odd
# groups), both head widths, one long document among short ones, one alone, hundreds of short ones.
MANY_ITEMS = [
    (1, 3000, 16, 4, 128, [2100] + _ragged(800, 9, 1)), (1, 4000, 10, 10, 64, _ragged(3990, 7, 2)),
    (1, 4000, 10, 10, 128, [4000]), (2, 3333, 24, 8, 64, _ragged(3300, 300, 3)), (1, 4100, 16, 2, 64, [4097]),
    (1, 2500, 20, 4, 128, _ragged(2500, 700, 4)),
]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens", MANY_ITEMS)
def test_more_items_than_sms(t, T, n_q, n_kv, d, lens):
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=T)
    _check(x, fwd, bwd, t, T, n_q, n_kv, d, lens)


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens", [(1, 2000, 16, 1, 128, [1500, 200, 100]), (1, 2600, 4, 1, 64, [100, 2300])])
def test_masked_places_in_key_tiles_that_several_items_share(t, T, n_q, n_kv, d, lens):
    """A long document's key tiles are summed in parts: NaN before and behind it stays outside."""
    x, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, seed=8)
    first = lens.index(max(lens))
    a, b = sum(lens[:first]), sum(lens[:first + 1])
    y = {k: [v.clone() for v in m] if k != "cu" else m for k, m in x.items()}
    for n in ("Q", "K", "V", "dO"):
        y[n][0][:a] = float("nan")
        y[n][0][b:] = float("nan")
    _, f2, b2 = _run(t, T, n_q, n_kv, d, lens, x=y)
    part = {k: [v[a:b] for v in m] if k != "cu" else m for k, m in x.items()}
    f = {"O": [f2["O"][0][a:b]], "lse": [f2["lse"][0][:, a:b]]}
    r = _reference(part, t, n_q, n_kv, d, [b - a], d ** -0.5, f)[0]
    _near(f["O"][0].view(b - a, -1, d), r["O"], r["dO"], "O")
    _near(f["lse"][0], r["lse"], r["dlse"], "lse")
    for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
        _near(b2[n][0][a:b].view(b - a, -1, d), r[n], r[e], n)


@pytest.mark.parametrize("T,n_q,n_kv,d", [(45, 2, 1, 64), (161, 3, 1, 128), (3001, 16, 4, 128)])
def test_results_in_a_wider_buffer(T, n_q, n_kv, d):
    """O as columns of a larger matrix: the columns beside it and the rows behind it keep their values."""
    lens = [T // 3, T - T // 3 - 5]
    x, fwd, bwd = _run(1, T, n_q, n_kv, d, lens, seed=T)
    big = torch.full((T + 70, n_q * d + 24), 7.0, dtype=BF16, device="cuda")
    out = ttl.packed_attn_fwd_buffers(1, T, n_q, n_kv, d, len(lens))
    out["O"] = [big[:T, 16:16 + n_q * d]]
    _, f2, b2 = _run(1, T, n_q, n_kv, d, lens, x=x, out_f=out)
    assert torch.equal(f2["O"][0], fwd["O"][0]) and torch.equal(b2["dQ"][0], bwd["dQ"][0])
    assert (big[T:] == 7).all() and (big[:, :16] == 7).all() and (big[:, 16 + n_q * d:] == 7).all()


def test_bad_document_bounds_with_many_items():
    t, T, n_q, n_kv, d = 1, 3000, 16, 4, 64
    x = _inputs(t, T, n_q, n_kv, d, [3000], 0)
    for cu in ([0, 2500, 100, 3000], [-5, 1000, 2000], [0, 1000, 50000], [4000, 5000], [2000, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        fwd = ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], cu, n_q=n_q, n_kv=n_kv, d=d)
        assert ttl.device_status() == ttl.TTL_ERR_DEVICE
        ttl.packed_attn_bwd(x["dO"], x["Q"], x["K"], x["V"], fwd, cu, n_q=n_q, n_kv=n_kv, d=d)
        assert ttl.device_status() == ttl.TTL_ERR_DEVICE


@pytest.mark.parametrize("T,n_q,n_kv,d,cu", [(200, 2, 1, 64, [40, 5000]), (200, 4, 2, 128, [0, 100, 5000]), (129, 2, 2, 64, [3, 300]),
                                             (3000, 16, 4, 64, [700, 1000, 50000]), (2500, 4, 1, 128, [5, 9000])])
def test_documents_beyond_the_pack_leave_the_rows_behind_it_alone(T, n_q, n_kv, d, cu):
    """cu_seqlens that end beyond T are reported, and nothing behind the T rows is read into a result or written."""
    x = _inputs(1, T, n_q, n_kv, d, [T], T)
    guard = 140
    wide = {n: torch.full((T + guard, x[n][0].shape[1]), float("nan"), dtype=BF16, device="cuda") for n in ("Q", "K", "V", "dO")}
    for n, m in wide.items():
        m[:T] = x[n][0]
    y = {n: [m[:T]] for n, m in wide.items()}
    y["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    cut = cu[:-1] + [T]
    y["ok"] = torch.tensor(cut, dtype=torch.int32, device="cuda")
    kw = dict(n_q=n_q, n_kv=n_kv, d=d)
    rows = {n: torch.full((T + guard, c), 7.0, dtype=BF16, device="cuda")
            for n, c in (("O", n_q * d), ("dQ", n_q * d), ("dK", n_kv * d), ("dV", n_kv * d))}
    lse = torch.full((n_q * T + guard,), 7.0, device="cuda")
    out_f = ttl.packed_attn_fwd_buffers(1, T, n_q, n_kv, d, len(cu) - 1)
    out_b = ttl.packed_attn_bwd_buffers(1, T, n_q, n_kv, d, len(cu) - 1)
    out_f["O"], out_f["lse"] = [rows["O"][:T]], [lse[:n_q * T].view(n_q, T)]
    for n in ("dQ", "dK", "dV"):
        out_b[n] = [rows[n][:T]]
    ttl.packed_attn_fwd(y["Q"], y["K"], y["V"], y["cu"], out=out_f, **kw)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    ttl.packed_attn_bwd(y["dO"], y["Q"], y["K"], y["V"], out_f, y["cu"], out=out_b, **kw)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    for n, m in rows.items():
        assert (m[T:] == 7).all(), n
    assert (lse[n_q * T:] == 7).all()
    # the last document cut to the pack is what the kernels take such bounds for: the same bits
    f2 = ttl.packed_attn_fwd(y["Q"], y["K"], y["V"], y["ok"], **kw)
    b2 = ttl.packed_attn_bwd(y["dO"], y["Q"], y["K"], y["V"], f2, y["ok"], **kw)
    assert ttl.device_status() == 0
    assert torch.equal(f2["O"][0], out_f["O"][0]) and torch.equal(f2["lse"][0], out_f["lse"][0])
    for n in ("dQ", "dK", "dV"):
        assert torch.equal(b2[n][0], out_b[n][0]), n


def _one_bad_value(T, n_q, n_kv, d, lens, which, at, bad=float("nan")):
    """Inputs with one value of `which` (head 0, column 3) at token `at` that is not finite, and the clean ones."""
    x = _inputs(1, T, n_q, n_kv, d, lens, T + at)
    y = {k: [v.clone() for v in m] if k != "cu" else m for k, m in x.items()}
    y[which][0][at, 3] = bad
    return x, y


# One work list and none, key tiles that several items share, both head widths, odd groups.
BESIDE = [(1, 700, 2, 1, 64, [100, 530, 60]), (1, 2600, 16, 4, 128, [130, 2100, 300]), (1, 2600, 6, 2, 64, [2, 2500, 60]),
          (1, 3000, 16, 1, 128, [2800, 150])]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens", BESIDE)
@pytest.mark.parametrize("which", ["V", "K", "Q", "dO"])
def test_a_value_that_is_not_finite_reaches_what_sees_it_and_nothing_else(t, T, n_q, n_kv, d, lens, which):
    """One NaN inside the longest document, in a tile's middle: the rows (and columns) that see it are NaN, all others
    are as near as without it."""
    first = lens.index(max(lens))
    a, b = sum(lens[:first]), sum(lens[:first + 1])
    for at in (a + 3, (a + b) // 2 + 5, b - 2):
        x, y = _one_bad_value(T, n_q, n_kv, d, lens, which, at)
        _, fwd, bwd = _run(t, T, n_q, n_kv, d, lens, x=x)
        _, f2, b2 = _run(t, T, n_q, n_kv, d, lens, x=y)
        # (the backward reference takes this run's O and lse, where a row's are numbers)
        own = {n: [torch.where(torch.isnan(f2[n][0]), fwd[n][0], f2[n][0])] for n in ("O", "lse")}
        ref = _reference(x, t, n_q, n_kv, d, lens, d ** -0.5, own)[0]
        grp, used = n_q // n_kv, sum(lens)
        see = {n: torch.zeros(T, h, d, dtype=torch.bool, device="cuda") for n, h in
               (("O", n_q), ("dQ", n_q), ("dK", n_kv), ("dV", n_kv))}
        lse = torch.zeros(n_q, T, dtype=torch.bool, device="cuda")
        if which == "V":        # column 3 of o; through dp and D: dq of those rows, dk of the keys that they see
            see["O"][at:b, :grp, 3] = True
            see["dQ"][at:b, :grp] = True
            see["dK"][a:b, 0] = True
        elif which == "K":      # scores of the rows at or behind it
            see["O"][at:b, :grp] = True
            lse[:grp, at:b] = True
            see["dQ"][at:b, :grp] = True
            see["dK"][a:b, 0] = True
            see["dV"][a:b, 0] = True
        elif which == "Q":      # its own row's scores
            see["O"][at, 0] = True
            lse[0, at] = True
            see["dQ"][at, 0] = True
            see["dK"][a:at + 1, 0] = True
            see["dV"][a:at + 1, 0] = True
        else:                   # its own row's D and dp, and column 3 of what it adds to dv
            see["dQ"][at, 0] = True
            see["dK"][a:at + 1, 0] = True
            see["dV"][a:at + 1, 0, 3] = True
        got = {"O": f2["O"][0], "dQ": b2["dQ"][0], "dK": b2["dK"][0], "dV": b2["dV"][0]}
        for n, e in (("O", "dO"), ("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
            g = got[n].view(T, -1, d)
            assert torch.isnan(g[see[n]]).all(), f"{n} at {at}"
            _near(g[~see[n]], ref[n][~see[n]], 2 * ref[e][~see[n]], f"{n} at {at}")
        assert torch.isnan(f2["lse"][0][lse]).all()
        rest = ~lse
        rest[:, used:] = False
        _near(f2["lse"][0][rest], ref["lse"][rest], ref["dlse"][rest], "lse")


@pytest.mark.parametrize("t,T,n_q,n_kv,d,lens,left", [(1, 2000, 16, 4, 128, [900, 700], 150), (2, 1000, 4, 2, 64, [500, 300], 77),
                                                      (1, 3000, 4, 1, 64, [2500], 201)])
@pytest.mark.parametrize("bad", [float("nan"), float("-inf")])
def test_rows_of_no_document_hold_anything(t, T, n_q, n_kv, d, lens, left, bad):
    """Uninitialised rows before and behind the documents."""
    x = _inputs(t, T, n_q, n_kv, d, lens, T)
    used = left + sum(lens)
    x["cu"] += left
    y = {k: [v.clone() for v in m] if k != "cu" else m for k, m in x.items()}
    for n in ("Q", "K", "V", "dO"):
        for m in y[n]:
            m[:left] = bad
            m[used:] = bad
    _, f2, b2 = _run(t, T, n_q, n_kv, d, lens, x=y)
    part = {k: [v[left:used].contiguous() for v in m] if k != "cu" else m for k, m in x.items()}
    f = {"O": [o[left:used] for o in f2["O"]], "lse": [l[:, left:used] for l in f2["lse"]]}
    n_ = used - left
    for i, r in enumerate(_reference(part, t, n_q, n_kv, d, lens, d ** -0.5, f)):
        _near(f["O"][i].reshape(n_, -1, d), r["O"], r["dO"], "O")
        _near(f["lse"][i], r["lse"], r["dlse"], "lse")
        for n, e in (("dQ", "eQ"), ("dK", "eK"), ("dV", "eV")):
            _near(b2[n][i][left:used].reshape(n_, -1, d), r[n], r[e], n)
            assert torch.count_nonzero(b2[n][i][:left]) == 0 and torch.count_nonzero(b2[n][i][used:]) == 0


def test_long_document_beside_a_value_that_is_not_finite():
    """65536 tokens, 16 query heads to a KV head, a NaN in dO at token 3: its tile's later keys are computed again over the
    whole document, which no wait may run out over; all other tiles keep their bits."""
    T, n_q, n_kv, d, at, grp = 65536, 48, 3, 64, 3, 16
    g = torch.Generator("cuda").manual_seed(1)
    mat = lambda c: [torch.randn(T, c, generator=g, device="cuda").to(BF16)]   # noqa: E731
    q, k, v, do = mat(n_q * d), mat(n_kv * d), mat(n_kv * d), mat(n_q * d)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    kw = dict(n_q=n_q, n_kv=n_kv, d=d)
    fwd = ttl.packed_attn_fwd(q, k, v, cu, **kw)
    clean = ttl.packed_attn_bwd(do, q, k, v, fwd, cu, **kw)
    bad = [do[0].clone()]
    bad[0][at, 3] = float("nan")
    got = ttl.packed_attn_bwd(bad, q, k, v, fwd, cu, **kw)
    assert ttl.device_status() == 0
    for n in ("dK", "dV"):
        a, b = clean[n][0].view(T, n_kv, d), got[n][0].view(T, n_kv, d)
        assert torch.equal(a[128:], b[128:]) and torch.equal(a[:, 1:], b[:, 1:]), n
    assert torch.isnan(got["dV"][0][:at + 1, 3]).all() and torch.isnan(got["dK"][0][:at + 1, :d]).all()
    # the tile's keys behind the NaN, of KV head 0
    rows = slice(at + 1, 128)
    kk, vv = k[0][rows, :d].to(F8), v[0][rows, :d].to(F8)
    hide = torch.arange(T, device="cuda")[:, None] < torch.arange(at + 1, 128, device="cuda")[None]
    r = {n: 0 for n in ("dV", "eV", "dK", "eK")}
    for c in range(grp):
        cols = slice(c * d, (c + 1) * d)
        qq, gg = q[0][:, cols].to(F8), do[0][:, cols].to(F8)
        ll, D = fwd["lse"][0][c].to(F8)[:, None], (gg * fwd["O"][0][:, cols].to(F8)).sum(1, keepdim=True)
        s = d ** -0.5 * qq @ kk.T
        p = torch.exp(s - ll).masked_fill(hide, 0.0)
        ep = d ** -0.5 * 2 * d * U * qq.abs() @ kk.abs().T + 16 * U * (1 + s.abs()) + 8 * U * (1 + ll.abs())
        dp = gg @ vv.T
        ds = d ** -0.5 * p * (dp - D)
        eds = d ** -0.5 * p * (ep * (dp - D).abs() + 2 * d * U * (gg.abs() @ vv.abs().T + (gg * fwd["O"][0][:, cols].to(F8)).abs().sum(1, keepdim=True)))
        r["dV"], r["eV"] = r["dV"] + p.T @ gg, r["eV"] + T * grp * U * p.T @ gg.abs() + (p * ep).T @ gg.abs()
        r["dK"], r["eK"] = r["dK"] + ds.T @ qq, r["eK"] + T * grp * U * ds.abs().T @ qq.abs() + eds.T @ qq.abs()
    for n, e in (("dV", "eV"), ("dK", "eK")):
        _near(got[n][0][rows, :d], r[n], 1.02 * r[e] + HALF * (r[n].abs() + r[e]), n)


def _edges_into_the_last_kernel(call):
    """The types of the edges between the kernels of a captured call behind one kernel of the caller's: 0 an ordinary
    dependency, 1 one that lets the later kernel's blocks be brought up early."""
    import ctypes
    x = torch.zeros(1000, device="cuda")
    x.add_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        x.add_(1)
        call()
    cuda = ctypes.CDLL("libcuda.so.1")
    n = ctypes.c_size_t(0)
    raw = ctypes.c_void_p(graph.raw_cuda_graph())
    assert cuda.cuGraphGetEdges_v2(raw, None, None, None, ctypes.byref(n)) == 0
    a, b, data = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)(), (ctypes.c_ubyte * (8 * n.value))()
    assert cuda.cuGraphGetEdges_v2(raw, a, b, data, ctypes.byref(n)) == 0
    return [data[8 * i + 2] for i in range(n.value)]


@pytest.mark.skipif(not hasattr(torch.cuda.CUDAGraph, "raw_cuda_graph"), reason="needs the graph itself")
@pytest.mark.parametrize("T,n_q,n_kv,d,types", [(200, 2, 1, 64, [0]), (300, 4, 1, 128, [0]), (4000, 20, 4, 64, [0, 1])])
def test_the_first_kernel_of_a_call_waits_for_the_callers(T, n_q, n_kv, d, types):
    x = _inputs(1, T, n_q, n_kv, d, [T], 1)
    out = ttl.packed_attn_fwd_buffers(1, T, n_q, n_kv, d, 1)
    call = lambda: ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], n_q=n_q, n_kv=n_kv, d=d, out=out)   # noqa: E731
    call()
    assert sorted(_edges_into_the_last_kernel(call)) == types


@pytest.mark.parametrize("n", [1024, 1025, 1500])
@pytest.mark.parametrize("T,n_q,n_kv,d", [(4000, 10, 10, 64), (3000, 16, 4, 128)])
def test_many_documents_and_more_items_than_sms(n, T, n_q, n_kv, d):
    """As many documents as the plan keeps in shared memory, one more, and far more: some fifty of any size, the rest empty."""
    lens = _ragged(T - 77, 50, n + T) + [0] * (n - 50)
    lens = [lens[i] for i in torch.randperm(n, generator=torch.Generator().manual_seed(n)).tolist()]
    x, fwd, bwd = _run(1, T, n_q, n_kv, d, lens, seed=n)
    _check(x, fwd, bwd, 1, T, n_q, n_kv, d, lens)


@pytest.mark.parametrize("n", [31, 32, 33, 64, 95, 1000])
def test_runs_of_empty_documents_inside_a_tile(n):
    for T, n_q, n_kv, d in ((600, 4, 2, 64), (2000, 24, 8, 128)):
        lens = [140] + [0] * n + [9] + [0] * 40 + [3, 1, 20] + [0] * n + [T - 200]
        x, fwd, bwd = _run(1, T, n_q, n_kv, d, lens, seed=n)
        _check(x, fwd, bwd, 1, T, n_q, n_kv, d, lens)


def test_thousands_of_empty_documents_cost_no_reading_of_each():
    T, n_q, n_kv, d = 8192, 32, 8, 128
    kw = dict(n_q=n_q, n_kv=n_kv, d=d)

    def best(empty):
        x = _inputs(1, T, n_q, n_kv, d, [700, 2303] + [0] * empty + [997, 2000, 2192], 4)
        out = ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], **kw)
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda._sleep(1000000)
            a.record()
            ttl.packed_attn_fwd(x["Q"], x["K"], x["V"], x["cu"], out=out, **kw)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    few, many = best(0), best(20000)
    assert many <= 2 * few, (few, many)
