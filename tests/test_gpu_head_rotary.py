"""Head norm and rotation by position vs a plain 64-bit implementation (GPU).

Bounds, per element, u = 2^-24.  A result is rounded to bf16 once (half a step, 2^-8).  Before that: the angle is off
by at most pi u (its conversion to fp32) and sine and cosine by 2 u each, a normed value by its reciprocal root (2 u, and half
the sum's error, at most 24 u) and two products: together below 40 u of the pair's |a| + |b|.  The gradient of x has
one such turn, the norm and a mean of products more: below 80 u of the sum of its terms' sizes.  A weight's gradient
is a sum of N terms in some order: N u of the terms' sizes, and 80 u of each.
"""
import math

import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8
F8, BF16 = torch.float64, torch.bfloat16


def _turn(x, cos, sin, inter):
    """x [T, heads, d], cos and sin [T, rot/2]."""
    n = cos.shape[1]
    y = x.clone()
    i = torch.arange(n, device=x.device)
    p, q = (2 * i, 2 * i + 1) if inter else (i, n + i)
    a, b, c, s = x[..., p], x[..., q], cos[:, None], sin[:, None]
    y[..., p], y[..., q] = a * c - b * s, b * c + a * s
    return y


def _pair_size(x, n, inter):
    """|a| + |b| of the pair each column belongs to."""
    one = torch.ones(x.shape[0], n, dtype=F8, device=x.device)
    y = x.abs()
    i = torch.arange(n, device=x.device)
    p, q = (2 * i, 2 * i + 1) if inter else (i, n + i)
    s = y[..., p] * one[:, None] + y[..., q]
    y[..., p], y[..., q] = s, s
    return y


def _places(T, cu, positions, axes):
    """Positions [pairs' axes, T] and the tokens that count, by the definition."""
    pos, inside = torch.arange(T, dtype=F8)[None], torch.ones(T, dtype=torch.bool)
    if cu is not None:
        pos, inside = torch.zeros(1, T, dtype=F8), torch.zeros(T, dtype=torch.bool)
        for a, b in zip(cu[:-1], cu[1:]):
            pos[0, a:b] = torch.arange(b - a, dtype=F8)
            inside[a:b] = True
    if positions is not None:
        pos = positions.cpu().to(F8).reshape(-1, T)
    return pos.cuda(), inside.cuda()


def _ref_fwd(x, gamma, d, cos, sin, inside, inter, eps):
    n = cos.shape[1]
    x = x.to(F8).view(x.shape[0], -1, d)
    if gamma is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gamma.to(F8)
    y = _turn(x, cos, sin, inter)
    keep = inside[:, None, None]
    return y * keep, (HALF * y.abs() + 41 * U * _pair_size(x, n, inter)) * keep


def _ref_bwd(dy, x, gamma, d, cos, sin, inside, inter, eps):
    n_, keep = cos.shape[1], inside[:, None, None]
    dy = dy.to(F8).view(dy.shape[0], -1, d)
    g, size = _turn(dy, cos, -sin, inter), _pair_size(dy, n_, inter)
    if gamma is None:
        return g * keep, (HALF * g.abs() + 41 * U * size) * keep, None, None
    x = x.to(F8).view(x.shape[0], -1, d)
    r = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    n, w = x * r, gamma.to(F8)
    h, hs = g * w, size * w.abs()
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    e = HALF * dx.abs() + 81 * U * r * (hs + n.abs() * (hs * n.abs()).mean(-1, keepdim=True))
    count = int(keep.sum()) * dy.shape[1]
    dg, gs = (g * n * keep).sum((0, 1)), (size * n.abs() * keep).sum((0, 1))
    return dx * keep, e * keep, dg, (count + 81) * U * gs


def _near(got, ref, bound, name):
    got = got.to(F8)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - bound * 1.01 - 1e-37
    assert (over <= 0).all(), f"{name}: {over.max().item():.3e} beyond the bound"


def _inputs(t, T, n_q, n_kv, d, norm, seed):
    g = torch.Generator().manual_seed(seed)

    def mats(n, std=1.0):
        return [(torch.randn(T, n // t * d, generator=g) * std).to(BF16).cuda() for _ in range(t)]

    x = {"Q": mats(n_q, 2.0), "K": mats(n_kv), "dQ": mats(n_q), "dK": mats(n_kv)}
    for n in ("gamma_q", "gamma_k"):
        x[n] = None if norm is None else (1 + 0.3 * torch.randn(d, generator=g)).to(norm).cuda()
    return x


def _run(x, rotary, t, T, n_q, n_kv, d, cu=None, positions=None, eps=1e-6, out_f=None, out_b=None, stream=None):
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, gamma_q=x["gamma_q"], gamma_k=x["gamma_k"], eps=eps, positions=positions,
              cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"), stream=stream)
    f = ttl.head_norm_rotary_fwd(x["Q"], x["K"], rotary, out=out_f, **kw)
    b = ttl.head_norm_rotary_bwd(x["dQ"], x["dK"], rotary, Q=x["Q"], K=x["K"], out=out_b, **kw)
    assert ttl.device_status() == 0
    return f, b


def _check(x, f, b, t, T, n_q, n_kv, d, freqs, axes, inter, cu, positions, eps=1e-6, norm=True):
    pos, inside = _places(T, cu, positions, axes)
    angle = torch.stack([pos[a] * w for a, w in zip(axes, freqs)], 1) if freqs else torch.zeros(T, 0, dtype=F8, device="cuda")
    cos, sin = angle.cos(), angle.sin()
    for n, heads in (("Q", n_q), ("K", n_kv)):
        w = x["gamma_" + n.lower()]
        dg, bound = 0, 0
        for i in range(t):
            y, e = _ref_fwd(x[n][i], w, d, cos, sin, inside, inter, eps)
            _near(f[n][i].view(T, -1, d), y, e, f"{n}[{i}]")
            dx, e, g, ge = _ref_bwd(x["d" + n][i], x[n][i], w, d, cos, sin, inside, inter, eps)
            _near(b["d" + n][i].view(T, -1, d), dx, e, f"d{n}[{i}]")
            if w is not None:
                dg, bound = dg + g, bound + ge
        if w is not None:
            _near(b["dgamma_" + n.lower()], dg, bound * t, "dgamma_" + n.lower())


# t, T, n_q, n_kv, d, rot, interleaved, weights, documents (None: one stretch), axes of the pairs
CASES = [
    (1, 1, 1, 1, 16, 16, False, None, None, 1), (1, 1, 1, 1, 128, 128, False, torch.bfloat16, [0, 1], 1),
    (2, 130, 4, 2, 64, 64, False, torch.bfloat16, [0, 1, 65, 130], 1), (2, 130, 4, 2, 64, 64, True, torch.float32, [3, 3, 90, 100], 1),
    (1, 77, 3, 1, 80, 80, False, torch.bfloat16, None, 2), (1, 77, 5, 5, 80, 48, True, None, None, 3),
    (4, 33, 8, 4, 96, 32, False, torch.float32, [0, 33], 1), (1, 515, 7, 2, 256, 256, False, torch.bfloat16, [10, 500], 1),
    (1, 300, 2, 1, 32, 16, True, torch.bfloat16, None, 1), (16, 9, 32, 16, 128, 64, False, torch.bfloat16, None, 1),
    (8, 700, 32, 8, 128, 128, False, torch.bfloat16, [0, 300, 300, 650], 1), (1, 64, 2, 2, 64, 0, False, torch.bfloat16, None, 1),
    (1, 64, 2, 2, 48, 0, False, None, None, 1), (1, 4099, 5, 5, 128, 128, True, torch.float32, None, 1),
    (1, 2000, 1, 40, 112, 112, False, torch.bfloat16, [], 1), (1, 20000, 2, 1, 64, 64, False, torch.bfloat16, [0, 12000, 19990], 1),
]


@pytest.mark.parametrize("t,T,n_q,n_kv,d,rot,inter,norm,cu,axes", CASES)
def test_forward_and_backward(t, T, n_q, n_kv, d, rot, inter, norm, cu, axes):
    if cu == []:
        cu = [0]                       # no document at all
    x = _inputs(t, T, n_q, n_kv, d, norm, T + d)
    freqs = ttl.rotary_freqs(rot)
    pair_axes = [i % axes for i in range(rot // 2)]
    positions = None
    if axes > 1:
        positions = torch.randint(-50, 3000, (axes, T), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    f, b = _run(x, ttl.Rotary(freqs, axes=pair_axes, interleaved=inter), t, T, n_q, n_kv, d, cu, positions)
    _check(x, f, b, t, T, n_q, n_kv, d, freqs, pair_axes, inter, cu, positions)


@pytest.mark.parametrize("start", [2 ** 31 - 200, -(2 ** 31), 10 ** 6, -5])
def test_far_positions(start):
    """Angles of positions near the ends of their type: whole turns are dropped exactly."""
    t, T, n_q, n_kv, d = 1, 150, 2, 1, 64
    x = _inputs(t, T, n_q, n_kv, d, torch.bfloat16, 3)
    freqs = ttl.rotary_freqs(d)
    positions = (start + torch.arange(T)).to(torch.int32).cuda()
    f, b = _run(x, ttl.Rotary(freqs), t, T, n_q, n_kv, d, None, positions)
    # (the 64-bit reference itself: a product of 2^31 is off by up to 2^-53 * 2^31 = 2.4e-7 radians, 4 u, and so
    # is the library's fraction of a turn, which 2^31 multiplies)
    _check(x, f, b, t, T, n_q, n_kv, d, freqs, [0] * (d // 2), False, None, positions)


def test_frequencies_of_any_size_and_sign():
    t, T, n_q, n_kv, d = 1, 90, 2, 1, 64
    x = _inputs(t, T, n_q, n_kv, d, None, 4)
    freqs = [0.0, -1.0, math.pi, 2 * math.pi, -2 * math.pi, 100.25, -1e-9, 1e-30] * 4
    f, b = _run(x, ttl.Rotary(freqs), t, T, n_q, n_kv, d)
    _check(x, f, b, t, T, n_q, n_kv, d, freqs, [0] * 32, False, None, None)


@pytest.mark.parametrize("norm", [None, torch.bfloat16])
def test_fused_projection_in_place_and_beside(norm):
    """Q and K as column ranges of one matrix; results in their place, or in a wider matrix: the same bits, and the
    columns beside them keep their values."""
    t, T, n_q, n_kv, d, cu = 2, 333, 8, 4, 64, [0, 200, 320]
    x = _inputs(t, T, n_q, n_kv, d, norm, 6)
    rotary = ttl.Rotary(ttl.rotary_freqs(d))
    f, b = _run(x, rotary, t, T, n_q, n_kv, d, cu)
    qc, kc = n_q // t * d, n_kv // t * d
    cut = lambda m: ([a[:, 8:8 + qc] for a in m], [a[:, 8 + qc:8 + qc + kc] for a in m])   # noqa: E731
    wide = lambda q, k: [torch.cat([torch.full((T, 8), 7.0, dtype=BF16, device="cuda"), q[i], k[i],   # noqa: E731
                                    torch.full((T, 16), 7.0, dtype=BF16, device="cuda")], 1) for i in range(t)]
    ins, grads = wide(x["Q"], x["K"]), wide(x["dQ"], x["dK"])
    y = dict(x)
    y["Q"], y["K"] = cut(ins)
    y["dQ"], y["dK"] = cut(grads)
    out_b = ttl.head_norm_rotary_bwd_buffers(t, T, n_q, n_kv, d, norm is not None)
    out_b["dQ"], out_b["dK"] = y["dQ"], y["dK"]
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, gamma_q=x["gamma_q"], gamma_k=x["gamma_k"],
              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    ttl.head_norm_rotary_bwd(y["dQ"], y["dK"], rotary, Q=y["Q"], K=y["K"], out=out_b, **kw)
    ttl.head_norm_rotary_fwd(y["Q"], y["K"], rotary, out={"Q": y["Q"], "K": y["K"]}, **kw)
    for i in range(t):
        for n in ("Q", "K"):
            assert torch.equal(y[n][i], f[n][i]) and torch.equal(y["d" + n][i], b["d" + n][i])
        for m in (ins[i], grads[i]):
            assert (m[:, :8] == 7).all() and (m[:, 8 + qc + kc:] == 7).all()
    if norm is not None:
        assert torch.equal(out_b["dgamma_q"], b["dgamma_q"]) and torch.equal(out_b["dgamma_k"], b["dgamma_k"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tokens_of_no_document_hold_anything(bad):
    t, T, n_q, n_kv, d, cu = 2, 260, 4, 2, 128, [7, 90, 90, 251]
    x = _inputs(t, T, n_q, n_kv, d, torch.float32, 8)
    freqs = ttl.rotary_freqs(d)
    f, b = _run(x, ttl.Rotary(freqs), t, T, n_q, n_kv, d, cu)
    y = {n: [m.clone() for m in v] if isinstance(v, list) else v for n, v in x.items()}
    for n in ("Q", "K", "dQ", "dK"):
        for m in y[n]:
            m[:7] = bad
            m[251:] = bad
    f2, b2 = _run(y, ttl.Rotary(freqs), t, T, n_q, n_kv, d, cu)
    for n in ("Q", "K"):
        assert all(torch.equal(p, q) for p, q in zip(f[n], f2[n])) and all(torch.equal(p, q) for p, q in zip(b["d" + n], b2["d" + n]))
        assert torch.count_nonzero(f2[n][0][:7]) == 0 and torch.count_nonzero(b2["d" + n][1][251:]) == 0
        assert torch.equal(b["dgamma_" + n.lower()], b2["dgamma_" + n.lower()])
    _check(x, f2, b2, t, T, n_q, n_kv, d, freqs, [0] * 64, False, cu, None)


def test_zero_heads_and_eps():
    """A head of zeros: its result and gradient are finite; a large eps counts."""
    t, T, n_q, n_kv, d = 1, 40, 2, 1, 64
    x = _inputs(t, T, n_q, n_kv, d, torch.bfloat16, 9)
    x["Q"][0][3] = 0
    x["K"][0][:] *= 1e-3
    freqs = ttl.rotary_freqs(d)
    for eps in (1e-6, 0.5):
        f, b = _run(x, ttl.Rotary(freqs), t, T, n_q, n_kv, d, eps=eps)
        _check(x, f, b, t, T, n_q, n_kv, d, freqs, [0] * 32, False, None, None, eps=eps)


def test_accumulate_and_no_tokens():
    t, T, n_q, n_kv, d = 1, 200, 4, 2, 64
    x = _inputs(t, T, n_q, n_kv, d, torch.bfloat16, 10)
    rotary = ttl.Rotary(ttl.rotary_freqs(d))
    f, b = _run(x, rotary, t, T, n_q, n_kv, d)
    out = ttl.head_norm_rotary_bwd_buffers(t, T, n_q, n_kv, d)
    out["dgamma_q"].fill_(2.0)
    out["dgamma_k"].fill_(-3.0)
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, gamma_q=x["gamma_q"], gamma_k=x["gamma_k"])
    ttl.head_norm_rotary_bwd(x["dQ"], x["dK"], rotary, Q=x["Q"], K=x["K"], accumulate=True, out=out, **kw)
    assert torch.equal(out["dgamma_q"], b["dgamma_q"] + 2.0) and torch.equal(out["dgamma_k"], b["dgamma_k"] - 3.0)
    none = {n: [m[:0] for m in x[n]] for n in ("Q", "K", "dQ", "dK")}
    ttl.head_norm_rotary_fwd(none["Q"], none["K"], rotary, **kw)
    out = ttl.head_norm_rotary_bwd(none["dQ"], none["dK"], rotary, Q=none["Q"], K=none["K"], **kw)
    assert torch.count_nonzero(out["dgamma_q"]) == 0 and torch.count_nonzero(out["dgamma_k"]) == 0
    assert ttl.device_status() == 0


def test_same_bits_again_and_from_a_graph_on_a_side_stream():
    t, T, n_q, n_kv, d, cu = 2, 1500, 8, 2, 128, [0, 400, 1499]
    x = _inputs(t, T, n_q, n_kv, d, torch.bfloat16, 11)
    rotary = ttl.Rotary(ttl.rotary_freqs(d))
    f, b = _run(x, rotary, t, T, n_q, n_kv, d, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f2, b2 = _run(x, rotary, t, T, n_q, n_kv, d, cu, stream=side)
    torch.cuda.synchronize()
    f3 = ttl.head_norm_rotary_fwd_buffers(t, T, n_q, n_kv, d)
    b3 = ttl.head_norm_rotary_bwd_buffers(t, T, n_q, n_kv, d)
    bounds = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, gamma_q=x["gamma_q"], gamma_k=x["gamma_k"], cu_seqlens=bounds)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        ttl.head_norm_rotary_fwd(x["Q"], x["K"], rotary, out=f3, **kw)
        ttl.head_norm_rotary_bwd(x["dQ"], x["dK"], rotary, Q=x["Q"], K=x["K"], out=b3, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert ttl.device_status() == 0
    for other_f, other_b in ((f2, b2), (f3, b3)):
        for n in ("Q", "K"):
            assert all(torch.equal(p, q) for p, q in zip(f[n], other_f[n]))
            assert all(torch.equal(p, q) for p, q in zip(b["d" + n], other_b["d" + n]))
            assert torch.equal(b["dgamma_" + n.lower()], other_b["dgamma_" + n.lower()])


def test_gradient_against_differences():
    t, T, n_q, n_kv, d, cu = 1, 60, 2, 1, 64, [0, 25, 58]
    x = _inputs(t, T, n_q, n_kv, d, torch.float32, 12)
    freqs = ttl.rotary_freqs(d)
    f, b = _run(x, ttl.Rotary(freqs, interleaved=True), t, T, n_q, n_kv, d, cu)
    pos, inside = _places(T, cu, None, [0])
    angle = pos[0][:, None] * torch.tensor(freqs, dtype=F8, device="cuda")
    gen = torch.Generator("cuda").manual_seed(5)
    for n in ("Q", "K"):
        w = x["gamma_" + n.lower()].to(F8)
        dx = torch.randn(x[n][0].shape, generator=gen, device="cuda", dtype=F8)
        dw = torch.randn(d, generator=gen, device="cuda", dtype=F8)

        def loss(e):
            y, _ = _ref_fwd(x[n][0].to(F8) + e * dx, w + e * dw, d, angle.cos(), angle.sin(), inside, True, 1e-6)
            return (y * x["d" + n][0].to(F8).view(T, -1, d)).sum()

        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        got = (b["d" + n][0].to(F8) * dx).sum() + (b["dgamma_" + n.lower()].to(F8) * dw).sum()
        # dx is rounded once, by at most half a step of each value: a random direction sees 4 sigma of its 2-norm;
        # the difference itself is off by its third derivative times 1e-8
        size = b["d" + n][0].to(F8).norm() + 1e-2
        assert (got - want).abs() <= 4 * HALF * size


def test_bad_document_bounds_are_reported():
    t, T, n_q, n_kv, d = 1, 200, 2, 1, 64
    x = _inputs(t, T, n_q, n_kv, d, torch.bfloat16, 0)
    rotary = ttl.Rotary(ttl.rotary_freqs(d))
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, gamma_q=x["gamma_q"], gamma_k=x["gamma_k"])
    for cu in ([0, 150, 100, 200], [-5, 100, 200], [0, 100, 5000], [300, 400], [200, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        ttl.head_norm_rotary_fwd(x["Q"], x["K"], rotary, cu_seqlens=cu, **kw)
        assert ttl.device_status() == ttl.TTL_ERR_DEVICE
        ttl.head_norm_rotary_bwd(x["dQ"], x["dK"], rotary, Q=x["Q"], K=x["K"], cu_seqlens=cu, **kw)
        assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    _run(x, rotary, t, T, n_q, n_kv, d, [0, 200])


def test_rows_beyond_32_bits():
    """A matrix of more than 2^31 elements: the last rows, of a few columns of it."""
    T, ld, d, n_q, n_kv = 70000, 40960, 64, 2, 1
    big = torch.empty(T, ld, dtype=BF16, device="cuda")
    x = _inputs(1, 300, n_q, n_kv, d, torch.bfloat16, 13)
    q, k = big[:, 1024:1024 + 2 * d], big[:, 40000 // 8 * 8:40000 // 8 * 8 + d]
    q.zero_()
    k.zero_()
    q[-300:], k[-300:] = x["Q"][0], x["K"][0]
    rotary = ttl.Rotary(ttl.rotary_freqs(d))
    kw = dict(n_q=n_q, n_kv=n_kv, d=d, gamma_q=x["gamma_q"], gamma_k=x["gamma_k"])
    want = ttl.head_norm_rotary_fwd([x["Q"][0]], [x["K"][0]], rotary,
                                    positions=torch.arange(T - 300, T, dtype=torch.int32, device="cuda"), **kw)
    ttl.head_norm_rotary_fwd([q], [k], rotary, out={"Q": [q], "K": [k]}, **kw)
    assert ttl.device_status() == 0
    assert torch.equal(q[-300:], want["Q"][0]) and torch.equal(k[-300:], want["K"][0])


# ---------------------------------------------------------------------------- values that are not finite

def _same(got, ref, bound, name):
    """NaN where the formula's result is NaN, its infinities, and everything else as near as without them."""
    got = got.to(F8)
    nan, inf = torch.isnan(ref), torch.isinf(ref)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaN at {torch.nonzero(torch.isnan(got) != nan)[:4].tolist()}"
    assert torch.equal(got[inf], ref[inf]), f"{name}: infinities"
    rest = ~(nan | inf)
    over = (got - ref).abs()[rest] - bound[rest] * 1.01 - 1e-37
    assert (over <= 0).all(), f"{name}: beyond the bound"


def _check_same(x, f, b, T, d, cos, sin, inter):
    inside = torch.ones(T, dtype=torch.bool, device="cuda")
    for n in ("Q", "K"):
        w = x["gamma_" + n.lower()]
        y, e = _ref_fwd(x[n][0], w, d, cos, sin, inside, inter, 1e-6)
        _same(f[n][0].view(T, -1, d), y, e, n)
        dx, e, dg, ge = _ref_bwd(x["d" + n][0], x[n][0], w, d, cos, sin, inside, inter, 1e-6)
        _same(b["d" + n][0].view(T, -1, d), dx, e, "d" + n)
        if w is not None:
            _same(b["dgamma_" + n.lower()], dg, ge, "dgamma_" + n.lower())


# columns, rotated ones and weights: parts of a head, none, all, and slots of 16 that leave lanes idle
MIXED = [(128, 64, None), (128, 64, torch.bfloat16), (64, 0, None), (64, 0, torch.float32), (80, 48, None), (256, 16, torch.float32),
         (64, 64, None), (128, 128, torch.bfloat16)]


@pytest.mark.parametrize("d,rot,norm", MIXED)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_value_that_is_not_finite_stays_in_its_pair(d, rot, norm, inter, bad):
    """In each column of a head, of the inputs or of the gradients: it reaches the column that it turns with, and through the norm its
    head; columns that do not turn keep theirs to themselves."""
    freqs = ttl.rotary_freqs(rot)
    rotary = ttl.Rotary(freqs, interleaved=inter)
    turned = lambda T: (torch.arange(T, dtype=F8, device="cuda")[:, None]   # noqa: E731
                        * torch.tensor(freqs, dtype=F8, device="cuda"))
    # every column, a token each
    for names in (("Q", "K"), ("dQ", "dK")):
        x = _inputs(1, d + 3, 2, 1, d, norm, d + rot)
        for n in names:
            for c in range(d):
                x[n][0][c + 1, c] = bad
        f, b = _run(x, rotary, 1, d + 3, 2, 1, d)
        a = turned(d + 3)
        _check_same(x, f, b, d + 3, d, a.cos(), a.sin(), inter)
    # one column alone, for the sums over tokens
    for c in sorted({0, 7, rot // 2, max(rot - 1, 0), min(rot, d - 1), min(rot + 8, d - 1), d - 9, d - 1}):
        for n in ("Q", "dQ"):
            x = _inputs(1, 6, 2, 1, d, norm, c)
            x[n][0][3, c] = bad
            f, b = _run(x, rotary, 1, 6, 2, 1, d)
            a = turned(6)
            _check_same(x, f, b, 6, d, a.cos(), a.sin(), inter)


# ---------------------------------------------------------------------------- large frequencies at far positions

_PI_BITS = 400


def _two_pi():
    """2 pi 2^400 as a whole number: 8 (4 atan(1/5) - atan(1/239))."""
    one = 1 << (_PI_BITS + 40)

    def atan_of(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return 8 * (4 * atan_of(5) - atan_of(239)) >> 40


def _reduced(freqs, positions):
    """Angles in (-2 pi, 2 pi) of each position and frequency, whole turns dropped in whole numbers."""
    turn = _two_pi()
    rows = []
    for p in positions:
        row = []
        for f in freqs:
            num, den = float(f).as_integer_ratio()        # (den a power of two)
            angle = p * num * (1 << _PI_BITS) % (turn * den)
            row.append(angle / (den << _PI_BITS))
        rows.append(row)
    return torch.tensor(rows, dtype=F8, device="cuda")


@pytest.mark.parametrize("start", [2 ** 24 - 40, 2 ** 31 - 81, -(2 ** 31), 10 ** 9 + 7])
@pytest.mark.parametrize("inter", [False, True])
def test_large_frequencies_at_far_positions(start, inter):
    """An angle of any accepted frequency and position, to the bound that holds for small ones."""
    t, T, n_q, n_kv, d = 1, 80, 2, 1, 64
    x = _inputs(t, T, n_q, n_kv, d, torch.float32, 31)
    freqs = [1.0, 100.0, -100.0, 12345.678, 99999.9, 2.0 ** 20, -(2.0 ** 20) + 0.37, math.pi * 1000, 1048575.999, 3e5, 1e-3, 0.1] * 3
    freqs = freqs[:32]
    positions = [start + i for i in range(T)]
    f, b = _run(x, ttl.Rotary(freqs, interleaved=inter), t, T, n_q, n_kv, d, None,
                torch.tensor(positions, dtype=torch.int32, device="cuda"))
    angle = _reduced(freqs, positions)
    inside = torch.ones(T, dtype=torch.bool, device="cuda")
    for n in ("Q", "K"):
        w = x["gamma_" + n.lower()]
        y, e = _ref_fwd(x[n][0], w, d, angle.cos(), angle.sin(), inside, inter, 1e-6)
        _near(f[n][0].view(T, -1, d), y, e, n)
        dx, e, dg, ge = _ref_bwd(x["d" + n][0], x[n][0], w, d, angle.cos(), angle.sin(), inside, inter, 1e-6)
        _near(b["d" + n][0].view(T, -1, d), dx, e, "d" + n)
        _near(b["dgamma_" + n.lower()], dg, ge, "dgamma_" + n.lower())


def _with_empty(total, n, seed):
    """n lengths, `total` tokens together: some fifty of any size, the rest empty, in any order."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, total + 1, (49,), generator=g).sort()[0].tolist()
    lens = [b - a for a, b in zip([0] + cuts, cuts + [total])] + [0] * (n - 50)
    return [lens[i] for i in torch.randperm(n, generator=g).tolist()]


@pytest.mark.parametrize("n", [512, 513, 2000])
@pytest.mark.parametrize("norm", [None, torch.bfloat16])
def test_many_documents(n, norm):
    """As many as a block keeps in shared memory, one more, and far more: empty ones among them."""
    t, T, n_q, n_kv, d = 2, 3100, 4, 2, 64
    cu = [5] + [5 + c for c in torch.tensor(_with_empty(3000, n, n)).cumsum(0).tolist()]
    x = _inputs(t, T, n_q, n_kv, d, norm, n)
    freqs = ttl.rotary_freqs(d)
    f, b = _run(x, ttl.Rotary(freqs), t, T, n_q, n_kv, d, cu)
    _check(x, f, b, t, T, n_q, n_kv, d, freqs, [0] * (d // 2), False, cu, None)


@pytest.mark.parametrize("d,rot", [(48, 0), (80, 48), (112, 112), (64, 64)])
@pytest.mark.parametrize("inter", [False, True])
def test_a_weight_that_is_infinite(d, rot, inter):
    """Widths that leave lanes idle among them: these add nothing to a head's sums."""
    freqs = ttl.rotary_freqs(rot)
    angle = torch.arange(9, dtype=F8, device="cuda")[:, None] * torch.tensor(freqs, dtype=F8, device="cuda")
    for c in (3, d - 5):
        x = _inputs(1, 9, 2, 1, d, torch.float32, c)
        x["gamma_q"][c], x["gamma_k"][c] = math.inf, -math.inf
        f, b = _run(x, ttl.Rotary(freqs, interleaved=inter), 1, 9, 2, 1, d)
        _check_same(x, f, b, 9, d, angle.cos(), angle.sin(), inter)
